// cache.cuh -- the paged 8-bit key/value cache of the serving calls: its
// descriptor, the e4m3 block format, and the split of attention work over the
// grid that its kernels and the merge kernel share.
//
// Format.  A page holds `page` consecutive tokens of one sequence; codes are
// e4m3, [n_pages, Hkv, page, d], and a (page, KV head) block of either array
// has one fp32 scale: value = code * scale.  The calls that write blocks use
// powers of two, the smallest 2^k >= 2^-64 that holds the block's largest
// magnitude within 448 (e4m3's largest value).  A power of two costs e4m3
// nothing but range (its relative step is the same over 2^-6 .. 448), makes
// x / scale and code * scale exact, and makes a block that grows a coarser
// scale later (appended to, or regrouped by an eviction) keep its codes' bits
// except where they fall below 2^-6 of the new scale.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "geometry.cuh"
#include "kernels.h"

namespace bdlm {

struct CacheDesc {
  uint8_t* k8;
  uint8_t* v8;
  float* ks;
  float* vs;
  const int32_t* table;  // [n_seqs, max_pages]
  const int32_t* lens;   // [n_seqs]
  int64_t n_pages;
  int n_seqs, max_pages, page, lp;  // page = 1 << lp
  int Hkv, d;
};

// New rows of the sequences: row_offsets [n_seqs + 1], or null for max_rows
// rows each; T rows in the tensors.
struct RowsDesc {
  const int32_t* off;
  int64_t T;
  int max_rows;
};

// Findings about contents that only the device can check: what is bad is left
// out of the result.  They are or-ed into a word of their own in the workspace
// header, so that the status word stays free for the first expired wait.
enum : uint32_t { kStatusBadPage = 0x7201, kStatusBadLen = 0x7202, kStatusBadRows = 0x7204 };
constexpr int kContentsWord = 1;  // (uint32; word 0: the status word)
static_assert(kContentsWord < kSchedWordFwd && (kContentsWord + 1) * 4 <= kHeaderClearBytes, "a word that training calls clear");

// Raises a kernel's dynamic shared memory limit on the current device, once per
// device (`done`: a bit for each).
cudaError_t raise_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done);

#if defined(__CUDACC__)

// Programmatic dependent launch: lets the next kernel of the stream start
// when it was launched so; waits for the kernel before this one to end.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct SeqView {
  int64_t row0;
  int rows, len;
};

// Rows and cached length of sequence s, held inside the tensors' bounds.
__device__ __forceinline__ SeqView seq_view(const CacheDesc& c, const RowsDesc& r, int s, uint32_t& bad) {
  SeqView v;
  if (r.off) {
    const int a = r.off[s], b = r.off[s + 1];
    const bool ok = a >= 0 && b >= a && b <= r.T && b - a <= r.max_rows;
    if (!ok) bad |= kStatusBadRows;
    v.row0 = ok ? a : 0;
    v.rows = ok ? b - a : 0;
  } else {
    v.row0 = (int64_t)s * r.max_rows;
    v.rows = r.max_rows;
  }
  const int64_t cap = (int64_t)c.max_pages << c.lp;
  const int len = c.lens[s];
  v.len = len < 0 ? 0 : len > cap ? (int)cap : len;
  if (v.len != len) bad |= kStatusBadLen;
  return v;
}

// Physical page of logical page j of sequence s, -1 (and flagged) when the
// table's entry is not a page of the pool.
__device__ __forceinline__ int page_id(const CacheDesc& c, int s, int j, uint32_t& bad) {
  const int p = c.table[(int64_t)s * c.max_pages + j];
  if (p >= 0 && p < c.n_pages) return p;
  bad |= kStatusBadPage;
  return -1;
}

// Of the eight groups of 16 keys of a unit, those that open a page (a bit each).
__device__ __forceinline__ uint32_t first_groups(int page) {
  return page == 16 ? 0xffu : page == 32 ? 0x55u : page == 64 ? 0x11u : 0x01u;
}

// The scale of a block whose largest magnitude has the fp32 bits `amax`
// (NaN when the block holds a value that is not finite).
__device__ __forceinline__ float block_scale(uint32_t amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  int k = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  if (k < -64) k = -64;
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ bool is_pow2(float s) {
  const uint32_t b = __float_as_uint(s);
  return (b & 0x807fffffu) == 0 && b != 0 && b < 0x7f800000u;
}

// Two values to e4m3 (nearest, ties to even; NaN to NaN, beyond 448 to 448).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Two e4m3 codes (low byte first) to a pair of halves: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// ------------------------------------------------------- division of work
// A segment is one row tile of one (sequence, KV head): the rows of the
// group's query heads flattened as token * group + head, tile_rows of them.
// Its keys are cut into units of 128: the cached ones, then the new rows'
// own block (folded into the last unit when it has at most kFoldRows rows).
// All units of all segments form one list, sequence by sequence, KV head by
// KV head, row tile by row tile; CTA c of G takes units
// [c U / G, (c + 1) U / G).  Every CTA so has the same work whatever the
// lengths; a segment that spans CTAs leaves one partial result per CTA, which
// the merge kernel joins in list order (no atomics: results do not depend on
// timing).  A CTA has at most two partials: its first segment (begun by
// another CTA) and its last (begun here, continued by another).
constexpr int kUnit = 128;
constexpr int kFoldRows = 32;

struct AttnSplit {
  int group;      // query heads per KV head
  int tile_rows;  // rows of a row tile
  int local;      // the rows also read their own block
  int extra;      // empty positions that open a segment
  int keyed;      // weights: one segment per (sequence, KV head) that holds all
                  // rows; a unit of keys counts once for each row tile
};

struct SegInfo {
  SeqView v;
  int rtiles, ktiles, ltiles;  // row tiles, cached units, own-block units that are not folded
  int units;                   // per segment
  int span;                    // its positions in the list
};

__device__ __forceinline__ SegInfo seg_info(const CacheDesc& c, const RowsDesc& r, const AttnSplit& a, int s,
                                            uint32_t& bad) {
  SegInfo g;
  g.v = seq_view(c, r, s, bad);
  g.rtiles = (g.v.rows * a.group + a.tile_rows - 1) / a.tile_rows;
  g.ktiles = (g.v.len + kUnit - 1) / kUnit;
  g.ltiles = a.local && g.v.rows > kFoldRows ? (g.v.rows + kUnit - 1) / kUnit : 0;
  const int n = g.ktiles + g.ltiles;
  g.units = n > 0 ? n : 1;
  if (a.keyed) {
    g.units = g.ktiles * g.rtiles;
    g.ltiles = g.rtiles;  // (positions of one unit of keys)
    g.rtiles = g.units > 0 ? 1 : 0;
  }
  g.span = g.units + a.extra;
  return g;
}

struct UnitPos {
  int s, h, rt, j;  // j: position in the segment; unit j - extra
};

// Positions of all segments (every lane of the calling warp gets the sum).
__device__ __forceinline__ int64_t total_units(const CacheDesc& c, const RowsDesc& r, const AttnSplit& a,
                                               uint32_t& bad) {
  const int lane = threadIdx.x & 31;
  int64_t sum = 0;
  for (int s = lane; s < c.n_seqs; s += 32) {
    const SegInfo g = seg_info(c, r, a, s, bad);
    sum += (int64_t)g.rtiles * c.Hkv * g.span;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The segment of list position u (0 <= u < total), by the whole warp.
__device__ __forceinline__ UnitPos locate_unit(const CacheDesc& c, const RowsDesc& r, const AttnSplit& a, int64_t u,
                                               uint32_t& bad) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int s0 = 0; s0 < c.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int64_t n = 0;
    int span = 1, rt = 1;
    if (s < c.n_seqs) {
      const SegInfo g = seg_info(c, r, a, s, bad);
      span = g.span;
      rt = g.rtiles;
      n = (int64_t)g.rtiles * c.Hkv * g.span;
    }
    int64_t cum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, cum, o);
      if (lane >= o) cum += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, u < before + cum);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int64_t left = u - (before + __shfl_sync(0xffffffffu, cum - n, l));
      span = __shfl_sync(0xffffffffu, span, l);
      rt = __shfl_sync(0xffffffffu, rt, l);
      const int64_t seg = left / span;
      UnitPos p;
      p.s = s0 + l;
      p.h = (int)(seg / rt);
      p.rt = (int)(seg % rt);
      p.j = (int)(left % span);
      return p;
    }
    before += __shfl_sync(0xffffffffu, cum, 31);
  }
  return UnitPos{0, 0, 0, 0};
}

// CTAs that take part: no more than there are units, so that none is empty.
__device__ __forceinline__ int split_ctas(int64_t U, int G) { return U < G ? (int)U : G; }
__device__ __forceinline__ int64_t split_begin(int64_t U, int G, int c) { return U * c / G; }
// What CTA `cta` of G takes: list positions [u0, u1) (u0 = u1: nothing), and the
// first position's segment (with `last`: the last position's); U and G: all
// positions, the CTAs that take part.  By a whole warp.  Up to 32 sequences are
// looked at once.
struct SplitOpen {
  int64_t u0, u1, U;
  int G;
  UnitPos pos;
  SegInfo seg;
};
template <bool last = false>
__device__ __forceinline__ SplitOpen split_open(const CacheDesc& c, const RowsDesc& r, const AttnSplit& a, int G, int cta,
                                                uint32_t& bad) {
  SplitOpen o;
  o.u0 = o.u1 = 0;
  o.pos = UnitPos{0, 0, 0, 0};
  o.seg = SegInfo{};
  if (c.n_seqs > 32) {
    const int64_t U = total_units(c, r, a, bad);
    G = split_ctas(U, G);
    o.U = U;
    o.G = G;
    if (cta < G) {
      o.u0 = split_begin(U, G, cta);
      o.u1 = split_begin(U, G, cta + 1);
      o.pos = locate_unit(c, r, a, last ? o.u1 - 1 : o.u0, bad);
      o.seg = seg_info(c, r, a, o.pos.s, bad);
    }
    return o;
  }
  const int lane = threadIdx.x & 31;
  SegInfo g{};
  int64_t n = 0;
  if (lane < c.n_seqs) {
    g = seg_info(c, r, a, lane, bad);
    n = (int64_t)g.rtiles * c.Hkv * g.span;
  }
  int64_t cum = n;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, cum, k);
    if (lane >= k) cum += x;
  }
  const int64_t U = __shfl_sync(0xffffffffu, cum, 31);
  G = split_ctas(U, G);
  o.U = U;
  o.G = G;
  if (cta >= G) return o;
  o.u0 = split_begin(U, G, cta);
  o.u1 = split_begin(U, G, cta + 1);
  const int64_t at = last ? o.u1 - 1 : o.u0;
  const int l = __ffs(__ballot_sync(0xffffffffu, at < cum)) - 1;
  const int64_t left = at - __shfl_sync(0xffffffffu, cum - n, l);
  o.seg.v.row0 = __shfl_sync(0xffffffffu, g.v.row0, l);
  o.seg.v.rows = __shfl_sync(0xffffffffu, g.v.rows, l);
  o.seg.v.len = __shfl_sync(0xffffffffu, g.v.len, l);
  o.seg.rtiles = __shfl_sync(0xffffffffu, g.rtiles, l);
  o.seg.ktiles = __shfl_sync(0xffffffffu, g.ktiles, l);
  o.seg.ltiles = __shfl_sync(0xffffffffu, g.ltiles, l);
  o.seg.units = __shfl_sync(0xffffffffu, g.units, l);
  o.seg.span = __shfl_sync(0xffffffffu, g.span, l);
  const int64_t seg = left / o.seg.span;
  o.pos.s = l;
  o.pos.h = (int)(seg / o.seg.rtiles);
  o.pos.rt = (int)(seg % o.seg.rtiles);
  o.pos.j = (int)(left % o.seg.span);
  return o;
}

// The units [b, e) of the segment at pos (whose info is g) that lie below list position u1, pos being at u.
__device__ __forceinline__ void split_units(const SegInfo& g, const AttnSplit& a, const UnitPos& pos, int64_t u, int64_t u1,
                                            int& b, int& e) {
  const int64_t n = u1 - u;
  const int end = n < g.span - pos.j ? pos.j + (int)n : g.span;
  b = pos.j > a.extra ? pos.j - a.extra : 0;
  e = end > a.extra ? end - a.extra : 0;
}
// The CTA whose range holds unit u.
__device__ __forceinline__ int split_owner(int64_t U, int G, int64_t u) { return (int)(((u + 1) * G - 1) / U); }

// The segment after (s, h, rt): its row tile, KV head or sequence advances;
// sequences without rows have none.  s = n_seqs when there is none left.
__device__ __forceinline__ void next_segment(const CacheDesc& c, const RowsDesc& r, const AttnSplit& a, UnitPos& p,
                                             SegInfo& g, uint32_t& bad) {
  p.j = 0;
  if (++p.rt < g.rtiles) return;
  p.rt = 0;
  if (++p.h < c.Hkv) return;
  p.h = 0;
  for (++p.s; p.s < c.n_seqs; ++p.s) {
    g = seg_info(c, r, a, p.s, bad);
    if (g.rtiles > 0) return;
  }
}

#endif  // __CUDACC__

}  // namespace bdlm
