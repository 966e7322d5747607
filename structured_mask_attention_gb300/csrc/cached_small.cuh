// cached_small.cuh -- what the attention kernels of up to 32 rows over the 8-bit cache on
// mma.sync tiles share (cached_small.cu, tree_small.cu): the products, the ring of K and V
// tiles and the warp that fills it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cached_attn.h"
#include "kernels.h"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kWarps = 4;  // warps that compute; one more loads

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// What rounding to half (bf16) left of two values, rounded the same way.
__device__ __forceinline__ uint32_t rest_half2(uint32_t hi, float a, float b) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half2(a - h.x, b - h.y);
}
__device__ __forceinline__ uint32_t rest_bf16x2(uint32_t hi, float a, float b) {
  return pack_bf16x2(a - bf_lo(hi), b - bf_hi(hi));
}

// Two bf16 values, those that are not finite as 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) { return w & __vcmpltu2(w & 0x7fff7fffu, 0x7f807f80u); }

// Barrier of the computing warps.
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// MMA columns.  The contraction index of S = Q K^T may visit the head
// dimension in any order that both operands share, keys may take any order
// that S's columns and V's rows share, and the columns of O may stand for the
// head dimension in any order.  So a thread takes 16 consecutive bytes of a key
// (16 codes) and uses them, word by word, as the fragments of four k-steps
// (word i, bytes 0-1 and 2-3: the two halves of step 4 h + i of 64-byte half h):
// every load is 16 bytes wide and no operand is transposed.  For P V, thread
// (g, t) takes HD / 8 codes of the keys at contraction indices 2 t, 2 t + 1,
// 2 t + 8, 2 t + 9 and pairs the codes of two keys by byte permutes: column tile j
// of O is element j of every thread's piece.  In the 128-byte swizzle of the
// tiles (HD = 128) MMA column c is key perm(c) = c / 2 + 4 (c % 2) of its eight
// and thread g's piece of V is chunk perm(g): the eight lanes of a load phase
// then touch all 32 banks.  (HD = 64, 64-byte swizzle: perm is the identity.)

// Key of MMA column c among its eight, and chunk of V of thread group c.
template <int HD>
__device__ __forceinline__ constexpr int perm(int x) {
  return HD == 128 ? (x >> 1) | ((x & 1) << 2) : x;
}

struct alignas(8) SInfo {  // of each 16 keys of a tile: K's scale, log2 and 2^-shift times the inverse of V's (scale 1 without a page)
  float s[8], lv[8], iv[8];
  int gone;     // bit x: no page
};

constexpr int NI = 16;  // info slots: the tiles in the ring, and a batch of four ahead

// The ring of K and V tiles of 128 keys in shared memory.  LY: its layout (NS slots of K and
// of V, kTile, kK, kV; kInfo, kBar).
template <class LY>
struct Ring {
  uint32_t base;
  uint8_t* mem;
  __device__ __forceinline__ explicit Ring(uint8_t* raw) {
    const uint32_t at = smem_u32(raw);
    base = (at + 1023u) & ~1023u;
    mem = raw + (base - at);
  }
  __device__ __forceinline__ uint32_t KF(uint32_t i) const { return base + LY::kBar + 8 * i; }
  __device__ __forceinline__ uint32_t KE(uint32_t i) const { return base + LY::kBar + 8 * (LY::NS + i); }
  __device__ __forceinline__ uint32_t VF(uint32_t i) const { return base + LY::kBar + 8 * (2 * LY::NS + i); }
  __device__ __forceinline__ uint32_t VE(uint32_t i) const { return base + LY::kBar + 8 * (3 * LY::NS + i); }
  __device__ __forceinline__ SInfo* infos() const { return reinterpret_cast<SInfo*>(mem + LY::kInfo); }
  __device__ __forceinline__ volatile int* abort_flag() const {
    return reinterpret_cast<volatile int*>(mem + LY::kBar + 4 * LY::NS * 8);
  }
  __device__ __forceinline__ void init() const {  // by one thread
    for (uint32_t i = 0; i < LY::NS; ++i) {
      mbar_init(KF(i), 1);
      mbar_init(VF(i), 1);
      mbar_init(KE(i), kWarps);
      mbar_init(VE(i), kWarps);
    }
    *abort_flag() = 0;
    fence_mbar_init();
  }
};

// A CTA's units [u0, u1), and where the first lies; every warp walks them on its own.
struct Pieces {
  int64_t u0, u1;
  UnitPos pos;
  SegInfo seg;
};
__device__ __forceinline__ Pieces open_pieces(const CachedParams& p, int cta, uint32_t& bad) {
  Pieces w{0, 0, UnitPos{0, 0, 0, 0}, {}};
  const CacheDesc& c = p.c;
  if (p.whole) {  // CTA per segment: (sequence, KV head, row tile), p.whole row tiles for each
    w.pos.rt = cta % p.whole;
    w.pos.h = cta / p.whole % c.Hkv;
    w.pos.s = cta / p.whole / c.Hkv;
    w.seg = seg_info(c, p.r, p.sp, w.pos.s, bad);
    w.u1 = w.pos.rt < w.seg.rtiles ? w.seg.span : 0;
  } else {
    const SplitOpen o = split_open(c, p.r, p.sp, p.G, cta, bad);
    w.u0 = o.u0;
    w.u1 = o.u1;
    w.pos = o.pos;
    w.seg = o.seg;
  }
  return w;
}

// The loading warp: fills the ring with the pieces' tiles.
template <int HD, class LY>
__device__ __forceinline__ void load_ring(const Ring<LY>& r, const CUtensorMap& tK8, const CUtensorMap& tV8,
                                          const CachedParams& p, Pieces& w, const Watchdog& wd, uint32_t bad) {
  const CacheDesc& c = p.c;
  const int lane = threadIdx.x & 31;
  const int64_t u1 = w.u1;
  UnitPos& pos = w.pos;
  SegInfo& seg = w.seg;
  uint32_t slot = 0, ph = 1, tc = 0;
  const uint32_t page_bytes = (uint32_t)(c.page * HD), page_groups = first_groups(c.page);
  bool ok = true;
  for (int64_t u = w.u0; ok && u < u1;) {
    int jb, je;
    split_units(seg, p.sp, pos, u, u1, jb, je);
    u += seg.span - pos.j;
    if (je == 0) break;
    const int len = seg.v.len, n = min(je, seg.ktiles) - jb, h = pos.h;
    const int32_t* table = c.table + (int64_t)pos.s * c.max_pages;
    // lane 8 a + x: page and scales of keys 16 x of tile a of a batch of 4 tiles, one batch ahead
    auto lookup = [&](int b) {
      const int tile = 4 * b + (lane >> 3), key = (jb + tile) * kUnit + 16 * (lane & 7);
      return tile < n && key < len ? __ldg(table + (key >> c.lp)) : -1;
    };
    // (a batch's entries are looked at a batch after they were asked for)
    auto checked = [&](int id, int b) {
      if (id >= 0 && id < c.n_pages) return id;
      const int tile = 4 * b + (lane >> 3), key = (jb + tile) * kUnit + 16 * (lane & 7);
      if (tile < n && key < len) bad |= kStatusBadPage;
      return -1;
    };
    auto scale_of = [&](const float* sc, int id) { return id >= 0 ? __ldg(sc + (int64_t)id * c.Hkv + h) : 1.f; };
    const int raw0 = lookup(0);
    int raw1 = lookup(1);
    int id = checked(raw0, 0);
    float sk = scale_of(c.ks, id), sv = scale_of(c.vs, id);
    for (int b = 0; ok && 4 * b < n; ++b) {
      const int id1 = checked(raw1, b + 1);
      const float sk1 = scale_of(c.ks, id1), sv1 = scale_of(c.vs, id1);
      const int raw2 = lookup(b + 2);
      // the batch's tiles, a group of eight lanes each
      const int grp = lane >> 3, x = lane & 7;
      const unsigned none = __ballot_sync(0xffffffffu, id < 0);
      SInfo& si = r.infos()[(tc + grp) % NI];
      if (4 * b + grp < n) {
        si.s[x] = sk;
        si.lv[x] = log2f(sv);
        si.iv[x] = kSmallUnshift / sv;
        if (x == 0) si.gone = (int)((none >> lane) & 0xffu);
      }
      __syncwarp();  // (before the arrivals that tell of them)
      const uint32_t bytes = (uint32_t)__popc(~(none >> (lane & 24)) & page_groups) * page_bytes;
      const bool loads = id >= 0 && ((page_groups >> x) & 1);
      const int blk = (int)((int64_t)id * c.Hkv + h);
      for (int a = 0; a < 4 && 4 * b + a < n; ++a, ++tc) {
        ok = mbar_wait(r.KE(slot), ph, wd, 70);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 8 * a) {
          if (bytes) mbar_arrive_expect_tx(r.KF(slot), bytes);
          else mbar_arrive(r.KF(slot));
        }
        __syncwarp();
        const bool mine = grp == a && loads;  // the lane of a page's first keys loads it
        if (mine) tma_load_3d(r.base + LY::kK + slot * LY::kTile + 16 * x * HD, &tK8, r.KF(slot), 0, 0, blk);
        ok = mbar_wait(r.VE(slot), ph, wd, 71);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 8 * a) {
          if (bytes) mbar_arrive_expect_tx(r.VF(slot), bytes);
          else mbar_arrive(r.VF(slot));
        }
        __syncwarp();
        if (mine) tma_load_3d(r.base + LY::kV + slot * LY::kTile + 16 * x * HD, &tV8, r.VF(slot), 0, 0, blk);
        if (++slot == LY::NS) slot = 0, ph ^= 1;
      }
      id = id1; raw1 = raw2; sk = sk1; sv = sv1;
    }
    if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
  }
  if (bad) atomicOr(p.status + kContentsWord, bad);
  // (copies that a timeout left in flight land before the CTA's shared memory is given up)
  if (*r.abort_flag()) drain_after_abort(200);
}

}  // namespace
}  // namespace bdlm
