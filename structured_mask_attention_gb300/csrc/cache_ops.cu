// cache_ops.cu -- the 8-bit cache's memory-bound calls: append (quantise new
// tokens into their pages) and evict (keep the most attended tokens, in other
// pages).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "cache_ops.h"
#include "kernels.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace bdlm {
namespace {

__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Eight e4m3 codes of eight values times inv (pow2 scale) or divided by s.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float s, float inv, bool pow2) {
  float y[8];
  if (pow2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], s);
  }
  return make_uint2(to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16,
                    to_e4m3x2(y[4], y[5]) | to_e4m3x2(y[6], y[7]) << 16);
}

__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float* f) {
  const uint32_t a = e4m3x2_to_half2(w), b = e4m3x2_to_half2(w >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}

// Four codes times r, rounded to codes again (r: a power of two, nothing above 448 comes out).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, __half2 r) {
  uint32_t q[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const uint32_t h = e4m3x2_to_half2(w >> (16 * y));
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&h), r);
    q[y] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
  }
  return q[0] | q[1] << 16;
}

// ------------------------------------------------------------------ append
// A CTA takes TT = max(page, 64) slots of one (sequence, KV head), K and V: 16
// values per thread and step (two 16-byte loads, HD / 16 lanes to a token),
// all in flight at once and held between the blocks' maxima and their codes,
// so the new tokens are read once.  Bound by HBM: 2 bytes read and 1 written per
// value: 131072 tokens of 8 heads of 128 (0.81 GB) take 147 us, 5.5 TB/s or 81 % of
// the measured copy rate; 16 sequences' blocks of 512 (43 MB) 14.3 us, half of it
// before the first bytes arrive; 64 single tokens 7 us, a launch.  (A CTA per
// block, one chunk per thread at a time: 203 us for the first.)
constexpr int kAppendThreads = 256;
template <int HD, int TT>
__global__ void __launch_bounds__(kAppendThreads* TT / 64) bdlm_cache_append_kernel(const AppendParams p) {
  constexpr int CH = HD / 16;                     // 16-value chunks of a token
  constexpr int kThreads = kAppendThreads * TT / 64;
  constexpr int NT = 2 * TT * CH / kThreads;      // chunks per thread, the first half K's
  __shared__ uint32_t s_amax[2][TT / 16];
  __shared__ float s_was[2][TT / 16];             // the blocks' scales before
  __shared__ int s_page[TT / 16];
  const CacheDesc& c = p.c;
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  uint32_t bad = 0;
  const SeqView v = seq_view(c, p.r, s, bad);
  const int64_t cap = (int64_t)c.max_pages << c.lp;
  int rows = v.rows;
  if (v.len + (int64_t)rows > cap) {
    bad |= kStatusBadLen;
    rows = (int)(cap - v.len);
  }
  const int base = (v.len & ~(TT - 1)) + (int)blockIdx.x * TT;  // first position
  const int first = base - v.len;                               // as a new token (negative: old tokens)
  if (blockIdx.x == 0 && h == 0 && tid == 0) {
    if (p.lens_out) p.lens_out[s] = v.len + rows;
    if (bad) atomicOr(p.status + kContentsWord, bad);
    bad = 0;
  }
  if (rows <= 0 || first >= rows) return;  // (without new rows a half-filled page, maybe another sequence's too, stays as it is)
  if (tid < TT / 16) {
    const int f = first + (tid << c.lp);  // new token of the block's first slot
    int id = -1;
    if (tid < (TT >> c.lp) && f < rows && f + c.page > 0) id = page_id(c, s, (base >> c.lp) + tid, bad);
    s_page[tid] = id;
    const int64_t b = (int64_t)max(id, 0) * c.Hkv + h;
    s_was[0][tid] = id >= 0 && f < 0 ? c.ks[b] : 0.f;
    s_was[1][tid] = id >= 0 && f < 0 ? c.vs[b] : 0.f;
    s_amax[0][tid] = s_amax[1][tid] = 0;
    if (bad) atomicOr(p.status + kContentsWord, bad);
  }
  uint4 x[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int kv = i >= NT / 2, k = (i % (NT / 2)) * kThreads + tid, tok = first + k / CH;
    const bool ok = tok >= 0 && tok < rows;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(kv ? p.V : p.K) +
                                                      ((v.row0 + (ok ? tok : 0)) * c.Hkv + h) * HD) + 2 * (k % CH);
    x[i][0] = ok ? __ldg(src) : make_uint4(0, 0, 0, 0);
    x[i][1] = ok ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int kv = i >= NT / 2, t = ((i % (NT / 2)) * kThreads + tid) / CH;
    // bf16 magnitudes compare like integers
    uint32_t m = 0;
#pragma unroll
    for (int y = 0; y < 2; ++y)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i][y].x & 0x7fff7fffu, x[i][y].y & 0x7fff7fffu),
                               __vmaxu2(x[i][y].z & 0x7fff7fffu, x[i][y].w & 0x7fff7fffu)));
    m = umax2(m & 0xffffu, m >> 16);
    // a warp's tokens belong to one block
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) atomicMax(&s_amax[kv][t >> c.lp], m << 16);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int kv = i >= NT / 2, k = (i % (NT / 2)) * kThreads + tid, t = k / CH, j = t >> c.lp, tok = first + t;
    const int id = s_page[j];
    if (id < 0 || tok >= rows) continue;
    float sc = block_scale(s_amax[kv][j]);
    const bool had = first + (j << c.lp) < 0;  // the block already holds tokens: its scale never shrinks, NaN stays
    const float was = s_was[kv][j];
    if (had) sc = (was != was || sc != sc) ? __uint_as_float(0x7fc00000u) : fmaxf(was, sc);
    const int64_t b = (int64_t)id * c.Hkv + h;
    uint4* code = reinterpret_cast<uint4*>((kv ? c.v8 : c.k8) + (b * c.page + (t & (c.page - 1))) * HD) + k % CH;
    if (k % CH == 0 && (t & (c.page - 1)) == (had ? v.len & (c.page - 1) : 0)) (kv ? c.vs : c.ks)[b] = sc;
    const bool pow2 = is_pow2(sc);
    const float inv = pow2 ? __uint_as_float(0x7f000000u - __float_as_uint(sc)) : 0.f;
    if (tok >= 0) {
      uint2 o[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t w[4] = {x[i][y].x, x[i][y].y, x[i][y].z, x[i][y].w};
        float f[8];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          f[2 * z] = __uint_as_float(w[z] << 16);
          f[2 * z + 1] = __uint_as_float(w[z] & 0xffff0000u);
        }
        o[y] = quantise8(f, sc, inv, pow2);
      }
      *code = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y);
    } else if (sc != was) {  // old codes to the new scale (true for NaN as well)
      const uint4 u = *code;
      float f[16];
      e4m3x4_to_float(u.x, f);
      e4m3x4_to_float(u.y, f + 4);
      e4m3x4_to_float(u.z, f + 8);
      e4m3x4_to_float(u.w, f + 12);
#pragma unroll
      for (int y = 0; y < 16; ++y) f[y] *= was;
      const uint2 lo = quantise8(*reinterpret_cast<const float(*)[8]>(f), sc, inv, pow2);
      const uint2 hi = quantise8(*reinterpret_cast<const float(*)[8]>(f + 8), sc, inv, pow2);
      *code = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

// ------------------------------------------------------------------- evict
// Selection, one cluster of CTAs per (sequence, KV head), each CTA a run of
// positions whose rank keys it holds in shared memory, so that the weights are
// read once.  A weight's rank key is an unsigned number of the same order (NaN
// the largest weight, -0 equal to 0); protected tokens take the largest key.
// Three passes over 11-, 11- and 10-bit digits find the key of the last token
// kept (every CTA adds up the cluster's histograms through distributed shared
// memory) and how many tokens of exactly that key are; those with the lowest
// positions are.  A prefix sum over threads and CTAs then places the kept
// tokens in order.  Bound by latency, not by the weights' bytes: of 16 us (8192
// weights of each of 128 heads, one CTA each) or 27 us (131072 of 8, eight CTAs
// each), 2 go by until the weights are there, 7 to 14 in the passes (counting,
// a cluster barrier, the counts of all CTAs, a scan) and the rest in placing
// the tokens.
constexpr int kSelThreads = 1024;
constexpr int kSelHeld = 44 * 1024;  // keys that a CTA holds; longer runs read the weights again
constexpr int kSelBins = 2048, kSelCopies = 5, kSelHist = kSelCopies * kSelBins;
constexpr int kSelRun = 16 * 1024;   // positions per CTA, while a cluster can grow

__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 -> 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The weight of a rank key (of a token that is neither protected nor NaN).
__device__ __forceinline__ float rank_weight(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Exclusive prefix sum over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int x, int* red, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) red[w] = v;
  __syncthreads();
  if (w == 0) {
    int z = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    red[lane] = z;
  }
  __syncthreads();
  *total = red[31];
  return v - x + (w ? red[w - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads, 1) bdlm_evict_select_kernel(const EvictParams p, int held) {
  extern __shared__ __align__(16) uint32_t sel_smem[];
  uint32_t* hist = sel_smem;                     // [kSelCopies][kSelBins]
  uint32_t* keys = sel_smem + kSelHist;          // [held]
  __shared__ int red[32];
  __shared__ uint32_t s_digit;
  __shared__ int s_need, s_count[2];
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const CacheDesc& c = p.c;
  const int s = blockIdx.y, h = blockIdx.x / C, tid = threadIdx.x;
  uint32_t bad = 0;
  launch_dependents();
  const SeqView v = seq_view(c, RowsDesc{nullptr, 0, 0}, s, bad);
  const int64_t cap = (int64_t)c.max_pages << c.lp;
  const float* w = p.W + ((int64_t)s * c.Hkv + h) * cap;
  float* wo = p.W_out + ((int64_t)s * c.Hkv + h) * cap;
  int32_t* kept = p.kept + ((int64_t)s * c.Hkv + h) * p.keep;
  const int len = v.len, left = len < p.keep ? len : p.keep;
  // this CTA's positions (runs of fours: the row of weights has a multiple of 16)
  const int run = ((len + C - 1) / C + 3) & ~3, b0 = min(rank * run, len), n = min(run, len - b0);
  const int top_sink = p.sinks - b0, first_recent = len - p.recent - b0;  // (as places in the run)
  auto weigh4 = [&](int i, float4 x) {  // keys of the run's places i .. i + 3
    uint4 k = make_uint4(rank_key(x.x), rank_key(x.y), rank_key(x.z), rank_key(x.w));
    if (i < top_sink || i + 3 >= first_recent) {
      if (i < top_sink || i >= first_recent) k.x = 0xffffffffu;
      if (i + 1 < top_sink || i + 1 >= first_recent) k.y = 0xffffffffu;
      if (i + 2 < top_sink || i + 2 >= first_recent) k.z = 0xffffffffu;
      if (i + 3 < top_sink || i + 3 >= first_recent) k.w = 0xffffffffu;
    }
    return k;
  };
  auto load4 = [&](int i) { return i < n ? *reinterpret_cast<const float4*>(w + b0 + i) : make_float4(0.f, 0.f, 0.f, 0.f); };
  constexpr int kRound = 4 * kSelThreads;
  const int here = min(n, held);
  for (int i = 4 * tid; i < here; i += 4 * kRound) {  // (four loads in flight)
    float4 x[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) x[y] = load4(i + y * kRound);
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (i + y * kRound < here) *reinterpret_cast<uint4*>(keys + i + y * kRound) = weigh4(i + y * kRound, x[y]);
  }
  auto keys_of = [&](int i) { return i < held ? *reinterpret_cast<const uint4*>(keys + i) : weigh4(i, load4(i)); };
  for (int i = tid; i < kSelHist; i += kSelThreads) hist[i] = 0;
  __syncthreads();
  uint32_t thr = 0, mask = 0;
  int need = left;  // tokens still to take among those that match thr under mask
  const bool cut = left < len;
  if (cut) {
    for (int pass = 0; pass < 3; ++pass) {
      const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, bins = 1 << bits;
      // the first pass counts every key, most of them in a few digits: its
      // warps share out kSelCopies - 1 histograms (the last copy is pass 1's)
      uint32_t* mine = hist + (pass == 1 ? kSelCopies - 1 : 0) * kSelBins;
      uint32_t* count = pass == 0 ? hist + ((tid >> 5) % (kSelCopies - 1)) * kSelBins : mine;
      for (int i = 4 * tid; i < n; i += kRound) {
        const uint4 k4 = keys_of(i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if ((k[y] & mask) == thr && i + y < n) atomicAdd(&count[(k[y] >> sh) & (bins - 1)], 1u);
      }
      if (pass == 0) {
        __syncthreads();
        for (int i = tid; i < kSelBins; i += kSelThreads)
          for (int y = 1; y < kSelCopies - 1; ++y) mine[i] += hist[y * kSelBins + i];
      }
      cl.sync();
      // two bins per thread, digits from the top: the one where the count reaches need
      // (all CTAs' counts asked for together, each CTA beginning with its own)
      const int top = bins - 1 - 2 * tid;
      int n0 = 0, n1 = 0;
      if (top > 0) {
        uint2 x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          x[r] = r < C ? *reinterpret_cast<const uint2*>(cl.map_shared_rank(mine, (rank + r) & (C - 1)) + top - 1)
                       : make_uint2(0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          n0 += (int)x[r].y;
          n1 += (int)x[r].x;
        }
      }
      int total;
      const int above = block_scan(n0 + n1, red, &total);
      if (above < need && above + n0 >= need) {
        s_digit = (uint32_t)top;
        s_need = need - above;
      } else if (above + n0 < need && above + n0 + n1 >= need) {
        s_digit = (uint32_t)top - 1;
        s_need = need - above - n0;
      }
      if (pass == 1) {  // every CTA of the cluster has read the first pass's counts
        for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
      }
      __syncthreads();
      thr |= s_digit << sh;
      mask |= (uint32_t)(bins - 1) << sh;
      need = s_need;
      __syncthreads();
    }
  }
  // kept tokens in order of position: a warp takes a run of positions, 4 per
  // lane at a time; a token's new slot is the number of larger keys before it
  // plus that of equal ones, of which the first `need` are kept
  const int lane = tid & 31, warp = tid >> 5;
  const int per = ((n + kRound - 1) / kRound) * 128;
  const int i0 = min(warp * per, n), i1 = min(i0 + per, n);
  auto sort4 = [&](int i, const uint4& k4, uint32_t& gt, uint32_t& eq) {  // a bit for each of 4 keys
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    gt = eq = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (i + y < i1 && (!cut || k[y] > thr)) gt |= 1u << y;
      if (i + y < i1 && cut && k[y] == thr) eq |= 1u << y;
    }
  };
  int gts = 0, eqs = 0;
  for (int i = i0 + 4 * lane; i < i1; i += 128) {
    uint32_t gt, eq;
    sort4(i, keys_of(i), gt, eq);
    gts += __popc(gt);
    eqs += __popc(eq);
  }
  gts = __reduce_add_sync(0xffffffffu, gts);
  eqs = __reduce_add_sync(0xffffffffu, eqs);
  int gt_all, eq_all;
  int eq0 = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? eqs : 0, red, &eq_all), 0);
  int gt0 = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? gts : 0, red, &gt_all), 0);
  if (tid == 0) {
    s_count[0] = gt_all;
    s_count[1] = eq_all;
  }
  cl.sync();
  for (int r = 0; r < rank; ++r) {
    const int* o = cl.map_shared_rank(s_count, r);
    gt0 += o[0];
    eq0 += o[1];
  }
  cl.barrier_arrive();  // (done with the other CTAs' memory)
  for (int ib = i0; ib < i1; ib += 128) {
    const int i = ib + 4 * lane;
    uint32_t gt = 0, eq = 0;
    uint4 k4 = make_uint4(0, 0, 0, 0);
    if (i < i1) {
      k4 = keys_of(i);
      sort4(i, k4, gt, eq);
    }
    const uint32_t mine = (uint32_t)__popc(gt) | (uint32_t)__popc(eq) << 16;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += z;
    }
    const uint32_t before = sum - mine, all = __shfl_sync(0xffffffffu, sum, 31);
    int g = gt0 + (int)(before & 0xffffu), e = eq0 + (int)(before >> 16);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const bool is_eq = (eq >> y) & 1, take = ((gt >> y) & 1) || (is_eq && e < need);
      if (take) {
        const int o = g + min(e, need);
        kept[o] = b0 + i + y;
        wo[o] = k[y] >= 0xfffffffeu ? w[b0 + i + y] : rank_weight(k[y]);
      }
      g += (gt >> y) & 1;
      e += is_eq;
    }
    gt0 += (int)(all & 0xffffu);
    eq0 += (int)(all >> 16);
  }
  const int step = C * kSelThreads;
  for (int i = left + rank * kSelThreads + tid; i < p.keep; i += step) kept[i] = -1;
  for (int64_t i = left + rank * kSelThreads + tid; i < cap; i += step) wo[i] = 0.f;
  if (h == 0 && rank == 0 && tid == 0) p.lens_out[s] = left;
  if (bad && tid == 0) atomicOr(p.status + kContentsWord, bad);
  cl.barrier_wait();  // no CTA leaves while another may still read its counts
}

// Moves the kept tokens of TT = max(page, 64) destination slots, K and V: one
// thread per token finds its old row and scales, then the CTA gathers all rows
// with 16-byte loads (HD / 16 lanes to a row), finds each destination block's
// scale and writes the codes, unchanged where the block's scale is the row's
// (e4m3 magnitudes compare like integers, so the maximum needs no conversion).
// It starts under the selection.  Bound by the chain position -> page -> scale
// and row that each CTA follows, at about 60 % of the issue slots: 30 us for 67 MB
// read and as many written (2048 tokens of 128 heads, or 32768 of 8), 4.5 TB/s.
constexpr int kMoveThreads = 256;
template <int HD, int TT>
__global__ void __launch_bounds__(kMoveThreads, TT == 128 ? 5 : 1) bdlm_evict_move_kernel(const EvictParams p) {
  constexpr int CH = HD / 16;                            // 16-byte chunks of a row
  constexpr int NT = 2 * TT * CH / kMoveThreads;         // chunks per thread, the first half K's
  __shared__ int64_t s_row[TT];                          // old row ((page, head) block * page + slot), -1: none
  __shared__ float s_scale[2][TT];
  __shared__ uint32_t s_amax[2][TT / 16];
  __shared__ int s_dst[TT / 16];
  const CacheDesc& c = p.c;
  const int s = blockIdx.z, h = blockIdx.y, t0 = (int)blockIdx.x * TT, tid = threadIdx.x;
  uint32_t bad = 0;
  const SeqView v = seq_view(c, RowsDesc{nullptr, 0, 0}, s, bad);
  const int left = v.len < p.keep ? v.len : p.keep;
  // (the selection may still run; every thread waits for it, so that this grid's end implies its end)
  dependency_wait();
  if (t0 >= left) return;
  float a = 0.f, b = 0.f;
  if (tid < TT) {
    const int slot = t0 + tid;
    int64_t row = -1;
    if (slot < left) {
      const int pos = p.kept[((int64_t)s * c.Hkv + h) * p.keep + slot];
      const int sp = page_id(c, s, pos >> c.lp, bad);
      if (sp >= 0) {
        const int64_t blk = (int64_t)sp * c.Hkv + h;
        row = blk * c.page + (pos & (c.page - 1));
        a = c.ks[blk];
        b = c.vs[blk];
      }
    }
    s_row[tid] = row;
  } else if (tid - TT < TT / 16) {
    const int j = tid - TT, slot = t0 + (j << c.lp);  // destination page j of this CTA
    int id = -1;
    if (j < (TT >> c.lp) && slot < left) {
      id = p.dst[(int64_t)s * c.max_pages + (slot >> c.lp)];
      if (id < 0 || id >= c.n_pages) {
        bad |= kStatusBadPage;
        id = -1;
      }
    }
    s_dst[j] = id;
    s_amax[0][j] = s_amax[1][j] = 0;
  }
  __syncthreads();
  uint4 x[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int kv = i >= NT / 2, k = (i % (NT / 2)) * kMoveThreads + tid;
    const int64_t row = s_row[k / CH];
    x[i] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>((kv ? c.v8 : c.k8) + row * HD) + k % CH)
                    : make_uint4(0, 0, 0, 0);
  }
  if (tid < TT) {  // (the scales arrive while the rows do)
    s_scale[0][tid] = a;
    s_scale[1][tid] = b;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int kv = i >= NT / 2, tok = ((i % (NT / 2)) * kMoveThreads + tid) / CH;
    // the largest of 16 magnitudes, two bytes at a time: of a 16-bit maximum the
    // high byte is the high bytes' maximum
    uint32_t hb = 0, lb = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint32_t w = (y == 0 ? x[i].x : y == 1 ? x[i].y : y == 2 ? x[i].z : x[i].w) & 0x7f7f7f7fu;
      hb = __vmaxu2(hb, w);
      lb = __vmaxu2(lb, w << 8);
    }
    const uint32_t m2 = __vmaxu2(hb, lb), top = umax2(m2 >> 24, (m2 >> 8) & 0xffu);
    const uint32_t hv = e4m3x2_to_half2(top);
    const float val = __half22float2(*reinterpret_cast<const __half2*>(&hv)).x * s_scale[kv][tok];
    uint32_t bits = s_row[tok] >= 0 ? __float_as_uint(val) & 0x7fffffffu : 0u;
    // a warp's rows belong to one destination page
    bits = __reduce_max_sync(0xffffffffu, bits);
    if ((tid & 31) == 0) atomicMax(&s_amax[kv][tok >> c.lp], bits);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int kv = i >= NT / 2, k = (i % (NT / 2)) * kMoveThreads + tid, tok = k / CH, j = tok >> c.lp;
    const int id = s_dst[j];
    if (t0 + tok >= left || id < 0) continue;
    const float ns = block_scale(s_amax[kv][j]), sc = s_scale[kv][tok];
    uint4 o = x[i];
    if (sc != ns) {
      const uint32_t ratio = __float_as_uint(sc) - __float_as_uint(ns) + 0x3f800000u;  // of two powers of two
      if (is_pow2(sc) && is_pow2(ns) && (int)ratio <= 0x47000000) {
        // times 2^j, j <= 15, in halves: exact from 2^-14 on, and what is smaller rounds to the code 0 either way
        const __half2 r = __float2half2_rn((int)ratio > 0x33000000 ? __uint_as_float(ratio) : 0.f);
        o = make_uint4(rescale4(x[i].x, r), rescale4(x[i].y, r), rescale4(x[i].z, r), rescale4(x[i].w, r));
      } else {
        const bool pow2 = is_pow2(ns);
        const float inv = pow2 ? __uint_as_float(0x7f000000u - __float_as_uint(ns)) : 0.f;
        uint2 q[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float f[8];
          e4m3x4_to_float(z ? x[i].z : x[i].x, f);
          e4m3x4_to_float(z ? x[i].w : x[i].y, f + 4);
#pragma unroll
          for (int y = 0; y < 8; ++y) f[y] *= sc;
          q[z] = quantise8(f, ns, inv, pow2);
        }
        o = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
      }
    }
    const int64_t blk = (int64_t)id * c.Hkv + h;
    *(reinterpret_cast<uint4*>((kv ? c.v8 : c.k8) + (blk * c.page + (tok & (c.page - 1))) * HD) + k % CH) = o;
    if (k % CH == 0 && (tok & (c.page - 1)) == 0) (kv ? c.vs : c.ks)[blk] = ns;
  }
  if (bad) atomicOr(p.status + kContentsWord, bad);
}

}  // namespace

cudaError_t raise_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t st, int* launches) {
  const int TT = p.c.page > 64 ? 128 : 64;
  // groups of TT slots that max_rows new tokens can touch
  const dim3 grid((unsigned)((p.r.max_rows + TT - 2) / TT + 1), (unsigned)p.c.Hkv, (unsigned)p.c.n_seqs);
  auto k = p.c.d == 128 ? (TT == 128 ? bdlm_cache_append_kernel<128, 128> : bdlm_cache_append_kernel<128, 64>)
                        : (TT == 128 ? bdlm_cache_append_kernel<64, 128> : bdlm_cache_append_kernel<64, 64>);
  k<<<grid, kAppendThreads * TT / 64, 0, st>>>(p);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t st, int* launches) {
  const int64_t cap = (int64_t)p.c.max_pages << p.c.lp;
  // a CTA for each kSelRun positions of the longest sequence, up to the portable
  // cluster size; more, down to kSelRun / 8 positions, while the GPU has room.  One
  // CTA against eight, 8 KV heads, the move included: 1 sequence of 131072 tokens
  // 143 / 53 us, of 16384 23 / 21, 2 of 40000 49 / 47; 16 of 8192 43 / 166
  int C = 1;
  while (C < 8 && (int64_t)C * kSelRun < cap) C *= 2;
  while (C < 8 && (int64_t)C * kSelRun / 8 < cap && (int64_t)p.c.n_seqs * p.c.Hkv * C * 2 <= 152) C *= 2;
  const int64_t run = ((cap + C - 1) / C + 3) & ~(int64_t)3;
  const int held = (int)(run < kSelHeld ? run : kSelHeld);
  const int bytes = (kSelHist + held) * (int)sizeof(uint32_t);
  static std::atomic<uint64_t> raised{0};
  cudaError_t e = raise_smem(reinterpret_cast<const void*>(bdlm_evict_select_kernel),
                             (kSelHist + kSelHeld) * (int)sizeof(uint32_t), raised);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.Hkv * C), (unsigned)p.c.n_seqs);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, bdlm_evict_select_kernel, p, held);
  if (e != cudaSuccess) return e;
  ++*launches;
  const int64_t most = p.keep < cap ? p.keep : cap;
  const int TT = p.c.page > 64 ? 128 : 64;
  const dim3 grid((unsigned)((most + TT - 1) / TT), (unsigned)p.c.Hkv, (unsigned)p.c.n_seqs);
  auto move = p.c.d == 128 ? (TT == 128 ? bdlm_evict_move_kernel<128, 128> : bdlm_evict_move_kernel<128, 64>)
                           : (TT == 128 ? bdlm_evict_move_kernel<64, 128> : bdlm_evict_move_kernel<64, 64>);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // may start before the selection's end
  at[0].val.programmaticStreamSerializationAllowed = 1;
  e = cudaLaunchKernelEx(&cfg, move, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
