// cache_ops.cu -- the 8-bit cache's memory-bound calls: append (quantise new
// tokens into their pages) and evict (keep the most attended tokens, in other
// pages).
#include <cuda_bf16.h>

#include "cache_ops.h"
#include "ptx.cuh"

namespace bdlm {
namespace {

__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Eight e4m3 codes of eight values times inv (pow2 scale) or divided by s.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float s, float inv, bool pow2) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = pow2 ? x[i] * inv : __fdiv_rn(x[i], s);
  return make_uint2(to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16,
                    to_e4m3x2(y[4], y[5]) | to_e4m3x2(y[6], y[7]) << 16);
}

__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float* f) {
  const uint32_t a = e4m3x2_to_half2(w), b = e4m3x2_to_half2(w >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}

// Largest of `v` over the `n` threads (a power of two, 8 .. 256) of an aligned
// group of the block; every thread of the block calls it.  What the group's
// threads read before it, they may write after it.
__device__ __forceinline__ uint32_t group_max(uint32_t v, int n, uint32_t* red) {
  const int lim = n < 32 ? n : 32;
  __syncwarp();
  for (int o = lim >> 1; o > 0; o >>= 1) v = umax2(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (n <= 32) return v;
  const int w = threadIdx.x >> 5, nw = n >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[w] = v;
  __syncthreads();
  const int w0 = w & ~(nw - 1);
  for (int i = 0; i < nw; ++i) v = umax2(v, red[w0 + i]);
  return v;
}

// ------------------------------------------------------------------ append
// A slab is one (sequence, touched page, KV head) of K or of V; page * HD / 64
// threads of a 256-thread block take it, 64 values each (eight 16-byte loads
// in flight), so the new tokens are read once and stay in registers between
// the block maximum and the codes.
constexpr int kAppendThreads = 256;
template <int HD>
__global__ void __launch_bounds__(kAppendThreads) bdlm_cache_append_kernel(const AppendParams p, int pages_per_seq) {
  __shared__ uint32_t red[kAppendThreads / 32];
  constexpr int CH = HD / 8;  // 8-value chunks of a token
  const CacheDesc& c = p.c;
  const int tps = c.page * HD / 64;  // threads per slab
  const int64_t slab = (int64_t)blockIdx.x * (kAppendThreads / tps) + threadIdx.x / tps;
  const int tl = threadIdx.x % tps;
  const int64_t n_slabs = (int64_t)c.n_seqs * pages_per_seq * c.Hkv * 2;
  uint32_t bad = 0;
  const bool in = slab < n_slabs;
  const int64_t id = in ? slab : 0;
  const int kv = (int)(id & 1);
  const int h = (int)((id >> 1) % c.Hkv);
  const int64_t sj = (id >> 1) / c.Hkv;
  const int j = (int)(sj % pages_per_seq), s = (int)(sj / pages_per_seq);
  const SeqView v = seq_view(c, p.r, s, bad);
  const int64_t cap = (int64_t)c.max_pages << c.lp;
  int rows = v.rows;
  if (v.len + (int64_t)rows > cap) {
    bad |= kStatusBadLen;
    rows = (int)(cap - v.len);
  }
  const int lpage = (v.len >> c.lp) + j;             // logical page
  const int first = (lpage << c.lp) - v.len;         // new-token index of its slot 0 (negative: old tokens before)
  const bool hit = in && rows > 0 && first < rows;
  const int pid = hit ? page_id(c, s, lpage, bad) : -1;
  if (in && tl == 0 && j == 0 && h == 0 && kv == 0 && p.lens_out) p.lens_out[s] = v.len + rows;
  const __nv_bfloat16* X = static_cast<const __nv_bfloat16*>(kv ? p.V : p.K);
  uint4 x[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = i * tps + tl, tok = first + ch / CH;
    const bool ok = pid >= 0 && tok >= 0 && tok < rows;
    x[i] = ok ? __ldg(reinterpret_cast<const uint4*>(X + ((v.row0 + tok) * c.Hkv + h) * HD) + ch % CH)
              : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) amax = umax2(amax, umax2(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
  }
  const int64_t b = (int64_t)max(pid, 0) * c.Hkv + h;
  float* sp = (kv ? c.vs : c.ks) + b;
  uint8_t* codes = (kv ? c.v8 : c.k8) + b * c.page * HD;
  float was = pid >= 0 && first < 0 ? *sp : 0.f;
  amax = group_max(amax << 16, tps, red);
  if (pid < 0) {
    if (bad && tl == 0) atomicOr(p.status, bad);
    return;
  }
  float sc = block_scale(amax);
  if (first < 0) {  // the block already holds tokens: its scale never shrinks (NaN stays)
    sc = (was != was || sc != sc) ? __uint_as_float(0x7fc00000u) : fmaxf(was, sc);
  }
  const bool pow2 = is_pow2(sc);
  const float inv = pow2 ? __uint_as_float(0x7f000000u - __float_as_uint(sc)) : 0.f;
  const bool regrade = first < 0 && sc != was;  // old codes to the new scale (true for NaN as well)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = i * tps + tl, tok = first + ch / CH;
    float f[8];
    if (tok >= 0 && tok < rows) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else if (tok < 0 && regrade) {
      const uint2 o = *(reinterpret_cast<const uint2*>(codes) + ch);
      e4m3x4_to_float(o.x, f);
      e4m3x4_to_float(o.y, f + 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= was;
    } else {
      continue;
    }
    *(reinterpret_cast<uint2*>(codes) + ch) = quantise8(f, sc, inv, pow2);
  }
  if (tl == 0) {
    *sp = sc;
    if (bad) atomicOr(p.status, bad);
  }
}

// ------------------------------------------------------------------- evict
// Selection, one block per (sequence, KV head).  A weight's rank key is an
// unsigned number of the same order (NaN the largest weight, -0 equal to 0);
// protected tokens take the largest key.  Four passes over 8-bit digits find
// the key of the last token kept and how many tokens of exactly that key
// are; those with the lowest positions are.
constexpr int kSelThreads = 1024;

__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 -> 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
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

__global__ void __launch_bounds__(kSelThreads) bdlm_evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int red[32];
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  const CacheDesc& c = p.c;
  const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  uint32_t bad = 0;
  const SeqView v = seq_view(c, RowsDesc{nullptr, 0, 0}, s, bad);
  const int64_t cap = (int64_t)c.max_pages << c.lp;
  const float* w = p.W + ((int64_t)s * c.Hkv + h) * cap;
  float* wo = p.W_out + ((int64_t)s * c.Hkv + h) * cap;
  int32_t* kept = p.kept + ((int64_t)s * c.Hkv + h) * p.keep;
  const int len = v.len, left = len < p.keep ? len : p.keep;
  auto key_of = [&](int i) { return i < p.sinks || i >= len - p.recent ? 0xffffffffu : rank_key(w[i]); };
  uint32_t thr = 0, mask = 0;
  int need = left;  // tokens still to take among those that match thr under mask
  if (left < len) {
    for (int sh = 24; sh >= 0; sh -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i = tid; i < len; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k & mask) == thr) atomicAdd(&hist[(k >> sh) & 255], 1);
      }
      __syncthreads();
      // digits from the top: the one where the count reaches need
      int n = tid < 256 ? hist[255 - tid] : 0, total;
      const int above = block_scan(n, red, &total);
      if (tid < 256 && above < need && above + n >= need) {
        s_digit = 255 - tid;
        s_need = need - above;
      }
      __syncthreads();
      thr |= s_digit << sh;
      mask |= 0xffu << sh;
      need = s_need;
    }
  }
  // kept tokens in order of position: a thread takes a run of positions
  const int per = (len + kSelThreads - 1) / kSelThreads;
  const int i0 = min(tid * per, len), i1 = min(i0 + per, len);
  int gt = 0, eq = 0;
  if (left < len)
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = key_of(i);
      gt += k > thr;
      eq += k == thr;
    }
  else
    gt = i1 - i0;
  int total;
  const int eq0 = block_scan(eq, red, &total);
  const int eq_take = min(max(need - eq0, 0), eq);
  int at = block_scan(gt + (left < len ? eq_take : 0), red, &total);
  int eq_left = eq_take;
  for (int i = i0; i < i1; ++i) {
    bool take = true;
    if (left < len) {
      const uint32_t k = key_of(i);
      take = k > thr || (k == thr && eq_left > 0);
      if (k == thr) --eq_left;
    }
    if (take) {
      kept[at] = i;
      wo[at] = w[i];
      ++at;
    }
  }
  for (int i = left + tid; i < p.keep; i += kSelThreads) kept[i] = -1;
  for (int64_t i = left + tid; i < cap; i += kSelThreads) wo[i] = 0.f;
  if (h == 0 && tid == 0) p.lens_out[s] = left;
  if (bad && tid == 0) atomicOr(p.status, bad);
}

// Moves one block of kept tokens: gathers their codes, finds the new scale,
// writes the codes in it.  The slab layout is append's.
template <int HD>
__global__ void __launch_bounds__(kAppendThreads) bdlm_evict_move_kernel(const EvictParams p, int pages_per_seq) {
  __shared__ uint32_t red[kAppendThreads / 32];
  constexpr int CH = HD / 8;
  const CacheDesc& c = p.c;
  const int tps = c.page * HD / 64;
  const int64_t slab = (int64_t)blockIdx.x * (kAppendThreads / tps) + threadIdx.x / tps;
  const int tl = threadIdx.x % tps;
  const int64_t n_slabs = (int64_t)c.n_seqs * pages_per_seq * c.Hkv * 2;
  uint32_t bad = 0;
  const bool in = slab < n_slabs;
  const int64_t id = in ? slab : 0;
  const int kv = (int)(id & 1);
  const int h = (int)((id >> 1) % c.Hkv);
  const int64_t sj = (id >> 1) / c.Hkv;
  const int j = (int)(sj % pages_per_seq), s = (int)(sj / pages_per_seq);
  const SeqView v = seq_view(c, RowsDesc{nullptr, 0, 0}, s, bad);
  const int left = v.len < p.keep ? v.len : p.keep;
  const int first = j << c.lp;
  int pid = -1;
  if (in && first < left) {
    pid = p.dst[(int64_t)s * c.max_pages + j];
    if (pid < 0 || pid >= c.n_pages) {
      bad |= kStatusBadPage;
      pid = -1;
    }
  }
  const int32_t* kept = p.kept + ((int64_t)s * c.Hkv + h) * p.keep;
  const uint8_t* from = kv ? c.v8 : c.k8;
  const float* scales = kv ? c.vs : c.ks;
  uint2 x[8];
  float sc[8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ch = i * tps + tl, slot = first + ch / CH;
    x[i] = make_uint2(0, 0);
    sc[i] = 0.f;
    if (pid >= 0 && slot < left) {
      const int pos = kept[slot];
      const int sp = page_id(c, s, pos >> c.lp, bad);
      if (sp >= 0) {
        const int64_t b = (int64_t)sp * c.Hkv + h;
        x[i] = __ldg(reinterpret_cast<const uint2*>(from + (b * c.page + (pos & (c.page - 1))) * HD) + ch % CH);
        sc[i] = __ldg(scales + b);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    e4m3x4_to_float(x[i].x, f);
    e4m3x4_to_float(x[i].y, f + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = umax2(amax, __float_as_uint(f[k] * sc[i]) & 0x7fffffffu);
  }
  amax = group_max(amax, tps, red);
  if (pid >= 0) {
    const float ns = block_scale(amax);
    const bool pow2 = is_pow2(ns);
    const float inv = pow2 ? __uint_as_float(0x7f000000u - __float_as_uint(ns)) : 0.f;
    const int64_t b = (int64_t)pid * c.Hkv + h;
    uint2* codes = reinterpret_cast<uint2*>((kv ? c.v8 : c.k8) + b * c.page * HD);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ch = i * tps + tl;
      if (first + ch / CH >= left) continue;
      float f[8];
      e4m3x4_to_float(x[i].x, f);
      e4m3x4_to_float(x[i].y, f + 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] *= sc[i];
      codes[ch] = quantise8(f, ns, inv, pow2);
    }
    if (tl == 0) (kv ? c.vs : c.ks)[b] = ns;
  }
  if (bad) atomicOr(p.status, bad);
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t st, int* launches) {
  const int per = (p.r.max_rows + p.c.page - 2) / p.c.page + 1;  // pages that max_rows new tokens can touch
  const int64_t slabs = (int64_t)p.c.n_seqs * per * p.c.Hkv * 2;
  const int in_block = kAppendThreads / (p.c.page * p.c.d / 64);
  const int64_t blocks = (slabs + in_block - 1) / in_block;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.c.d == 128) bdlm_cache_append_kernel<128><<<(unsigned)blocks, kAppendThreads, 0, st>>>(p, per);
  else bdlm_cache_append_kernel<64><<<(unsigned)blocks, kAppendThreads, 0, st>>>(p, per);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_cache_evict(const EvictParams& p, cudaStream_t st, int* launches) {
  bdlm_evict_select_kernel<<<dim3(p.c.Hkv, p.c.n_seqs), kSelThreads, 0, st>>>(p);
  ++*launches;
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t cap = (int64_t)p.c.max_pages << p.c.lp;
  const int64_t most = p.keep < cap ? p.keep : cap;
  const int per = (int)((most + p.c.page - 1) / p.c.page);
  const int64_t slabs = (int64_t)p.c.n_seqs * per * p.c.Hkv * 2;
  const int in_block = kAppendThreads / (p.c.page * p.c.d / 64);
  const int64_t blocks = (slabs + in_block - 1) / in_block;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (p.c.d == 128) bdlm_evict_move_kernel<128><<<(unsigned)blocks, kAppendThreads, 0, st>>>(p, per);
  else bdlm_evict_move_kernel<64><<<(unsigned)blocks, kAppendThreads, 0, st>>>(p, per);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace bdlm
