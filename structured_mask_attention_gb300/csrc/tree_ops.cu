// tree_ops.cu -- drafted trees beside the attention over the 8-bit cache: what each row
// of a tree sees, and which drafted tokens the target's probabilities accept.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "kernels.h"
#include "tree_ops.h"

namespace cg = cooperative_groups;

namespace bdlm {
namespace {

// ------------------------------------------------------------------ mask
// A CTA per sequence.  A warp closes 32 consecutive rows over their parents inside
// the group by doubling (5 steps of shuffles): the rows of the group above a row, as
// bits, how many they are, and the first ancestor below the group (a parent comes
// before its child, so ancestors lie in this group or in earlier ones).  A row then
// collects one word from each group that its ancestors touch.  Bound by latency.
constexpr int kMaskThreads = 256;

__global__ void __launch_bounds__(kMaskThreads) bdlm_tree_mask_kernel(const TreeMaskParams p) {
  extern __shared__ int mask_smem[];
  uint32_t* in = reinterpret_cast<uint32_t*>(mask_smem);  // [max_rows] ancestors inside the row's group, and itself
  int* top = mask_smem + p.r.max_rows;                    // the first ancestor in an earlier group, -1: none
  int* num = top + p.r.max_rows;                          // bits of `in`
  const int s = blockIdx.x, lane = threadIdx.x & 31;
  uint32_t bad = 0;
  const SeqView v = seq_view(p.c, p.r, s, bad);
  for (int g0 = (threadIdx.x >> 5) * 32; g0 < v.rows; g0 += kMaskThreads) {
    const int i = g0 + lane;
    int par = i < v.rows ? __ldg(p.parents + v.row0 + i) : -1;
    if (par < -1 || par >= i) {  // (such a row counts as one without a parent)
      bad |= kStatusBadTree;
      par = -1;
    }
    uint32_t m = 1u << lane;
    int q = par >= g0 ? par - g0 : -1, t = par >= g0 ? -1 : par, n = 1;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int from = q < 0 ? lane : q;
      const uint32_t qm = __shfl_sync(0xffffffffu, m, from);
      const int qq = __shfl_sync(0xffffffffu, q, from), qt = __shfl_sync(0xffffffffu, t, from);
      const int qn = __shfl_sync(0xffffffffu, n, from);
      if (q >= 0) {
        m |= qm;
        n += qn;
        t = qt;
        q = qq;
      }
    }
    if (i < v.rows) {
      in[i] = m;
      top[i] = t;
      num[i] = n;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < v.rows; i += kMaskThreads) {
    uint32_t* out = p.vis + (v.row0 + i) * p.words;
    int depth = 0, at = i;
    for (int w = p.words - 1; w >= 0; --w) {  // (ancestors come in falling order)
      uint32_t x = 0;
      if (at >= 0 && (at >> 5) == w) {
        x = in[at];
        depth += num[at];
        at = top[at];
      }
      out[w] = x;
    }
    p.positions[v.row0 + i] = v.len + depth - 1;
  }
  if (bad) atomicOr(p.status + kContentsWord, bad);
}

// ---------------------------------------------------------------- verify
// A cluster of CTAs per sequence.  Warp 0 of every CTA walks the tree from row 0
// (all CTAs the same way, from the same numbers, so that nothing but sums has to be
// exchanged): the children of the current row in row order, against
//   r_k = max(p - c_k q, 0), of total Z_k, after k rejected ones.
// (Rejecting a child replaces r / Z by max(r / Z - q, 0) over its total.  Times Z,
// and with clamping nested, that is c_{k+1} = c_k + Z_k from c_0 = 0, Z_0 = 1: one
// number for each row instead of a vector.)  The first test needs p and q of one
// token each; Z_k, and the token behind the path, pass over the vocabulary, which the
// cluster's CTAs and their warps take in consecutive runs.
//
// Probabilities are summed as whole numbers of 2^-62 (exact from 2^-38 on, cut off
// below): sums do not depend on their order, so results do not on the number of
// CTAs, and the token is the first whose running sum passes u total to the bit.
// Bound by HBM, and for few sequences by its chain of latencies.
constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;
constexpr double kOne = 4611686018427387904.0;  // 2^62

// A probability in units of 2^-62 (outside [0, 1]: the nearer end; NaN: 0).
__device__ __forceinline__ uint64_t fixed(float x) {
  return __float2ull_rz(fminf(fmaxf(x, 0.f), 1.f) * 4611686018427387904.f);
}

template <typename T>
struct Probs;
template <>
struct Probs<float> {
  static constexpr int N = 4;  // values of 16 bytes
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void vec(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
};
template <>
struct Probs<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void vec(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// One pass over max(p - c q, 0) of a vocabulary row.
struct PassRow {
  const void *p, *q;  // q null: p alone
  uint64_t ci, cf;    // c = ci + cf 2^-64
  int sh;             // elements between the 16-byte boundary below the row's start and its start
  bool same;          // q has the same shift
  int64_t V;
};

__device__ __forceinline__ uint64_t residual(uint64_t P, uint64_t Q, const PassRow& w) {
  if (w.ci == 1 && w.cf == 0) return P > Q ? P - Q : 0;  // (the first rejected child)
  if (__umul64hi(Q, w.ci) != 0) return 0;
  const uint64_t x = Q * w.ci, y = x + __umul64hi(Q, w.cf);
  return y >= x && P > y ? P - y : 0;
}

// The N values of vector k (elements k N - sh on); outside the row: 0.
template <typename T>
__device__ __forceinline__ void load_vec(const PassRow& w, int64_t k, uint64_t (&r)[Probs<T>::N]) {
  constexpr int N = Probs<T>::N;
  const int64_t x0 = k * N - w.sh;
  const T *p = static_cast<const T*>(w.p) + x0, *q = static_cast<const T*>(w.q) + x0;
  float a[N], b[N];
  const bool in = x0 >= 0 && x0 + N <= w.V;
  if (in) {
    Probs<T>::vec(p, a);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = x0 + i >= 0 && x0 + i < w.V ? Probs<T>::one(p + i) : 0.f;
  }
  if (w.q) {
    if (in && w.same) {
      Probs<T>::vec(q, b);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) b[i] = x0 + i >= 0 && x0 + i < w.V ? Probs<T>::one(q + i) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = w.q ? residual(fixed(a[i]), fixed(b[i]), w) : fixed(a[i]);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What the walk holds of a sequence's rows, and where it stands.
struct TreeRows {
  int *par, *tok, *gone;  // gone: the rejected tokens of the current row (chosen drafts)
  float *u, *p, *q;
};
struct Walk {
  int cur, last, took, gone;
  double c, z;
  int want;  // 0: the path is complete; 1: the total of max(p - c q, 0) is needed
};

// The first child of row cur behind row `last`, -1: none.  By a warp.
__device__ __forceinline__ int next_child(const int* par, int rows, int cur, int last) {
  const int lane = threadIdx.x & 31;
  for (int j0 = max(cur, last) + 1; j0 < rows; j0 += 32) {
    const unsigned hit = __ballot_sync(0xffffffffu, j0 + lane < rows && par[j0 + lane] == cur);
    if (hit) return j0 + __ffs(hit) - 1;
  }
  return -1;
}

// Goes on until the path is complete or a total is needed.  By a warp; `path`
// (null: another CTA's warp writes it) gets the accepted rows.
__device__ __forceinline__ void advance(Walk& w, const TreeRows& t, int rows, bool drawn, int max_path, int32_t* path) {
  const int lane = threadIdx.x & 31;
  w.want = 0;
  for (;;) {
    if (w.took >= max_path) return;
    const int j = next_child(t.par, rows, w.cur, w.last);
    if (j < 0) return;
    if (w.z < 0.0) {  // (drawn) a child was rejected, and another one is left
      w.want = 1;
      return;
    }
    const int x = t.tok[j];
    const double p = t.p[j], q = t.q[j];
    double left = drawn ? __dsub_rn(p, __dmul_rn(w.c, q)) : p, weight = drawn ? __dmul_rn((double)t.u[j], q) : (double)t.u[j];
    if (left < 0.0) left = 0.0;
    if (!drawn) {
      bool was = false;
      for (int k = lane; k < w.gone; k += 32) was |= t.gone[k] == x;
      if (__any_sync(0xffffffffu, was)) left = 0.0;
    }
    if (__dmul_rn(weight, w.z) < left) {
      if (lane == 0 && path) path[w.took] = j;
      ++w.took;
      w.cur = j;
      w.last = -1;
      w.gone = 0;
      w.c = 0.0;
      w.z = 1.0;
      continue;
    }
    w.last = j;
    if (drawn) {
      w.c = __dadd_rn(w.c, w.z);
      w.z = -1.0;  // not known
    } else if (left > 0.0) {
      w.z = __dsub_rn(w.z, left);
      if (lane == 0) t.gone[w.gone] = x;
      ++w.gone;
      __syncwarp();
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) bdlm_tree_verify_kernel(const VerifyParams p) {
  constexpr int N = Probs<T>::N;
  extern __shared__ int verify_smem[];
  __shared__ uint64_t s_cta[2][kVerifyCluster], s_warp[kVerifyWarps];
  __shared__ PassRow s_row;
  __shared__ int s_want, s_gone;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), s = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t bad = 0;
  const RowsView v = rows_view(p.r, s, bad);
  int32_t* path = p.path + (int64_t)s * p.max_path;
  const bool drawn = p.draft != nullptr;
  TreeRows t;
  t.par = verify_smem;
  t.tok = t.par + p.r.max_rows;
  t.gone = t.tok + p.r.max_rows;
  t.u = reinterpret_cast<float*>(t.gone + p.r.max_rows);
  t.p = t.u + p.r.max_rows;
  t.q = t.p + p.r.max_rows;
  for (int i = tid; i < v.rows; i += kVerifyThreads) {
    int par = i > 0 ? __ldg(p.parents + v.row0 + i) : -1;
    const int x = i > 0 ? __ldg(p.tokens + v.row0 + i) : 0;
    const float u = i > 0 ? __ldg(p.uniforms + v.row0 + i) : 0.f;
    if (par < -1 || par >= i || x < 0 || x >= p.V) {  // (never accepted)
      if (i > 0) bad |= kStatusBadTree;
      par = -1;
    }
    const int64_t row = v.row0 + (par < 0 ? 0 : par);
    const float pp = par < 0 ? 0.f : Probs<T>::one(static_cast<const T*>(p.target) + row * p.target_stride + x);
    const float qq = par < 0 || !drawn ? 0.f : Probs<T>::one(static_cast<const T*>(p.draft) + row * p.draft_stride + x);
    t.par[i] = par < 0 ? -1 : par;
    t.tok[i] = x;
    t.u[i] = fmaxf(u, 0.f);
    t.p[i] = fminf(fmaxf(pp, 0.f), 1.f);
    t.q[i] = fminf(fmaxf(qq, 0.f), 1.f);
  }
  if (bad && rank == 0) atomicOr(p.status + kContentsWord, bad);
  __syncthreads();
  if (v.rows == 0) {  // (all CTAs of the cluster alike)
    if (rank == 0) {
      for (int i = tid; i < p.max_path; i += kVerifyThreads) path[i] = -1;
      if (tid == 0) p.accepted[s] = 0, p.next_token[s] = -1;
    }
    return;
  }
  Walk w{0, -1, 1, 0, 0.0, 1.0, 0};
  if (rank == 0 && tid == 0) {
    path[0] = 0;
    p.next_token[s] = -1;
  }
  const float us = p.sample[s];
  bool fallback = false;
  for (int pass = 0;; ++pass) {
    if (warp == 0) {
      if (!fallback) advance(w, t, v.rows, drawn, p.max_path, rank == 0 ? path : nullptr);
      if (lane == 0) {
        const int64_t row = v.row0 + w.cur;
        s_want = w.want;
        s_gone = drawn || fallback ? 0 : w.gone;
        s_row.p = static_cast<const T*>(p.target) + row * p.target_stride;
        s_row.q = drawn && w.c > 0.0 && !fallback ? static_cast<const T*>(p.draft) + row * p.draft_stride : nullptr;
        const double ci = floor(w.c);
        s_row.ci = (uint64_t)ci;
        s_row.cf = __double2ull_rz((w.c - ci) * 18446744073709551616.0);
        s_row.sh = (int)((reinterpret_cast<uintptr_t>(s_row.p) & 15) / sizeof(T));
        s_row.same = s_row.sh == (int)((reinterpret_cast<uintptr_t>(s_row.q) & 15) / sizeof(T));
        s_row.V = p.V;
      }
    }
    __syncthreads();
    const PassRow row = s_row;
    const int want = s_want, gone = s_gone;
    // this warp's run of vectors
    const int64_t nv = (p.V + row.sh + N - 1) / N;
    const int64_t c0 = nv * rank / C, c1 = nv * (rank + 1) / C;
    const int64_t v0 = c0 + (c1 - c0) * warp / kVerifyWarps, v1 = c0 + (c1 - c0) * (warp + 1) / kVerifyWarps;
    uint64_t sum = 0;
#pragma unroll 4
    for (int64_t k = v0 + lane; k < v1; k += 32) {
      uint64_t r[N];
      load_vec<T>(row, k, r);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += r[i];
    }
    // (rejected tokens are left out: each is in the list once)
    for (int i = lane; i < gone; i += 32) {
      const int64_t k = (t.gone[i] + row.sh) / N;
      if (k >= v0 && k < v1) sum -= fixed(Probs<T>::one(static_cast<const T*>(row.p) + t.gone[i]));
    }
    sum = warp_sum(sum);
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kVerifyWarps; ++i) mine += s_warp[i];
    // (two buffers: a CTA may still read the last pass's totals; it has when it arrives here)
    if (tid < C) *cl.map_shared_rank(&s_cta[pass & 1][rank], tid) = mine;
    cl.sync();
    uint64_t total = 0, before = 0;
    for (int i = 0; i < C; ++i) {
      if (i < rank) before += s_cta[pass & 1][i];
      total += s_cta[pass & 1][i];
    }
    if (want) {
      w.z = (double)total / kOne;
      continue;
    }
    if (total == 0 && !fallback) {  // nothing is left: from p itself
      fallback = true;
      continue;
    }
    // the first token whose running sum passes u total
    const float u = fminf(fmaxf(us, 0.f), 0.99999994f);
    const uint64_t goal = __umul64hi(__float2ull_rz(u * 18446744073709551616.f), total);
    for (int i = 0; i < warp; ++i) before += s_warp[i];
    if (goal >= before && goal - before < sum) {
      uint64_t run = before;
      int found = -1;
      for (int64_t k0 = v0; k0 < v1 && found < 0; k0 += 32) {
        uint64_t r[N], part = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = 0;
        if (k0 + lane < v1) load_vec<T>(row, k0 + lane, r);
        const int64_t x0 = (k0 + lane) * N - row.sh;
        for (int g = 0; g < gone; ++g)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (x0 + i == t.gone[g]) r[i] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) part += r[i];
        uint64_t upto = part;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run + upto > goal);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            uint64_t at = run + upto - part;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              at += r[i];
              if (found < 0 && at > goal) found = (int)(x0 + i);
            }
            p.next_token[s] = found;
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (rank == 0 && tid == 0) {
      p.accepted[s] = w.took;
      if (total == 0) atomicOr(p.status + kContentsWord, kStatusBadTree);
    }
    if (rank == 0 && warp == 0)
      for (int i = w.took + lane; i < p.max_path; i += 32) path[i] = -1;
    return;
  }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t st, int* launches) {
  bdlm_tree_mask_kernel<<<p.c.n_seqs, kMaskThreads, 12 * (size_t)p.r.max_rows, st>>>(p);
  ++*launches;
  return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_verify(const VerifyParams& p, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  auto k = bdlm_tree_verify_kernel<T>;
  const cudaError_t e = raise_smem(reinterpret_cast<const void*>(k), 24 * kMaxTreeRows, raised);
  if (e != cudaSuccess) return e;
  int C = 1;
  while (C < kVerifyCluster && p.n_seqs * C < 4 * sms) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C, (unsigned)p.n_seqs);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = 24 * (size_t)p.r.max_rows;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

cudaError_t launch_tree_verify(const VerifyParams& p, int sms, cudaStream_t st, int* launches) {
  const cudaError_t e = p.bf16 ? launch_verify<__nv_bfloat16>(p, sms, st) : launch_verify<float>(p, sms, st);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
