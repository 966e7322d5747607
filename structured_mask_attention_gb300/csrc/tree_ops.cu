// tree_ops.cu -- drafted trees beside the attention over the 8-bit cache: what each row
// of a tree sees, and which drafted tokens the target's probabilities accept.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <utility>

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
// Sums carry the rounding of every addition beside them, about twice fp32's
// width: a running sum that is off by d picks another token for a share d of all random
// numbers, for each token of the vocabulary, 1e-4 of all calls with fp32 sums.  Lanes'
// sums join as whole numbers of 2^-62, whose order does not matter.  (Whole numbers from
// the start: 98 us for the drawn trees below with the conversion instruction, 64 with
// shifts, 39 this way; fp64 has two additions a clock and SM.)
// Bound by a chain of latencies: row offsets, parents, the rows' p and q (2 thousand
// cycles), the walk (2, and 0.4 for each accepted row), 5 for a pass and its join by
// the cluster, 1 to find the token; and by HBM for its passes where sequences are many.
// 64 trees of 16 rows drawn with up to 3 children, V = 131072 in fp32 (66 MB, more for
// 2nd and 3rd passes): 39 us, the last sequences 3 passes; 16 trees of 64 chosen rows, V
// = 100003 in bf16: 16 us; one chain of 8, V = 32000: 10 us.  CTAs of 512 / 256 / 128
// threads: 48 / 39 / 41 us; up to 2 / 4 CTAs for each SM: 41 / 39 (80 registers leave room for three:
// of 512 CTAs 456 are resident, at least 7 of 64 clusters begin when others have ended; a sequence that ends
// early leaves its place).
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;
constexpr double kOne = 4611686018427387904.0;  // 2^62: the whole numbers' unit

// A number of fp32's width twice over: s + e.
struct Wide {
  float s, e;
};
// In units of 2^-62, what is below cut off.  A single value, at most 1:
__device__ __forceinline__ uint64_t fixed(Wide x) {
  constexpr float k = 4611686018427387904.f;
  return (uint64_t)(__float2ll_rz(x.s * k) + __float2ll_rz(x.e * k));
}
// A lane's sum, below 4, where a signed number ends at 2: 2 of it are set as a bit.
__device__ __forceinline__ uint64_t fixed_sum(Wide x) {
  const bool top = x.s >= 2.f;
  if (top) x.s -= 2.f;
  return fixed(x) + (top ? 1ull << 63 : 0ull);
}
// sum += x, both parts of every rounding kept.
__device__ __forceinline__ void add(Wide& sum, Wide x) {
  const float t = __fadd_rn(sum.s, x.s), b = __fsub_rn(t, sum.s);
  const float r = __fadd_rn(__fsub_rn(x.s, b), __fsub_rn(sum.s, __fsub_rn(t, b)));
  sum.e = __fadd_rn(sum.e, __fadd_rn(r, x.e));
  sum.s = t;
}

template <typename T>
struct Probs;
template <>
struct Probs<float> {
  static constexpr int N = 4;  // values of 16 bytes
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ float value(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ void put(uint4& v, int i, float x) {
    (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = __float_as_uint(x);
  }
};
template <>
struct Probs<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ float value(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ void put(uint4& v, int i, float x) {
    const uint32_t b = __float_as_uint(x) >> 16;  // (x is a bf16 value)
    (i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w) |= i & 1 ? b << 16 : b;
  }
};

// What a pass adds up over a vocabulary row: p, or max(p - c q, 0) with c = 1 (the first
// rejected child) or any c = ch + cl.
enum PassKind { kPlain, kFirst, kAny };
struct PassRow {
  const void *p, *q;
  float ch, cl;
  int kind;
  int sh;     // elements between the 16-byte boundary below the row's start and its start
  int aside;  // q has another shift: its vectors are put together from single values
  int V;
};

// The 16 bytes of vector k (elements k N - sh on); outside the row: 0.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const void* row, int x0, int V, bool aside) {
  constexpr int N = Probs<T>::N;
  const T* p = static_cast<const T*>(row) + x0;
  if (x0 >= 0 && x0 + N <= V && !aside) return __ldg(reinterpret_cast<const uint4*>(p));
  uint4 v = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (x0 + i >= 0 && x0 + i < V) Probs<T>::put(v, i, Probs<T>::one(p + i));
  return v;
}

// Exact for c = 1 (the difference of two fp32 numbers and its rounding); any c: to about 2^-46 of p and c q.
template <int KIND>
__device__ __forceinline__ Wide residual(float p, float q, const PassRow& w) {
  p = __saturatef(p);  // (NaN: 0)
  if (KIND == kPlain) return Wide{p, 0.f};
  q = __saturatef(q);
  Wide r;
  if (KIND == kFirst) {
    r.s = __fsub_rn(p, q);
    r.e = __fsub_rn(__fsub_rn(p, r.s), q);
    return r.s > 0.f ? r : Wide{0.f, 0.f};
  }
  const float h = __fmul_rn(w.ch, q), l = __fmaf_rn(w.cl, q, __fmaf_rn(w.ch, q, -h));  // c q = h + l
  r.s = __fsub_rn(p, h);
  const float b = __fsub_rn(r.s, p);
  r.e = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(r.s, b)), __fadd_rn(h, b)), l);
  return __fadd_rn(r.s, r.e) > 0.f ? r : Wide{0.f, 0.f};
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A warp's run of vectors [v0, v1) is cut into four quarters of whole 32-vector tiles.
__device__ __forceinline__ int quarter(int v0, int v1, int i) {
  return min(v1, v0 + ((v1 - v0 + 127) >> 7) * 32 * i);
}

// A lane's sums of the quarters: a tile of each at a time, all loads in flight.
template <typename T, int KIND>
__device__ __forceinline__ void sum_run(const PassRow& w, int v0, int v1, uint64_t (&sum)[4]) {
  constexpr int N = Probs<T>::N;
  const int lane = threadIdx.x & 31, len = ((v1 - v0 + 127) >> 7) * 32;
  Wide x[4] = {};
#pragma unroll 1
  for (int k = lane; k < len; k += 32) {
    uint4 a[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = v0 + u * len + k, x0 = at < v1 ? at * N - w.sh : w.V;
      a[u] = load_vec<T>(w.p, x0, w.V, false);
      if (KIND != kPlain) b[u] = load_vec<T>(w.q, x0, w.V, w.aside);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int y = 0; y < N; ++y)
        add(x[u], residual<KIND>(Probs<T>::value(a[u], y), KIND == kPlain ? 0.f : Probs<T>::value(b[u], y), w));
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) sum[u] = fixed_sum(x[u]);
}

// What the walk holds of a sequence's rows, and where it stands.
struct TreeRows {
  int *par, *tok, *gone;  // gone: the rejected tokens of the current row (chosen drafts)
  float *u, *p, *q;       // (u with a sign, -0 too: the row is accepted as a first child)
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
    if (drawn && w.z < 0.0) {  // a child was rejected, and another one is left
      w.want = 1;
      return;
    }
    const int x = t.tok[j];
    const float u = t.u[j];
    bool ok;
    double left = t.p[j];
    if (w.last < 0) {
      ok = __float_as_int(u) < 0;
    } else {
      const double q = t.q[j], ua = fabsf(u);
      if (drawn) {
        left = __dsub_rn(left, __dmul_rn(w.c, q));
      } else {
        bool was = false;
        for (int k = lane; k < w.gone; k += 32) was |= t.gone[k] == x;
        if (__any_sync(0xffffffffu, was)) left = 0.0;
      }
      ok = __dmul_rn(drawn ? __dmul_rn(ua, q) : ua, w.z) < (left > 0.0 ? left : 0.0);
    }
    if (ok) {
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
__global__ void __launch_bounds__(kVerifyThreads, 3) bdlm_tree_verify_kernel(const VerifyParams p) {
  constexpr int N = Probs<T>::N;
  extern __shared__ int verify_smem[];
  __shared__ uint64_t s_cta[2][kVerifyCluster], s_warp[kVerifyWarps];
  __shared__ PassRow s_row;
  __shared__ int s_want, s_gone;
  cg::cluster_group cl = cg::this_cluster();
  auto begun = cl.barrier_arrive();  // (waited for before the first write into another CTA's shared memory)
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
    const float pc = fminf(fmaxf(pp, 0.f), 1.f), qc = fminf(fmaxf(qq, 0.f), 1.f), uc = fabsf(fmaxf(u, 0.f));
    // the test against p itself, for all rows side by side (u q is exact in 64 bits); its answer is u's sign
    const bool first = drawn ? (double)uc * (double)qc < (double)pc : uc < pc;
    t.u[i] = first ? -uc : uc;
    t.p[i] = pc;
    t.q[i] = qc;
  }
  if (bad && rank == 0) atomicOr(p.status + kContentsWord, bad);
  cl.barrier_wait(std::move(begun));
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
        const bool rest = drawn && w.c > 0.0 && !fallback;
        s_row.p = static_cast<const T*>(p.target) + row * p.target_stride;
        s_row.q = rest ? static_cast<const T*>(p.draft) + row * p.draft_stride : nullptr;
        s_row.kind = !rest ? kPlain : w.c == 1.0 ? kFirst : kAny;
        s_row.ch = (float)w.c;
        s_row.cl = (float)(w.c - (double)s_row.ch);
        s_row.sh = (int)((reinterpret_cast<uintptr_t>(s_row.p) & 15) / sizeof(T));
        s_row.aside = s_row.sh != (int)((reinterpret_cast<uintptr_t>(s_row.q) & 15) / sizeof(T));
        s_row.V = (int)p.V;
      }
    }
    __syncthreads();
    const PassRow row = s_row;
    const int want = s_want, gone = s_gone;
    // this warp's run of vectors
    const int nv = (row.V + row.sh + N - 1) / N, per = (nv + C * kVerifyWarps - 1) / (C * kVerifyWarps);
    const int v0 = min(nv, (rank * kVerifyWarps + warp) * per), v1 = min(nv, v0 + per);
    uint64_t part[4];
    if (row.kind == kPlain) sum_run<T, kPlain>(row, v0, v1, part);
    else if (row.kind == kFirst) sum_run<T, kFirst>(row, v0, v1, part);
    else sum_run<T, kAny>(row, v0, v1, part);
    // (rejected tokens are left out: each is in the list once)
    for (int i = lane; i < gone; i += 32) {
      const int k = (t.gone[i] + row.sh) / N;
      if (k < v0 || k >= v1) continue;
      const uint64_t x = fixed(Wide{__saturatef(Probs<T>::one(static_cast<const T*>(row.p) + t.gone[i])), 0.f});
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (k >= quarter(v0, v1, y) && k < quarter(v0, v1, y + 1)) part[y] -= x;
    }
    const uint64_t sum = warp_sum(part[0] + part[1] + part[2] + part[3]);
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
      int y = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) {  // the quarter
        const uint64_t z = warp_sum(part[i]);
        if (y == i && goal - run >= z) run += z, y = i + 1;
      }
      const int e = quarter(v0, v1, y + 1);
      // the token, a tile after the other (its sums may differ from the run's in the last unit: then the last token
      // that has any)
      int token = -1, last = -1;
#pragma unroll 1
      for (int k0 = quarter(v0, v1, y); k0 < e && token < 0; k0 += 32) {
        const int x0 = k0 + lane < e ? (k0 + lane) * N - row.sh : row.V;
        const uint4 a = load_vec<T>(row.p, x0, row.V, false);
        const uint4 b = row.kind == kPlain ? make_uint4(0, 0, 0, 0) : load_vec<T>(row.q, x0, row.V, row.aside);
        uint64_t r[N], mine = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float pv = Probs<T>::value(a, i), qv = Probs<T>::value(b, i);
          r[i] = fixed(row.kind == kPlain   ? residual<kPlain>(pv, qv, row)
                       : row.kind == kFirst ? residual<kFirst>(pv, qv, row)
                                            : residual<kAny>(pv, qv, row));
          for (int g = 0; g < gone; ++g)
            if (x0 + i == t.gone[g]) r[i] = 0;
          mine += r[i];
          if (r[i] != 0) last = x0 + i;
        }
        uint64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t z = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += z;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, run + upto > goal);
        if (hit) {
          uint64_t at = run + upto - mine;
          int x = -1;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            at += r[i];
            if (x < 0 && at > goal) x = x0 + i;
          }
          token = __shfl_sync(0xffffffffu, x, __ffs(hit) - 1);
        } else {
          run += __shfl_sync(0xffffffffu, upto, 31);
        }
      }
      if (token < 0) token = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) p.next_token[s] = token;
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
  while (C < kVerifyCluster && p.n_seqs * C * 2 <= 4 * sms) C *= 2;
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
