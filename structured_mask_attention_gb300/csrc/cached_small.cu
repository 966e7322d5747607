// cached_small.cu -- attention of up to 32 rows over the 8-bit cache (cached_small.cuh),
// and the merge of partial results.
#include "cached_small.cuh"

namespace bdlm {
namespace {

// Joins the partial results of the segments that span CTAs.  Block c takes
// the segment that CTA c of the attention kernel began and did not finish (a
// CTA has one such at most): its partials lie in slot 2 c + 1 and in slot
// 2 c' of the CTAs c' that continue it, and are joined in that order.  A
// block takes 16 of the tile's rows; neighbouring threads read neighbouring
// rows (the partials' layout), and the rows leave through shared memory.
// Bound by latency: it is launched under the attention kernel's tail and takes
// 9 to 17 us alone with nothing in L2 (15 us for 22 MB of partials of 256-row
// tiles), where they are as a rule.
constexpr int kMergeThreads = 128, kMergeRows = 16;
template <int HD>
__global__ void __launch_bounds__(kMergeThreads) bdlm_cached_merge_kernel(const CachedParams p) {
  constexpr int N = HD / 4 * kMergeRows / kMergeThreads;  // float4 per thread
  __shared__ __align__(16) float out[kMergeRows][HD + 4];
  uint32_t bad = 0;
  const CacheDesc& c = p.c;
  const int cta = blockIdx.x;
  const SplitOpen o = split_open<true>(c, p.r, p.sp, p.G, cta, bad);
  // (the kernel before this one may still run; every thread waits for it, so
  // that this grid's end implies that one's)
  dependency_wait();
  if (cta >= o.G - 1) return;
  const int64_t U = o.U, u0 = o.u0, u1 = o.u1;
  const int G = o.G;
  const UnitPos pos = o.pos;
  const SegInfo seg = o.seg;
  const int64_t begin = u1 - 1 - pos.j, last = begin + seg.span - 1;
  // begun by another CTA (its first unit lies before or behind this CTA's range), or finished here
  if (begin + p.sp.extra < u0 || begin + p.sp.extra >= u1 || last < u1) return;
  const int c1 = split_owner(U, G, last);
  const int R = p.sp.tile_rows, row0 = blockIdx.y * kMergeRows;
  const int r = threadIdx.x % kMergeRows, row = row0 + r, c4 = threadIdx.x / kMergeRows;
  const int rows = seg.v.rows * p.sp.group - pos.rt * R;  // of this tile
  if (row0 >= rows) return;
  const int64_t pf = part_floats(R, HD);
  const float* parts = p.part + 2 * (int64_t)cta * pf;
  auto slot = [&](int x) { return parts + (2 * (int64_t)(x - cta) + (x == cta ? 1 : 0)) * pf; };
  float M = -INFINITY;
#pragma unroll 4
  for (int x = cta; x <= c1; ++x) M = fmaxf(M, slot(x)[R * HD + row]);
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int x = cta; x <= c1; ++x) {
    const float* q = slot(x);
    const float w = ex2_approx(q[R * HD + row] - base);
    L = fmaf(w, q[R * (HD + 1) + row], L);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 o = reinterpret_cast<const float4*>(q)[(c4 + i * (kMergeThreads / kMergeRows)) * R + row];
      a[i].x = fmaf(w, o.x, a[i].x); a[i].y = fmaf(w, o.y, a[i].y);
      a[i].z = fmaf(w, o.z, a[i].z); a[i].w = fmaf(w, o.w, a[i].w);
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    *reinterpret_cast<float4*>(&out[r][4 * (c4 + i * (kMergeThreads / kMergeRows))]) =
        make_float4(a[i].x * inv, a[i].y * inv, a[i].z * inv, a[i].w * inv);
  auto place = [&](int rr, int64_t& at, int& head) {  // packed row and query head of tile row row0 + rr
    const int fr = pos.rt * R + row0 + rr, tok = fr / p.sp.group;
    head = pos.h * p.sp.group + fr - tok * p.sp.group;
    at = seg.v.row0 + tok;
  };
  int64_t at;
  int head;
  if (c4 == 0 && row < rows) {
    place(r, at, head);
    p.LSE[(int64_t)head * p.r.T + at] = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int k = threadIdx.x + i * kMergeThreads, rr = k / (HD / 4), col = (k % (HD / 4)) * 4;
    if (row0 + rr >= rows) continue;
    place(rr, at, head);
    const float4 o = *reinterpret_cast<const float4*>(&out[rr][col]);
    const int64_t o0 = (at * p.Hq + head) * HD + col;
    if (p.o_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.O) + o0) = o;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + o0) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
}

}  // namespace

template <int HD, bool FINE>
static cudaError_t launch_rows(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  return p.sp.tile_rows == 16 ? launch<HD, 1, 1, FINE, false>(m, p, st) : launch<HD, 1, 2, FINE, false>(m, p, st);
}

cudaError_t launch_cached_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? (p.o_f32 ? launch_rows<128, true>(m, p, st) : launch_rows<128, false>(m, p, st))
                                     : (p.o_f32 ? launch_rows<64, true>(m, p, st) : launch_rows<64, false>(m, p, st));
  if (e == cudaSuccess) ++*launches;
  return e;
}

cudaError_t launch_cached_merge(const CachedParams& p, cudaStream_t st, int* launches) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.G, (unsigned)(p.sp.tile_rows / kMergeRows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // may start before the attention kernel's end
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = p.c.d == 128 ? cudaLaunchKernelEx(&cfg, bdlm_cached_merge_kernel<128>, p)
                                     : cudaLaunchKernelEx(&cfg, bdlm_cached_merge_kernel<64>, p);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
