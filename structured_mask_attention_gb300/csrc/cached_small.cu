// cached_small.cu -- attention of few rows over the 8-bit cache: mma.sync
// tiles of 16 rows, and the merge of partial results.
//
// One token of a sequence gives Hq / Hkv rows per KV head, a handful against
// thousands of keys: every cached byte is read once and used for one or two
// 16-row MMA tiles, so the kernel's only bound is the stream of codes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cached_attn.h"
#include "kernels.h"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kWarps = 4;

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
// Codes: read once, kept out of L1.
__device__ __forceinline__ uint4 ldg16_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg8_stream(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
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

// Online-softmax state of a warp's 16 x HD tile.  A thread (g = lane / 4,
// t = lane % 4) holds rows g and g + 8; its O values are HD / 4 consecutive
// columns of each row (see pv_step).
template <int HD>
struct State {
  float o[HD / 8][4];
  float m[2], l[2];  // l: this thread's part of the row sum
};

// Scores of one group of N8 * 8 keys -> probabilities in place; the running
// maximum moves, O and l are rescaled when it does.
//
// Value scales.  A cached key's score comes with log2 of its value block's
// scale added: p' = exp2(s + log2 vs - m) is then the weight of the codes
// themselves (O = sum p' code, at the fp16 precision of the largest weight
// whatever the scales), and the row sum takes p' / vs (iv).  In units of
// exp2(m), O / l is the attention's output and m + log2 l its LSE.
template <int HD, int N8>
__device__ __forceinline__ void softmax_step(State<HD>& st, float (&s)[N8][4], const float (&iv)[N8 / 2]) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < N8; ++i) mx = fmaxf(mx, fmaxf(s[i][2 * r], s[i][2 * r + 1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(st.m[r], mx);
    const float base = mn == -INFINITY ? 0.f : mn;  // no key yet: every p below is 0
    const float alpha = ex2_approx(st.m[r] - base);
    if (__any_sync(0xffffffffu, mn != st.m[r])) {
#pragma unroll
      for (int j = 0; j < HD / 8; ++j) {
        st.o[j][2 * r] *= alpha;
        st.o[j][2 * r + 1] *= alpha;
      }
      st.l[r] *= alpha;
    }
    st.m[r] = mn;
    float sum[N8 / 2] = {};
#pragma unroll
    for (int i = 0; i < N8; ++i) {
      s[i][2 * r] = ex2_approx(s[i][2 * r] - base);
      s[i][2 * r + 1] = ex2_approx(s[i][2 * r + 1] - base);
      sum[i / 2] += s[i][2 * r] + s[i][2 * r + 1];
    }
#pragma unroll
    for (int i = 0; i < N8 / 2; ++i) st.l[r] = fmaf(sum[i], iv[i], st.l[r]);
  }
}

// MMA columns.  The contraction index of S = Q K^T may visit the head
// dimension in any order that both operands share, and the columns of O may
// stand for the head dimension in any order: a thread takes 16 consecutive
// bytes of a key (16 codes) and uses them, word by word, as the fragments of
// four k-steps (word i, bytes 0-1 and 2-3: the two halves of step 4 h + i of
// 64-byte half h), so every load is 16 bytes wide and no operand is
// transposed.  For P V, thread (g, t) takes codes HD/8 g .. + HD/8 - 1 of keys
// 2 t, 2 t + 1, 2 t + 8, 2 t + 9 and pairs the codes of two keys by byte
// permutes: column tile j of O is then element j of every thread's piece, and
// O's fragment of thread t holds columns HD/4 t .. HD/4 (t + 1) - 1 in order.
//
// P is rounded to fp16 (2^-11) for cached keys and bf16 for own ones, below a
// bf16 output's own rounding.  FINE, for an fp32 output: P goes in two (three)
// parts, each what the rounding of the one before left, so that O is off by
// fp32 sums alone.
template <int HD, bool FINE>
__global__ void __launch_bounds__(32 * kWarps, kSmallCtasPerSm) bdlm_cached_small_kernel(const CachedParams p) {
  constexpr int KH = HD / 64;  // 64-byte halves of a key's codes
  constexpr int VW = HD / 32;  // words of a thread's piece of a value row
  extern __shared__ __align__(16) float red[];
  float(*red_o)[kSmallRows][HD + 4] = reinterpret_cast<float(*)[kSmallRows][HD + 4]>(red);
  float(*red_ml)[kSmallRows][2] =
      reinterpret_cast<float(*)[kSmallRows][2]>(red + kWarps * kSmallRows * (HD + 4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t bad = 0;
  const CacheDesc& c = p.c;
  const int cta = blockIdx.x;
  int64_t u0 = 0, u1 = 0;
  UnitPos pos{0, 0, 0, 0};
  SegInfo seg;
  launch_dependents();
  if (p.whole) {  // CTA per segment: (sequence, KV head, row tile), p.whole row tiles for each
    pos.rt = cta % p.whole;
    pos.h = cta / p.whole % c.Hkv;
    pos.s = cta / p.whole / c.Hkv;
    seg = seg_info(c, p.r, p.sp, pos.s, bad);
    u1 = pos.rt < seg.rtiles ? seg.span : 0;
  } else {
    const int64_t U = total_units(c, p.r, p.sp, bad);
    const int G = split_ctas(U, p.G);
    if (cta < G) {
      u0 = split_begin(U, G, cta);
      u1 = split_begin(U, G, cta + 1);
      pos = locate_unit(c, p.r, p.sp, u0, bad);
      seg = seg_info(c, p.r, p.sp, pos.s, bad);
    }
  }
  {
    for (int64_t u = u0; u < u1;) {
      int jb, je;
      split_units(seg, p.sp, pos, u, u1, jb, je);
      u += seg.span - pos.j;
      if (je == 0) break;  // only the segment's opening lies here: the next CTA begins it
      // ---- the tile's rows: fp16, each scaled by a power of two that puts
      // its largest magnitude in [2^14, 2^15): exact down to 2^-28 of it
      uint32_t q[KH * 4][4];
      float cq[2];
      int64_t qoff[2];
      bool live[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int fr = pos.rt * kSmallRows + g + 8 * r, tok = fr / p.sp.group;
        live[r] = tok < seg.v.rows;
        const int head = pos.h * p.sp.group + fr - tok * p.sp.group;
        qoff[r] = ((seg.v.row0 + (live[r] ? tok : 0)) * p.Hq + head) * HD;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.Q) + qoff[r];
        uint32_t w[KH][8];
        uint32_t amax = 0;
#pragma unroll
        for (int h = 0; h < KH; ++h) {
          const uint4 x = live[r] ? ldg16(src + 64 * h + 16 * t) : make_uint4(0, 0, 0, 0);
          const uint4 y = live[r] ? ldg16(src + 64 * h + 16 * t + 8) : make_uint4(0, 0, 0, 0);
          w[h][0] = x.x; w[h][1] = x.y; w[h][2] = x.z; w[h][3] = x.w;
          w[h][4] = y.x; w[h][5] = y.y; w[h][6] = y.z; w[h][7] = y.w;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = max(amax, max(w[h][i] & 0x7fffu, (w[h][i] >> 16) & 0x7fffu));
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int e = 14 + 127 - (int)(amax >> 7);  // bf16 exponent field
        if (amax >= 0x7f80u || amax == 0) e = 0;
        e = min(e, 126);
        const float f = __uint_as_float((uint32_t)(e + 127) << 23);
        cq[r] = p.sl2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int h = 0; h < KH; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            q[4 * h + i][r] = pack_half2(bf_lo(w[h][2 * i]) * f, bf_hi(w[h][2 * i]) * f);
            q[4 * h + i][2 + r] = pack_half2(bf_lo(w[h][2 * i + 1]) * f, bf_hi(w[h][2 * i + 1]) * f);
          }
      }
      State<HD> st;
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[j][i] = 0.f;
      st.m[0] = st.m[1] = -INFINITY;
      st.l[0] = st.l[1] = 0.f;

      // ---- cached keys: this warp's 32 of every unit of 128
      const int kc = min(je, seg.ktiles);
      uint4 kw[4][KH];
      uint32_t vw[2][4][VW];
      int pid[2] = {-1, -1}, npid[2] = {-1, -1};
      auto pages = [&](int j, int (&id)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = j * kUnit + warp * 32 + 16 * x;
          id[x] = j < kc && key < seg.v.len ? page_id(c, pos.s, key >> c.lp, bad) : -1;
        }
      };
      auto row_at = [&](int64_t page, int key) -> int64_t {
        return ((page * c.Hkv + pos.h) * c.page + (key & (c.page - 1))) * HD;
      };
      auto load_k = [&](int j, const int (&id)[2]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = j * kUnit + warp * 32 + 8 * i + g;
          const bool ok = id[i >> 1] >= 0 && key < seg.v.len;
          const uint8_t* src = c.k8 + (ok ? row_at(id[i >> 1], key) + 16 * t : 0);
#pragma unroll
          for (int h = 0; h < KH; ++h) kw[i][h] = ok ? ldg16_stream(src + 64 * h) : make_uint4(0, 0, 0, 0);
        }
      };
      auto load_v = [&](int j, const int (&id)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = j * kUnit + warp * 32 + 16 * x + 2 * t + (i & 1) + 8 * (i >> 1);
            const bool ok = id[x] >= 0 && key < seg.v.len;
            const uint8_t* src = c.v8 + (ok ? row_at(id[x], key) + (HD / 8) * g : 0);
            if (HD == 128) {
              const uint4 v = ok ? ldg16_stream(src) : make_uint4(0, 0, 0, 0);
              vw[x][i][0] = v.x; vw[x][i][1] = v.y; vw[x][i][VW - 2] = v.z; vw[x][i][VW - 1] = v.w;
            } else {
              const uint2 v = ok ? ldg8_stream(src) : make_uint2(0, 0);
              vw[x][i][0] = v.x; vw[x][i][1] = v.y;
            }
          }
      };
      if (jb < kc) {
        pages(jb, pid);
        load_k(jb, pid);
        load_v(jb, pid);
      }
      for (int j = jb; j < kc; ++j) {
        pages(j + 1, npid);
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
          for (int h = 0; h < KH; ++h) {
            const uint32_t w[4] = {kw[i][h].x, kw[i][h].y, kw[i][h].z, kw[i][h].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(s[i], q[4 * h + k][0], q[4 * h + k][1], q[4 * h + k][2], q[4 * h + k][3],
                      e4m3x2_to_half2(w[k]), e4m3x2_to_half2(w[k] >> 16));
          }
        }
        load_k(j + 1, npid);  // (ids of -1 past the end: nothing is read)
        float iv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int64_t b = (int64_t)max(pid[x], 0) * c.Hkv + pos.h;
          const float ks = pid[x] >= 0 ? __ldg(c.ks + b) : 0.f;
          const float vs = pid[x] >= 0 ? __ldg(c.vs + b) : 1.f;
          const float lv = log2f(vs);
          iv[x] = 1.f / vs;
          const int key = j * kUnit + warp * 32 + 16 * x + 2 * t;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool ok = pid[x] >= 0 && key + 8 * i + (e & 1) < seg.v.len;
              s[2 * x + i][e] = ok ? fmaf(s[2 * x + i][e], cq[e >> 1] * ks, lv) : -INFINITY;
            }
        }
        softmax_step<HD, 4>(st, s, iv);
        uint32_t pa[2][4], pr[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = s[2 * x + (i >> 1)][2 * (i & 1)], b = s[2 * x + (i >> 1)][2 * (i & 1) + 1];
            pa[x][i] = pack_half2(a, b);
            if (FINE) pr[x][i] = rest_half2(pa[x][i], a, b);
          }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // bytes 2 hf, 2 hf + 1 of word w: column tiles 4 w + 2 hf, + 1
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t lo = __byte_perm(vw[x][0][w], vw[x][1][w], hf ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(vw[x][2][w], vw[x][3][w], hf ? 0x7362 : 0x5140);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t b0 = e4m3x2_to_half2(lo >> (16 * y)), b1 = e4m3x2_to_half2(hi >> (16 * y));
                mma_f16(st.o[4 * w + 2 * hf + y], pa[x][0], pa[x][1], pa[x][2], pa[x][3], b0, b1);
                if (FINE) mma_f16(st.o[4 * w + 2 * hf + y], pr[x][0], pr[x][1], pr[x][2], pr[x][3], b0, b1);
              }
            }
          }
        load_v(j + 1, npid);
        pid[0] = npid[0];
        pid[1] = npid[1];
      }

      // ---- the rows' own block (bf16), in groups of 16 keys
      if (p.sp.local) {
        int k0 = 0, k1 = 0;  // own keys of this piece
        if (seg.ltiles == 0) {
          if (je == seg.units) k1 = seg.v.rows;
        } else {
          k0 = max(jb - seg.ktiles, 0) * kUnit;
          k1 = min(max(je - seg.ktiles, 0) * kUnit, seg.v.rows);
        }
        for (int key0 = k0 + 16 * warp; key0 < k1; key0 += 16 * kWarps) {
          float s[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
          for (int h = 0; h < HD / 32; ++h) {
            uint4 a[2], b[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              a[r] = live[r] ? ldg16(static_cast<const __nv_bfloat16*>(p.Q) + qoff[r] + 32 * h + 8 * t)
                             : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int key = key0 + 8 * i + g;
              b[i] = key < seg.v.rows
                         ? ldg16(static_cast<const __nv_bfloat16*>(p.K) +
                                 ((seg.v.row0 + key) * c.Hkv + pos.h) * HD + 32 * h + 8 * t)
                         : make_uint4(0, 0, 0, 0);
              mma_bf16(s[i], a[0].x, a[1].x, a[0].y, a[1].y, b[i].x, b[i].y);
              mma_bf16(s[i], a[0].z, a[1].z, a[0].w, a[1].w, b[i].z, b[i].w);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[i][e] = key0 + 8 * i + 2 * t + (e & 1) < seg.v.rows ? s[i][e] * p.sl2 : -INFINITY;
          const float one[1] = {1.f};
          softmax_step<HD, 2>(st, s, one);
          uint32_t pa[4], pr[4], pq[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = s[i >> 1][2 * (i & 1)], b = s[i >> 1][2 * (i & 1) + 1];
            pa[i] = pack_bf16x2(a, b);
            if (FINE) {
              pr[i] = rest_bf16x2(pa[i], a, b);
              pq[i] = rest_bf16x2(pr[i], a - bf_lo(pa[i]), b - bf_hi(pa[i]));
            }
          }
#pragma unroll
          for (int w = 0; w < HD / 64; ++w) {  // 8 columns of the thread's HD / 8 (16 bytes) at a time
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + 2 * t + (i & 1) + 8 * (i >> 1);
              v[i] = key < seg.v.rows
                         ? ldg16(static_cast<const __nv_bfloat16*>(p.V) +
                                 ((seg.v.row0 + key) * c.Hkv + pos.h) * HD + (HD / 8) * g + 8 * w)
                         : make_uint4(0, 0, 0, 0);
            }
            const uint32_t x0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, x1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
            const uint32_t y0[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, y1[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t sel = y ? 0x7632 : 0x5410;
                const uint32_t b0 = __byte_perm(x0[k], x1[k], sel), b1 = __byte_perm(y0[k], y1[k], sel);
                mma_bf16(st.o[8 * w + 2 * k + y], pa[0], pa[1], pa[2], pa[3], b0, b1);
                if (FINE) {
                  mma_bf16(st.o[8 * w + 2 * k + y], pr[0], pr[1], pr[2], pr[3], b0, b1);
                  mma_bf16(st.o[8 * w + 2 * k + y], pq[0], pq[1], pq[2], pq[3], b0, b1);
                }
              }
            }
          }
        }
      }

      // ---- the four warps' states joined through shared memory
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = st.l[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) {
          red_ml[warp][g + 8 * r][0] = st.m[r];
          red_ml[warp][g + 8 * r][1] = l;
        }
        // tile j, element e: column (HD / 4) t + (HD / 8) e + j
        float* o = &red_o[warp][g + 8 * r][(HD / 4) * t];
#pragma unroll
        for (int j = 0; j < HD / 8; j += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(o + (HD / 8) * e + j) =
                make_float4(st.o[j][2 * r + e], st.o[j + 1][2 * r + e], st.o[j + 2][2 * r + e], st.o[j + 3][2 * r + e]);
      }
      __syncthreads();
      {
        const int row = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * 4;
        float M = -INFINITY, w[kWarps], L = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) M = fmaxf(M, red_ml[x][row][0]);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          w[x] = M == -INFINITY ? 0.f : ex2_approx(red_ml[x][row][0] - M);
          L = fmaf(w[x], red_ml[x][row][1], L);
        }
        const int fr = pos.rt * kSmallRows + row, tok = fr / p.sp.group;
        const bool whole = jb == 0 && je == seg.units;
        float* slot = p.part + (2 * (int64_t)cta + (jb == 0 ? 1 : 0)) * part_floats(kSmallRows, HD);
        if (tok < seg.v.rows) {
          const int head = pos.h * p.sp.group + fr - tok * p.sp.group;
          const int64_t o0 = ((seg.v.row0 + tok) * p.Hq + head) * HD;
          const float inv = whole ? (L != 0.f ? 1.f / L : 0.f) : 1.f;
#pragma unroll
          for (int k = 0; k < HD / 32; ++k) {
            const int col = c0 + 32 * k;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
              const float4 b = *reinterpret_cast<const float4*>(&red_o[x][row][col]);
              a.x = fmaf(w[x], b.x, a.x); a.y = fmaf(w[x], b.y, a.y);
              a.z = fmaf(w[x], b.z, a.z); a.w = fmaf(w[x], b.w, a.w);
            }
            a.x *= inv; a.y *= inv; a.z *= inv; a.w *= inv;
            if (!whole) reinterpret_cast<float4*>(slot)[(col >> 2) * kSmallRows + row] = a;
            else if (p.o_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.O) + o0 + col) = a;
            else
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + o0 + col) =
                  make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
          }
          if ((threadIdx.x & 7) == 0) {
            if (whole) p.LSE[(int64_t)head * p.r.T + seg.v.row0 + tok] = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
            else {
              slot[kSmallRows * HD + row] = M;
              slot[kSmallRows * HD + kSmallRows + row] = L;
            }
          }
        }
      }
      __syncthreads();
      if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
    }
  }
  if (bad) atomicOr(p.status, bad);
}

// Joins the partial results of the segments that span CTAs.  Block c takes
// the segment that CTA c of the attention kernel began and did not finish (a
// CTA has one such at most): its partials lie in slot 2 c + 1 and in slot
// 2 c' of the CTAs c' that continue it, and are joined in that order.  A
// block takes 16 of the tile's rows; neighbouring threads read neighbouring
// rows (the partials' layout), and the rows leave through shared memory.
constexpr int kMergeThreads = 128, kMergeRows = 16;
template <int HD>
__global__ void __launch_bounds__(kMergeThreads) bdlm_cached_merge_kernel(const CachedParams p) {
  constexpr int N = HD / 4 * kMergeRows / kMergeThreads;  // float4 per thread
  __shared__ __align__(16) float out[kMergeRows][HD + 4];
  uint32_t bad = 0;
  const CacheDesc& c = p.c;
  const int cta = blockIdx.x;
  const int64_t U = total_units(c, p.r, p.sp, bad);
  const int G = split_ctas(U, p.G);
  // (the kernel before this one may still run; every thread waits for it, so
  // that this grid's end implies that one's)
  dependency_wait();
  if (cta >= G - 1) return;
  const int64_t u0 = split_begin(U, G, cta), u1 = split_begin(U, G, cta + 1);
  const UnitPos pos = locate_unit(c, p.r, p.sp, u1 - 1, bad);
  const SegInfo seg = seg_info(c, p.r, p.sp, pos.s, bad);
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

cudaError_t launch_cached_small(const CachedParams& p, cudaStream_t st, int* launches) {
  // (at most 34.3 KB: within the default limit)
  const int bytes = (kWarps * kSmallRows * (p.c.d + 4) + kWarps * kSmallRows * 2) * (int)sizeof(float);
  auto k = p.c.d == 128 ? (p.o_f32 ? bdlm_cached_small_kernel<128, true> : bdlm_cached_small_kernel<128, false>)
                        : (p.o_f32 ? bdlm_cached_small_kernel<64, true> : bdlm_cached_small_kernel<64, false>);
  k<<<p.G, 32 * kWarps, bytes, st>>>(p);
  ++*launches;
  return cudaGetLastError();
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
