// cached_small.cu -- attention of up to 32 rows over the 8-bit cache on mma.sync
// tiles, and the merge of partial results.
//
// One token of a sequence, or a short block, gives Hq / Hkv rows per token and
// KV head, a handful against thousands of keys: the stream of codes bounds the
// call, and a tcgen05 tile of 128 rows would be mostly padding.  A CTA of four
// warps takes 16 or 32 rows (MT 16-row tiles); its warps are MT row tiles by
// 4 / MT groups of keys.  A fifth warp keeps a ring of K and V tiles of 128 keys
// filled by TMA, codes as they lie, so that 128 KB per SM (two CTAs) are in flight
// whatever the warps do; they turn codes into fp16 on the way from shared
// memory to the MMA.
// Bound by HBM: 32 sequences of up to 32768 tokens (1.30 GB of codes), a token
// each, 32 / 8 heads of 128, take 208 us with the merge: 6.2 TB/s, 92 % of the
// measured copy rate.  (With loads issued by the computing warps themselves it
// was 334 us.)  With fp32 outputs, whose weights go in two parts: 247 us (ptxas
// reports 60 bytes of spills, 332 with tiles of 32 rows).  S from two e4m3 parts of Q
// by e4m3 m16n8k32 instead, without K's conversion: 259 us against 227 when it was
// tried.  One sequence of 256 tokens: 8 us, less than the call takes on the host.
#include "cached_small.cuh"

namespace bdlm {
namespace {

constexpr int kThreads = 32 * (kWarps + 1);

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
// themselves (O = sum p' code, whatever the scales), and the row sum takes
// p' / vs (iv).  In units of exp2(m), O / l is the attention's output and
// m + log2 l its LSE.  The weights carry 2^kSmallShift (iv its inverse).
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
    const float alpha = ex2_approx(st.m[r] - base), less = __fadd_ru(base, -kSmallShift);
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
      s[i][2 * r] = ex2_approx(s[i][2 * r] - less);
      s[i][2 * r + 1] = ex2_approx(s[i][2 * r + 1] - less);
      sum[i / 2] += s[i][2 * r] + s[i][2 * r + 1];
    }
#pragma unroll
    for (int i = 0; i < N8 / 2; ++i) st.l[r] = fmaf(sum[i], iv[i], st.l[r]);
  }
}

// P is rounded to fp16 for cached keys (2^-11, of weights down to 2^-29 of the
// largest); own keys, whose bf16 values would not fit fp16, take it in two bf16
// parts (2^-16), the second what the first's rounding left.  FINE, for an fp32
// output: P goes in two (own keys: three) parts, so that O is off by
// fp32 sums alone; and the products of 16 keys are added to O by the threads: the
// tensor cores cut their sums off instead of rounding them, always towards zero,
// which over 600 products in a row came to 9e-6 of O.
template <int HD>
struct LayS {
  static constexpr int NS = HD == 128 ? 2 : 4;    // slots of K and of V
  static constexpr int kTile = 128 * HD;
  static constexpr int kK = 0, kV = NS * kTile;
  static constexpr int kRed = 2 * NS * kTile;     // [kWarps][16][HD + 4] fp32; before, each warp's Q fragments
  static constexpr int kML = kRed + kWarps * 16 * (HD + 4) * 4;  // [kWarps][16][2]
  static constexpr int kInfo = kML + kWarps * 16 * 2 * 4;
  static constexpr int kBar = (kInfo + NI * (int)sizeof(SInfo) + 15) & ~15;
  static constexpr int kBytes = kBar + 4 * NS * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;    // (aligned to 1024)
};

template <int HD, int MT, bool FINE>
__global__ void __launch_bounds__(kThreads, kSmallCtasPerSm)
    bdlm_cached_small_kernel(const __grid_constant__ CUtensorMap tK8, const __grid_constant__ CUtensorMap tV8,
                             const CachedParams p) {
  using LY = LayS<HD>;
  constexpr int NS = LY::NS;
  constexpr int KH = HD / 64;   // 64-byte halves of a key's codes
  constexpr int VW = HD / 32;   // words of a thread's piece of a value row
  constexpr int KG = kWarps / MT;         // key groups
  constexpr int kStep = 128 / KG / 32;    // 32-key steps of a warp per tile
  constexpr int kRows = 16 * MT;
  extern __shared__ uint8_t smem_raw[];
  const Ring<LY> ring(smem_raw);
  const uint32_t base = ring.base;
  uint8_t* bp = ring.mem;
  float(*red_o)[16][HD + 4] = reinterpret_cast<float(*)[16][HD + 4]>(bp + LY::kRed);
  float(*red_ml)[16][2] = reinterpret_cast<float(*)[16][2]>(bp + LY::kML);
  const SInfo* infos = ring.infos();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) ring.init();
  __syncthreads();
  launch_dependents();
  const Watchdog wd{p.status, p.limit_ns, ring.abort_flag()};
  uint32_t bad = 0;
  const CacheDesc& c = p.c;
  const int cta = blockIdx.x;
  Pieces own = open_pieces(p, cta, bad);
  if (warp == kWarps) {
    load_ring<HD>(ring, tK8, tV8, p, own, wd, bad);
    return;
  }

  // ---------------------------------------------------- the computing warps
  // After a timeout (ok false) they go on without waiting, so that all of them
  // meet at the same barriers; the call reports the timeout.
  const int mt = warp / KG, kg = warp % KG;
  uint32_t slot = 0, ph = 0, tc = 0;
  bool ok = true;
  const int64_t u1 = own.u1;
  UnitPos& pos = own.pos;
  SegInfo& seg = own.seg;
  for (int64_t u = own.u0; u < u1;) {
    int jb, je;
    split_units(seg, p.sp, pos, u, u1, jb, je);
    u += seg.span - pos.j;
    if (je == 0) break;  // only the segment's opening lies here: the next CTA begins it
    // ---- the warp's rows: fp16, each scaled by a power of two that puts its
    // largest magnitude in [2^14, 2^15): exact down to 2^-28 of it
    // (their fragments stay in the warp's part of the reduction buffer: registers
    // go to the keys in flight)
    const uint32_t qs = base + LY::kRed + warp * (16 * (HD + 4) * 4) + lane * 16;
    float cq[2];
    int64_t qoff[2];
    bool live[2];
    uint32_t q[KH * 4][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int fr = pos.rt * kRows + 16 * mt + g + 8 * r, tok = fr / p.sp.group;
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
#pragma unroll
    for (int k = 0; k < KH * 4; ++k) st_shared_v4(qs + k * 512, q[k][0], q[k][1], q[k][2], q[k][3]);
    __syncwarp();
    State<HD> st;
#pragma unroll
    for (int j = 0; j < HD / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[j][i] = 0.f;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;

    // ---- cached keys
    const int kc = min(je, seg.ktiles);
    for (int j = jb; j < kc; ++j, ++tc) {
      const int left = seg.v.len - j * kUnit;  // keys of the tile
      if (ok) ok = mbar_wait(ring.KF(slot), ph, wd, 72);
      const SInfo& si = infos[tc % NI];
      const int gone = si.gone;
      const bool full = left >= kUnit && gone == 0;
#pragma unroll 1
      for (int step = 0; step < kStep; ++step) {
        const int kb = (kg * kStep + step) * 32;  // first key of the step in the tile
        float s[4][4];
        const uint32_t sk = base + LY::kK + slot * LY::kTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int h = 0; h < KH; ++h) {
          uint32_t w[4][4];  // four columns' halves; their sums advance side by side
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = kb + 8 * i + perm<HD>(g);
            const uint4 k4 = lds16(sk + (HD == 128 ? row * 128 + (((4 * h + t) ^ (row & 7)) << 4)
                                                   : row * 64 + ((t ^ ((row >> 1) & 3)) << 4)));
            w[i][0] = k4.x; w[i][1] = k4.y; w[i][2] = k4.z; w[i][3] = k4.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 a = lds16(qs + (4 * h + k) * 512);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16(s[i], a.x, a.y, a.z, a.w, e4m3x2_to_half2(w[i][k]), e4m3x2_to_half2(w[i][k] >> 16));
          }
        }
        float iv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int b = (kb >> 4) + x;
          const float ks = si.s[b], lv = si.lv[b];
          iv[x] = si.iv[b];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[2 * x + i][e] = fmaf(s[2 * x + i][e], cq[e >> 1] * ks, lv);
          if (!full)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (kb + 16 * x + 8 * i + perm<HD>(2 * t + (e & 1)) >= left || ((gone >> b) & 1)) s[2 * x + i][e] = -INFINITY;
        }
        if (step == kStep - 1) {  // K's slot and its info are read
          __syncwarp();
          if (lane == 0) mbar_arrive(ring.KE(slot));
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
        if (step == 0 && ok) ok = mbar_wait(ring.VF(slot), ph, wd, 73);
        const uint32_t sv = base + LY::kV + slot * LY::kTile;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = kb + 16 * x + 8 * (i >> 1) + perm<HD>(2 * t + (i & 1));
            if (HD == 128) {
              const uint4 v = lds16(sv + row * 128 + ((perm<HD>(g) ^ (row & 7)) << 4));
              vw[i][0] = v.x; vw[i][1] = v.y; vw[i][VW - 2] = v.z; vw[i][VW - 1] = v.w;
            } else {
              const uint2 v = lds8(sv + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
              vw[i][0] = v.x; vw[i][1] = v.y;
            }
            if (!full && (row >= left || ((gone >> (row >> 4)) & 1))) {  // stale codes
#pragma unroll
              for (int w = 0; w < VW; ++w) vw[i][w] = 0;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // bytes 2 hf, 2 hf + 1 of word w: column tiles 4 w + 2 hf, + 1
              const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t b0 = e4m3x2_to_half2(lo >> (16 * y)), b1 = e4m3x2_to_half2(hi >> (16 * y));
                float (&o)[4] = st.o[4 * w + 2 * hf + y];
                if (FINE) {
                  float z[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(z, pa[x][0], pa[x][1], pa[x][2], pa[x][3], b0, b1);
                  mma_f16(z, pr[x][0], pr[x][1], pr[x][2], pr[x][3], b0, b1);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[e] += z[e];
                } else {
                  mma_f16(o, pa[x][0], pa[x][1], pa[x][2], pa[x][3], b0, b1);
                }
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.VE(slot));
      if (++slot == NS) slot = 0, ph ^= 1;
    }

    // ---- the rows' own block (bf16), in groups of 16 keys
    static_assert(kSmallRows <= kFoldRows, "the own block follows the last cached unit");
    if (p.sp.local && je == seg.units) {
      for (int key0 = 16 * kg; key0 < seg.v.rows; key0 += 16 * KG) {
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
        const float one[1] = {kSmallUnshift};
        softmax_step<HD, 2>(st, s, one);
        uint32_t pa[4], pr[4], pq[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = s[i >> 1][2 * (i & 1)], b = s[i >> 1][2 * (i & 1) + 1];
          pa[i] = pack_bf16x2(a, b);
          pr[i] = rest_bf16x2(pa[i], a, b);
          if (FINE) pq[i] = rest_bf16x2(pr[i], a - bf_lo(pa[i]), b - bf_hi(pa[i]));
        }
#pragma unroll
        for (int w = 0; w < HD / 64; ++w) {  // 8 columns of the thread's HD / 8 (16 bytes) at a time
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 2 * t + (i & 1) + 8 * (i >> 1);
            v[i] = key < seg.v.rows
                       ? ldg16(static_cast<const __nv_bfloat16*>(p.V) +
                               ((seg.v.row0 + key) * c.Hkv + pos.h) * HD + (HD / 8) * perm<HD>(g) + 8 * w)
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
              // (the weights' rests may be 0 or negative: infinite values meet the first part alone)
              const uint32_t c0 = finite2(b0), c1 = finite2(b1);
              float (&o)[4] = st.o[8 * w + 2 * k + y];
              if (FINE) {
                float z[4] = {0.f, 0.f, 0.f, 0.f};
                mma_bf16(z, pa[0], pa[1], pa[2], pa[3], b0, b1);
                mma_bf16(z, pr[0], pr[1], pr[2], pr[3], c0, c1);
                mma_bf16(z, pq[0], pq[1], pq[2], pq[3], c0, c1);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += z[e];
              } else {
                mma_bf16(o, pa[0], pa[1], pa[2], pa[3], b0, b1);
                mma_bf16(o, pr[0], pr[1], pr[2], pr[3], c0, c1);
              }
            }
          }
        }
      }
    }

    // ---- the warps' states through shared memory, a row tile's key groups joined
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float l = st.l[r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t == 0) {
        red_ml[warp][g + 8 * r][0] = st.m[r];
        red_ml[warp][g + 8 * r][1] = l;
      }
      // tile j, element e: column HD / 8 perm<HD>(2 t + e) + j
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* o = &red_o[warp][g + 8 * r][(HD / 8) * perm<HD>(2 * t + e)];
#pragma unroll
        for (int j = 0; j < HD / 8; j += 4)
          *reinterpret_cast<float4*>(o + j) =
              make_float4(st.o[j][2 * r + e], st.o[j + 1][2 * r + e], st.o[j + 2][2 * r + e], st.o[j + 3][2 * r + e]);
      }
    }
    compute_sync();
    const bool whole = jb == 0 && je == seg.units;
    float* part = p.part + (2 * (int64_t)cta + (jb == 0 ? 1 : 0)) * part_floats(kRows, HD);
#pragma unroll 1
    for (int item = threadIdx.x; item < kRows * 8; item += 32 * kWarps) {
      const int row = item >> 3, c0 = (item & 7) * 4, w0 = (row >> 4) * KG, r = row & 15;
      float M = -INFINITY, w[KG], L = 0.f;
#pragma unroll
      for (int x = 0; x < KG; ++x) M = fmaxf(M, red_ml[w0 + x][r][0]);
#pragma unroll
      for (int x = 0; x < KG; ++x) {
        w[x] = M == -INFINITY ? 0.f : ex2_approx(red_ml[w0 + x][r][0] - M);
        L = fmaf(w[x], red_ml[w0 + x][r][1], L);
      }
      const int fr = pos.rt * kRows + row, tok = fr / p.sp.group;
      if (tok >= seg.v.rows) continue;
      const int head = pos.h * p.sp.group + fr - tok * p.sp.group;
      const int64_t o0 = ((seg.v.row0 + tok) * p.Hq + head) * HD;
      const float inv = whole ? (L != 0.f ? kSmallUnshift / L : 0.f) : kSmallUnshift;
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) {
        const int col = c0 + 32 * k;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < KG; ++x) {
          const float4 b = *reinterpret_cast<const float4*>(&red_o[w0 + x][r][col]);
          a.x = fmaf(w[x], b.x, a.x); a.y = fmaf(w[x], b.y, a.y);
          a.z = fmaf(w[x], b.z, a.z); a.w = fmaf(w[x], b.w, a.w);
        }
        a.x *= inv; a.y *= inv; a.z *= inv; a.w *= inv;
        if (!whole) reinterpret_cast<float4*>(part)[(col >> 2) * kRows + row] = a;
        else if (p.o_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.O) + o0 + col) = a;
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + o0 + col) =
              make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      }
      if ((item & 7) == 0) {
        if (whole) p.LSE[(int64_t)head * p.r.T + seg.v.row0 + tok] = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        else {
          part[kRows * HD + row] = M;
          part[kRows * HD + kRows + row] = L;
        }
      }
    }
    compute_sync();
    if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
  }
}

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

template <int HD, int MT, bool FINE>
static cudaError_t launch(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e = raise_smem(reinterpret_cast<const void*>(bdlm_cached_small_kernel<HD, MT, FINE>),
                                   LayS<HD>::kAlloc, raised);
  if (e != cudaSuccess) return e;
  bdlm_cached_small_kernel<HD, MT, FINE><<<p.G, kThreads, LayS<HD>::kAlloc, st>>>(m.k8, m.v8, p);
  return cudaGetLastError();
}
template <int HD, bool FINE>
static cudaError_t launch_mt(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  return p.sp.tile_rows == 16 ? launch<HD, 1, FINE>(m, p, st) : launch<HD, 2, FINE>(m, p, st);
}

cudaError_t launch_cached_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? (p.o_f32 ? launch_mt<128, true>(m, p, st) : launch_mt<128, false>(m, p, st))
                                     : (p.o_f32 ? launch_mt<64, true>(m, p, st) : launch_mt<64, false>(m, p, st));
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
