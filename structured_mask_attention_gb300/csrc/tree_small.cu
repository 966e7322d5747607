// tree_small.cu -- attention of up to 32 rows of drafted trees over the 8-bit cache: an own
// row sees the own rows that its visibility words name.
//
// As in cached_small.cu the stream of codes is what the call cannot do without, and a warp's
// work on 32 keys (their conversion, two products, a softmax) has to fit under it.  So the
// products take the keys (S^T = K Q^T) and the head dimension (O^T = V^T P^T) as their 16
// rows and the call's rows as their columns, 8 at a time: 5 rows of 4 heads are 24 columns
// where tiles of 16 rows would be 32, each code becomes fp16 once for all of them, and a
// warp's state of 24 rows takes 96 registers.  The accumulators of S^T have a key's rows
// side by side and P^T wants a row's keys: movmatrix turns an 8 x 8 block.  Each of four
// warps has 32 keys of every tile of 128 and all rows.  Rows' references follow the maxima
// in steps (kRowsStep), so that as a rule a group of keys costs comparisons and a vote
// instead of exchanges between the threads that hold a row.
// State and fragments of 24 or 32 rows take 200 registers and more, which ten warps on the
// SM's four register files do not have (three share one: 168 each): the loader gets a
// warpgroup of its own (three of its warps leave) and hands its registers over.
//
// In a graph, warm, 32 sequences, 32 / 8 heads of 128: chains of 5 (24 columns) behind at most
// 2048 / 8192 / 32768 tokens 43 / 82 / 223 us, where tiles of 16 rows, one to each of two warps,
// took 50 / 114 / 363 and both to each warp 53 / 108 / 299; chains of 8 behind 32768 285 (both
// tiles to each warp: 311); one token 198 (cached_small.cu's tiles: 202); fp32 outputs, chains of
// 5, 329 (470); d = 64, chains of 5 behind 16384, 86 (both: 115).
// What bounds chains of 5, 1.28 GB at 5.7 TB/s or 85 % of the measured copy rate: HBM beside the
// instructions' latencies, which two computing warps per scheduler see.  Tried where segments
// were split less evenly (234 us; with all codes from L2 204): the next tile's scores beside
// this one's weights and three slots of K and V, 259; the three slots alone 249 (they take the
// first-level cache); the loop written out twice 293 (instructions no longer fit); 24 / 40 / 64
// registers for the loader instead of 56, 245 / 236 / 237.
#include "cached_small.cuh"

namespace bdlm {
namespace {

constexpr int kRowsThreads = 256;
// NT: tiles of 8 rows.  32 rows of 128 columns: their state alone takes 128 registers.
template <int HD, int NT>
struct RowsRegs {
  static constexpr int kLaunch = 128, kLoad = HD == 128 && NT == 4 ? 24 : 56, kCompute = 2 * kLaunch - kLoad;
};
// A reference may lie this much (log2 units) below a row's maximum, and the weights' shift leaves
// room for it: p' stays below 2^15.9.  (cached_small.cu: the exact maximum and a shift of 15.)
constexpr float kRowsStep = 1.9f, kRowsShift = 14.0f, kRowsUnshift = 1.0f / (1 << (int)kRowsShift);

__device__ __forceinline__ void st_shared_v2(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// Four codes as two pairs of halves.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// The first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// An 8 x 8 matrix of 16-bit values, row g of it in lanes 4 g to 4 g + 3, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// The rows' online-softmax state.  A thread (g = lane / 4, t = lane % 4) has rows 8 n + 2 t
// + e, e = 0, 1: reference, its keys' part of the sum, and the HD / 8 columns of O of its
// piece of a value row; element 2 f + e of o[j][n] is column 2 j + f of them.
template <int HD, int NT>
struct Columns {
  float o[HD / 16][NT][4];
  float m[NT][2], l[NT][2];
};

// Moves the references where a score is kRowsStep and more above one, to the rows'
// maxima; O and l are rescaled then.
template <int HD, int NT, int X>
__device__ __forceinline__ void move_references(Columns<HD, NT>& st, const float (&s)[NT][X][4]) {
  float mx[NT][2];
  bool above = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[n][e] = fmaxf(s[n][0][e], s[n][0][2 + e]);
#pragma unroll
      for (int x = 1; x < X; ++x) mx[n][e] = fmaxf(mx[n][e], fmaxf(s[n][x][e], s[n][x][2 + e]));
      above |= mx[n][e] > __fadd_rd(st.m[n][e], kRowsStep);
    }
  if (!__any_sync(0xffffffffu, above)) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float alpha[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y = mx[n][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
      y = fmaxf(y, st.m[n][e]);
      alpha[e] = ex2_approx(st.m[n][e] - (y == -INFINITY ? 0.f : y));  // no key yet: 0
      st.m[n][e] = y;
      st.l[n][e] *= alpha[e];
    }
#pragma unroll
    for (int j = 0; j < HD / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[j][n][i] *= alpha[i & 1];
  }
}

// Scores -> weights in place, and the row sums.
template <int HD, int NT, int X>
__device__ __forceinline__ void weights(Columns<HD, NT>& st, float (&s)[NT][X][4], const float (&iv)[X]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float less = __fadd_ru(st.m[n][e] == -INFINITY ? 0.f : st.m[n][e], -kRowsShift);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        float &a = s[n][x][e], &b = s[n][x][2 + e];
        a = ex2_approx(a - less);
        b = ex2_approx(b - less);
        st.l[n][e] = fmaf(a + b, iv[x], st.l[n][e]);
      }
    }
}

// (the ring, the fragments and the reduction in as little shared memory as will do: the rest is the first-level cache)
template <int HD>
struct LayR {
  static constexpr int NS = HD == 128 ? 2 : 4;  // slots of K and of V
  static constexpr int kTile = 128 * HD;
  static constexpr int kK = 0, kV = NS * kTile;
  static constexpr int kRed = 2 * NS * kTile;                   // [kWarps][8][64 + 4] fp32; before, the query fragments
  static constexpr int kML = kRed + kWarps * 8 * (64 + 4) * 4;  // [kWarps][32][2]
  static constexpr int kInfo = kML + kWarps * 32 * 2 * 4;
  static constexpr int kBar = (kInfo + NI * (int)sizeof(SInfo) + 15) & ~15;
  static constexpr int kBytes = kBar + 4 * NS * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;  // (aligned to 1024)
  static_assert(kInfo % 8 == 0 && sizeof(SInfo) % 8 == 0, "pairs of a tile's numbers are read at once");
  static_assert(NS + 4 <= NI, "the ring's tiles and a batch have info slots");
  static_assert(kSmallCtasPerSm * (kAlloc + 1024) <= 228 * 1024, "CTAs per SM");
};

template <int HD, int NT, bool FINE>
__global__ void __launch_bounds__(kRowsThreads, kSmallCtasPerSm)
    bdlm_tree_small_kernel(const __grid_constant__ CUtensorMap tK8, const __grid_constant__ CUtensorMap tV8,
                          const CachedParams p) {
  using LY = LayR<HD>;
  constexpr int NS = LY::NS;
  constexpr int KH = HD / 64;   // 64-byte halves of a key's codes
  constexpr int VW = HD / 32;   // words of a thread's piece of a value row
  constexpr int KG = kWarps;    // key groups
  constexpr int kRows = NT <= 2 ? 16 : 32;  // the call's row tile
  constexpr int kFrag = KH * 4 * 512;       // bytes of 16 rows' query fragments
  static_assert((NT + 1) / 2 * kFrag <= LY::kML - LY::kRed, "the fragments fit the reduction buffer");
  extern __shared__ uint8_t smem_raw[];
  const Ring<LY> ring(smem_raw);
  const uint32_t base = ring.base;
  uint8_t* bp = ring.mem;
  float(*red_o)[8][64 + 4] = reinterpret_cast<float(*)[8][64 + 4]>(bp + LY::kRed);
  float(*red_ml)[32][2] = reinterpret_cast<float(*)[32][2]>(bp + LY::kML);
  const SInfo* infos = ring.infos();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) ring.init();
  __syncthreads();
  launch_dependents();
  const Watchdog wd{p.status, p.limit_ns, ring.abort_flag()};
  uint32_t bad = 0;
  const CacheDesc& c = p.c;
  const int cta = blockIdx.x;
  Pieces own = open_pieces(p, cta, bad);
  if (threadIdx.x < 128) {
    setmaxnreg_dec<RowsRegs<HD, NT>::kLoad>();
    if (threadIdx.x >= 32) return;
    load_ring<HD>(ring, tK8, tV8, p, own, wd, bad);
    return;
  }

  // ---------------------------------------------------- the computing warps
  // After a timeout (ok false) they go on without waiting, so that all of them
  // meet at the same barriers; the call reports the timeout.
  setmaxnreg_inc<RowsRegs<HD, NT>::kCompute>();
  const int warp = (int)(threadIdx.x >> 5) - 4;
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
    // ---- the rows, 8 prepared by each warp: fp16, each scaled by a power of two that puts
    // its largest magnitude in [2^14, 2^15): exact down to 2^-28 of it
    auto place = [&](int row, int& tok) -> int {  // the query head; tok: the token of the sequence
      const int fr = pos.rt * kRows + row;
      tok = fr / p.sp.group;
      return pos.h * p.sp.group + fr - tok * p.sp.group;
    };
    auto query = [&](int row) -> const __nv_bfloat16* {  // null: no such row
      int tok;
      const int head = place(row, tok);
      if (tok >= seg.v.rows) return nullptr;
      return static_cast<const __nv_bfloat16*>(p.Q) + ((seg.v.row0 + tok) * p.Hq + head) * HD;
    };
    // the fragments of tiles 2 y, 2 y + 1 lie side by side, a last one alone
    auto frag = [&](int n, int k) -> uint32_t {
      const uint32_t pair = base + LY::kRed + (n >> 1) * kFrag;
      return n == NT - 1 && n % 2 == 0 ? pair + k * 256 + lane * 8 : pair + k * 512 + lane * 16 + (n & 1) * 8;
    };
    if (warp < NT) {
      const __nv_bfloat16* src = query(8 * warp + g);
      uint32_t w[KH][8];
      uint32_t amax = 0;
#pragma unroll
      for (int h = 0; h < KH; ++h) {
        const uint4 y = src ? ldg16(src + 64 * h + 16 * t) : make_uint4(0, 0, 0, 0);
        const uint4 z = src ? ldg16(src + 64 * h + 16 * t + 8) : make_uint4(0, 0, 0, 0);
        w[h][0] = y.x; w[h][1] = y.y; w[h][2] = y.z; w[h][3] = y.w;
        w[h][4] = z.x; w[h][5] = z.y; w[h][6] = z.z; w[h][7] = z.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, max(w[h][i] & 0x7fffu, (w[h][i] >> 16) & 0x7fffu));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = 14 + 127 - (int)(amax >> 7);  // bf16 exponent field
      if (amax >= 0x7f80u || amax == 0) e = 0;
      e = min(e, 126);
      const float f = __uint_as_float((uint32_t)(e + 127) << 23);
      if (t == 0) red_ml[0][8 * warp + g][0] = p.sl2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int h = 0; h < KH; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v2(frag(warp, 4 * h + i), pack_half2(bf_lo(w[h][2 * i]) * f, bf_hi(w[h][2 * i]) * f),
                       pack_half2(bf_lo(w[h][2 * i + 1]) * f, bf_hi(w[h][2 * i + 1]) * f));
    }
    compute_sync();
    float cq[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) cq[n][e] = red_ml[0][8 * n + 2 * t + e][0];
    Columns<HD, NT> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < HD / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[j][n][i] = 0.f;
      st.m[n][0] = st.m[n][1] = -INFINITY;
      st.l[n][0] = st.l[n][1] = 0.f;
    }

    // ---- cached keys, 32 of each tile to a warp
    const int kc = min(je, seg.ktiles), kb = warp * 32;
#pragma unroll 1
    for (int j = jb; j < kc; ++j, ++tc) {
      const int left = seg.v.len - j * kUnit;  // keys of the tile
      if (ok) ok = mbar_wait(ring.KF(slot), ph, wd, 72);
      const uint32_t sk = base + LY::kK + slot * LY::kTile, sv = base + LY::kV + slot * LY::kTile;
      float s[NT][2][4];
#pragma unroll
      for (int h = 0; h < KH; ++h) {
        uint32_t w[4][4];  // four keys' halves; their sums advance side by side
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = kb + 8 * i + perm<HD>(g);
          const uint4 k4 = lds16(sk + (HD == 128 ? row * 128 + (((4 * h + t) ^ (row & 7)) << 4)
                                                 : row * 64 + ((t ^ ((row >> 1) & 3)) << 4)));
          w[i][0] = k4.x; w[i][1] = k4.y; w[i][2] = k4.z; w[i][3] = k4.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t b[NT][2];
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            if (n + 1 < NT) {
              const uint4 v = lds16(frag(n, 4 * h + k));
              b[n][0] = v.x; b[n][1] = v.y; b[n + 1][0] = v.z; b[n + 1][1] = v.w;
            } else {
              const uint2 v = lds8(frag(n, 4 * h + k));
              b[n][0] = v.x; b[n][1] = v.y;
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_half2(w[2 * x][k], a0, a2);
            e4m3x4_to_half2(w[2 * x + 1][k], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (h == 0 && k == 0) mma_f16_first(s[n][x], a0, a1, a2, a3, b[n][0], b[n][1]);
              else mma_f16(s[n][x], a0, a1, a2, a3, b[n][0], b[n][1]);
            }
          }
        }
      }
      const SInfo& si = infos[tc % NI];
      const unsigned gone = (unsigned)si.gone;
      const bool full = left >= kUnit && gone == 0;
      const int b16 = kb >> 4;
      const float2 ks = *reinterpret_cast<const float2*>(&si.s[b16]);
      const float2 lv = *reinterpret_cast<const float2*>(&si.lv[b16]);
      const float2 iv2 = *reinterpret_cast<const float2*>(&si.iv[b16]);
      constexpr float up = 1 << (int)(kSmallShift - kRowsShift);
      const float iv[2] = {iv2.x * up, iv2.y * up};
      __syncwarp();  // K's slot and its info are read
      if (lane == 0) mbar_arrive(ring.KE(slot));
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][0][e] = fmaf(s[n][0][e], cq[n][e & 1] * ks.x, lv.x);
          s[n][1][e] = fmaf(s[n][1][e], cq[n][e & 1] * ks.y, lv.y);
        }
      if (!full) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            if (kb + 16 * x + 8 * f + perm<HD>(g) >= left || ((gone >> (b16 + x)) & 1))
#pragma unroll
              for (int n = 0; n < NT; ++n) s[n][x][2 * f] = s[n][x][2 * f + 1] = -INFINITY;
      }
      move_references<HD, NT, 2>(st, s);
      weights<HD, NT, 2>(st, s, iv);
      uint32_t pa[NT][2][2], pr[NT][2][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // (keys as rows -> keys as the contraction)
            const float a = s[n][x][2 * i], b = s[n][x][2 * i + 1];
            const uint32_t w = pack_half2(a, b);
            pa[n][x][i] = transpose8(w);
            if (FINE) pr[n][x][i] = transpose8(rest_half2(w, a, b));
          }
      if (ok) ok = mbar_wait(ring.VF(slot), ph, wd, 73);
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
        }
        if (!full) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = kb + 16 * x + 8 * (i >> 1) + perm<HD>(2 * t + (i & 1));
            if (row < left && !((gone >> (row >> 4)) & 1)) continue;
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[i][w] = 0;  // stale codes
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // bytes 2 hf, 2 hf + 1 of word w: columns 4 w + 2 hf, + 1
            const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], hf ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(vw[2][w], vw[3][w], hf ? 0x7362 : 0x5140);
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_half2(lo, a0, a1);
            e4m3x4_to_half2(hi, a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float (&o)[4] = st.o[2 * w + hf][n];
              if (FINE) {
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(sum, a0, a1, a2, a3, pa[n][x][0], pa[n][x][1]);
                mma_f16(sum, a0, a1, a2, a3, pr[n][x][0], pr[n][x][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += sum[e];
              } else {
                mma_f16(o, a0, a1, a2, a3, pa[n][x][0], pa[n][x][1]);
              }
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ring.VE(slot));
      if (++slot == NS) slot = 0, ph ^= 1;
    }

    // ---- the rows' own block (bf16), in groups of 16 keys
    if (p.sp.local && je == seg.units) {
#pragma unroll 1
      for (int key0 = 16 * warp; key0 < seg.v.rows; key0 += 16 * KG) {
        float s[NT][1][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0][0] = s[n][0][1] = s[n][0][2] = s[n][0][3] = 0.f;
#pragma unroll
        for (int h = 0; h < HD / 32; ++h) {
          uint4 a[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = key0 + 8 * i + g;
            a[i] = key < seg.v.rows
                       ? ldg16(static_cast<const __nv_bfloat16*>(p.K) +
                               ((seg.v.row0 + key) * c.Hkv + pos.h) * HD + 32 * h + 8 * t)
                       : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const __nv_bfloat16* src = query(8 * n + g);
            const uint4 b = src ? ldg16(src + 32 * h + 8 * t) : make_uint4(0, 0, 0, 0);
            mma_bf16(s[n][0], a[0].x, a[1].x, a[0].y, a[1].y, b.x, b.y);
            mma_bf16(s[n][0], a[0].z, a[1].z, a[0].w, a[1].w, b.z, b.w);
          }
        }
        uint32_t sees[NT][2];  // the bits of these 16 keys
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int tok;
            place(8 * n + 2 * t + e, tok);
            const bool row = tok < seg.v.rows;
            sees[n][e] = row ? __ldg(p.vis + (seg.v.row0 + tok) * p.words + (key0 >> 5)) >> (key0 & 31) : 0;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int k = 8 * f + g;
              float& x = s[n][0][2 * f + e];
              x = key0 + k < seg.v.rows && (sees[n][e] >> k) & 1 ? x * p.sl2 : -INFINITY;
            }
          }
        const float one[1] = {kRowsUnshift};
        move_references<HD, NT, 1>(st, s);
        weights<HD, NT, 1>(st, s, one);
        uint32_t b0[NT][2], b1[NT][2], b2[NT][2];  // the weights in two or three bf16 parts
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = s[n][0][2 * i], b = s[n][0][2 * i + 1];
            const uint32_t w0 = pack_bf16x2(a, b), w1 = rest_bf16x2(w0, a, b);
            b0[n][i] = transpose8(w0);
            b1[n][i] = transpose8(w1);
            if (FINE) b2[n][i] = transpose8(rest_bf16x2(w1, a - bf_lo(w0), b - bf_hi(w0)));
          }
        bool odd = false;  // a value that is not finite
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
            // (rows that do not see an infinite value or NaN must not meet it)
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
              const uint32_t all = i < 2 ? __byte_perm(x0[k], x1[k], sel) : __byte_perm(y0[k], y1[k], sel);
              a[i] = finite2(all);
              odd |= a[i] != all;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float (&o)[4] = st.o[4 * w + k][n];
              if (FINE) {
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                mma_bf16(sum, a[0], a[1], a[2], a[3], b0[n][0], b0[n][1]);
                mma_bf16(sum, a[0], a[1], a[2], a[3], b1[n][0], b1[n][1]);
                mma_bf16(sum, a[0], a[1], a[2], a[3], b2[n][0], b2[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += sum[e];
              } else {
                mma_bf16(o, a[0], a[1], a[2], a[3], b0[n][0], b0[n][1]);
                mma_bf16(o, a[0], a[1], a[2], a[3], b1[n][0], b1[n][1]);
              }
            }
          }
        }
        if (__any_sync(0xffffffffu, odd)) {  // values that are not finite, to the rows that see them
#pragma unroll 1
          for (int k = 0; k < min(16, seg.v.rows - key0); ++k) {
            const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(p.V) +
                                     ((seg.v.row0 + key0 + k) * c.Hkv + pos.h) * HD + (HD / 8) * perm<HD>(g);
#pragma unroll
            for (int j = 0; j < HD / 8; ++j) {
              const float x = __bfloat162float(V[j]);
              if (isfinite(x)) continue;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if ((sees[n][e] >> k) & 1) st.o[j >> 1][n][2 * (j & 1) + e] += x;
            }
          }
        }
      }
    }

    // ---- the warps' states through shared memory, a row tile's key groups joined
    const bool whole = jb == 0 && je == seg.units;
    float* part = p.part + (2 * (int64_t)cta + (jb == 0 ? 1 : 0)) * part_floats(kRows, HD);
    compute_sync();  // (the query fragments are read)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[n][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (g == 0) {
          red_ml[warp][8 * n + 2 * t + e][0] = st.m[n][e];
          red_ml[warp][8 * n + 2 * t + e][1] = l;
        }
      }
    // 8 rows, and 8 of each piece's columns, at a time: a thread joins four columns of a row
    const int r = (warp * 32 + lane) >> 4, c4 = lane & 15;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int half = 0; half < HD / 64; ++half) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* o = &red_o[warp][2 * t + e][8 * perm<HD>(g)];
#pragma unroll
          for (int y = 0; y < 4; y += 2) {
            const float(&a)[4] = st.o[4 * half + y][n], (&b)[4] = st.o[4 * half + y + 1][n];
            *reinterpret_cast<float4*>(o + 2 * y) = make_float4(a[e], a[2 + e], b[e], b[2 + e]);
          }
        }
        compute_sync();
        const int row = 8 * n + r;
        int tok;
        const int head = place(row, tok);
        if (tok < seg.v.rows) {
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int x = 0; x < KG; ++x) M = fmaxf(M, red_ml[x][row][0]);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < KG; ++x) {
            const float w = M == -INFINITY ? 0.f : ex2_approx(red_ml[x][row][0] - M);
            L = fmaf(w, red_ml[x][row][1], L);
            const float4 b = *reinterpret_cast<const float4*>(&red_o[x][r][4 * c4]);
            a.x = fmaf(w, b.x, a.x); a.y = fmaf(w, b.y, a.y);
            a.z = fmaf(w, b.z, a.z); a.w = fmaf(w, b.w, a.w);
          }
          const float inv = whole ? (L != 0.f ? kRowsUnshift / L : 0.f) : kRowsUnshift;
          a.x *= inv; a.y *= inv; a.z *= inv; a.w *= inv;
          const int col = (HD / 8) * (c4 >> 1) + 8 * half + 4 * (c4 & 1);
          const int64_t at = ((seg.v.row0 + tok) * p.Hq + head) * HD + col;
          if (!whole) reinterpret_cast<float4*>(part)[(col >> 2) * kRows + row] = a;
          else if (p.o_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.O) + at) = a;
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.O) + at) =
                make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
          if (half == 0 && c4 == 0) {
            if (whole) {
              p.LSE[(int64_t)head * p.r.T + seg.v.row0 + tok] =
                  L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
            } else {
              part[kRows * HD + row] = M;
              part[kRows * HD + kRows + row] = L;
            }
          }
        }
        compute_sync();
      }
    }
    if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
  }
}

template <int HD, int NT, bool FINE>
cudaError_t launch(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  auto k = bdlm_tree_small_kernel<HD, NT, FINE>;
  // the register split needs the block's full allotment: refuse to launch otherwise
  static const cudaError_t ready = [&] {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, k);
    if (e != cudaSuccess) return e;
    return fa.numRegs == RowsRegs<HD, NT>::kLaunch ? cudaSuccess : cudaErrorInvalidConfiguration;
  }();
  if (ready != cudaSuccess) return ready;
  const cudaError_t e = raise_smem(reinterpret_cast<const void*>(k), LayR<HD>::kAlloc, raised);
  if (e != cudaSuccess) return e;
  k<<<p.G, kRowsThreads, LayR<HD>::kAlloc, st>>>(m.k8, m.v8, p);
  return cudaGetLastError();
}

}  // namespace

template <int HD, bool FINE>
static cudaError_t launch_rows(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  const int rows = p.sp.group * p.r.max_rows;  // (p.sp.tile_rows: 16 for up to 16 of them, else 32)
  return rows <= 8    ? launch<HD, 1, FINE>(m, p, st)
         : rows <= 16 ? launch<HD, 2, FINE>(m, p, st)
         : rows <= 24 ? launch<HD, 3, FINE>(m, p, st)
                      : launch<HD, 4, FINE>(m, p, st);
}

cudaError_t launch_tree_small(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? (p.o_f32 ? launch_rows<128, true>(m, p, st) : launch_rows<128, false>(m, p, st))
                                     : (p.o_f32 ? launch_rows<64, true>(m, p, st) : launch_rows<64, false>(m, p, st));
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
