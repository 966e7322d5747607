// cached_small.cuh -- attention of up to 32 rows over the 8-bit cache on mma.sync
// tiles.  TREE: an own row sees the own rows that its visibility words name
// (cached_small.cu has the instances without, tree_small.cu those with).
//
// One token of a sequence, or a short block, gives Hq / Hkv rows per token and
// KV head, a handful against thousands of keys: the stream of codes bounds the
// call, and a tcgen05 tile of 128 rows would be mostly padding.  A CTA of four
// warps takes 16 or 32 rows (RT 16-row tiles to a warp, RG groups of them); its warps
// are RG row groups by 4 / RG groups of keys.  A fifth warp keeps a ring of K and V tiles of 128 keys
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
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cached_attn.h"
#include "kernels.h"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kWarps = 4;  // warps that compute; one more loads
// With two row tiles to a warp (RT = 2) its state takes 200 registers and more, and of ten
// warps on the SM's four register files three share one: 168 each.  So the loader
// gets a warpgroup of its own (three of its warps leave) and hands its registers over.
template <int RT>
struct Roles {
  static constexpr bool kSplit = RT > 1;
  static constexpr int kThreads = kSplit ? 256 : 32 * (kWarps + 1);
  static constexpr int kFirst = kSplit ? 4 : 0;  // the first computing warp
  static constexpr int kLoader = kSplit ? 0 : kWarps;
  static constexpr int kRegs = 128, kRegsLoad = 24, kRegsCompute = 232;  // (split)
  static_assert(128 * (kRegsLoad + kRegsCompute) <= 256 * kRegs, "register split exceeds the block");
};

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
//
// P is rounded to fp16 for cached keys (2^-11, of weights down to 2^-29 of the
// largest); own keys, whose bf16 values would not fit fp16, take it in two bf16
// parts (2^-16), the second what the first's rounding left.  FINE, for an fp32
// output: P goes in two (own keys: three) parts, so that O is off by
// fp32 sums alone; and the products of 16 keys are added to O by the threads: the
// tensor cores cut their sums off instead of rounding them, always towards zero,
// which over 600 products in a row came to 9e-6 of O.
struct SInfo {  // of each 16 keys of a tile: K's scale, log2 and 2^-shift times the inverse of V's (scale 1 without a page)
  float s[8], lv[8], iv[8];
  int gone;     // bit x: no page
};

constexpr int NI = 16;  // info slots: the tiles in the ring, and a batch of four ahead

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

template <int HD, int RT, int RG, bool FINE, bool TREE>
__global__ void __launch_bounds__(Roles<RT>::kThreads, kSmallCtasPerSm)
    bdlm_cached_small_kernel(const __grid_constant__ CUtensorMap tK8, const __grid_constant__ CUtensorMap tV8,
                             const CachedParams p) {
  using LY = LayS<HD>;
  constexpr int NS = LY::NS;
  constexpr int KH = HD / 64;   // 64-byte halves of a key's codes
  constexpr int VW = HD / 32;   // words of a thread's piece of a value row
  constexpr int KG = kWarps / RG;         // key groups
  constexpr int kStep = 128 / KG / 32;    // 32-key steps of a warp per tile
  constexpr int kRows = 16 * RT * RG;
  constexpr int kFrag = KH * 4 * 512;     // bytes of a row tile's query fragments
  static_assert(RT * kFrag <= 16 * (HD + 4) * 4, "the fragments fit a warp's part of the reduction buffer");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  float(*red_o)[16][HD + 4] = reinterpret_cast<float(*)[16][HD + 4]>(bp + LY::kRed);
  float(*red_ml)[16][2] = reinterpret_cast<float(*)[16][2]>(bp + LY::kML);
  SInfo* infos = reinterpret_cast<SInfo*>(bp + LY::kInfo);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + LY::kBar + 4 * NS * 8);
  auto KF = [&](uint32_t i) -> uint32_t { return base + LY::kBar + 8 * i; };
  auto KE = [&](uint32_t i) -> uint32_t { return base + LY::kBar + 8 * (NS + i); };
  auto VF = [&](uint32_t i) -> uint32_t { return base + LY::kBar + 8 * (2 * NS + i); };
  auto VE = [&](uint32_t i) -> uint32_t { return base + LY::kBar + 8 * (3 * NS + i); };
  using R = Roles<RT>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < NS; ++i) {
      mbar_init(KF(i), 1);
      mbar_init(VF(i), 1);
      mbar_init(KE(i), kWarps);
      mbar_init(VE(i), kWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  launch_dependents();
  const Watchdog wd{p.status, p.limit_ns, abort_flag};
  uint32_t bad = 0;
  const CacheDesc& c = p.c;
  // every warp walks the CTA's pieces on its own
  const int cta = blockIdx.x;
  int64_t u0 = 0, u1 = 0;
  UnitPos pos{0, 0, 0, 0};
  SegInfo seg;
  if (p.whole) {  // CTA per segment: (sequence, KV head, row tile), p.whole row tiles for each
    pos.rt = cta % p.whole;
    pos.h = cta / p.whole % c.Hkv;
    pos.s = cta / p.whole / c.Hkv;
    seg = seg_info(c, p.r, p.sp, pos.s, bad);
    u1 = pos.rt < seg.rtiles ? seg.span : 0;
  } else {
    const SplitOpen o = split_open(c, p.r, p.sp, p.G, cta, bad);
    u0 = o.u0;
    u1 = o.u1;
    pos = o.pos;
    seg = o.seg;
  }

  if (R::kSplit ? threadIdx.x < 128 : (int)(threadIdx.x >> 5) == R::kLoader) {
    if (R::kSplit) {
      setmaxnreg_dec<R::kRegsLoad>();
      if (threadIdx.x >= 32) return;
    }
    // -------------------------------------------------- loader
    uint32_t slot = 0, ph = 1, tc = 0;
    const uint32_t page_bytes = (uint32_t)(c.page * HD), page_groups = first_groups(c.page);
    bool ok = true;
    for (int64_t u = u0; ok && u < u1;) {
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
        SInfo& si = infos[(tc + grp) % NI];
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
          ok = mbar_wait(KE(slot), ph, wd, 70);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 8 * a) {
            if (bytes) mbar_arrive_expect_tx(KF(slot), bytes);
            else mbar_arrive(KF(slot));
          }
          __syncwarp();
          const bool mine = grp == a && loads;  // the lane of a page's first keys loads it
          if (mine) tma_load_3d(base + LY::kK + slot * LY::kTile + 16 * x * HD, &tK8, KF(slot), 0, 0, blk);
          ok = mbar_wait(VE(slot), ph, wd, 71);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 8 * a) {
            if (bytes) mbar_arrive_expect_tx(VF(slot), bytes);
            else mbar_arrive(VF(slot));
          }
          __syncwarp();
          if (mine) tma_load_3d(base + LY::kV + slot * LY::kTile + 16 * x * HD, &tV8, VF(slot), 0, 0, blk);
          if (++slot == NS) slot = 0, ph ^= 1;
        }
        id = id1; raw1 = raw2; sk = sk1; sv = sv1;
      }
      if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
    }
    if (bad) atomicOr(p.status + kContentsWord, bad);
    // (copies that a timeout left in flight land before the CTA's shared memory is given up)
    if (*abort_flag) drain_after_abort(200);
    return;
  }

  // ---------------------------------------------------- the computing warps
  // After a timeout (ok false) they go on without waiting, so that all of them
  // meet at the same barriers; the call reports the timeout.
  if (R::kSplit) setmaxnreg_inc<R::kRegsCompute>();
  const int warp = (int)(threadIdx.x >> 5) - R::kFirst;
  const int rg = warp / KG, kg = warp % KG;
  auto perm = [](int x) { return HD == 128 ? (x >> 1) | ((x & 1) << 2) : x; };
  uint32_t slot = 0, ph = 0, tc = 0;
  bool ok = true;
  for (int64_t u = u0; u < u1;) {
    int jb, je;
    split_units(seg, p.sp, pos, u, u1, jb, je);
    u += seg.span - pos.j;
    if (je == 0) break;  // only the segment's opening lies here: the next CTA begins it
    // ---- the warp's rows: fp16, each scaled by a power of two that puts its
    // largest magnitude in [2^14, 2^15): exact down to 2^-28 of it
    // (their fragments stay in the warp's part of the reduction buffer: registers
    // go to the keys in flight)
    const uint32_t qs = base + LY::kRed + warp * (16 * (HD + 4) * 4) + lane * 16;
    // row r (of two: g, g + 8) of the warp's row tile x, as a token of the sequence and a query head
    auto token = [&](int x, int r) { return (pos.rt * kRows + 16 * (RT * rg + x) + g + 8 * r) / p.sp.group; };
    auto query = [&](int x, int r) -> const __nv_bfloat16* {  // null: no such row
      const int fr = pos.rt * kRows + 16 * (RT * rg + x) + g + 8 * r, tok = fr / p.sp.group;
      if (tok >= seg.v.rows) return nullptr;
      const int head = pos.h * p.sp.group + fr - tok * p.sp.group;
      return static_cast<const __nv_bfloat16*>(p.Q) + ((seg.v.row0 + tok) * p.Hq + head) * HD;
    };
    float cq[RT][2];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      uint32_t q[KH * 4][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const __nv_bfloat16* src = query(x, r);
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
        cq[x][r] = p.sl2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int h = 0; h < KH; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            q[4 * h + i][r] = pack_half2(bf_lo(w[h][2 * i]) * f, bf_hi(w[h][2 * i]) * f);
            q[4 * h + i][2 + r] = pack_half2(bf_lo(w[h][2 * i + 1]) * f, bf_hi(w[h][2 * i + 1]) * f);
          }
      }
#pragma unroll
      for (int k = 0; k < KH * 4; ++k) st_shared_v4(qs + x * kFrag + k * 512, q[k][0], q[k][1], q[k][2], q[k][3]);
    }
    __syncwarp();
    State<HD> st[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
#pragma unroll
      for (int j = 0; j < HD / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st[x].o[j][i] = 0.f;
      st[x].m[0] = st[x].m[1] = -INFINITY;
      st[x].l[0] = st[x].l[1] = 0.f;
    }

    // ---- cached keys
    const int kc = min(je, seg.ktiles);
    for (int j = jb; j < kc; ++j, ++tc) {
      const int left = seg.v.len - j * kUnit;  // keys of the tile
      if (ok) ok = mbar_wait(KF(slot), ph, wd, 72);
      const SInfo& si = infos[tc % NI];
      const int gone = si.gone;
      const bool full = left >= kUnit && gone == 0;
#pragma unroll 1
      for (int step = 0; step < kStep; ++step) {
        const int kb = (kg * kStep + step) * 32;  // first key of the step in the tile
        float s[RT][4][4];
        const uint32_t sk = base + LY::kK + slot * LY::kTile;
#pragma unroll
        for (int y = 0; y < RT; ++y)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[y][i][0] = s[y][i][1] = s[y][i][2] = s[y][i][3] = 0.f;
#pragma unroll
        for (int h = 0; h < KH; ++h) {
          uint32_t w[4][4];  // four columns' halves; their sums advance side by side
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = kb + 8 * i + perm(g);
            const uint4 k4 = lds16(sk + (HD == 128 ? row * 128 + (((4 * h + t) ^ (row & 7)) << 4)
                                                   : row * 64 + ((t ^ ((row >> 1) & 3)) << 4)));
            w[i][0] = k4.x; w[i][1] = k4.y; w[i][2] = k4.z; w[i][3] = k4.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 a[RT];
#pragma unroll
            for (int y = 0; y < RT; ++y) a[y] = lds16(qs + y * kFrag + (4 * h + k) * 512);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = e4m3x2_to_half2(w[i][k]), b1 = e4m3x2_to_half2(w[i][k] >> 16);
#pragma unroll
              for (int y = 0; y < RT; ++y) mma_f16(s[y][i], a[y].x, a[y].y, a[y].z, a[y].w, b0, b1);
            }
          }
        }
        float iv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int b = (kb >> 4) + x;
          const float ks = si.s[b], lv = si.lv[b];
          iv[x] = si.iv[b];
#pragma unroll
          for (int y = 0; y < RT; ++y)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[y][2 * x + i][e] = fmaf(s[y][2 * x + i][e], cq[y][e >> 1] * ks, lv);
          if (!full)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (kb + 16 * x + 8 * i + perm(2 * t + (e & 1)) >= left || ((gone >> b) & 1))
#pragma unroll
                  for (int y = 0; y < RT; ++y) s[y][2 * x + i][e] = -INFINITY;
        }
        if (step == kStep - 1) {  // K's slot and its info are read
          __syncwarp();
          if (lane == 0) mbar_arrive(KE(slot));
        }
        uint32_t pa[RT][2][4], pr[RT][2][4];
#pragma unroll
        for (int y = 0; y < RT; ++y) {
          softmax_step<HD, 4>(st[y], s[y], iv);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = s[y][2 * x + (i >> 1)][2 * (i & 1)], b = s[y][2 * x + (i >> 1)][2 * (i & 1) + 1];
              pa[y][x][i] = pack_half2(a, b);
              if (FINE) pr[y][x][i] = rest_half2(pa[y][x][i], a, b);
            }
        }
        if (step == 0 && ok) ok = mbar_wait(VF(slot), ph, wd, 73);
        const uint32_t sv = base + LY::kV + slot * LY::kTile;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = kb + 16 * x + 8 * (i >> 1) + perm(2 * t + (i & 1));
            if (HD == 128) {
              const uint4 v = lds16(sv + row * 128 + ((perm(g) ^ (row & 7)) << 4));
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
#pragma unroll
                for (int z = 0; z < RT; ++z) {
                  float (&o)[4] = st[z].o[4 * w + 2 * hf + y];
                  const uint32_t(&a)[4] = pa[z][x];
                  if (FINE) {
                    const uint32_t(&r)[4] = pr[z][x];
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(sum, a[0], a[1], a[2], a[3], b0, b1);
                    mma_f16(sum, r[0], r[1], r[2], r[3], b0, b1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] += sum[e];
                  } else {
                    mma_f16(o, a[0], a[1], a[2], a[3], b0, b1);
                  }
                }
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(VE(slot));
      if (++slot == NS) slot = 0, ph ^= 1;
    }

    // ---- the rows' own block (bf16), in groups of 16 keys
    if (p.sp.local && je == seg.units) {
#pragma unroll 1
      for (int key0 = 16 * kg; key0 < seg.v.rows; key0 += 16 * KG) {
        float s[RT][2][4];
#pragma unroll
        for (int y = 0; y < RT; ++y)
#pragma unroll
          for (int i = 0; i < 2; ++i) s[y][i][0] = s[y][i][1] = s[y][i][2] = s[y][i][3] = 0.f;
#pragma unroll
        for (int h = 0; h < HD / 32; ++h) {
          uint4 b[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = key0 + 8 * i + g;
            b[i] = key < seg.v.rows
                       ? ldg16(static_cast<const __nv_bfloat16*>(p.K) +
                               ((seg.v.row0 + key) * c.Hkv + pos.h) * HD + 32 * h + 8 * t)
                       : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int y = 0; y < RT; ++y) {
            uint4 a[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const __nv_bfloat16* src = query(y, r);
              a[r] = src ? ldg16(src + 32 * h + 8 * t) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma_bf16(s[y][i], a[0].x, a[1].x, a[0].y, a[1].y, b[i].x, b[i].y);
              mma_bf16(s[y][i], a[0].z, a[1].z, a[0].w, a[1].w, b[i].z, b[i].w);
            }
          }
        }
        uint32_t sees[RT][2];  // (TREE) the bits of these 16 keys
        uint32_t pa[RT][4], pr[RT][4], pq[RT][4];
#pragma unroll
        for (int y = 0; y < RT; ++y) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int tok = TREE ? token(y, r) : 0;
            sees[y][r] = TREE && tok < seg.v.rows
                             ? __ldg(p.vis + (seg.v.row0 + tok) * p.words + (key0 >> 5)) >> (key0 & 31)
                             : 0;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = 8 * i + 2 * t + (e & 1);
              s[y][i][e] = key0 + k < seg.v.rows && (!TREE || (sees[y][e >> 1] >> k) & 1) ? s[y][i][e] * p.sl2 : -INFINITY;
            }
          const float one[1] = {kSmallUnshift};
          softmax_step<HD, 2>(st[y], s[y], one);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = s[y][i >> 1][2 * (i & 1)], b = s[y][i >> 1][2 * (i & 1) + 1];
            pa[y][i] = pack_bf16x2(a, b);
            pr[y][i] = rest_bf16x2(pa[y][i], a, b);
            if (FINE) pq[y][i] = rest_bf16x2(pr[y][i], a - bf_lo(pa[y][i]), b - bf_hi(pa[y][i]));
          }
        }
        bool odd = false;  // (TREE) a value that is not finite
#pragma unroll
        for (int w = 0; w < HD / 64; ++w) {  // 8 columns of the thread's HD / 8 (16 bytes) at a time
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 2 * t + (i & 1) + 8 * (i >> 1);
            v[i] = key < seg.v.rows
                       ? ldg16(static_cast<const __nv_bfloat16*>(p.V) +
                               ((seg.v.row0 + key) * c.Hkv + pos.h) * HD + (HD / 8) * perm(g) + 8 * w)
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
              // (the weights' rests may be 0 or negative: infinite values meet the first part alone;
              // TREE: rows that do not see them must not meet them either)
              const uint32_t c0 = finite2(b0), c1 = finite2(b1), d0 = TREE ? c0 : b0, d1 = TREE ? c1 : b1;
              if (TREE) odd |= c0 != b0 || c1 != b1;
#pragma unroll
              for (int z = 0; z < RT; ++z) {
                float (&o)[4] = st[z].o[8 * w + 2 * k + y];
                if (FINE) {
                  float sum[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_bf16(sum, pa[z][0], pa[z][1], pa[z][2], pa[z][3], d0, d1);
                  mma_bf16(sum, pr[z][0], pr[z][1], pr[z][2], pr[z][3], c0, c1);
                  mma_bf16(sum, pq[z][0], pq[z][1], pq[z][2], pq[z][3], c0, c1);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[e] += sum[e];
                } else {
                  mma_bf16(o, pa[z][0], pa[z][1], pa[z][2], pa[z][3], d0, d1);
                  mma_bf16(o, pr[z][0], pr[z][1], pr[z][2], pr[z][3], c0, c1);
                }
              }
            }
          }
        }
        if (TREE && __any_sync(0xffffffffu, odd)) {  // values that are not finite, to the rows that see them
#pragma unroll 1
          for (int k = 0; k < min(16, seg.v.rows - key0); ++k) {
            const __nv_bfloat16* V =
                static_cast<const __nv_bfloat16*>(p.V) + ((seg.v.row0 + key0 + k) * c.Hkv + pos.h) * HD;
#pragma unroll
            for (int j = 0; j < HD / 8; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = __bfloat162float(V[(HD / 8) * perm(2 * t + e) + j]);
                if (isfinite(x)) continue;
#pragma unroll
                for (int z = 0; z < RT; ++z) {
                  if ((sees[z][0] >> k) & 1) st[z].o[j][e] += x;
                  if ((sees[z][1] >> k) & 1) st[z].o[j][2 + e] += x;
                }
              }
          }
        }
      }
    }

    // ---- the warps' states through shared memory, a row tile's key groups joined
    const bool whole = jb == 0 && je == seg.units;
    float* part = p.part + (2 * (int64_t)cta + (jb == 0 ? 1 : 0)) * part_floats(kRows, HD);
#pragma unroll
    for (int y = 0; y < RT; ++y) {  // (the warps' tiles y of their row groups)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = st[y].l[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) {
          red_ml[warp][g + 8 * r][0] = st[y].m[r];
          red_ml[warp][g + 8 * r][1] = l;
        }
        // tile j, element e: column HD / 8 perm(2 t + e) + j
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* o = &red_o[warp][g + 8 * r][(HD / 8) * perm(2 * t + e)];
#pragma unroll
          for (int j = 0; j < HD / 8; j += 4)
            *reinterpret_cast<float4*>(o + j) = make_float4(st[y].o[j][2 * r + e], st[y].o[j + 1][2 * r + e],
                                                            st[y].o[j + 2][2 * r + e], st[y].o[j + 3][2 * r + e]);
        }
      }
      compute_sync();
#pragma unroll 1
      for (int item = 32 * warp + lane; item < RG * 16 * 8; item += 32 * kWarps) {
        const int r = (item >> 3) & 15, c0 = (item & 7) * 4, w0 = (item >> 7) * KG;
        const int row = 16 * (RT * (item >> 7) + y) + r;  // of the CTA's rows
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
          if (whole)
            p.LSE[(int64_t)head * p.r.T + seg.v.row0 + tok] = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
          else {
            part[kRows * HD + row] = M;
            part[kRows * HD + kRows + row] = L;
          }
        }
      }
      compute_sync();
    }
    if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
  }
}

template <int HD, int RT, int RG, bool FINE, bool TREE>
cudaError_t launch(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  auto k = bdlm_cached_small_kernel<HD, RT, RG, FINE, TREE>;
  if (Roles<RT>::kSplit) {
    // the register split needs the block's full allotment: refuse to launch otherwise
    static const cudaError_t ready = [&] {
      cudaFuncAttributes fa;
      const cudaError_t e = cudaFuncGetAttributes(&fa, k);
      if (e != cudaSuccess) return e;
      return fa.numRegs == Roles<RT>::kRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
    }();
    if (ready != cudaSuccess) return ready;
  }
  const cudaError_t e = raise_smem(reinterpret_cast<const void*>(k), LayS<HD>::kAlloc, raised);
  if (e != cudaSuccess) return e;
  k<<<p.G, Roles<RT>::kThreads, LayS<HD>::kAlloc, st>>>(m.k8, m.v8, p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace bdlm
