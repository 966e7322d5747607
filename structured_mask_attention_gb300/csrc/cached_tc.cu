// cached_tc.cu -- attention of a block's rows over the 8-bit cache on the
// sm_103a tensor cores.
//
// S = Q K^T without touching K's codes: a bf16 query has 8 significant bits, so
// it is the sum of an e4m3 value of 4 bits and an e5m2 value of 3, and
// S = Qhi K^T + Qlo K^T are two kind::f8f6f4 products that cost together what
// one bf16 product would (8-bit types run at twice its rate), with K's tiles taken
// as TMA leaves them.  (Each row of Q is first scaled by a power of two that
// puts its largest magnitude into [128, 256): exact for elements down to
// 2^-13 of it, off by at most 2^-21 of it below; split_f8.)  Scores meet the key
// blocks' scales in the softmax, one multiplication per block that the
// exponent's fma absorbs.
// P V runs in fp16: an e4m3 code is exact in fp16 and one instruction turns
// two, so a warpgroup converts V's codes, without their scales, while the tensor
// cores work on the tile before.  The scales join the scores: with log2 of its
// value block's scale added to a key's score, p' = exp2(s + log2 vs - m) is the
// weight of the codes themselves, whatever the scales (in fp16 with a shift that
// cached_attn.h explains), and the row sum takes p' / vs: a few operations per
// block of keys and row.  (In bf16, V's values code * scale cost five
// instructions for two, as much issue as the softmax; P in two e4m3 parts
// would triple the exponentials' cost.)  For an fp32 output P goes in two
// parts, the second what the first's rounding left.
//
// A CTA per SM takes its share of the units of 128 keys (cache.cuh).  Two
// arrangements of the same roles:
//   pairs (KS = false): 256 rows, two sub-tiles of 128 that share every key
//     tile; for more than 128 rows, where the tensor cores bound the call;
//   split (KS = true): 128 rows, the two sub-tiles take alternate key tiles
//     with a softmax state each and are joined at the end; for up to 128 rows,
//     where the stream of codes does.
// Roles (16 warps): warp 0 loads K, warp 2 loads V (both walk the page table,
// 4 tiles ahead), one lane of warp 1 issues the MMAs in the order that keeps
// one sub-tile's product running during the other's softmax, warps 4-7 and
// 8-11 are the softmax of sub-tiles 0 and 1 (one row per thread), warps 12-15
// convert V.  TMEM: S of sub-tile t at 128 t (P over it), O at 256 + 128 t.
// The rows' own block (bf16 keys) follows the cached tiles of the last unit or
// has units of its own; its Q is bf16, its V is converted in place, over a scale
// that the K loader finds (P in bf16 beside bf16 values would be off by 2^-8: O of
// blocks of 32 / 128 was off by 1.95 / 2.14e-3 of its size, of which bf16 outputs
// alone are 1.66).
//
// What bounds it (16 / 8 heads of 128, merge included): a block of 512 over one
// sequence of 131072 tokens takes 487 us, 1.13 PFLOP/s or 61 % of the measured
// bf16 rate; a pair's tile period is about 4000 cycles against 2150 of its
// products alone: the chain S -> softmax (2500) -> P V of each sub-tile, and the
// issuing thread's waits in between.  Blocks of 128 over 4 sequences, 40 / 8
// heads: 224 us, 0.77 PFLOP/s (three tiles of 256 for 640 rows: a sixth is
// padding).  Blocks of 32 over 16 sequences of 8192 at most (split, 64 rows of
// 128): 86 us.  There, by the CTAs' clocks with cold caches, 21 thousand cycles
// pass before the first scores (2 to start, 9 until the walk has read lengths and
// offsets, 7 to place the queries, 3 until K is there), 10 more in the first tile
// (instructions that no CTA has run yet), 2 for each of 33 units, and 10 to 16 for
// the end of a segment and the beginning of the next (1 to 2 of them): 102 to 156 in
// all, 132 in the mean, 69 us.
// Registers: ptxas reports 60 to 176 bytes of spills in the bf16 instances and 208
// to 420 in the fp32 ones.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <type_traits>

#include "cached_attn.h"
#include "cached_tc.cuh"
#include "kernels.h"

namespace bdlm {
namespace {

constexpr int kThreads = 512;
constexpr int kRegsControl = 72, kRegsConvert = 40, kRegsSoftmax = 200;
constexpr int kLaunchRegs = 128;
static_assert(128 * (kRegsControl + kRegsConvert) + 256 * kRegsSoftmax <= kThreads * kLaunchRegs,
              "register split exceeds the block");
// (fp32 outputs) Key tiles that a sub-tile adds up on the tensor cores.  1 / 2 / 4 /
// all of about 90: O off by 1.0 / 1.2 / 1.6 / 8.9e-6 of its size over 19357 keys
// (fp32 products in torch: 2.6e-6); blocks of 128 of the case above as fp32, with 1 /
// 2 / 4: 670 / 596 / 564 us.
constexpr int kFineTiles = 2;
constexpr int NK = 3;             // K slots: 128 keys of codes, or one 64-column panel of own keys
constexpr int NI = 16;            // tile-info slots (more than any two roles are apart, and a batch of four)
constexpr int kSlot = 128 * 128;  // bytes of a K slot, of a V slot and of a bf16 panel

enum { B_QF = 0, B_KF = 2, B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + 2, B_WF = B_VE + 2, B_WE = B_WF + 2,
       B_SF = B_WE + 2, B_PF = B_SF + 2, B_OD = B_PF + 2, B_OE = B_OD + 2, B_ML = B_OE + 2,
       B_KI = B_ML + 1, B_PCF = B_KI + NI, B_PCE = B_PCF + 4, B_COUNT = B_PCE + 4 };

// What the softmax and the conversion need of a tile.  s, lv, iv: K's scale, log2
// and 2^-shift times the inverse of V's (scale 1 where there is no page), [0][x] of keys 32 x ..
// 32 x + 15 and [1][x] of the 16 behind them.
struct alignas(16) KInfo {
  float s[2][4], lv[2][4], iv[2][4];
  int fine;  // scales differ inside 32 keys, or some keys' page is missing
  int gone;  // bit x: the page of keys 16 x .. 16 x + 15 is missing
};

template <int HD>
struct Lay {
  static constexpr int kQ = 0;                    // two regions of 128 rows x HD bf16 (or its two 8-bit parts)
  static constexpr int kQBytes = 128 * HD * 2;
  static constexpr int kK = 2 * kQBytes;
  static constexpr int kV = kK + NK * kSlot;      // codes of V, 2 slots
  static constexpr int kW = kV + 2 * kSlot;       // fp16 V, 2 slots of HD / 64 panels
  static constexpr int kWBytes = kSlot * (HD / 64);
  static constexpr int kBar = kW + 2 * kWBytes;
  static constexpr int kKI = kBar + ((8 * B_COUNT + 8 + 15) & ~15);
  static constexpr int kML = kKI + NI * (int)sizeof(KInfo);
  static constexpr int kCQ = kML + 2 * 128 * 8;
  static constexpr int kPC = kCQ + 256 * 4;
  static constexpr int kBytes = kPC + 4 * 64;
  // 1024 bytes to align; at least 120 KB so that no second CTA shares the SM (each holds all of TMEM)
  static constexpr int kAlloc = kBytes + 1024 > 120 * 1024 ? kBytes + 1024 : 120 * 1024;
};
static_assert(Lay<128>::kAlloc <= 232448, "shared memory");

// One CTA's share of a segment, as the roles read it from a ring in shared
// memory (warp 3 fills it, so that no other role carries the walk over the
// segments in its registers).
struct Piece {
  int64_t row0;        // the sequence's first row
  int s, h, rt;        // sequence, KV head, row tile
  int len, rows;       // cached tokens and new rows of the sequence
  int nk, k0;          // cached tiles, the first; nk = -1: no more pieces
  int nl, l0;          // own tiles, the first
  int whole, first;    // the whole segment; its beginning
};
constexpr int NP = 4;  // ring slots

// A tile's 128 query rows (first: the first as token * group + head of the
// group), by the TEAM threads of one or both sub-tiles: 16-byte copies, all in
// flight at once, then, for the 8-bit parts, each thread turns the 32 bytes that it
// copied to where their 16 + 16 codes go.  Loops that are not unrolled: this
// runs once or twice in a CTA's life, and instructions that no CTA has fetched
// yet cost more (about 25 cycles each) than the loops' own.
template <int HD, int TEAM, bool E4M3>
__device__ __forceinline__ void put_rows(const CachedParams& p, const Piece* pp, int tid, int first, uint32_t dst,
                                         float* factor) {
  constexpr int PER = E4M3 ? HD / 16 : HD / 8;  // lanes to a row
  const int i = tid % PER, group = p.sp.group, h = pp->h, rows = pp->rows;
  const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(p.Q) + (pp->row0 * p.Hq + h * group) * HD + i * (HD / PER);
#pragma unroll 1
  for (int r = tid / PER; r < 128; r += TEAM / PER) {
    const int fr = first + r, tok = fr / group;
    const int bytes = tok < rows ? 16 : 0;
    const __nv_bfloat16* src = Q + (bytes ? ((int64_t)tok * p.Hq + fr - tok * group) * HD : 0);
    if (E4M3) {
      const uint32_t at = dst + e4m3_chunk<HD>(r, i);
      cp_async16(at, src, bytes);
      cp_async16(at + 128 * HD, src + 8, bytes);
    } else {
      cp_async16(dst + (i >> 3) * kSlot + r * 128 + (((i & 7) ^ (r & 7)) << 4), src, bytes);
    }
  }
  cp_async_wait_all();
  if (E4M3) {
#pragma unroll 1
    for (int r = tid / PER; r < 128; r += TEAM / PER) {
      const uint32_t at = dst + e4m3_chunk<HD>(r, i);
      const uint4 x = ld_shared_v4(at), y = ld_shared_v4(at + 128 * HD);
      const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      uint32_t amax = 0, hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = __vmaxu2(amax, w[k] & 0x7fff7fffu);
      amax = max(amax & 0xffffu, amax >> 16);
#pragma unroll
      for (int o = PER / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float inv;
      const float f = row_factor(amax, inv);
      split_f8(w, f, hi, lo);
      st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(at + 128 * HD, lo[0], lo[1], lo[2], lo[3]);
      if (i == 0) factor[r] = p.sl2 * inv;
    }
  }
}

// The same as a call, for pairs: inlined there, it costs the softmax's loop its
// registers (block of 512: 518 against 481 us; split, as a call: block of 32 92
// against 86 us).
template <int HD, int TEAM, bool E4M3>
__device__ __noinline__ void put_rows_call(const CachedParams& p, const Piece* pp, int tid, int first, uint32_t dst,
                                           float* factor) {
  put_rows<HD, TEAM, E4M3>(p, pp, tid, first, dst, factor);
}

// 2^x of a whole x in fp32's normal range.
__device__ __forceinline__ float exp2_int(float x) { return __uint_as_float((uint32_t)((int)x + 127) << 23); }

// log2 of the scale that own tile l's values get: V / scale is fp16, exact for
// bf16 values down to 2^-25 of the tile's largest magnitude, which comes to
// [2^8, 2^9) as in a cached block.  Only the sequence's own rows count, and of
// them finite values (others stay what they are in fp16).  By the K loader's warp,
// which would come late to the next tile's keys if each round of loads took its way
// to L2: the lines are asked for first (block of 512: 501 -> 487 us).
template <int HD>
__device__ __forceinline__ float own_scale(const CachedParams& p, const Piece* pp, int l, int lane) {
  constexpr int PER = HD / 8, STEP = 32 / PER;  // lanes to a row, rows at a time
  const int first = (pp->l0 + l) * kUnit, n = min(pp->rows - first, kUnit);
  const __nv_bfloat16* V =
      static_cast<const __nv_bfloat16*>(p.V) + ((pp->row0 + first) * p.c.Hkv + pp->h) * HD + (lane % PER) * 8;
  if (n > 16 * STEP)
    for (int r = lane; r < n; r += 32)
#pragma unroll
      for (int x = 0; x < HD / 64; ++x)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(V - (lane % PER) * 8 + (int64_t)r * p.c.Hkv * HD + x * 64));
  uint32_t m = 0;
#pragma unroll 1
  for (int r0 = lane / PER; r0 < n; r0 += 8 * STEP) {  // (eight loads in flight)
    uint4 w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int r = r0 + x * STEP;
      w[x] = r < n ? __ldg(reinterpret_cast<const uint4*>(V + (int64_t)r * p.c.Hkv * HD)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint32_t v[4] = {w[x].x & 0x7fff7fffu, w[x].y & 0x7fff7fffu, w[x].z & 0x7fff7fffu, w[x].w & 0x7fff7fffu};
#pragma unroll
      for (int y = 0; y < 4; ++y) m = __vmaxu2(m, v[y] & __vcmpltu2(v[y], 0x7f807f80u));
    }
  }
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  return (float)max((int)(m >> 7) - 127 - 8, -96);
}

__device__ __forceinline__ float max32(const uint32_t (&a)[32]) {
  float u[10];
#pragma unroll
  for (int c = 0; c < 10; ++c)
    u[c] = fmax3(__uint_as_float(a[3 * c]), __uint_as_float(a[3 * c + 1]), __uint_as_float(a[3 * c + 2]));
  const float x = fmax3(u[0], u[1], u[2]), y = fmax3(u[3], u[4], u[5]), z = fmax3(u[6], u[7], u[8]);
  return fmax3(fmax3(x, y, z), u[9], fmaxf(__uint_as_float(a[30]), __uint_as_float(a[31])));
}

__device__ __forceinline__ void mask32(uint32_t (&a)[32], int hi) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (c >= hi) a[c] = __float_as_uint(-INFINITY);
}

// 32 scores of two key blocks of unlike scales: times their factors, plus
// their shifts, or -inf where a block's page is missing.
__device__ __forceinline__ void scores16(uint32_t (&a)[32], float f, float lf, float g, float lg, int gone) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const float x = fmaf(__uint_as_float(a[c]), c < 16 ? f : g, c < 16 ? lf : lg);
    a[c] = (gone >> (c >> 4)) & 1 ? __float_as_uint(-INFINITY) : __float_as_uint(x);
  }
}

// p = exp2(s f + n) of 32 scores in place, and the sums of the first and the
// last 16.  The exponentials are issued side by side (volatile: in this order),
// not each followed by its use.
__device__ __forceinline__ void exp32(uint32_t (&a)[32], float f, float n, float& s0, float& s1) {
  const uint64_t f2x = f2(f, f), n2 = f2(n, n);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float x0, x1;
    f2_split(f2_fma(f2(__uint_as_float(a[c]), __uint_as_float(a[c + 1])), f2x, n2), x0, x1);
    a[c] = __float_as_uint(x0);
    a[c + 1] = __float_as_uint(x1);
  }
#pragma unroll
  for (int c = 0; c < 32; ++c) asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+r"(a[c]));
  uint64_t r[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) r[y] = f2(__uint_as_float(a[8 * y]), __uint_as_float(a[8 * y + 1]));
#pragma unroll
  for (int c = 2; c < 8; c += 2)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      r[y] = f2_add(r[y], f2(__uint_as_float(a[8 * y + c]), __uint_as_float(a[8 * y + c + 1])));
  float x, y;
  f2_split(f2_add(r[0], r[1]), x, y);
  s0 = x + y;
  f2_split(f2_add(r[2], r[3]), x, y);
  s1 = x + y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// P lies over the S columns that it replaces, 32 keys by 32 keys: 16 packed
// columns, then 16 of the second part (FINE).  Column of the 16 keys of PV
// k-step kk:
__device__ __forceinline__ uint32_t p_col(int kk) { return (uint32_t)((kk >> 1) * 32 + (kk & 1) * 8); }

// Packs 32 values to fp16 at 16 columns of TMEM; REST: the values become what the rounding left.
template <bool REST>
__device__ __forceinline__ void store_p(uint32_t (&a)[32], uint32_t taddr) {
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const float x = __uint_as_float(a[c]), y = __uint_as_float(a[c + 1]);
    uint32_t w;  // (saturating: from scores of 2^20 on their rounding may exceed the margin below 2^16)
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(y), "f"(x));
    pk[c / 2] = w;
    if (REST) {
      const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&w));
      a[c] = __float_as_uint(x - z.x);
      a[c + 1] = __float_as_uint(y - z.y);
    }
  }
  tmem_st16(taddr, pk);
}

template <int HD, bool KS, bool FINE>
__global__ void __launch_bounds__(kThreads, 1)
    bdlm_cached_tc_kernel(const __grid_constant__ CUtensorMap tK8, const __grid_constant__ CUtensorMap tK,
                          const __grid_constant__ CUtensorMap tV, const CachedParams p) {
  using LY = Lay<HD>;
  constexpr int KP = HD / 64;        // 64-column panels of a bf16 tile
  constexpr int SWQ = HD == 128 ? 2 : 4;
  constexpr uint32_t SBO8 = 8 * HD;  // bytes between 8-row groups of an e4m3 tile
  constexpr int kTileRows = KS ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  auto BAR = [&](int i) -> uint32_t { return base + LY::kBar + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bp + LY::kBar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + LY::kBar + 8 * B_COUNT + 4);
  KInfo* kinfo = reinterpret_cast<KInfo*>(bp + LY::kKI);
  float2* ml = reinterpret_cast<float2*>(bp + LY::kML);  // split: both sub-tiles' states of the rows, [2][128]
  // the rows' score factors
  float* row_cq = reinterpret_cast<float*>(bp + LY::kCQ);
  Piece* pieces = reinterpret_cast<Piece*>(bp + LY::kPC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(BAR(B_KF + i), 1);
      mbar_init(BAR(B_KE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(B_QF + i), KS ? 256 : 128);
      mbar_init(BAR(B_VF + i), 1);
      mbar_init(BAR(B_VE + i), 128);
      mbar_init(BAR(B_WF + i), 128);
      mbar_init(BAR(B_WE + i), 1);
      mbar_init(BAR(B_SF + i), 1);
      mbar_init(BAR(B_PF + i), 128);
      mbar_init(BAR(B_OD + i), 1);
      mbar_init(BAR(B_OE + i), KS ? 256 : 128);
    }
    mbar_init(BAR(B_ML), 256);
    for (int i = 0; i < NP; ++i) {
      mbar_init(BAR(B_PCF + i), 1);
      mbar_init(BAR(B_PCE + i), 32 + 32 + 1 + 256 + 128);  // K and V loader, MMA thread, softmax, conversion
    }
    for (int i = 0; i < NI; ++i) mbar_init(BAR(B_KI + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  launch_dependents();
  const Watchdog wd{p.status, p.limit_ns, abort_flag};
  const CacheDesc& c = p.c;
  // the n-th piece (null: none left, or gave up); its slot stays this thread's until done(n)
  auto piece = [&](uint32_t n) -> const Piece* {
    if (!mbar_wait(BAR(B_PCF + (n % NP)), (n / NP) & 1, wd, 10)) return nullptr;
    const Piece* q = pieces + n % NP;
    return q->nk < 0 ? nullptr : q;
  };
  auto done = [&](uint32_t n) { mbar_arrive(BAR(B_PCE + (n % NP))); };

  if (warp < 4) {
    setmaxnreg_dec<kRegsControl>();
    auto load = [&](auto is_v) {
      // ---------------------------------------------- loaders: K (warp 0), V (warp 2)
      // Lane 8 a + x looks up the page (K's loader: and the scales) of keys
      // 16 x of tile a of a batch of 4 tiles; the lookups of the next batch are
      // in flight while this one is loaded.
      constexpr bool isV = decltype(is_v)::value;
      uint32_t bad = 0;
      uint32_t slot = 0, sph = 1, tc = 0;  // slot and its phase parity to wait for, tiles so far
      constexpr int nslots = isV ? 2 : NK;
      const uint32_t page_bytes = (uint32_t)(c.page * HD), page_groups = first_groups(c.page);
      bool ok = true;
      for (uint32_t np = 0; ok; ++np) {
        const Piece* pp = piece(np);
        if (__any_sync(0xffffffffu, pp == nullptr)) break;
        const int len = pp->len, nk = pp->nk, k0 = pp->k0, h = pp->h;
        const int32_t* table = c.table + (int64_t)pp->s * c.max_pages;
        auto lookup = [&](int b) {  // page of this lane's 16 keys of batch b, -1: none
          const int tile = 4 * b + (lane >> 3), key = (k0 + tile) * kUnit + 16 * (lane & 7);
          return tile < nk && key < len ? __ldg(table + (key >> c.lp)) : -1;
        };
        // (a batch's entries are looked at a batch after they were asked for)
        auto checked = [&](int id, int b) {
          if (id >= 0 && id < c.n_pages) return id;
          const int tile = 4 * b + (lane >> 3), key = (k0 + tile) * kUnit + 16 * (lane & 7);
          if (tile < nk && key < len) bad |= kStatusBadPage;
          return -1;
        };
        auto scale_of = [&](const float* sc, int id) { return id >= 0 ? __ldg(sc + (int64_t)id * c.Hkv + h) : 1.f; };
        const int raw0 = lookup(0);
        int raw1 = lookup(1);
        int id = checked(raw0, 0);
        float sk = 1.f, sv = 1.f, sk1 = 1.f, sv1 = 1.f;
        if (!isV) sk = scale_of(c.ks, id), sv = scale_of(c.vs, id);
        for (int b = 0; ok && 4 * b < nk; ++b) {
          const int id1 = checked(raw1, b + 1);
          if (!isV) sk1 = scale_of(c.ks, id1), sv1 = scale_of(c.vs, id1);
          const int raw2 = lookup(b + 2);
          // the batch's tiles, a group of eight lanes each
          const int grp = lane >> 3, x = lane & 7, key = (k0 + 4 * b) * kUnit + 16 * lane;
          const bool on = 4 * b + grp < nk;
          const unsigned none = __ballot_sync(0xffffffffu, id < 0);
          if (!isV) {
            const float pk = __shfl_xor_sync(0xffffffffu, sk, 1), pv = __shfl_xor_sync(0xffffffffu, sv, 1);
            const unsigned gone = __ballot_sync(0xffffffffu, id < 0 && key < len);
            const unsigned odd = __ballot_sync(0xffffffffu, (key | 16) < len && (sk != pk || sv != pv));
            KInfo& ki = kinfo[(tc + grp) % NI];
            if (on) {
              ki.s[x & 1][x >> 1] = sk;
              ki.lv[x & 1][x >> 1] = log2f(sv);
              ki.iv[x & 1][x >> 1] = kTcUnshift / sv;
            }
            if (on && x == 0) {
              ki.fine = (((gone | odd) >> lane) & 0xffu) != 0;
              ki.gone = (int)((gone >> lane) & 0xffu);
            }
            __syncwarp();
            if (on && x == 0) mbar_arrive(BAR(B_KI + (tc + grp) % NI));
          }
          const uint32_t bytes = (uint32_t)__popc(~(none >> (lane & 24)) & page_groups) * page_bytes;
          const bool loads = id >= 0 && ((page_groups >> x) & 1);
          const int64_t blk = (int64_t)id * c.Hkv + h;
          for (int a = 0; a < 4 && 4 * b + a < nk; ++a, ++tc) {
            ok = mbar_wait(BAR((isV ? B_VE : B_KE) + slot), sph, wd, 20 + warp);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t fb = BAR((isV ? B_VF : B_KF) + slot);
            if (lane == 8 * a) {
              if (bytes) mbar_arrive_expect_tx(fb, bytes);
              else mbar_arrive(fb);
            }
            __syncwarp();
            if (grp == a && loads) {  // the lane of a page's first keys loads it
              const uint32_t dst = base + (isV ? LY::kV : LY::kK) + slot * kSlot + 16 * x * HD;
              if (isV) bulk_load(dst, c.v8 + blk * page_bytes, page_bytes, fb);
              else tma_load_3d(dst, &tK8, fb, 0, 0, (int)blk);
            }
            if (++slot == (uint32_t)nslots) slot = 0, sph ^= 1;
          }
          id = id1; raw1 = raw2; sk = sk1; sv = sv1;
        }
        // own tiles: K by panels through the K slots; V straight into the fp16 slot that its tile has
        const int nl = pp->nl;
        for (int l = 0; ok && l < nl; ++l, ++tc) {
          const int row = (int)(pp->row0 + (int64_t)(pp->l0 + l) * kUnit);
          if (!isV) {
            KInfo& ki = kinfo[tc % NI];
            const float lv = own_scale<HD>(p, pp, l, lane);
            if (lane < 4) ki.s[0][lane] = 1.f, ki.iv[0][lane] = exp2_int(-lv) * kTcUnshift, ki.lv[0][lane] = lv;
            if (lane == 0) ki.fine = ki.gone = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_KI + tc % NI));
          }
          if (isV) {
            ok = mbar_wait(BAR(B_VE + slot), sph, wd, 24);
            if (ok) ok = mbar_wait(BAR(B_WE + slot), sph, wd, 25);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(BAR(B_VF + slot), LY::kWBytes);
              for (int pn = 0; pn < KP; ++pn)
                tma_load_3d(base + LY::kW + slot * LY::kWBytes + pn * kSlot, &tV, BAR(B_VF + slot), 64 * pn, h, row);
            }
            slot ^= 1;
            if (slot == 0) sph ^= 1;
          } else {
            for (int pn = 0; ok && pn < KP; ++pn) {
              ok = mbar_wait(BAR(B_KE + slot), sph, wd, 26);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(BAR(B_KF + slot), kSlot);
                tma_load_3d(base + LY::kK + slot * kSlot, &tK, BAR(B_KF + slot), 64 * pn, h, row);
              }
              if (++slot == NK) slot = 0, sph ^= 1;
            }
          }
        }
        done(np);
      }
      if (bad) atomicOr(p.status + kContentsWord, bad);
    };
    if (warp == 0) {
      load(std::false_type{});
    } else if (warp == 2) {
      load(std::true_type{});
    } else if (warp == 3) {
      // ---------------------------------------------- walk over the CTA's pieces
      uint32_t bad = 0;
      const SplitOpen open = split_open(c, p.r, p.sp, p.G, blockIdx.x, bad);
      int64_t u = open.u0;
      const int64_t u1 = open.u1;
      UnitPos pos = open.pos;
      SegInfo seg = open.seg;
      if (lane == 0) {
        for (uint32_t n = 0;; ++n) {
          if (n >= NP && !mbar_wait(BAR(B_PCE + n % NP), (n / NP - 1) & 1, wd, 11)) break;
          Piece& q = pieces[n % NP];
          if (u >= u1) {
            q.nk = -1;
            mbar_arrive(BAR(B_PCF + n % NP));
            break;
          }
          int jb, je;
          split_units(seg, p.sp, pos, u, u1, jb, je);
          u += seg.span - pos.j;
          if (je == 0) {  // only the segment's opening lies here: the next CTA begins it
            q.nk = -1;
            mbar_arrive(BAR(B_PCF + n % NP));
            break;
          }
          const int kt = seg.ktiles;
          q.row0 = seg.v.row0;
          q.s = pos.s; q.h = pos.h; q.rt = pos.rt;
          q.len = seg.v.len; q.rows = seg.v.rows;
          q.k0 = jb;
          q.nk = max(min(je, kt) - jb, 0);
          q.l0 = max(jb - kt, 0);
          q.nl = seg.ltiles > 0 ? max(je - kt, 0) - q.l0 : (p.sp.local && je == seg.units ? 1 : 0);
          q.first = jb == 0;
          q.whole = jb == 0 && je == seg.units;
          mbar_arrive(BAR(B_PCF + n % NP));
          if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
        }
      }
      if (bad) atomicOr(p.status + kContentsWord, bad);  // (each lane has looked at other sequences)
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issue
      if (lane == 0) {
        constexpr uint32_t kId8[2] = {idesc_f8(128, 128, kE4m3, kE4m3), idesc_f8(128, 128, kE5m2, kE4m3)};  // Q's parts
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdO = idesc_bf16(128, HD, false, true) & ~((1u << 7) | (1u << 10));  // fp16 P and V
        uint32_t ks = 0, kph = 0;            // next K slot and its full parity
        // bit t of a mask: the parity of sub-tile t's next phase (in pairs both bits are equal, bit 0 alone is kept)
        uint32_t qph = 0;                    // Q (split: bit 0 of Q8, bit 1 of bf16 Q)
        uint32_t pph = 0;                    // P
        uint32_t oph = 3;                    // O left by the last piece (first wait passes)
        uint32_t wc = 0;                     // V tiles multiplied so far
        auto bit = [](uint32_t m, int t) { return (m >> (KS ? t : 0)) & 1; };
        auto flip = [](uint32_t& m, int t) {
          if (KS || t == 1) m ^= 1u << (KS ? t : 0);  // pairs: sub-tile 1 comes last
        };
        bool ok = true;
        uint32_t k0 = 0, k1 = 0;             // slots of the tile whose S is being issued
        // the tile's keys are there
        auto take_k = [&](bool own) {
          k0 = ks;
          if (!mbar_wait(BAR(B_KF + ks), kph, wd, 30)) return false;
          if (++ks == NK) ks = 0, kph ^= 1;
          if (KP == 2 && own) {
            k1 = ks;
            if (!mbar_wait(BAR(B_KF + ks), kph, wd, 30)) return false;
            if (++ks == NK) ks = 0, kph ^= 1;
          }
          tc_fence_after();
          return true;
        };
        auto free_k = [&](bool own) {
          tc_commit(BAR(B_KE + k0));
          if (KP == 2 && own) tc_commit(BAR(B_KE + k1));
        };
        auto issue_s = [&](int t, bool own) {
          const uint32_t d = tmem + t * 128;
          if (!own) {
            constexpr uint32_t H = desc_hi(SWQ, SBO8);
            const uint32_t q = desc_lo(base + LY::kQ + (KS ? 0 : t) * LY::kQBytes, 16);
            const uint32_t k = desc_lo(base + LY::kK + k0 * kSlot, 16);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) mma_ss<true>(d, q + kk * 2, H, k + kk * 2, H, kId8[0], kk > 0);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) mma_ss<true>(d, q + 8 * HD + kk * 2, H, k + kk * 2, H, kId8[1], 1);
          } else {
            constexpr uint32_t H = desc_hi(2, 1024);
#pragma unroll
            for (int pn = 0; pn < KP; ++pn) {
              const uint32_t q = desc_lo(base + LY::kQ + (KS ? 1 : t) * LY::kQBytes + pn * kSlot, 16);
              const uint32_t k = desc_lo(base + LY::kK + (pn ? k1 : k0) * kSlot, 16);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_ss<false>(d, q + kk * 2, H, k + kk * 2, H, kIdS, (pn | kk) > 0);
            }
          }
          tc_commit(BAR(B_SF + t));
        };
        // O_t += P_t V of V tile w
        // (col: 0 the first part of P, 16 the second)
        auto pv = [&](int t, uint32_t w, uint32_t col, bool first) {
          const uint32_t v = desc_lo(base + LY::kW + (w & 1) * LY::kWBytes, kSlot);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + 256 + t * 128, tmem + t * 128 + col + p_col(kk), v + kk * 128, desc_hi(2, 1024), kIdO,
                   (kk > 0 || !first) ? 1u : 0u);
        };
        // (first: the piece's first product; fresh: the last piece's O may still be read)
        auto issue_pv = [&](int t, uint32_t w, bool first, bool fresh) {
          if (!mbar_wait(BAR(B_PF + t), bit(pph, t), wd, 31)) return false;
          flip(pph, t);
          if (fresh) {
            if (!mbar_wait(BAR(B_OE + t), bit(oph, t), wd, 32)) return false;
            flip(oph, t);
          }
          if ((KS || t == 0) && !mbar_wait(BAR(B_WF + (w & 1)), (w >> 1) & 1, wd, 33)) return false;
          tc_fence_after();
          pv(t, w, 0, first);
          if (FINE) pv(t, w, 16, false);
          return true;
        };
        for (uint32_t np = 0; ok; ++np) {
          const Piece* pp = piece(np);
          if (!pp) break;
          const int nk = pp->nk, n = nk + pp->nl;
          done(np);
          if (n == 0) continue;
          auto own = [&](int j) { return j >= nk; };
          // Q of sub-tile t (split: of kind t) has to be there before the first tile of each kind
          auto wait_q = [&](int t) {
            const bool r = mbar_wait(BAR(B_QF + t), bit(qph, t), wd, 35);
            flip(qph, t);
            if (r) tc_fence_after();
            return r;
          };
          if (KS) {
            auto start_s = [&](int j) {
              if ((j == 0 || j == nk) && !wait_q(own(j) ? 1 : 0)) return false;
              if (!take_k(own(j))) return false;
              issue_s(j & 1, own(j));
              free_k(own(j));
              return true;
            };
            ok = start_s(0) && (n < 2 || start_s(1));
            int j = 0;
            // (as in pairs, below: while the tile after next is a cached one)
            const bool opened = nk > 3;
            if (opened) {
              ok = ok && mbar_wait(BAR(B_OE + 0), oph & 1, wd, 32) && mbar_wait(BAR(B_OE + 1), (oph >> 1) & 1, wd, 32);
              oph ^= 3;
              auto lean = [&](auto sub) {
                constexpr int t = decltype(sub)::value;
                const uint32_t acc = j > 0, vs = wc & 1, vt = desc_lo(base + LY::kW + vs * LY::kWBytes, kSlot);
                const uint32_t kt = desc_lo(base + LY::kK + ks * kSlot, 16), q = desc_lo(base + LY::kQ, 16);
                constexpr uint32_t HV = desc_hi(2, 1024), HQ = desc_hi(SWQ, SBO8);
                constexpr int n8 = HD / 32;
                if (!(mbar_wait(BAR(B_WF + vs), (wc >> 1) & 1, wd, 33) && mbar_wait(BAR(B_KF + ks), kph, wd, 30) &&
                      mbar_wait(BAR(B_PF + t), bit(pph, t), wd, 31)))
                  return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_ts(tmem + 256 + t * 128, tmem + t * 128 + p_col(kk), vt + kk * 128, HV, kIdO, kk > 0 ? 1u : acc);
#pragma unroll
                for (int kk = 0; kk < (FINE ? 8 : 0); ++kk)
                  mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 16 + p_col(kk), vt + kk * 128, HV, kIdO, 1);
                tc_commit(BAR(B_WE + vs));
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                  mma_ss<true>(tmem + t * 128, q + (kk / n8) * 8 * HD + (kk % n8) * 2, HQ, kt + (kk % n8) * 2, HQ, kId8[kk / n8],
                               kk > 0);
                tc_commit(BAR(B_SF + t));
                tc_commit(BAR(B_KE + ks));
                if (++ks == NK) ks = 0, kph ^= 1;
                ++wc;
                return true;
              };
              for (; ok && j + 3 < nk; j += 2) {
                ok = lean(std::integral_constant<int, 0>{}) && lean(std::integral_constant<int, 1>{});
                pph ^= 3;
              }
            }
            for (; ok && j < n; ++j, ++wc) {
              const int t = j & 1;
              ok = issue_pv(t, wc, j < 2, j < 2 && !opened);
              if (!ok) break;
              tc_commit(BAR(B_WE + (wc & 1)));
              if (j + 2 >= n) tc_commit(BAR(B_OD + t));
              else ok = start_s(j + 2);
            }
          } else {
            ok = wait_q(0) && take_k(own(0));
            if (ok) issue_s(0, own(0));
            ok = ok && wait_q(1);
            if (ok) {
              issue_s(1, own(0));
              free_k(own(0));
            }
            int j = 0;
            // cached tiles that a cached tile follows: the waits, products and
            // commits alone (whatever else this thread does idles the tensor
            // cores: their queue holds about one product)
            if (nk > 1) {
              ok = ok && mbar_wait(BAR(B_OE + 0), oph & 1, wd, 32) && mbar_wait(BAR(B_OE + 1), oph & 1, wd, 32);
              oph ^= 1;
              for (; ok && j + 1 < nk; ++j, ++wc) {
                const uint32_t acc = j > 0, vt = desc_lo(base + LY::kW + (wc & 1) * LY::kWBytes, kSlot);
                const uint32_t kt = desc_lo(base + LY::kK + ks * kSlot, 16), q = desc_lo(base + LY::kQ, 16);
                constexpr uint32_t HV = desc_hi(2, 1024), HQ = desc_hi(SWQ, SBO8);
                ok = mbar_wait(BAR(B_WF + (wc & 1)), (wc >> 1) & 1, wd, 33) && mbar_wait(BAR(B_KF + ks), kph, wd, 30) &&
                     mbar_wait(BAR(B_PF + 0), pph & 1, wd, 31);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_ts(tmem + 256, tmem + p_col(kk), vt + kk * 128, HV, kIdO, kk > 0 ? 1u : acc);
#pragma unroll
                for (int kk = 0; kk < (FINE ? 8 : 0); ++kk)
                  mma_ts(tmem + 256, tmem + 16 + p_col(kk), vt + kk * 128, HV, kIdO, 1);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                  constexpr int n8 = HD / 32;
                  mma_ss<true>(tmem, q + (kk / n8) * 8 * HD + (kk % n8) * 2, HQ, kt + (kk % n8) * 2, HQ, kId8[kk / n8], kk > 0);
                }
                tc_commit(BAR(B_SF + 0));
                ok = mbar_wait(BAR(B_PF + 1), pph & 1, wd, 31);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_ts(tmem + 384, tmem + 128 + p_col(kk), vt + kk * 128, HV, kIdO, kk > 0 ? 1u : acc);
#pragma unroll
                for (int kk = 0; kk < (FINE ? 8 : 0); ++kk)
                  mma_ts(tmem + 384, tmem + 144 + p_col(kk), vt + kk * 128, HV, kIdO, 1);
                tc_commit(BAR(B_WE + (wc & 1)));
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                  constexpr int n8 = HD / 32;
                  mma_ss<true>(tmem + 128, q + (LY::kQBytes >> 4) + (kk / n8) * 8 * HD + (kk % n8) * 2, HQ,
                               kt + (kk % n8) * 2, HQ, kId8[kk / n8], kk > 0);
                }
                tc_commit(BAR(B_SF + 1));
                tc_commit(BAR(B_KE + ks));
                if (++ks == NK) ks = 0, kph ^= 1;
                pph ^= 1;
              }
            }
            const bool opened = nk > 1;
            for (; ok && j < n; ++j, ++wc) {
              const bool last = j == n - 1, swap = j + 1 == nk && !last;
              ok = issue_pv(0, wc, j == 0, j == 0 && !opened);
              if (!ok) break;
              if (last) tc_commit(BAR(B_OD + 0));
              if (!last) {
                ok = (!swap || wait_q(0)) && take_k(own(j + 1));
                if (!ok) break;
                issue_s(0, own(j + 1));
              }
              ok = issue_pv(1, wc, j == 0, j == 0 && !opened);
              if (!ok) break;
              tc_commit(BAR(B_WE + (wc & 1)));
              if (last) {
                tc_commit(BAR(B_OD + 1));
              } else {
                ok = !swap || wait_q(1);
                if (!ok) break;
                issue_s(1, own(j + 1));
                free_k(own(j + 1));
              }
            }
          }
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------ softmax (thread = row of sub-tile t)
    setmaxnreg_inc<kRegsSoftmax>();
    const int t = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + tl + t * 128, tO = tmem + tl + 256;
    uint32_t sc = 0, tcount = 0, itn[2] = {0, 0}, mlc = 0, qfc = 0;
    bool ok = true;
    for (uint32_t np = 0; ok; ++np) {
      const Piece* pp = piece(np);
      if (__any_sync(0xffffffffu, pp == nullptr)) break;
      const int nk = pp->nk, nl = pp->nl, n = nk + nl;
      // this thread's row: its token and query head (worked out again where it is needed)
      struct Row {
        int64_t at;  // row of the packed tensors
        int head;
        bool live;
      };
      auto my_row = [&]() {
        const int fr = pp->rt * kTileRows + (KS ? 0 : t * 128) + row, tok = fr / p.sp.group;
        Row r;
        r.live = tok < pp->rows;
        r.head = pp->h * p.sp.group + fr - tok * p.sp.group;
        r.at = pp->row0 + (r.live ? tok : 0);
        return r;
      };
      // Q's rows to shared memory, HD / 16 (HD / 8) lanes to a row: 8 bits in two
      // parts with the rows' factors, or bf16.  Pairs: the sub-tile's 128 rows by its
      // threads; split: the tile's 128 rows by both sub-tiles' threads.
      constexpr int kTeam = KS ? 256 : 128;
      const int tid = (KS ? t * 128 : 0) + row, first = pp->rt * kTileRows + (KS ? 0 : t * 128);
      auto put_q8 = [&]() {
        if (KS) put_rows<HD, kTeam, true>(p, pp, tid, first, base + LY::kQ, row_cq);
        else put_rows_call<HD, kTeam, true>(p, pp, tid, first, base + LY::kQ + t * LY::kQBytes, row_cq + t * 128);
      };
      auto put_q16 = [&]() {
        if (KS) put_rows<HD, kTeam, false>(p, pp, tid, first, base + LY::kQ + LY::kQBytes, nullptr);
        else put_rows_call<HD, kTeam, false>(p, pp, tid, first, base + LY::kQ + t * LY::kQBytes, nullptr);
      };
      float cq = p.sl2;
      if (n > 0) {
        if (KS ? nk > 0 : true) {
          if (KS || nk > 0) put_q8();
          else put_q16();
          fence_proxy_async_smem();
          mbar_arrive(BAR(B_QF + (KS ? 0 : t)));
        }
        if (KS && nl > 0) {
          put_q16();
          fence_proxy_async_smem();
          mbar_arrive(BAR(B_QF + 1));
        }
        if (nk > 0) {  // the factor of this thread's row, found by another thread
          ok = mbar_wait(BAR(B_QF + (KS ? 0 : t)), qfc & 1, wd, 42);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          cq = row_cq[(KS ? 0 : t * 128) + row];
        }
        if (!KS || nk > 0) ++qfc;
      }
      float m_ref = -INFINITY, l = 0.f;
      // FINE: the tensor cores cut their sums off instead of rounding them, always
      // towards zero (9e-6 of O over 600 products in a row); so every kFineTiles
      // tiles O moves to sums that this thread keeps, and begins again at 0
      float m_sum = -INFINITY;
      int since = 0;
      bool summed = false;
      float4* sums = reinterpret_cast<float4*>(p.fine + ((int64_t)blockIdx.x * 2 + t) * 128 * HD) + row;
      // back: O takes in the sums; else: the sums take in O
      auto move_o = [&](bool back) {
        const float f = summed && m_ref != -INFINITY ? ex2_approx(m_sum - m_ref) : 0.f;
#pragma unroll 1
        for (int c4 = 0; c4 < HD / 32; ++c4) {
          uint32_t o[32];
          tmem_ld32(tO + t * 128 + c4 * 32, o);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            float4* at = sums + (c4 * 8 + x) * 128;
            float4 v = summed ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
            v.x = fmaf(v.x, f, __uint_as_float(o[4 * x]));
            v.y = fmaf(v.y, f, __uint_as_float(o[4 * x + 1]));
            v.z = fmaf(v.z, f, __uint_as_float(o[4 * x + 2]));
            v.w = fmaf(v.w, f, __uint_as_float(o[4 * x + 3]));
            if (!back) *at = v;
            o[4 * x] = back ? __float_as_uint(v.x) : 0u;
            o[4 * x + 1] = back ? __float_as_uint(v.y) : 0u;
            o[4 * x + 2] = back ? __float_as_uint(v.z) : 0u;
            o[4 * x + 3] = back ? __float_as_uint(v.w) : 0u;
          }
          tmem_st32(tO + t * 128 + c4 * 32, o);
        }
        m_sum = m_ref;
        summed = true;
      };
      // keys left from the piece's first cached (own) tile on
      const int left_k = pp->len - pp->k0 * kUnit, left_l = pp->rows - pp->l0 * kUnit;
      for (int j = KS ? t : 0; j < n; j += KS ? 2 : 1, ++sc) {
        const bool own = j >= nk;
        const uint32_t ti = tcount + (uint32_t)j;
        ok = mbar_wait(BAR(B_KI + ti % NI), (ti / NI) & 1, wd, 41);
        // (read before the wait for S: shared memory is slow to answer beside the MMAs)
        const KInfo& ki = kinfo[ti % NI];
        const float4 ks4 = *reinterpret_cast<const float4*>(ki.s[0]);
        const float4 lv4 = *reinterpret_cast<const float4*>(ki.lv[0]);
        const float4 iv4 = *reinterpret_cast<const float4*>(ki.iv[0]);
        const int fine = ki.fine;
        if (ok) ok = mbar_wait(BAR(B_SF + t), sc & 1, wd, 40);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // (O is complete up to the tile before: S of this one was issued behind its product)
        if (FINE && since++ == kFineTiles) {
          move_o(false);
          since = 1;
        }
        const int hi = own ? left_l - (j - nk) * kUnit : left_k - j * kUnit;
        const float rf = own ? p.sl2 : cq;
        float f[4] = {rf * ks4.x, rf * ks4.y, rf * ks4.z, rf * ks4.w}, lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w};
        const float iv[4] = {iv4.x, iv4.y, iv4.z, iv4.w};
        uint32_t a[4][32];  // the row's 128 scores
        tmem_ld32x4(tS, tS + 32, tS + 64, tS + 96, a[0], a[1], a[2], a[3]);
        if (fine) {
          const int gone = ki.gone;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            scores16(a[x], f[x], lv[x], rf * ki.s[1][x], ki.lv[1][x], gone >> (2 * x));
            f[x] = 1.f;
            lv[x] = 0.f;
          }
        }
        if (hi < kUnit) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            // (tiny queries on a block of tiny scale: 0 times -inf would be NaN)
            if (f[x] == 0.f) f[x] = FLT_MIN;
            mask32(a[x], hi - 32 * x);
          }
        }
        const float mx = fmaxf(fmaxf(fmaf(max32(a[0]), f[0], lv[0]), fmaf(max32(a[1]), f[1], lv[1])),
                               fmaxf(fmaf(max32(a[2]), f[2], lv[2]), fmaf(max32(a[3]), f[3], lv[3])));
        bool rescale = false;
        float alpha = 1.f;
        if (m_ref == -INFINITY) {
          m_ref = mx;  // first keys of this row (O holds zeros)
        } else if (mx > m_ref + kRescale) {
          alpha = ex2_approx(m_ref - mx);
          m_ref = mx;
          rescale = true;
        }
        const float nm = m_ref == -INFINITY ? 0.f : kTcShift - m_ref;
        l *= alpha;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float s0, s1;
          exp32(a[x], f[x], nm + lv[x], s0, s1);
          l = fine ? fmaf(s0, iv[x], fmaf(s1, ki.iv[1][x], l)) : fmaf(s0 + s1, iv[x], l);
          store_p<FINE>(a[x], tS + 32 * x);
          if (FINE) store_p<false>(a[x], tS + 32 * x + 16);
        }
        // O is complete up to the tile before (S of this one was issued behind its product)
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int c4 = 0; c4 < HD / 32; ++c4) {
            uint32_t o[32];
            tmem_ld32(tO + t * 128 + c4 * 32, o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
            tmem_st32(tO + t * 128 + c4 * 32, o);
          }
        }
        tc_fence_before();
        mbar_arrive(BAR(B_PF + t));
        if (!KS && j == nk - 1 && nl > 0) {  // the cached keys are through with Q's codes
          put_q16();
          fence_proxy_async_smem();
          mbar_arrive(BAR(B_QF + t));
          ++qfc;
        }
      }
      if (!ok) break;
      tcount += (uint32_t)n;

      // ---- the piece's result
      float w0 = 1.f, w1 = 0.f, M = m_ref, L = l;
      const int n0 = KS ? (n + 1) / 2 : n, n1 = KS ? n / 2 : n;
      if (KS && n > 0) {
        // both sub-tiles' states of this row (O's first product of the piece waited
        // for all threads to leave the last piece's, so ml is free)
        ok = mbar_wait(BAR(B_OD + 0), itn[0] & 1, wd, 44);
        if (ok && n1 > 0) ok = mbar_wait(BAR(B_OD + 1), itn[1] & 1, wd, 45);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (FINE && summed) {
          tc_fence_after();
          move_o(true);
          tc_fence_before();
        }
        ml[t * 128 + row] = make_float2(m_ref, l);
        mbar_arrive(BAR(B_ML));
        ok = mbar_wait(BAR(B_ML), mlc & 1, wd, 46);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++mlc;
        const float2 x0 = ml[row], x1 = ml[128 + row];
        M = fmaxf(x0.x, x1.x);
        const float b = M == -INFINITY ? 0.f : M;
        w0 = ex2_approx(x0.x - b);
        w1 = n1 > 0 ? ex2_approx(x1.x - b) : 0.f;
        L = x0.y * w0 + (n1 > 0 ? x1.y * w1 : 0.f);
        ++itn[0];
        if (n1 > 0) ++itn[1];
      } else if (!KS && n > 0) {
        ok = mbar_wait(BAR(B_OD + t), itn[0] & 1, wd, 47);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++itn[0];
        if (FINE && summed) {
          tc_fence_after();
          move_o(true);
        }
      }
      tc_fence_after();
      const bool whole = pp->whole;
      const float inv = whole ? (L != 0.f ? kTcUnshift / L : 0.f) : kTcUnshift;
      const Row r = my_row();
      const bool live = r.live;
      const float s0 = w0 * inv, s1 = w1 * inv;
      float* slot = p.part + (2 * (int64_t)blockIdx.x + (pp->first ? 1 : 0)) * part_floats(kTileRows, HD);
      const int prow = (KS ? 0 : t * 128) + row;
      const int64_t oofs = (r.at * p.Hq + r.head) * HD;
      done(np);  // (the rest is in registers)
      // split: sub-tile t's threads write columns HD / 2 t ..; both read both accumulators
      constexpr int kCols = KS ? HD / 2 : HD;
      const int col0 = KS ? t * (HD / 2) : 0;
#pragma unroll 1
      for (int c4 = 0; c4 < kCols / 32; ++c4) {
        const int col = col0 + c4 * 32;
        uint32_t o[32];
        if (n > 0) tmem_ld32(tO + (KS ? 0 : t * 128) + col, o);
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = n0 > 0 ? __float_as_uint(__uint_as_float(o[x]) * s0) : 0u;
        if (KS && n1 > 0) {
          uint32_t o1[32];
          tmem_ld32(tO + 128 + col, o1);
#pragma unroll
          for (int x = 0; x < 32; ++x)
            o[x] = __float_as_uint(fmaf(__uint_as_float(o1[x]), s1, __uint_as_float(o[x])));
        }
        if (!live) continue;  // (nobody reads a partial result's rows without a token)
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            reinterpret_cast<float4*>(slot)[(col / 4 + x) * kTileRows + prow] =
                make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]), __uint_as_float(o[4 * x + 2]),
                            __uint_as_float(o[4 * x + 3]));
        } else {
          if (p.o_f32) {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.O) + oofs + col);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              d[x] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]), __uint_as_float(o[4 * x + 2]),
                                 __uint_as_float(o[4 * x + 3]));
          } else {
            uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.O) + oofs + col);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              d[x] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * x]), __uint_as_float(o[8 * x + 1])),
                                pack_bf16x2(__uint_as_float(o[8 * x + 2]), __uint_as_float(o[8 * x + 3])),
                                pack_bf16x2(__uint_as_float(o[8 * x + 4]), __uint_as_float(o[8 * x + 5])),
                                pack_bf16x2(__uint_as_float(o[8 * x + 6]), __uint_as_float(o[8 * x + 7])));
          }
        }
      }
      tc_fence_before();
      if (n > 0) {
        if (KS) {
          mbar_arrive(BAR(B_OE + 0));
          if (n1 > 0) mbar_arrive(BAR(B_OE + 1));
        } else {
          mbar_arrive(BAR(B_OE + t));
        }
      }
      if (!KS || t == 0) {
        if (whole) {
          if (live) p.LSE[(int64_t)r.head * p.r.T + r.at] = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        } else {
          slot[(int64_t)kTileRows * HD + prow] = M;
          slot[(int64_t)kTileRows * (HD + 1) + prow] = L;
        }
      }
    }
  } else {
    // ------------------------------------------------ V's codes, own keys' values -> fp16
    setmaxnreg_dec<kRegsConvert>();
    const int i = threadIdx.x - 384;
    constexpr int CH = HD / 16;             // 16-code chunks of a key
    uint32_t w = 0;
    bool ok = true;
    for (uint32_t np = 0; ok; ++np) {
      const Piece* pp = piece(np);
      if (!pp) break;
      const int nk = pp->nk, n = nk + pp->nl;
      const int left_k = pp->len - pp->k0 * kUnit, left_l = pp->rows - pp->l0 * kUnit;
      done(np);
      for (int j = 0; j < n; ++j, ++w) {
        const uint32_t slot = w & 1, ph = (w >> 1) & 1;
        ok = mbar_wait(BAR(B_VF + slot), ph, wd, 50) && mbar_wait(BAR(B_WE + slot), ph ^ 1, wd, 51) &&
             mbar_wait(BAR(B_KI + w % NI), (w / NI) & 1, wd, 52);
        if (!ok) break;
        const uint32_t dst = base + LY::kW + slot * LY::kWBytes;
        if (j < nk) {
          const uint4* src = reinterpret_cast<const uint4*>(bp + LY::kV + slot * kSlot) + i;
          const int left = left_k - j * kUnit;
          const int gone = kinfo[w % NI].gone;
          const bool full = left >= kUnit && gone == 0;
          const int c16 = i % CH, key0 = i / CH;
          // 8-value chunks 2 c16, 2 c16 + 1 of a key; the second panel's threads write them in the other order,
          // so that the 8 lanes of a store phase cover all banks
          const uint32_t at0 = dst + (c16 >> 2) * kSlot, ch = (uint32_t)(c16 & 3) * 2;
          const bool odd = c16 >= 4;
          constexpr int XB = 4;  // loads in flight
#pragma unroll
          for (int x0 = 0; x0 < CH; x0 += XB) {
            uint4 v[XB];
#pragma unroll
            for (int x = 0; x < XB; ++x) v[x] = src[(x0 + x) * 128];
#pragma unroll
            for (int x = 0; x < XB; ++x) {
              const int key = key0 + (x0 + x) * (128 / CH);
              if (!full && (key >= left || ((gone >> (key >> 4)) & 1))) v[x] = make_uint4(0, 0, 0, 0);  // stale codes
              const uint32_t a[2] = {odd ? v[x].z : v[x].x, odd ? v[x].w : v[x].y};
              const uint32_t b[2] = {odd ? v[x].x : v[x].z, odd ? v[x].y : v[x].w};
              const uint32_t at = at0 + key * 128, sw = (uint32_t)key & 7u;
              st_shared_v4(at + (((ch + (odd ? 1 : 0)) ^ sw) << 4), e4m3x2_to_half2(a[0]), e4m3x2_to_half2(a[0] >> 16),
                           e4m3x2_to_half2(a[1]), e4m3x2_to_half2(a[1] >> 16));
              st_shared_v4(at + (((ch + (odd ? 0 : 1)) ^ sw) << 4), e4m3x2_to_half2(b[0]), e4m3x2_to_half2(b[0] >> 16),
                           e4m3x2_to_half2(b[1]), e4m3x2_to_half2(b[1] >> 16));
            }
          }
        } else {
          // own tile, loaded as bf16: key i's values over the tile's scale, in place (rows behind the sequence's
          // belong to others: zero)
          const bool mine = i < left_l - (j - nk) * kUnit;
          const float f = exp2_int(-kinfo[w % NI].lv[0][0]);
#pragma unroll 2
          for (int x = 0; x < HD / 8; ++x) {
            const uint32_t at = dst + (x >> 3) * kSlot + i * 128 + (((x ^ i) & 7) << 4);
            const uint4 v = ld_shared_v4(at);
            const uint32_t b[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              h[y] = mine ? pack_f16x2(__uint_as_float(b[y] << 16) * f, __uint_as_float(b[y] & 0xffff0000u) * f) : 0u;
            st_shared_v4(at, h[0], h[1], h[2], h[3]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(BAR(B_WF + slot));
        mbar_arrive(BAR(B_VE + slot));
      }
    }
  }

  __syncthreads();
  if (*abort_flag) drain_after_abort(200);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool KS, bool FINE>
cudaError_t launch(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  auto k = bdlm_cached_tc_kernel<HD, KS, FINE>;
  // the register split needs the block's full allotment: refuse to launch otherwise
  static const cudaError_t ready = [&] {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, k);
    if (e != cudaSuccess) return e;
    return fa.numRegs == kLaunchRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
  }();
  if (ready != cudaSuccess) return ready;
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e = raise_smem(reinterpret_cast<const void*>(k), Lay<HD>::kAlloc, raised);
  if (e != cudaSuccess) return e;
  k<<<p.G, kThreads, Lay<HD>::kAlloc, st>>>(m.k8, m.k, m.v, p);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_d(const CachedMaps& m, const CachedParams& p, cudaStream_t st) {
  if (p.sp.tile_rows == 128)
    return p.o_f32 ? launch<HD, true, true>(m, p, st) : launch<HD, true, false>(m, p, st);
  return p.o_f32 ? launch<HD, false, true>(m, p, st) : launch<HD, false, false>(m, p, st);
}

}  // namespace

cudaError_t launch_cached_tc(const CachedMaps& m, const CachedParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? launch_d<128>(m, p, st) : launch_d<64>(m, p, st);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
