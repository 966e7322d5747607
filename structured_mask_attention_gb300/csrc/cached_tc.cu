// cached_tc.cu -- attention of a block's rows over the 8-bit cache on the
// sm_103a tensor cores.
//
// S = Q K^T without touching K's codes: a bf16 query has 8 significant bits, so
// it is the exact sum of two e4m3 values of 4 bits each, and
// S = Qhi K^T + Qlo K^T are two kind::f8f6f4 products that cost together what
// one bf16 product would (e4m3 runs at twice its rate), with K's tiles taken
// as TMA leaves them.  (Each row of Q is first scaled by a power of two that
// puts its largest magnitude into [128, 256): exact for elements down to
// 2^-10 of it, off by at most 2^-18 of it below.)  Scores meet the key
// blocks' scales in the softmax, one multiplication per block that the
// exponent's fma absorbs.
// P V runs in bf16: P needs 8 bits, and the values code * scale (a power of two)
// are exact in bf16, so a warpgroup turns V's codes into a bf16 tile in shared
// memory while the tensor cores work on the tile before (16384 values against
// 32768 exponentials per 128 keys; splitting P in two e4m3 parts instead
// would triple the exponentials' cost).
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
// has units of its own; its Q is bf16, its V tile needs no conversion.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cached_attn.h"
#include "ptx.cuh"

namespace bdlm {
namespace {

constexpr int kThreads = 512;
constexpr int kRegsControl = 56, kRegsConvert = 72, kRegsSoftmax = 192;
constexpr int kLaunchRegs = 128;
static_assert(128 * (kRegsControl + kRegsConvert) + 256 * kRegsSoftmax <= kThreads * kLaunchRegs,
              "register split exceeds the block");
constexpr float kRescale = 8.0f;  // log2 units: the reference maximum moves in steps of at least this
constexpr int NK = 3;             // K slots: 128 keys of codes, or one 64-column panel of own keys
constexpr int NI = 8;             // tile-info slots (more than any two roles are apart)
constexpr int kSlot = 128 * 128;  // bytes of a K slot, of a V slot and of a bf16 panel

enum { B_QF = 0, B_KF = 2, B_KE = B_KF + NK, B_VF = B_KE + NK, B_VE = B_VF + 2, B_WF = B_VE + 2, B_WE = B_WF + 2,
       B_SF = B_WE + 2, B_PF = B_SF + 2, B_OD = B_PF + 2, B_OE = B_OD + 2, B_FD = B_OE + 2, B_P2 = B_FD + 2,
       B_ML = B_P2 + 2, B_KI = B_ML + 1, B_VI = B_KI + NI, B_COUNT = B_VI + NI };

struct KInfo {   // what the softmax needs of a tile
  float s[8];    // scale of each 16 keys
  int fine;      // scales differ inside 32 keys, or some keys are missing pages
  int gone;      // bit x: keys 16 x .. 16 x + 15 have no page
};
struct VInfo {
  float s[8];    // 0 where there is no page
};

template <int HD>
struct Lay {
  static constexpr int kQ = 0;                    // two regions of 128 rows x HD bf16 (or two e4m3 parts)
  static constexpr int kQBytes = 128 * HD * 2;
  static constexpr int kK = 2 * kQBytes;
  static constexpr int kV = kK + NK * kSlot;      // codes of V, 2 slots
  static constexpr int kW = kV + 2 * kSlot;       // bf16 V, 2 slots of HD / 64 panels
  static constexpr int kWBytes = kSlot * (HD / 64);
  static constexpr int kBar = kW + 2 * kWBytes;
  static constexpr int kKI = kBar + ((8 * B_COUNT + 16 + 15) & ~15);
  static constexpr int kVI = kKI + NI * (int)sizeof(KInfo);
  static constexpr int kML = kVI + NI * (int)sizeof(VInfo);
  static constexpr int kCQ = kML + 2 * 128 * 8;
  static constexpr int kBytes = kCQ + 128 * 4;
  // 1024 bytes to align; at least 120 KB so that no second CTA shares the SM (each holds all of TMEM)
  static constexpr int kAlloc = kBytes + 1024 > 120 * 1024 ? kBytes + 1024 : 120 * 1024;
};
static_assert(Lay<128>::kAlloc <= 232448, "shared memory");

// One CTA's share of a segment.
struct Piece {
  UnitPos pos;
  SegInfo seg;
  int nk, k0;   // cached tiles, the first
  int nl, l0;   // own tiles, the first
  bool whole, first;
};

struct PieceIter {
  int64_t u, u1;
  UnitPos pos;
  SegInfo seg;
};

// By a whole warp.
__device__ __forceinline__ PieceIter piece_begin(const CachedParams& p, uint32_t& bad) {
  PieceIter it;
  const int64_t U = total_units(p.c, p.r, p.sp, bad);
  const int G = split_ctas(U, p.G), cta = blockIdx.x;
  it.u = it.u1 = 0;
  if (cta < G) {
    it.u = split_begin(U, G, cta);
    it.u1 = split_begin(U, G, cta + 1);
    it.pos = locate_unit(p.c, p.r, p.sp, it.u, bad);
    it.seg = seg_info(p.c, p.r, p.sp, it.pos.s, bad);
  }
  return it;
}

// By any thread.
__device__ __forceinline__ bool piece_next(const CachedParams& p, PieceIter& it, Piece& pc, uint32_t& bad) {
  if (it.u >= it.u1) return false;
  const int jb = it.pos.j, je = (int)imin64(it.seg.units, jb + (it.u1 - it.u));
  pc.pos = it.pos;
  pc.seg = it.seg;
  const int kt = it.seg.ktiles;
  pc.k0 = jb;
  pc.nk = max(min(je, kt) - jb, 0);
  pc.l0 = max(jb - kt, 0);
  pc.nl = it.seg.ltiles > 0 ? max(je - kt, 0) - pc.l0 : (p.sp.local && je == it.seg.units ? 1 : 0);
  pc.first = jb == 0;
  pc.whole = jb == 0 && je == it.seg.units;
  it.u += je - jb;
  if (it.u < it.u1) next_segment(p.c, p.r, p.sp, it.pos, it.seg, bad);
  return true;
}

// 128-byte (SW = 2) or 64-byte (SW = 4) swizzled operand; see sdesc_sw128.
template <int SW>
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | ((uint64_t)SW << 61);
}

// D[tmem] (+)= A[smem] B[smem], e4m3 in, fp32 accumulator, K = 32.
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// fp32 accumulator, e4m3 A and B (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Contiguous copy into shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
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

// p = exp2(s f - m) of 32 scores in place; returns their sum.
__device__ __forceinline__ float exp32(uint32_t (&a)[32], float f, float nm) {
  const uint64_t f2x = f2(f, f), n2 = f2(nm, nm);
  float r0 = 0.f, r1 = 0.f;
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float x0, x1;
    f2_split(f2_fma(f2(__uint_as_float(a[c]), __uint_as_float(a[c + 1])), f2x, n2), x0, x1);
    x0 = ex2_approx(x0);
    x1 = ex2_approx(x1);
    r0 += x0;
    r1 += x1;
    a[c] = __float_as_uint(x0);
    a[c + 1] = __float_as_uint(x1);
  }
  return r0 + r1;
}

// Packs 32 values to bf16 at 16 columns of TMEM; REST: the values become what the rounding left.
template <bool REST>
__device__ __forceinline__ void store_p(uint32_t (&a)[32], uint32_t taddr) {
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const float x = __uint_as_float(a[c]), y = __uint_as_float(a[c + 1]);
    const uint32_t w = pack_bf16x2(x, y);
    pk[c / 2] = w;
    if (REST) {
      a[c] = __float_as_uint(x - __uint_as_float(w << 16));
      a[c + 1] = __float_as_uint(y - __uint_as_float(w & 0xffff0000u));
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
  VInfo* vinfo = reinterpret_cast<VInfo*>(bp + LY::kVI);
  // split only: both sub-tiles' states of the rows, and the rows' score factors
  float2* ml = reinterpret_cast<float2*>(bp + LY::kML);  // [2][128]
  float* row_cq = reinterpret_cast<float*>(bp + LY::kCQ);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(BAR(B_KF + i), 1);
      mbar_init(BAR(B_KE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(B_QF + i), 128);
      mbar_init(BAR(B_VF + i), 1);
      mbar_init(BAR(B_VE + i), 128);
      mbar_init(BAR(B_WF + i), 128);
      mbar_init(BAR(B_WE + i), 1);
      mbar_init(BAR(B_SF + i), 1);
      mbar_init(BAR(B_PF + i), 128);
      mbar_init(BAR(B_OD + i), 1);
      mbar_init(BAR(B_OE + i), KS ? 256 : 128);
      mbar_init(BAR(B_FD + i), 1);
      mbar_init(BAR(B_P2 + i), 128);
    }
    mbar_init(BAR(B_ML), 256);
    for (int i = 0; i < NI; ++i) {
      mbar_init(BAR(B_KI + i), 1);
      mbar_init(BAR(B_VI + i), 1);
    }
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
  const Watchdog wd{p.status, p.limit_ns, abort_flag};
  const CacheDesc& c = p.c;
  uint32_t bad = 0;

  if (warp < 4) {
    setmaxnreg_dec<kRegsControl>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------- loaders: K (warp 0), V (warp 2)
      // Lane 8 a + x looks up the page and scale of keys 16 x of tile a of a
      // batch of 4 tiles; the lookups of the next batch are in flight while
      // this one is loaded.
      const bool isV = warp == 2;
      const float* scales = isV ? c.vs : c.ks;
      PieceIter it = piece_begin(p, bad);
      Piece pc;
      uint32_t slot = 0, sph = 1, tc = 0;  // slot and its phase parity to wait for, tiles so far
      const int nslots = isV ? 2 : NK;
      bool ok = true;
      while (ok && piece_next(p, it, pc, bad)) {
        const int len = pc.seg.v.len;
        auto lookup = [&](int b) {  // page of this lane's 16 keys of batch b, -1: none
          const int tile = 4 * b + (lane >> 3), key = (pc.k0 + tile) * kUnit + 16 * (lane & 7);
          return tile < pc.nk && key < len ? page_id(c, pc.pos.s, key >> c.lp, bad) : -1;
        };
        auto scale_of = [&](int id) { return id >= 0 ? __ldg(scales + (int64_t)id * c.Hkv + pc.pos.h) : 0.f; };
        int id = lookup(0), id1 = lookup(1);
        float sc = scale_of(id);
        for (int b = 0; ok && 4 * b < pc.nk; ++b) {
          const float sc1 = scale_of(id1);
          const int id2 = lookup(b + 2);
          for (int a = 0; a < 4 && 4 * b + a < pc.nk; ++a, ++tc) {
            const int key0 = (pc.k0 + 4 * b + a) * kUnit;
            ok = mbar_wait(BAR((isV ? B_VE : B_KE) + slot), sph, wd, 20 + warp);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int x = lane & 7;
            const int cid = __shfl_sync(0xffffffffu, id, 8 * a + x);
            const float csc = __shfl_sync(0xffffffffu, sc, 8 * a + x);
            const unsigned none = __ballot_sync(0xffffffffu, cid < 0) & 0xffu;
            const uint32_t fb = BAR((isV ? B_VF : B_KF) + slot);
            if (isV) {
              if (lane < 8) vinfo[tc % NI].s[x] = csc;
            } else {
              const float peer = __shfl_xor_sync(0xffffffffu, csc, 1);
              const unsigned gone = __ballot_sync(0xffffffffu, cid < 0 && key0 + 16 * x < len) & 0xffu;
              const unsigned odd = __ballot_sync(0xffffffffu, cid >= 0 && key0 + 16 * (x | 1) < len && csc != peer) & 0xffu;
              if (lane < 8) kinfo[tc % NI].s[x] = csc;
              if (lane == 0) {
                kinfo[tc % NI].fine = (gone | odd) != 0;
                kinfo[tc % NI].gone = (int)gone;
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR((isV ? B_VI : B_KI) + tc % NI));
            // pages of the tile that hold keys: lane q loads page q
            const int per = kUnit >> c.lp, step = c.page >> 4;  // pages per tile, 16-key groups per page
            int n = 0;
            for (int q = 0; q < per; ++q) n += !((none >> (q * step)) & 1u);
            if (lane == 0) {
              if (n) mbar_arrive_expect_tx(fb, (uint32_t)(n * c.page * HD));
              else mbar_arrive(fb);
            }
            __syncwarp();
            const int pid = __shfl_sync(0xffffffffu, cid, (lane * step) & 7);
            if (lane < per && pid >= 0) {
              const uint32_t dst = base + (isV ? LY::kV : LY::kK) + slot * kSlot + lane * c.page * HD;
              const int64_t blk = (int64_t)pid * c.Hkv + pc.pos.h;
              if (isV) bulk_load(dst, c.v8 + blk * c.page * HD, (uint32_t)(c.page * HD), fb);
              else tma_load_3d(dst, &tK8, fb, 0, 0, (int)blk);
            }
            if (++slot == (uint32_t)nslots) slot = 0, sph ^= 1;
          }
          id = id1; id1 = id2; sc = sc1;
        }
        // own tiles: K by panels through the K slots; V straight into the bf16 slot that its tile has
        for (int l = 0; ok && l < pc.nl; ++l, ++tc) {
          const int row = (int)(pc.seg.v.row0 + (int64_t)(pc.l0 + l) * kUnit);
          if (lane == 0) {
            if (!isV)
              for (int x = 0; x < 8; ++x) kinfo[tc % NI].s[x] = 1.f;
            if (!isV) kinfo[tc % NI].fine = kinfo[tc % NI].gone = 0;
            mbar_arrive(BAR((isV ? B_VI : B_KI) + tc % NI));
          }
          if (isV) {
            ok = mbar_wait(BAR(B_VE + slot), sph, wd, 24);
            if (ok) ok = mbar_wait(BAR(B_WE + slot), sph, wd, 25);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(BAR(B_VF + slot), LY::kWBytes);
              for (int pn = 0; pn < KP; ++pn)
                tma_load_3d(base + LY::kW + slot * LY::kWBytes + pn * kSlot, &tV, BAR(B_VF + slot), 64 * pn, pc.pos.h, row);
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
                tma_load_3d(base + LY::kK + slot * kSlot, &tK, BAR(B_KF + slot), 64 * pn, pc.pos.h, row);
              }
              if (++slot == NK) slot = 0, sph ^= 1;
            }
          }
        }
      }
      if (bad) atomicOr(p.status, bad);
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issue
      PieceIter it = piece_begin(p, bad);
      if (lane == 0) {
        constexpr uint32_t kId8 = idesc_e4m3(128, 128);
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdO = idesc_bf16(128, HD, false, true);
        Piece pc;
        uint32_t ks = 0, kph = 0;            // next K slot and its full parity
        uint32_t qph[2] = {0, 0};            // parity of Q's next full phase (split: of Q8, of bf16 Q)
        uint32_t wc = 0;                     // V tiles multiplied so far
        uint32_t st[2] = {0, 0};             // tiles of each sub-tile so far
        uint32_t itn[2] = {0, 0};            // pieces of each sub-tile so far
        bool ok = true;
        // slots of the tile whose S is being issued; waits for its keys
        uint32_t cur[2], ncur = 0;
        auto take_k = [&](bool own) {
          ncur = own ? KP : 1;
          for (uint32_t i = 0; i < ncur; ++i) {
            cur[i] = ks;
            if (!mbar_wait(BAR(B_KF + ks), kph, wd, 30)) return false;
            if (++ks == NK) ks = 0, kph ^= 1;
          }
          tc_fence_after();
          return true;
        };
        auto free_k = [&]() {
          for (uint32_t i = 0; i < ncur; ++i) tc_commit(BAR(B_KE + cur[i]));
        };
        auto issue_s = [&](int t, bool own) {
          if (!own) {
            const uint32_t q = base + LY::kQ + (KS ? 0 : t) * LY::kQBytes;
            const uint64_t hi = sdesc<SWQ>(q, 16, SBO8), lo = sdesc<SWQ>(q + 128 * HD, 16, SBO8);
            const uint64_t k = sdesc<SWQ>(base + LY::kK + cur[0] * kSlot, 16, SBO8);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) tc_mma_f8(tmem + t * 128, desc_add(hi, kk * 32), desc_add(k, kk * 32), kId8, kk > 0);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) tc_mma_f8(tmem + t * 128, desc_add(lo, kk * 32), desc_add(k, kk * 32), kId8, 1);
          } else {
            const uint32_t q = base + LY::kQ + (KS ? 1 : t) * LY::kQBytes;
#pragma unroll
            for (int pn = 0; pn < KP; ++pn) {
              const uint64_t a = sdesc_sw128(q + pn * kSlot, 16, 1024);
              const uint64_t k = sdesc_sw128(base + LY::kK + cur[pn] * kSlot, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_ss(tmem + t * 128, desc_add(a, kk * 32), desc_add(k, kk * 32), kIdS, (pn | kk) > 0);
            }
          }
          tc_commit(BAR(B_SF + t));
        };
        // O_t += P_t V of V tile w
        auto pv = [&](int t, uint32_t w, uint32_t col, bool first) {
          const uint64_t v = sdesc_sw128(base + LY::kW + (w & 1) * LY::kWBytes, kSlot, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(tmem + 256 + t * 128, tmem + t * 128 + col + kk * 8, desc_add(v, kk * 2048), kIdO,
                      (kk > 0 || !first) ? 1u : 0u);
        };
        auto issue_pv = [&](int t, uint32_t w, bool first) {
          if (!mbar_wait(BAR(B_PF + t), st[t] & 1, wd, 31)) return false;
          if (first && itn[t] > 0 && !mbar_wait(BAR(B_OE + t), (itn[t] - 1) & 1, wd, 32)) return false;
          if (!mbar_wait(BAR(B_WF + (w & 1)), (w >> 1) & 1, wd, 33)) return false;
          tc_fence_after();
          pv(t, w, 0, first);
          if (FINE) {
            pv(t, w, 64, false);
            tc_commit(BAR(B_FD + t));
            if (!mbar_wait(BAR(B_P2 + t), st[t] & 1, wd, 34)) return false;
            tc_fence_after();
            pv(t, w, 0, false);
          }
          ++st[t];
          return true;
        };
        while (ok && piece_next(p, it, pc, bad)) {
          const int n = pc.nk + pc.nl;
          if (n == 0) continue;
          auto own = [&](int j) { return j >= pc.nk; };
          // Q of sub-tile t (split: of kind t) has to be there before the first tile of each kind
          auto wait_q = [&](int t) {
            const bool r = mbar_wait(BAR(B_QF + t), qph[t], wd, 35);
            qph[t] ^= 1;
            if (r) tc_fence_after();
            return r;
          };
          if (KS) {
            auto start_s = [&](int j) {
              if ((j == 0 || j == pc.nk) && !wait_q(own(j) ? 1 : 0)) return false;
              if (!take_k(own(j))) return false;
              issue_s(j & 1, own(j));
              free_k();
              return true;
            };
            ok = start_s(0) && (n < 2 || start_s(1));
            for (int j = 0; ok && j < n; ++j, ++wc) {
              const int t = j & 1;
              ok = issue_pv(t, wc, j < 2);
              if (!ok) break;
              tc_commit(BAR(B_WE + (wc & 1)));
              if (j + 2 >= n) {
                tc_commit(BAR(B_OD + t));
                ++itn[t];
              } else {
                ok = start_s(j + 2);
              }
            }
          } else {
            ok = wait_q(0) && take_k(own(0));
            if (ok) issue_s(0, own(0));
            ok = ok && wait_q(1);
            if (ok) {
              issue_s(1, own(0));
              free_k();
            }
            for (int j = 0; ok && j < n; ++j, ++wc) {
              const bool last = j == n - 1, swap = j + 1 == pc.nk && pc.nk > 0 && !last;
              ok = issue_pv(0, wc, j == 0);
              if (!ok) break;
              if (last) tc_commit(BAR(B_OD + 0));
              if (!last) {
                ok = (!swap || wait_q(0)) && take_k(own(j + 1));
                if (!ok) break;
                issue_s(0, own(j + 1));
              }
              ok = issue_pv(1, wc, j == 0);
              if (!ok) break;
              tc_commit(BAR(B_WE + (wc & 1)));
              if (last) {
                tc_commit(BAR(B_OD + 1));
              } else {
                ok = !swap || wait_q(1);
                if (!ok) break;
                issue_s(1, own(j + 1));
                free_k();
              }
            }
            ++itn[0];
            ++itn[1];
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
    PieceIter it = piece_begin(p, bad);
    Piece pc;
    uint32_t sc = 0, tcount = 0, itn[2] = {0, 0}, mlc = 0, q8c = 0;
    bool ok = true;
    while (ok && piece_next(p, it, pc, bad)) {
      const int n = pc.nk + pc.nl;
      const int64_t fr = (int64_t)pc.pos.rt * kTileRows + (KS ? 0 : t * 128) + row;
      const int64_t tok = fr / p.sp.group;
      const bool live = tok < pc.seg.v.rows;
      const int head = pc.pos.h * p.sp.group + (int)(fr - tok * p.sp.group);
      const int64_t grow = pc.seg.v.row0 + (live ? tok : 0);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.Q) + (grow * p.Hq + head) * HD;
      float cq = p.sl2;

      // Q's row to shared memory: e4m3 in two parts, or bf16
      auto put_q8 = [&]() {
        const uint32_t dst = base + LY::kQ + (KS ? 0 : t) * LY::kQBytes;
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) amax = max(amax, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
        }
        int e = 7 + 127 - (int)(amax >> 7);
        if (amax >= 0x7f80u || amax == 0) e = 0;
        const bool nan = amax >= 0x7f80u;  // e4m3 has no infinity: a row that is not finite reads NaN
        e = min(e, 126);
        const float f = nan ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(e + 127) << 23);
        cq = p.sl2 * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 2
        for (int i = 0; i < HD / 16; ++i) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(q) + 2 * i + y) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t h[4], l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = __uint_as_float(w[k] << 16) * f, b = __uint_as_float(w[k] & 0xffff0000u) * f;
              h[k] = to_e4m3x2(a, b);
              const uint32_t hh = e4m3x2_to_half2(h[k]);
              const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&hh));
              l[k] = to_e4m3x2(a - r.x, b - r.y);
            }
            hi[2 * y] = h[0] | h[1] << 16; hi[2 * y + 1] = h[2] | h[3] << 16;
            lo[2 * y] = l[0] | l[1] << 16; lo[2 * y + 1] = l[2] | l[3] << 16;
          }
          const uint32_t at = HD == 128 ? (uint32_t)(row * 128 + ((i ^ (row & 7)) << 4))
                                        : (uint32_t)(row * 64 + ((i ^ ((row >> 1) & 3)) << 4));
          st_shared_v4(dst + at, hi[0], hi[1], hi[2], hi[3]);
          st_shared_v4(dst + 128 * HD + at, lo[0], lo[1], lo[2], lo[3]);
        }
      };
      auto put_q16 = [&]() {
        const uint32_t dst = base + LY::kQ + (KS ? 1 : t) * LY::kQBytes;
#pragma unroll 4
        for (int i = 0; i < HD / 8; ++i) {
          const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
          st_shared_v4(dst + (i >> 3) * kSlot + row * 128 + (((i & 7) ^ (row & 7)) << 4), x.x, x.y, x.z, x.w);
        }
      };
      if (n > 0) {
        if (KS) {
          // sub-tile 0's threads write the codes, sub-tile 1's the bf16 rows
          if (t == 0 && pc.nk > 0) {
            put_q8();
            row_cq[row] = cq;
            fence_proxy_async_smem();
            mbar_arrive(BAR(B_QF + 0));
          }
          if (t == 1 && pc.nl > 0) {
            put_q16();
            fence_proxy_async_smem();
            mbar_arrive(BAR(B_QF + 1));
          }
        } else {
          if (pc.nk > 0) put_q8();
          else put_q16();
          fence_proxy_async_smem();
          mbar_arrive(BAR(B_QF + t));
        }
      }
      float m_ref = -INFINITY, l = 0.f;
      bool have_cq = !KS || t == 0;
      for (int j = KS ? t : 0; j < n; j += KS ? 2 : 1, ++sc) {
        const bool own = j >= pc.nk;
        const uint32_t ti = tcount + (uint32_t)j;
        ok = mbar_wait(BAR(B_SF + t), sc & 1, wd, 40);
        if (ok) ok = mbar_wait(BAR(B_KI + ti % NI), (ti / NI) & 1, wd, 41);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (KS && !have_cq && !own) {
          // the factor that sub-tile 0's thread found (this phase of QF cannot
          // be followed by the next before the piece's end, which needs this thread)
          ok = mbar_wait(BAR(B_QF + 0), q8c & 1, wd, 42);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          cq = row_cq[row];
          have_cq = true;
        }
        const KInfo& ki = kinfo[ti % NI];
        uint32_t a0[32], a1[32], a2[32], a3[32];
        tmem_ld32x4(tS, tS + 32, tS + 64, tS + 96, a0, a1, a2, a3);
        const int key0 = own ? (pc.l0 + j - pc.nk) * kUnit : (pc.k0 + j) * kUnit;
        const int hi = (own ? pc.seg.v.rows : pc.seg.v.len) - key0;
        const float rf = own ? p.sl2 : cq;
        float f0 = rf * ki.s[0], f1 = rf * ki.s[2], f2_ = rf * ki.s[4], f3 = rf * ki.s[6];
        if (ki.fine) {  // a scale for each 16 keys, keys without a page
          const int gone = ki.gone;
#pragma unroll
          for (int c8 = 0; c8 < 32; ++c8) {
            const int x = c8 >> 4;
            a0[c8] = (gone >> x) & 1 ? __float_as_uint(-INFINITY) : __float_as_uint(__uint_as_float(a0[c8]) * (rf * ki.s[x]));
            a1[c8] = (gone >> (2 + x)) & 1 ? __float_as_uint(-INFINITY) : __float_as_uint(__uint_as_float(a1[c8]) * (rf * ki.s[2 + x]));
            a2[c8] = (gone >> (4 + x)) & 1 ? __float_as_uint(-INFINITY) : __float_as_uint(__uint_as_float(a2[c8]) * (rf * ki.s[4 + x]));
            a3[c8] = (gone >> (6 + x)) & 1 ? __float_as_uint(-INFINITY) : __float_as_uint(__uint_as_float(a3[c8]) * (rf * ki.s[6 + x]));
          }
          f0 = f1 = f2_ = f3 = 1.f;
        }
        if (hi < kUnit) {
          mask32(a0, hi);
          mask32(a1, hi - 32);
          mask32(a2, hi - 64);
          mask32(a3, hi - 96);
          if (hi <= 32) f1 = f0;  // (blocks behind the end have no scale: any finite factor keeps -inf)
          if (hi <= 64) f2_ = f0;
          if (hi <= 96) f3 = f0;
        }
        const float mx = fmaxf(fmaxf(max32(a0) * f0, max32(a1) * f1), fmaxf(max32(a2) * f2_, max32(a3) * f3));
        bool rescale = false;
        float alpha = 1.f;
        if (m_ref == -INFINITY) {
          m_ref = mx;  // first keys of this row (O holds zeros)
        } else if (mx > m_ref + kRescale) {
          alpha = ex2_approx(m_ref - mx);
          m_ref = mx;
          rescale = true;
        }
        const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
        float sum = exp32(a0, f0, nm);
        sum += exp32(a1, f1, nm);
        sum += exp32(a2, f2_, nm);
        sum += exp32(a3, f3, nm);
        l = fmaf(l, alpha, sum);
        store_p<FINE>(a0, tS);
        store_p<FINE>(a1, tS + 16);
        store_p<FINE>(a2, tS + 32);
        store_p<FINE>(a3, tS + 48);
        if (FINE) {
          store_p<true>(a0, tS + 64);
          store_p<true>(a1, tS + 80);
          store_p<true>(a2, tS + 96);
          store_p<true>(a3, tS + 112);
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
        if (FINE) {  // the third part, once the first two are multiplied
          ok = mbar_wait(BAR(B_FD + t), sc & 1, wd, 43);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          store_p<false>(a0, tS);
          store_p<false>(a1, tS + 16);
          store_p<false>(a2, tS + 32);
          store_p<false>(a3, tS + 48);
          tc_fence_before();
          mbar_arrive(BAR(B_P2 + t));
        }
        if (!KS && j == pc.nk - 1 && pc.nl > 0) {  // the cached keys are through with Q's codes
          put_q16();
          fence_proxy_async_smem();
          mbar_arrive(BAR(B_QF + t));
        }
      }
      if (!ok) break;
      tcount += (uint32_t)n;
      if (pc.nk > 0) ++q8c;

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
      }
      tc_fence_after();
      const float inv = L != 0.f ? 1.f / L : 0.f;
      const float s0 = pc.whole ? w0 * inv : w0, s1 = pc.whole ? w1 * inv : w1;
      float* slot = p.part + (2 * (int64_t)blockIdx.x + (pc.first ? 1 : 0)) * part_floats(kTileRows, HD);
      const int prow = (KS ? 0 : t * 128) + row;
      const int64_t oofs = (grow * p.Hq + head) * HD;
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
        if (live) {
          if (!pc.whole || p.o_f32) {
            float4* d = reinterpret_cast<float4*>(pc.whole ? static_cast<float*>(p.O) + oofs + col
                                                           : slot + (int64_t)prow * HD + col);
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
      if (live && (!KS || t == 0)) {
        if (pc.whole) {
          p.LSE[(int64_t)head * p.r.T + grow] = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        } else {
          slot[(int64_t)kTileRows * HD + prow] = M;
          slot[(int64_t)kTileRows * (HD + 1) + prow] = L;
        }
      }
    }
  } else {
    // ------------------------------------------------ V's codes -> bf16
    setmaxnreg_dec<kRegsConvert>();
    const int i = threadIdx.x - 384;
    constexpr int CH = HD / 16;             // 16-code chunks of a key
    PieceIter it = piece_begin(p, bad);
    Piece pc;
    uint32_t w = 0;
    bool ok = true;
    while (ok && piece_next(p, it, pc, bad)) {
      for (int j = 0; j < pc.nk + pc.nl; ++j, ++w) {
        const uint32_t slot = w & 1, ph = (w >> 1) & 1;
        ok = mbar_wait(BAR(B_VF + slot), ph, wd, 50) && mbar_wait(BAR(B_WE + slot), ph ^ 1, wd, 51) &&
             mbar_wait(BAR(B_VI + w % NI), (w / NI) & 1, wd, 52);
        if (!ok) break;
        const uint32_t dst = base + LY::kW + slot * LY::kWBytes;
        if (j < pc.nk) {
          const uint32_t src = base + LY::kV + slot * kSlot;
          const int left = pc.seg.v.len - (pc.k0 + j) * kUnit;
          const VInfo& vi = vinfo[w % NI];
#pragma unroll 4
          for (int x = 0; x < CH; ++x) {
            const int id = x * 128 + i, key = id / CH, c16 = id % CH;
            uint4 v = ld_shared_v4(src + id * 16);
            float s = vi.s[key >> 4];
            if (key >= left || s == 0.f) {  // stale codes (or none) may be anything
              v = make_uint4(0, 0, 0, 0);
              s = 0.f;
            }
            const uint32_t wd4[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[8];
            const uint64_t s2 = f2(s, s);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t h = e4m3x2_to_half2(wd4[k] >> (16 * y));
                const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&h));
                float z0, z1;
                f2_split(f2_mul(f2(z.x, z.y), s2), z0, z1);
                o[2 * k + y] = pack_bf16x2(z0, z1);
              }
            // 8-value chunks 2 c16, 2 c16 + 1 of the key; the second panel's threads write them in the other
            // order, so that the 8 lanes of a store phase cover all banks
            const uint32_t at = dst + (c16 >> 2) * kSlot + key * 128;
            const uint32_t ch = (uint32_t)(c16 & 3) * 2, sw = (uint32_t)key & 7u;
            const bool odd = c16 >= 4;
            st_shared_v4(at + (((ch + (odd ? 1 : 0)) ^ sw) << 4), odd ? o[4] : o[0], odd ? o[5] : o[1], odd ? o[6] : o[2], odd ? o[7] : o[3]);
            st_shared_v4(at + (((ch + (odd ? 0 : 1)) ^ sw) << 4), odd ? o[0] : o[4], odd ? o[1] : o[5], odd ? o[2] : o[6], odd ? o[3] : o[7]);
          }
        } else {
          // own tile, loaded as bf16: rows behind the sequence's belong to others
          const int left = pc.seg.v.rows - (pc.l0 + j - pc.nk) * kUnit;
          if (i >= left)
            for (int x = 0; x < HD / 8; ++x) st_shared_v4(dst + (x >> 3) * kSlot + i * 128 + (x & 7) * 16, 0, 0, 0, 0);
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
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<HD>::kAlloc);
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
