// weights_tc.cu -- the attention weight that cached tokens receive, on the
// sm_103a tensor cores.
//
//   W[j] += sum over rows i of exp(s_ij - LSE_i)
// needs the sum of each *key* over all rows, so the scores are computed
// transposed: K's tile of 128 keys is the first operand (its e4m3 codes as TMA
// left them), the rows' queries the second (two 8-bit parts, cached_tc.cu), and
// S^T has a key per TMEM lane.  A thread then owns a key: its block's scale is
// a constant, the rows' factors and LSEs are read from shared memory by all
// threads together, the sum stays in two registers, and no two threads ever
// add to the same weight (no atomics).  All rows of a (sequence, KV head) are
// handled by the CTA that owns the key tile, 256 at a time.
// Bound: for few rows the stream of K's codes (32 sequences of 32768 tokens at
// most, 32 / 8 heads of 128, one token each: 126 us for 0.69 GB, 5.5 TB/s or
// 81 % of the measured copy rate; what the issuing thread does for a tile, 700
// cycles, is the rest of it: more K slots, more score buffers and weights added in
// L2 instead of read first were all level); from about 128 rows on the exponentials (one per
// row and key) and the products (blocks of 128 over 4 such sequences, 16 / 8
// heads: 45 us, 0.76 PFLOP/s; the tensor pipe 30 %, the exponentials' 36 % busy, a
// third of the time begins and ends the CTAs' two segments).  Not kept: both
// parts' products side by side as 2 N columns, added by the threads (162 us
// against 158 when it was tried).
// Roles (12 warps): warp 0 loads K, one lane of warp 1 issues the MMAs, warp 3
// walks the CTA's share of the list; warps 4-7 and 8-11 prepare the queries
// together and then take alternate key tiles (256 TMEM columns each).
#include "cache_ops.h"
#include "cached_tc.cuh"
#include "kernels.h"

namespace bdlm {
namespace {

constexpr int kThreads = 384;
constexpr int NK = 6;              // K slots of 128 keys
constexpr int NI = 16;             // tile-info slots (the K and S slots ahead of a reader, and a batch of four)
constexpr int NP = 4;              // piece slots
constexpr int kChunk = 256;        // rows at a time
constexpr int kSlot = 128 * 128;

enum { B_KF = 0, B_KE = NK, B_SF = 2 * NK, B_SE = B_SF + 2, B_QF = B_SE + 2, B_QD, B_KI, B_PCF = B_KI + NI,
       B_PCE = B_PCF + NP, B_COUNT = B_PCE + NP };

struct WInfo {
  float s[8];  // K's scale of each 16 keys
  int gone;    // bit x: no page
};
struct WPiece {
  int64_t row0;
  int s, h, len, rows;
  int j0, n;  // first key tile, tiles (-1: no more pieces)
};

template <int HD>
struct LayW {
  static constexpr int kQ = 0;                      // two parts of 256 rows
  static constexpr int kPart = kChunk * HD;
  static constexpr int kK = 2 * kPart;
  static constexpr int kRow = kK + NK * kSlot;      // two buffers of row pairs {c0, c1, n0, n1}
  static constexpr int kInfo = kRow + 2 * kChunk * 8;
  static constexpr int kPC = kInfo + NI * (int)sizeof(WInfo);
  static constexpr int kBar = (kPC + NP * (int)sizeof(WPiece) + 15) & ~15;
  static constexpr int kBytes = kBar + 8 * B_COUNT + 16;
  static constexpr int kAlloc = kBytes + 1024 > 120 * 1024 ? kBytes + 1024 : 120 * 1024;
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    bdlm_cache_weights_kernel(const __grid_constant__ CUtensorMap tK8, const WeightsParams p) {
  using LY = LayW<HD>;
  constexpr int SW = HD == 128 ? 2 : 4;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  auto BAR = [&](int i) -> uint32_t { return base + LY::kBar + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bp + LY::kBar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + LY::kBar + 8 * B_COUNT + 4);
  WInfo* infos = reinterpret_cast<WInfo*>(bp + LY::kInfo);
  WPiece* pieces = reinterpret_cast<WPiece*>(bp + LY::kPC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(BAR(B_KF + i), 1);
      mbar_init(BAR(B_KE + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(B_SF + i), 1);
      mbar_init(BAR(B_SE + i), 128);
    }
    mbar_init(BAR(B_QF), 256);
    mbar_init(BAR(B_QD), 1);
    for (int i = 0; i < NI; ++i) mbar_init(BAR(B_KI + i), 1);
    for (int i = 0; i < NP; ++i) {
      mbar_init(BAR(B_PCF + i), 1);
      mbar_init(BAR(B_PCE + i), 32 + 1 + 256);
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
  auto piece = [&](uint32_t n) -> const WPiece* {
    if (!mbar_wait(BAR(B_PCF + (n % NP)), (n / NP) & 1, wd, 60)) return nullptr;
    const WPiece* q = pieces + n % NP;
    return q->n < 0 ? nullptr : q;
  };
  auto done = [&](uint32_t n) { mbar_arrive(BAR(B_PCE + (n % NP))); };

  if (warp == 0) {
    // ---------------------------------------------- K loader
    uint32_t bad = 0, slot = 0, sph = 1, tc = 0;
    const uint32_t page_bytes = (uint32_t)(c.page * HD), page_groups = first_groups(c.page);
    bool ok = true;
    for (uint32_t np = 0; ok; ++np) {
      const WPiece* pp = piece(np);
      if (__any_sync(0xffffffffu, pp == nullptr)) break;
      const int len = pp->len, n = pp->n, j0 = pp->j0, h = pp->h;
      const int chunks = (pp->rows * p.sp.group + kChunk - 1) / kChunk;
      const int32_t* table = c.table + (int64_t)pp->s * c.max_pages;
      // lane 8 a + x: keys 16 x of tile a of a batch of 4 tiles, one batch ahead
      auto lookup = [&](int b) {
        const int tile = 4 * b + (lane >> 3), key = (j0 + tile) * kUnit + 16 * (lane & 7);
        return tile < n && key < len ? __ldg(table + (key >> c.lp)) : -1;
      };
      // (a batch's entries are looked at a batch after they were asked for)
      auto checked = [&](int id, int b) {
        if (id >= 0 && id < c.n_pages) return id;
        const int tile = 4 * b + (lane >> 3), key = (j0 + tile) * kUnit + 16 * (lane & 7);
        if (tile < n && key < len) bad |= kStatusBadPage;
        return -1;
      };
      auto scale_of = [&](int id) { return id >= 0 ? __ldg(c.ks + (int64_t)id * c.Hkv + h) : 0.f; };
      for (int ch = 0; ok && ch < chunks; ++ch) {
        const int raw0 = lookup(0);
        int raw1 = lookup(1);
        int id = checked(raw0, 0);
        float sc = scale_of(id);
        for (int b = 0; ok && 4 * b < n; ++b) {
          const int id1 = checked(raw1, b + 1);
          const float sc1 = scale_of(id1);
          const int raw2 = lookup(b + 2);
          // the batch's tiles, a group of eight lanes each
          const int grp = lane >> 3, x = lane & 7;
          const bool on = 4 * b + grp < n;
          const unsigned none = __ballot_sync(0xffffffffu, id < 0);
          WInfo& wi = infos[(tc + grp) % NI];
          if (on) wi.s[x] = sc;
          if (on && x == 0) wi.gone = (int)((none >> lane) & 0xffu);
          __syncwarp();
          if (on && x == 0) mbar_arrive(BAR(B_KI + (tc + grp) % NI));
          const uint32_t bytes = (uint32_t)__popc(~(none >> (lane & 24)) & page_groups) * page_bytes;
          const bool loads = id >= 0 && ((page_groups >> x) & 1);
          const int blk = (int)((int64_t)id * c.Hkv + h);
          for (int a = 0; a < 4 && 4 * b + a < n; ++a, ++tc) {
            ok = mbar_wait(BAR(B_KE + slot), sph, wd, 61);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 8 * a) {
              if (bytes) mbar_arrive_expect_tx(BAR(B_KF + slot), bytes);
              else mbar_arrive(BAR(B_KF + slot));
            }
            __syncwarp();
            if (grp == a && loads)  // the lane of a page's first keys loads it
              tma_load_3d(base + LY::kK + slot * kSlot + 16 * x * HD, &tK8, BAR(B_KF + slot), 0, 0, blk);
            if (++slot == NK) slot = 0, sph ^= 1;
          }
          id = id1; raw1 = raw2; sc = sc1;
        }
      }
      done(np);
    }
    if (bad) atomicOr(p.status + kContentsWord, bad);
  } else if (warp == 1) {
    // ---------------------------------------------- MMA issue
    if (lane == 0) {
      uint32_t slot = 0, kph = 0, qph = 0, tc = 0;
      bool ok = true;
      for (uint32_t np = 0; ok; ++np) {
        const WPiece* pp = piece(np);
        if (!pp) break;
        const int flat = pp->rows * p.sp.group, n = pp->n;
        done(np);
        for (int r0 = 0; ok && r0 < flat; r0 += kChunk) {
          const int N = (min(flat - r0, kChunk) + 31) & ~31;
          const uint32_t id = idesc_f8(128, N, kE4m3, kE4m3), id_lo = idesc_f8(128, N, kE4m3, kE5m2);
          ok = mbar_wait(BAR(B_QF), qph, wd, 62);
          qph ^= 1;
          if (!ok) break;
          tc_fence_after();
          for (int j = 0; j < n; ++j, ++tc) {
            const uint32_t buf = tc & 1;
            ok = mbar_wait(BAR(B_KF + slot), kph, wd, 64) && mbar_wait(BAR(B_SE + buf), ((tc >> 1) & 1) ^ 1, wd, 63);
            if (!ok) break;
            tc_fence_after();
            constexpr uint32_t H = desc_hi(SW, 8 * HD);
            const uint32_t k = desc_lo(base + LY::kK + slot * kSlot, 16), q = desc_lo(base + LY::kQ, 16);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk) mma_ss<true>(tmem + buf * 256, k + kk * 2, H, q + kk * 2, H, id, kk > 0);
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk)
              mma_ss<true>(tmem + buf * 256, k + kk * 2, H, q + (LY::kPart >> 4) + kk * 2, H, id_lo, 1);
            tc_commit(BAR(B_SF + buf));
            if (++slot == NK) slot = 0, kph ^= 1;
          }
          tc_commit(BAR(B_QD));
        }
      }
    }
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
        WPiece q;
        q.n = -1;
        while (u < u1 && q.n <= 0) {
          // key tiles whose first position lies in [u, u1)
          int b, e;
          split_units(seg, p.sp, pos, u, u1, b, e);
          const int w = seg.ltiles;
          q.j0 = (b + w - 1) / w;
          q.n = (e + w - 1) / w - q.j0;
          q.row0 = seg.v.row0;
          q.s = pos.s; q.h = pos.h; q.len = seg.v.len; q.rows = seg.v.rows;
          u += seg.span - pos.j;
          if (u < u1) next_segment(c, p.r, p.sp, pos, seg, bad);
        }
        if (q.n <= 0) q.n = -1;
        if (n >= NP && !mbar_wait(BAR(B_PCE + n % NP), (n / NP - 1) & 1, wd, 65)) break;
        pieces[n % NP] = q;
        mbar_arrive(BAR(B_PCF + n % NP));
        if (q.n < 0) break;
      }
    }
    if (bad) atomicOr(p.status + kContentsWord, bad);  // (each lane has looked at other sequences)
  } else if (warp >= 4) {
    // ---------------------------------------------- queries, then a key per thread
    const int t = (warp - 4) >> 2, tid = threadIdx.x - 128;
    const int key = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + t * 256;
    uint32_t tc = 0, sph = 0, qd = 0;
    bool ok = true;
    for (uint32_t np = 0; ok; ++np) {
      const WPiece* pp = piece(np);
      if (__any_sync(0xffffffffu, pp == nullptr)) break;
      const int flat = pp->rows * p.sp.group, n = pp->n, j0 = pp->j0, len = pp->len, h = pp->h;
      const int64_t row0 = pp->row0;
      float* W = p.W + ((int64_t)pp->s * c.Hkv + h) * ((int64_t)c.max_pages << c.lp);
      done(np);
      for (int r0 = 0; r0 < flat; r0 += kChunk) {
        const int cnt = min(flat - r0, kChunk), N = (cnt + 31) & ~31;
        // The rows' constants have two buffers, by the chunk's parity: the products'
        // end (B_QD) frees the query tiles, but one sub-tile may still be reading the
        // constants for its last key tile while the other writes the next chunk's.  It
        // comes to chunk c + 2, and chunk c's buffer, behind B_QF of chunk c + 1, where
        // all 256 threads arrive when they have left chunk c.
        float* const rows_c = reinterpret_cast<float*>(bp + LY::kRow) + (qd & 1) * 2 * kChunk;
        // ---- HD / 16 lanes take a row, 16 values each
        constexpr int PER = HD / 16;
        constexpr int RB = 4, RS = 256 / PER;  // rows in flight per thread, rows per pass
        const int i = tid % PER;
        for (int rb = tid / PER; rb < N; rb += RB * RS) {
          uint4 x[RB], y[RB];
          float lse[RB];
#pragma unroll
          for (int k = 0; k < RB; ++k) {
            const int r = rb + k * RS, fr = r0 + r, tok = fr / p.sp.group, head = h * p.sp.group + fr - tok * p.sp.group;
            const bool live = r < cnt;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.Q) +
                                                              ((row0 + (live ? tok : 0)) * p.Hq + head) * HD + 16 * i);
            x[k] = live ? __ldg(src) : make_uint4(0, 0, 0, 0);
            y[k] = live ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
            lse[k] = live && i == 0 ? __ldg(p.LSE + (int64_t)head * p.r.T + row0 + tok) : -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < RB; ++k) {
            const int r = rb + k * RS;
            if (r >= N) break;  // (N and RS are such that a warp's lanes agree)
            // a row without a key, or none at all, adds nothing, whatever its query holds
            const uint32_t on = __shfl_sync(0xffffffffu, lse[k], lane & ~(PER - 1)) == -INFINITY ? 0u : 0xffffffffu;
            const uint32_t w[8] = {x[k].x & on, x[k].y & on, x[k].z & on, x[k].w & on,
                                   y[k].x & on, y[k].y & on, y[k].z & on, y[k].w & on};
            const float nl = lse[k] == -INFINITY ? -INFINITY : lse[k] * -1.4426950408889634f;
            uint32_t amax = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) amax = __vmaxu2(amax, w[q] & 0x7fff7fffu);
            amax = max(amax & 0xffffu, amax >> 16);
#pragma unroll
            for (int o = PER / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            float inv;
            const float f = row_factor(amax, inv);
            uint32_t hi[4], lo[4];
            split_f8(w, f, hi, lo);
            const uint32_t at = base + LY::kQ + e4m3_chunk<HD>(r, i);
            st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(at + LY::kPart, lo[0], lo[1], lo[2], lo[3]);
            if (i == 0) {
              float* rp = rows_c + (r >> 1) * 4 + (r & 1);
              rp[0] = p.sl2 * inv;
              rp[2] = nl;
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(BAR(B_QF));
        // (the rows' constants are read by every thread: all have written theirs)
        ok = mbar_wait(BAR(B_QF), qd & 1, wd, 66);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float4* rowc = reinterpret_cast<const float4*>(rows_c);
        // (a tile's weights are read a tile ahead)
        auto old = [&](int j) { return j < n && (j0 + j) * kUnit + key < len ? W[(j0 + j) * kUnit + key] : 0.f; };
        float next = old((int)((tc ^ (uint32_t)t) & 1));
        for (int j = 0; j < n; ++j, ++tc) {
          if ((tc & 1) != (uint32_t)t) continue;
          const int at = (j0 + j) * kUnit + key;
          const float was = next;
          next = old(j + 2);
          ok = mbar_wait(BAR(B_KI + tc % NI), (tc / NI) & 1, wd, 67);
          const float ks = infos[tc % NI].s[key >> 4];
          const bool mine = at < len && !((infos[tc % NI].gone >> (key >> 4)) & 1);
          if (ok) ok = mbar_wait(BAR(B_SF + t), sph, wd, 68);
          sph ^= 1;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // (the products are done with K's slot; the issuing thread, which bounds short rows, is spared a commit)
          if ((tid & 127) == 0) mbar_arrive(BAR(B_KE + tc % NK));
          tc_fence_after();
          const uint64_t ks2 = f2(ks, ks);
          uint64_t sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
          auto add32 = [&](const uint32_t (&a)[32], int x) {
            float4 rc[16];  // {c0, c1, n0, n1} of two rows
#pragma unroll
            for (int y = 0; y < 16; ++y) rc[y] = rowc[(x >> 1) + y];
            float e[32];
#pragma unroll
            for (int y = 0; y < 16; ++y)
              f2_split(f2_fma(f2_mul(f2(__uint_as_float(a[2 * y]), __uint_as_float(a[2 * y + 1])), ks2),
                              f2(rc[y].x, rc[y].y), f2(rc[y].z, rc[y].w)),
                       e[2 * y], e[2 * y + 1]);
#pragma unroll
            for (int y = 0; y < 32; ++y) e[y] = ex2_approx(e[y]);
#pragma unroll
            for (int y = 0; y < 16; ++y) sum[y & 1] = f2_add(sum[y & 1], f2(e[2 * y], e[2 * y + 1]));
          };
          int x = 0;
          for (; x + 64 <= N; x += 64) {
            uint32_t a[32], b[32];
            tmem_ld32x2(tS + x, tS + x + 32, a, b);
            add32(a, x);
            add32(b, x + 32);
          }
          if (x < N) {
            uint32_t a[32];
            tmem_ld32(tS + x, a);
            add32(a, x);
          }
          tc_fence_before();
          mbar_arrive(BAR(B_SE + t));
          float s0, s1;
          f2_split(f2_add(sum[0], sum[1]), s0, s1);
          if (mine) W[at] = was + (s0 + s1);
        }
        if (!ok) break;
        // the chunk's products are through with the queries
        ok = mbar_wait(BAR(B_QD), qd & 1, wd, 69);
        ++qd;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
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

}  // namespace

template <int HD>
static cudaError_t launch(const CUtensorMap& k8, const WeightsParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e =
      raise_smem(reinterpret_cast<const void*>(bdlm_cache_weights_kernel<HD>), LayW<HD>::kAlloc, raised);
  if (e != cudaSuccess) return e;
  bdlm_cache_weights_kernel<HD><<<p.G, kThreads, LayW<HD>::kAlloc, st>>>(k8, p);
  return cudaGetLastError();
}

cudaError_t launch_cache_weights(const CUtensorMap& k8, const WeightsParams& p, cudaStream_t st, int* launches) {
  const cudaError_t e = p.c.d == 128 ? launch<128>(k8, p, st) : launch<64>(k8, p, st);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace bdlm
