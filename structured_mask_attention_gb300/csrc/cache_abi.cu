// cache_abi.cu -- the C entry points of the 8-bit cache (include/bdlm_attn.h):
// argument validation and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <initializer_list>

#include "abi_internal.h"
#include "cache.cuh"
#include "cache_ops.h"
#include "cached_attn.h"
#include "kernels.h"
#include "tree_ops.h"

using namespace bdlm;

namespace {

#define CACHE_CHECK(expr)         \
  do {                            \
    bdlm_status _s = (expr);      \
    if (_s != BDLM_OK) return _s; \
  } while (0)

constexpr size_t kHeader = 256;
constexpr int kSmsMax = 160;  // workspace sizing: at least the SM count of a GB300 (152)

template <typename F>
bdlm_status guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& ex) {
    return abi_fail(BDLM_ERR_INVALID_ARG, "internal exception: %s", ex.what());
  } catch (...) {
    return abi_fail(BDLM_ERR_INVALID_ARG, "internal exception");
  }
}

bdlm_status check_ptr(const char* name, const void* p, unsigned align) {
  if (!p) return abi_fail(BDLM_ERR_INVALID_ARG, "%s is null", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return abi_fail(BDLM_ERR_ALIGN, "%s is not %u-byte aligned", name, align);
  return BDLM_OK;
}

bdlm_status check_cache(const bdlm_cache* c, CacheDesc* d) {
  if (!c) return abi_fail(BDLM_ERR_INVALID_ARG, "cache is null");
  if (c->d != 64 && c->d != 128) return abi_fail(BDLM_ERR_SHAPE, "head dim d=%d must be 64 or 128", c->d);
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
    return abi_fail(BDLM_ERR_SHAPE, "page=%d must be 16, 32, 64 or 128 tokens", c->page);
  if (c->Hkv <= 0 || c->Hkv > 4096) return abi_fail(BDLM_ERR_SHAPE, "Hkv=%d must be in [1, 4096]", c->Hkv);
  if (c->n_seqs <= 0 || c->n_seqs > 65535) return abi_fail(BDLM_ERR_SHAPE, "n_seqs=%d must be in [1, 65535]", c->n_seqs);
  if (c->n_pages <= 0 || c->n_pages > 0x7fffffff || c->n_pages * c->Hkv > 0x7fffffff)
    return abi_fail(BDLM_ERR_SHAPE, "n_pages=%lld: n_pages * Hkv must be in [1, 2^31)", (long long)c->n_pages);
  if (c->max_pages <= 0 || (int64_t)c->max_pages * c->page > (int64_t)1 << 30)
    return abi_fail(BDLM_ERR_SHAPE, "max_pages=%d: max_pages * page must be in [1, 2^30]", c->max_pages);
  CACHE_CHECK(check_ptr("cache k8", c->k8, 16));
  CACHE_CHECK(check_ptr("cache v8", c->v8, 16));
  CACHE_CHECK(check_ptr("cache k_scale", c->k_scale, 4));
  CACHE_CHECK(check_ptr("cache v_scale", c->v_scale, 4));
  CACHE_CHECK(check_ptr("cache page_table", c->page_table, 4));
  CACHE_CHECK(check_ptr("cache lens", c->lens, 4));
  int lp = 4;
  while ((1 << lp) < c->page) ++lp;
  *d = CacheDesc{static_cast<uint8_t*>(c->k8), static_cast<uint8_t*>(c->v8), c->k_scale, c->v_scale, c->page_table,
                 c->lens, c->n_pages, c->n_seqs, c->max_pages, c->page, lp, c->Hkv, c->d};
  return BDLM_OK;
}

bdlm_status check_rows(const CacheDesc& c, const int32_t* off, int64_t T, int64_t max_rows, RowsDesc* r) {
  if (max_rows <= 0 || max_rows > (int64_t)1 << 24)
    return abi_fail(BDLM_ERR_SHAPE, "max_rows=%lld must be in [1, 2^24]", (long long)max_rows);
  if (T < 0 || T > (int64_t)1 << 30) return abi_fail(BDLM_ERR_SHAPE, "rows=%lld must be in [0, 2^30]", (long long)T);
  if (off) {
    CACHE_CHECK(check_ptr("row_offsets", off, 4));
  } else if (T != max_rows * c.n_seqs) {
    return abi_fail(BDLM_ERR_SHAPE, "without row_offsets the tensors hold n_seqs * max_rows = %lld rows, not %lld",
                    (long long)(max_rows * c.n_seqs), (long long)T);
  }
  *r = RowsDesc{off, T, (int)max_rows};
  return BDLM_OK;
}

bdlm_status check_heads(const CacheDesc& c, const RowsDesc& r, int Hq, float scale) {
  if (Hq <= 0 || Hq > 4096 || Hq % c.Hkv)
    return abi_fail(BDLM_ERR_SHAPE, "Hq=%d must be a positive multiple of Hkv=%d, at most 4096", Hq, c.Hkv);
  if ((int64_t)r.max_rows * (Hq / c.Hkv) > (int64_t)1 << 29)
    return abi_fail(BDLM_ERR_SHAPE, "max_rows * Hq / Hkv exceeds 2^29");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return abi_fail(BDLM_ERR_INVALID_ARG, "scale=%g must be finite and > 0", scale);
  return BDLM_OK;
}

// An output must not share memory with an input that other CTAs still read.
bdlm_status check_apart(const char* out, const void* a, int64_t na, const char* in, const void* b, int64_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  if (x && y && x < y + nb && y < x + na) return abi_fail(BDLM_ERR_INVALID_ARG, "%s overlaps %s", out, in);
  return BDLM_OK;
}

bdlm_status check_lens_out(const int32_t* lens_out, const bdlm_cache* c) {
  const int64_t ns = 4 * (int64_t)c->n_seqs;
  CACHE_CHECK(check_apart("lens_out", lens_out, ns, "the cache's lens (read throughout the call)", c->lens, ns));
  return check_apart("lens_out", lens_out, ns, "page_table", c->page_table, ns * c->max_pages);
}

bdlm_status check_space(void* ws, size_t bytes, size_t need) {
  if (!ws) return abi_fail(BDLM_ERR_WORKSPACE, "workspace is null (need %zu bytes)", need);
  CACHE_CHECK(check_ptr("workspace", ws, 16));
  if (bytes < need) return abi_fail(BDLM_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  return BDLM_OK;
}

size_t attn_space(int64_t flat, int d) {
  const int tile = cached_tile_rows(flat);  // (a tree's may be 128 where this is 256: less)
  return (size_t)cached_ctas(tile, kSmsMax) * (2 * part_floats(tile, d) + fine_floats(tile, d)) * sizeof(float);
}

// Codes: boxes of one (page, KV head) block, swizzled by the row's bytes.
bdlm_status encode_codes(EncodeTiledFn fn, CUtensorMap* m, const CacheDesc& c, uint8_t* codes) {
  cuuint64_t dims[3] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)(c.n_pages * c.Hkv)};
  cuuint64_t strides[2] = {(cuuint64_t)c.d, (cuuint64_t)c.d * c.page};
  cuuint32_t box[3] = {(cuuint32_t)c.d, (cuuint32_t)c.page, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return abi_fail(BDLM_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  return BDLM_OK;
}

// [T, H, d] bf16: boxes of 64 columns, one head, 128 rows.
bdlm_status encode_rows(EncodeTiledFn fn, CUtensorMap* m, const void* p, int64_t T, int H, int d) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
  cuuint32_t box[3] = {64, 1, 128};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return abi_fail(BDLM_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  return BDLM_OK;
}
size_t kept_space(int n_seqs, int Hkv, int64_t keep) { return (size_t)n_seqs * Hkv * keep * sizeof(int32_t); }

// bdlm_cache_append, and with a path bdlm_cache_commit.
bdlm_status append_call(const void* K, const void* V, const bdlm_cache* cache, const int32_t* path, int64_t max_path,
                        const int32_t* accepted, const int32_t* row_offsets, int64_t rows, int64_t max_rows,
                        int32_t* lens_out, void* workspace, size_t ws_bytes, bdlm_stream stream) {
  CacheDesc c;
  RowsDesc r;
  CACHE_CHECK(check_cache(cache, &c));
  CACHE_CHECK(check_rows(c, row_offsets, rows, max_rows, &r));
  const int64_t ns = 4 * (int64_t)cache->n_seqs;
  if (path && (max_path <= 0 || max_path > (int64_t)1 << 24))
    return abi_fail(BDLM_ERR_SHAPE, "max_path=%lld must be in [1, 2^24]", (long long)max_path);
  if (rows > 0) {
    CACHE_CHECK(check_ptr("K", K, 16));
    CACHE_CHECK(check_ptr("V", V, 16));
  }
  if (lens_out) CACHE_CHECK(check_ptr("lens_out", lens_out, 4));
  CACHE_CHECK(check_lens_out(lens_out, cache));
  CACHE_CHECK(check_apart("lens_out", lens_out, ns, "row_offsets", row_offsets, ns + 4));
  CACHE_CHECK(check_apart("lens_out", lens_out, ns, "path", path, ns * max_path));
  CACHE_CHECK(check_apart("lens_out", lens_out, ns, "accepted", accepted, ns));
  CACHE_CHECK(check_space(workspace, ws_bytes, kHeader));
  int sms;
  CACHE_CHECK(abi_device(&sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int launches = 0;
  void* tm = abi_timer_begin(path ? ABI_T_COMMIT : ABI_T_APPEND, st);
  uint32_t* status = static_cast<uint32_t*>(workspace);
  cudaError_t e = path ? launch_cache_commit(CommitParams{c, r, K, V, path, accepted, (int)max_path, lens_out, status}, st,
                                             &launches)
                       : launch_cache_append(AppendParams{c, r, K, V, lens_out, status}, st, &launches);
  abi_timer_end(tm);
  return abi_finish(e, launches, path ? "cache commit launch" : "cache append launch");
}

// bdlm_attn_cached, and with visibility words bdlm_attn_tree.
bdlm_status attn_call(const void* Qn, const void* Kn, const void* Vn, const int32_t* visible, int64_t words,
                      const bdlm_cache* cache, const int32_t* row_offsets, int64_t rows, int64_t max_rows, int Hq,
                      float scale, void* O, bdlm_dtype o_dtype, float* LSE, void* workspace, size_t ws_bytes,
                      bdlm_stream stream) {
  CachedParams p;
  CACHE_CHECK(check_cache(cache, &p.c));
  CACHE_CHECK(check_rows(p.c, row_offsets, rows, max_rows, &p.r));
  CACHE_CHECK(check_heads(p.c, p.r, Hq, scale));
  if (o_dtype != BDLM_BF16 && o_dtype != BDLM_F32) return abi_fail(BDLM_ERR_INVALID_ARG, "bad o_dtype %d", (int)o_dtype);
  if (!Kn != !Vn) return abi_fail(BDLM_ERR_INVALID_ARG, "Kn and Vn: give both or neither");
  if (visible && max_rows > 32 * words)
    return abi_fail(BDLM_ERR_SHAPE, "%lld words hold the bits of fewer rows than max_rows=%lld", (long long)words,
                    (long long)max_rows);
  if (rows == 0) return BDLM_OK;
  CACHE_CHECK(check_ptr("Qn", Qn, 16));
  if (Kn) {
    CACHE_CHECK(check_ptr("Kn", Kn, 16));
    CACHE_CHECK(check_ptr("Vn", Vn, 16));
  }
  CACHE_CHECK(check_ptr("O", O, 16));
  CACHE_CHECK(check_ptr("LSE", LSE, 4));
  const int64_t nq = rows * Hq * p.c.d, nkv = rows * p.c.Hkv * p.c.d, no = nq * (o_dtype == BDLM_F32 ? 4 : 2);
  CACHE_CHECK(check_apart("O", O, no, "Qn", Qn, 2 * nq));
  CACHE_CHECK(check_apart("O", O, no, "Kn", Kn, 2 * nkv));
  CACHE_CHECK(check_apart("O", O, no, "Vn", Vn, 2 * nkv));
  const int64_t nl = 4 * rows * Hq;
  CACHE_CHECK(check_apart("LSE", LSE, nl, "O", O, no));
  CACHE_CHECK(check_apart("LSE", LSE, nl, "Qn", Qn, 2 * nq));
  CACHE_CHECK(check_apart("LSE", LSE, nl, "Kn", Kn, 2 * nkv));
  CACHE_CHECK(check_apart("LSE", LSE, nl, "Vn", Vn, 2 * nkv));
  CACHE_CHECK(check_apart("O", O, no, "visible", visible, 4 * rows * words));
  CACHE_CHECK(check_apart("LSE", LSE, nl, "visible", visible, 4 * rows * words));
  const int64_t flat = max_rows * (Hq / p.c.Hkv);
  CACHE_CHECK(check_space(workspace, ws_bytes, kHeader + attn_space(flat, p.c.d)));
  int sms;
  CACHE_CHECK(abi_device(&sms));
  p.sp.group = Hq / p.c.Hkv;
  p.sp.local = Kn != nullptr;
  p.Q = Qn;
  p.K = Kn;
  p.V = Vn;
  p.Hq = Hq;
  p.sl2 = scale * 1.4426950408889634f;
  p.vis = reinterpret_cast<const uint32_t*>(visible);
  p.words = (int)words;
  p.O = O;
  p.o_f32 = o_dtype == BDLM_F32;
  p.LSE = LSE;
  p.status = static_cast<uint32_t*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader);
  p.limit_ns = abi_wait_limit_ns();
  p.sp.tile_rows = visible ? tree_tile_rows(flat) : cached_tile_rows(flat);
  const bool small = p.sp.tile_rows <= kSmallRows;
  p.sp.extra = !small ? kTcExtra : visible ? kTreeExtra : Kn ? kSmallExtraOwn : kSmallExtra;
  p.sp.keyed = 0;
  p.whole = 0;
  p.G = cached_ctas(p.sp.tile_rows, std::min(sms, kSmsMax));
  p.fine = p.part + (int64_t)p.G * 2 * part_floats(p.sp.tile_rows, p.c.d);
  const int64_t rt = (flat + p.sp.tile_rows - 1) / p.sp.tile_rows;
  if (small && (int64_t)p.c.max_pages * p.c.page <= kWholeKeys && rt * p.c.Hkv * p.c.n_seqs <= 0x7fffffff) {
    p.whole = (int)rt;
    p.G = (int)(rt * p.c.Hkv * p.c.n_seqs);
  }
  CachedMaps maps;
  EncodeTiledFn enc;
  CACHE_CHECK(abi_encoder(&enc));
  CACHE_CHECK(encode_codes(enc, &maps.k8, p.c, p.c.k8));
  if (small) {
    CACHE_CHECK(encode_codes(enc, &maps.v8, p.c, p.c.v8));
  } else {
    // without own keys these maps are not used: any valid tensor encodes
    CACHE_CHECK(encode_rows(enc, &maps.k, Kn ? Kn : Qn, rows, Kn ? p.c.Hkv : Hq, p.c.d));
    CACHE_CHECK(encode_rows(enc, &maps.v, Vn ? Vn : Qn, rows, Vn ? p.c.Hkv : Hq, p.c.d));
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int launches = 0;
  void* tm = abi_timer_begin(ABI_T_ATTN_CACHED, st);
  cudaError_t e = visible ? (small ? launch_tree_small(maps, p, st, &launches) : launch_tree_tc(maps, p, st, &launches))
                  : small ? launch_cached_small(maps, p, st, &launches)
                          : launch_cached_tc(maps, p, st, &launches);
  abi_timer_end(tm);
  if (e == cudaSuccess && !p.whole) {
    tm = abi_timer_begin(ABI_T_CACHED_MERGE, st);
    e = launch_cached_merge(p, st, &launches);
    abi_timer_end(tm);
  }
  return abi_finish(e, launches, "cached attention launch");
}

// Row offsets of a call without a cache.
bdlm_status check_tree_rows(int n_seqs, const int32_t* off, int64_t T, int64_t max_rows, RowsDesc* r) {
  if (n_seqs <= 0 || n_seqs > 65535) return abi_fail(BDLM_ERR_SHAPE, "n_seqs=%d must be in [1, 65535]", n_seqs);
  CacheDesc c{};
  c.n_seqs = n_seqs;
  CACHE_CHECK(check_rows(c, off, T, max_rows, r));
  if (max_rows > kMaxTreeRows)
    return abi_fail(BDLM_ERR_SHAPE, "max_rows=%lld: a tree has at most %d rows", (long long)max_rows, kMaxTreeRows);
  return BDLM_OK;
}

}  // namespace

extern "C" {

size_t bdlm_workspace_size_cache(int n_seqs, int Hq, int Hkv, int d, int64_t max_rows, int64_t keep) {
  if (n_seqs <= 0 || n_seqs > 65535 || Hkv <= 0 || Hkv > 4096 || Hq < 0 || Hq > 4096 || Hq % Hkv ||
      (d != 64 && d != 128) || max_rows < 0 || max_rows > (int64_t)1 << 24 || keep < 0 || keep > (int64_t)1 << 30)
    return 0;
  const int64_t flat = max_rows * (Hq / Hkv);
  return kHeader + std::max(flat > 0 ? attn_space(flat, d) : 0, kept_space(n_seqs, Hkv, keep));
}

bdlm_status bdlm_cache_append(const void* K, const void* V, const bdlm_cache* cache, const int32_t* row_offsets,
                              int64_t rows, int64_t max_rows, int32_t* lens_out, void* workspace, size_t ws_bytes,
                              bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    return append_call(K, V, cache, nullptr, 0, nullptr, row_offsets, rows, max_rows, lens_out, workspace, ws_bytes,
                       stream);
  });
}

bdlm_status bdlm_cache_commit(const void* K, const void* V, const bdlm_cache* cache, const int32_t* path,
                              int64_t max_path, const int32_t* accepted, const int32_t* row_offsets, int64_t rows,
                              int64_t max_rows, int32_t* lens_out, void* workspace, size_t ws_bytes,
                              bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    CACHE_CHECK(check_ptr("path", path, 4));
    CACHE_CHECK(check_ptr("accepted", accepted, 4));
    return append_call(K, V, cache, path, max_path, accepted, row_offsets, rows, max_rows, lens_out, workspace, ws_bytes,
                       stream);
  });
}

bdlm_status bdlm_attn_cached(const void* Qn, const void* Kn, const void* Vn, const bdlm_cache* cache,
                             const int32_t* row_offsets, int64_t rows, int64_t max_rows, int Hq, float scale, void* O,
                             bdlm_dtype o_dtype, float* LSE, void* workspace, size_t ws_bytes, bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    return attn_call(Qn, Kn, Vn, nullptr, 0, cache, row_offsets, rows, max_rows, Hq, scale, O, o_dtype, LSE, workspace,
                     ws_bytes, stream);
  });
}

bdlm_status bdlm_attn_tree(const void* Qn, const void* Kn, const void* Vn, const int32_t* visible, int64_t words,
                           const bdlm_cache* cache, const int32_t* row_offsets, int64_t rows, int64_t max_rows, int Hq,
                           float scale, void* O, bdlm_dtype o_dtype, float* LSE, void* workspace, size_t ws_bytes,
                           bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    if (words <= 0 || words > (int64_t)1 << 19)
      return abi_fail(BDLM_ERR_SHAPE, "words=%lld must be in [1, 2^19]", (long long)words);
    if (rows != 0) {
      if (!Kn || !Vn) return abi_fail(BDLM_ERR_INVALID_ARG, "Kn and Vn: a tree's rows see themselves, give both");
      CACHE_CHECK(check_ptr("visible", visible, 4));
    }
    return attn_call(Qn, Kn, Vn, visible, words, cache, row_offsets, rows, max_rows, Hq, scale, O, o_dtype, LSE,
                     workspace, ws_bytes, stream);
  });
}

bdlm_status bdlm_cache_weights(const void* Qn, const float* LSE, const bdlm_cache* cache, const int32_t* row_offsets,
                               int64_t rows, int64_t max_rows, int Hq, float scale, float* weights, void* workspace,
                               size_t ws_bytes, bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    WeightsParams p;
    CACHE_CHECK(check_cache(cache, &p.c));
    CACHE_CHECK(check_rows(p.c, row_offsets, rows, max_rows, &p.r));
    CACHE_CHECK(check_heads(p.c, p.r, Hq, scale));
    if (rows == 0) return BDLM_OK;
    CACHE_CHECK(check_ptr("Qn", Qn, 16));
    CACHE_CHECK(check_ptr("LSE", LSE, 4));
    CACHE_CHECK(check_ptr("weights", weights, 16));
    const int64_t nw = 4 * (int64_t)cache->n_seqs * cache->Hkv * cache->max_pages * cache->page;
    CACHE_CHECK(check_apart("weights", weights, nw, "Qn", Qn, 2 * rows * Hq * p.c.d));
    CACHE_CHECK(check_apart("weights", weights, nw, "LSE", LSE, 4 * rows * Hq));
    CACHE_CHECK(check_space(workspace, ws_bytes, kHeader));
    // a sequence's units are counted in 32 bits
    const int64_t tiles = (max_rows * (Hq / p.c.Hkv) + 127) / 128, units = ((int64_t)p.c.max_pages * p.c.page + 127) / 128;
    if (tiles * units > (int64_t)1 << 30)
      return abi_fail(BDLM_ERR_SHAPE, "%lld row tiles by %lld key tiles of 128 exceed 2^30", (long long)tiles,
                      (long long)units);
    int sms;
    CACHE_CHECK(abi_device(&sms));
    p.Q = Qn;
    p.LSE = LSE;
    p.Hq = Hq;
    p.sl2 = scale * 1.4426950408889634f;
    p.W = weights;
    p.sp = AttnSplit{Hq / p.c.Hkv, 128, 0, kTcExtra, 1};
    p.G = std::min(sms, kSmsMax);
    p.status = static_cast<uint32_t*>(workspace);
    p.limit_ns = abi_wait_limit_ns();
    EncodeTiledFn enc;
    CUtensorMap k8;
    CACHE_CHECK(abi_encoder(&enc));
    CACHE_CHECK(encode_codes(enc, &k8, p.c, p.c.k8));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int launches = 0;
    void* tm = abi_timer_begin(ABI_T_WEIGHTS, st);
    cudaError_t e = launch_cache_weights(k8, p, st, &launches);
    abi_timer_end(tm);
    return abi_finish(e, launches, "cache weights launch");
  });
}

bdlm_status bdlm_cache_evict(const bdlm_cache* cache, const float* weights, const int32_t* dst_table, int64_t keep,
                             int64_t sinks, int64_t recent, int32_t* lens_out, float* weights_out, int32_t* kept,
                             void* workspace, size_t ws_bytes, bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    EvictParams p;
    CACHE_CHECK(check_cache(cache, &p.c));
    if (keep <= 0 || keep > (int64_t)1 << 30) return abi_fail(BDLM_ERR_SHAPE, "keep=%lld must be in [1, 2^30]", (long long)keep);
    if (sinks < 0 || recent < 0 || sinks > keep || recent > keep || sinks + recent > keep)
      return abi_fail(BDLM_ERR_SHAPE, "sinks=%lld and recent=%lld must be >= 0 and at most keep=%lld together",
                      (long long)sinks, (long long)recent, (long long)keep);
    CACHE_CHECK(check_ptr("weights", weights, 16));
    CACHE_CHECK(check_ptr("weights_out", weights_out, 16));
    CACHE_CHECK(check_ptr("dst_table", dst_table, 4));
    CACHE_CHECK(check_ptr("lens_out", lens_out, 4));
    if (kept) CACHE_CHECK(check_ptr("kept", kept, 4));
    const int64_t heads = (int64_t)cache->n_seqs * cache->Hkv, nw = 4 * heads * cache->max_pages * cache->page;
    const int64_t nt = 4 * (int64_t)cache->n_seqs * cache->max_pages, ns = 4 * (int64_t)cache->n_seqs;
    CACHE_CHECK(check_apart("weights_out", weights_out, nw, "weights", weights, nw));
    CACHE_CHECK(check_lens_out(lens_out, cache));
    CACHE_CHECK(check_apart("lens_out", lens_out, ns, "dst_table", dst_table, nt));
    CACHE_CHECK(check_apart("dst_table (tokens move to other pages)", dst_table, nt, "page_table", cache->page_table, nt));
    CACHE_CHECK(check_apart("kept", kept, 4 * heads * keep, "weights", weights, nw));
    CACHE_CHECK(check_apart("kept", kept, 4 * heads * keep, "weights_out", weights_out, nw));
    CACHE_CHECK(check_space(workspace, ws_bytes, kHeader + (kept ? 0 : kept_space(cache->n_seqs, cache->Hkv, keep))));
    int sms;
    CACHE_CHECK(abi_device(&sms));
    p.dst = dst_table;
    p.W = weights;
    p.W_out = weights_out;
    p.kept = kept ? kept : reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kHeader);
    p.lens_out = lens_out;
    p.keep = (int)keep;
    p.sinks = (int)sinks;
    p.recent = (int)recent;
    p.status = static_cast<uint32_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int launches = 0;
    void* tm = abi_timer_begin(ABI_T_EVICT, st);
    cudaError_t e = launch_cache_evict(p, st, &launches);
    abi_timer_end(tm);
    return abi_finish(e, launches, "cache evict launch");
  });
}

bdlm_status bdlm_tree_mask(const int32_t* parents, const bdlm_cache* cache, const int32_t* row_offsets, int64_t rows,
                           int64_t max_rows, int32_t* visible, int64_t words, int32_t* positions, void* workspace,
                           size_t ws_bytes, bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    TreeMaskParams p;
    CACHE_CHECK(check_cache(cache, &p.c));
    CACHE_CHECK(check_tree_rows(p.c.n_seqs, row_offsets, rows, max_rows, &p.r));
    if (words <= 0 || words > (int64_t)1 << 19)
      return abi_fail(BDLM_ERR_SHAPE, "words=%lld must be in [1, 2^19]", (long long)words);
    if (max_rows > 32 * words)
      return abi_fail(BDLM_ERR_SHAPE, "%lld words hold the bits of fewer rows than max_rows=%lld", (long long)words,
                      (long long)max_rows);
    if (rows == 0) return BDLM_OK;
    CACHE_CHECK(check_ptr("parents", parents, 4));
    CACHE_CHECK(check_ptr("visible", visible, 4));
    CACHE_CHECK(check_ptr("positions", positions, 4));
    const int64_t ns = 4 * (int64_t)cache->n_seqs, nr = 4 * rows;
    const struct { const char* name; const void* at; int64_t bytes; } in[3] = {
        {"parents", parents, nr}, {"row_offsets", row_offsets, ns + 4}, {"the cache's lens", cache->lens, ns}};
    for (const auto& x : in) {
      CACHE_CHECK(check_apart("visible", visible, nr * words, x.name, x.at, x.bytes));
      CACHE_CHECK(check_apart("positions", positions, nr, x.name, x.at, x.bytes));
    }
    CACHE_CHECK(check_apart("positions", positions, nr, "visible", visible, nr * words));
    CACHE_CHECK(check_space(workspace, ws_bytes, kHeader));
    int sms;
    CACHE_CHECK(abi_device(&sms));
    p.parents = parents;
    p.vis = reinterpret_cast<uint32_t*>(visible);
    p.words = (int)words;
    p.positions = positions;
    p.status = static_cast<uint32_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int launches = 0;
    void* tm = abi_timer_begin(ABI_T_TREE_MASK, st);
    cudaError_t e = launch_tree_mask(p, st, &launches);
    abi_timer_end(tm);
    return abi_finish(e, launches, "tree mask launch");
  });
}

size_t bdlm_workspace_size_verify(int n_seqs, int64_t max_rows, int64_t V) {
  if (n_seqs <= 0 || n_seqs > 65535 || max_rows <= 0 || max_rows > kMaxTreeRows || V <= 0 || V > (int64_t)1 << 30) return 0;
  return kHeader;
}

bdlm_status bdlm_tree_verify(const int32_t* parents, const int32_t* tokens, const void* target, const void* draft,
                             bdlm_dtype p_dtype, int64_t V, int64_t target_stride, int64_t draft_stride,
                             const float* uniforms, const float* sample, int n_seqs, const int32_t* row_offsets,
                             int64_t rows, int64_t max_rows, int32_t* path, int64_t max_path, int32_t* accepted,
                             int32_t* next_token, void* workspace, size_t ws_bytes, bdlm_stream stream) {
  return guarded([&]() -> bdlm_status {
    VerifyParams p;
    CACHE_CHECK(check_tree_rows(n_seqs, row_offsets, rows, max_rows, &p.r));
    if (p_dtype != BDLM_BF16 && p_dtype != BDLM_F32) return abi_fail(BDLM_ERR_INVALID_ARG, "bad p_dtype %d", (int)p_dtype);
    if (V <= 0 || V > (int64_t)1 << 30) return abi_fail(BDLM_ERR_SHAPE, "V=%lld must be in [1, 2^30]", (long long)V);
    if (max_path <= 0 || max_path > (int64_t)1 << 24)
      return abi_fail(BDLM_ERR_SHAPE, "max_path=%lld must be in [1, 2^24]", (long long)max_path);
    const int64_t e = p_dtype == BDLM_F32 ? 4 : 2, ns = 4 * (int64_t)n_seqs, nr = 4 * rows;
    const struct { const char* name; const void* at; int64_t stride; } probs[2] = {{"target", target, target_stride},
                                                                                 {"draft", draft, draft_stride}};
    for (const auto& x : probs) {
      if (&x == &probs[1] && !draft) break;
      if (rows > 0) CACHE_CHECK(check_ptr(x.name, x.at, (unsigned)e));
      if (x.stride < V || x.stride > (int64_t)1 << 40)
        return abi_fail(BDLM_ERR_SHAPE, "%s's rows are %lld values apart, at least V=%lld are needed", x.name,
                        (long long)x.stride, (long long)V);
      if (rows > 1 && x.stride > ((int64_t)1 << 58) / rows)  // (their bytes are counted in 64 bits below)
        return abi_fail(BDLM_ERR_SHAPE, "%s's rows end past 2^58 values", x.name);
    }
    if (rows > 0) {
      CACHE_CHECK(check_ptr("parents", parents, 4));
      CACHE_CHECK(check_ptr("tokens", tokens, 4));
      CACHE_CHECK(check_ptr("uniforms", uniforms, 4));
    }
    CACHE_CHECK(check_ptr("sample", sample, 4));
    CACHE_CHECK(check_ptr("path", path, 4));
    CACHE_CHECK(check_ptr("accepted", accepted, 4));
    CACHE_CHECK(check_ptr("next_token", next_token, 4));
    const struct { const char* name; const void* at; int64_t bytes; } out[3] = {
        {"path", path, ns * max_path}, {"accepted", accepted, ns}, {"next_token", next_token, ns}};
    const struct { const char* name; const void* at; int64_t bytes; } in[7] = {
        {"parents", parents, nr},
        {"tokens", tokens, nr},
        {"target", target, rows > 0 ? ((rows - 1) * target_stride + V) * e : 0},
        {"draft", draft, rows > 0 ? ((rows - 1) * draft_stride + V) * e : 0},
        {"uniforms", uniforms, nr},
        {"sample", sample, ns},
        {"row_offsets", row_offsets, ns + 4}};
    for (int i = 0; i < 3; ++i) {
      for (const auto& x : in) CACHE_CHECK(check_apart(out[i].name, out[i].at, out[i].bytes, x.name, x.at, x.bytes));
      for (int j = 0; j < i; ++j)
        CACHE_CHECK(check_apart(out[i].name, out[i].at, out[i].bytes, out[j].name, out[j].at, out[j].bytes));
    }
    CACHE_CHECK(check_space(workspace, ws_bytes, kHeader));
    int sms;
    CACHE_CHECK(abi_device(&sms));
    p.n_seqs = n_seqs;
    p.parents = parents;
    p.tokens = tokens;
    p.target = target;
    p.draft = draft;
    p.bf16 = p_dtype == BDLM_BF16;
    p.V = V;
    p.target_stride = target_stride;
    p.draft_stride = draft_stride;
    p.uniforms = uniforms;
    p.sample = sample;
    p.path = path;
    p.max_path = (int)max_path;
    p.accepted = accepted;
    p.next_token = next_token;
    p.status = static_cast<uint32_t*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int launches = 0;
    void* tm = abi_timer_begin(ABI_T_VERIFY, st);
    cudaError_t err = launch_tree_verify(p, sms, st, &launches);
    abi_timer_end(tm);
    return abi_finish(err, launches, "tree verify launch");
  });
}

}  // extern "C"
