// C ABI of the cache calls (declared in include/mla.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/mla.h"
#include "mla_cache.cuh"
#include "mla_common.cuh"

using namespace mla;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

mla_status_t validate(const mla_cache_t* c) {
  if (!c || c->num_pages < 1 || c->page_table_stride < 1 || c->page_size < 1) return MLA_ERR_INVALID_ARG;
  if ((c->dtype != MLA_BF16 && c->dtype != MLA_E4M3) || !aligned(c->kept, 4)) return MLA_ERR_INVALID_ARG;
  if ((c->page_size & (c->page_size - 1)) != 0 || c->page_size < kMinPageSize || c->page_size > kMaxPageSize)
    return MLA_ERR_UNSUPPORTED;
  if ((long long)c->page_table_stride * c->page_size > (1ll << 30) || c->num_pages > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

int shift_of(const mla_cache_t* c) {
  int s = 0;
  while ((1 << s) < c->page_size) ++s;
  return s;
}
int elt_of(const mla_cache_t* c) { return c->dtype == MLA_E4M3 ? 1 : 2; }
bool pools_ok(const void* ckv, const void* kpe) { return ckv && kpe && aligned(ckv, 16) && aligned(kpe, 16); }
// an int array of n entries: present and aligned, or not needed
bool ints_ok(const int32_t* p, long long n) { return (p || n == 0) && aligned(p, 4); }

mla_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

}  // namespace

extern "C" {

mla_status_t mla_cache_append(const void* c_new, long long c_stride, const void* kpe_new, long long kpe_stride,
                              const int32_t* token_start, int num_tokens, const int32_t* page_table,
                              const int32_t* seq_lens, int B, void* ckv_cache, void* kpe_cache, const mla_cache_t* cache,
                              const mla_append_t* a, uint32_t* status, cudaStream_t stream) {
  mla_status_t st = validate(cache);
  if (st != MLA_OK) return st;
  if (!a || num_tokens < 0 || B < 0) return MLA_ERR_INVALID_ARG;
  if (B > kMaxCacheRows || num_tokens > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  if (a->in_dtype != MLA_BF16 && a->in_dtype != MLA_F32) return MLA_ERR_INVALID_ARG;
  const int es = a->in_dtype == MLA_F32 ? 4 : 2;
  if (!std::isfinite(a->kv_descale) || a->kv_descale <= 0.f || !std::isfinite(1.f / a->kv_descale) ||
      (cache->dtype == MLA_BF16 && a->kv_descale != 1.f))
    return MLA_ERR_INVALID_ARG;
  if (a->norm_weight && (!aligned(a->norm_weight, 16) || !(a->norm_eps >= 0.f) || !std::isfinite(a->norm_eps)))
    return MLA_ERR_INVALID_ARG;
  if (a->rope_table && (!aligned(a->rope_table, 4) || a->rope_positions < 1)) return MLA_ERR_INVALID_ARG;
  if (a->rope_interleaved != 0 && a->rope_interleaved != 1) return MLA_ERR_INVALID_ARG;
  if (a->cp_world < 0 || a->cp_interleave < 0) return MLA_ERR_INVALID_ARG;
  if (a->cp_world > 1 && (a->cp_rank < 0 || a->cp_rank >= a->cp_world || !a->global_seq_lens || !aligned(a->global_seq_lens, 4)))
    return MLA_ERR_INVALID_ARG;
  if (!token_start && num_tokens > 0 && (B == 0 || num_tokens % B != 0)) return MLA_ERR_INVALID_ARG;
  if (!aligned(token_start, 4) || !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0 || B == 0) return MLA_OK;  // nobody's tokens
  if (!c_new || !kpe_new || !pools_ok(ckv_cache, kpe_cache) || !page_table || !seq_lens) return MLA_ERR_INVALID_ARG;
  if (!aligned(c_new, 16) || c_stride < kDLatent || (c_stride * es) % 16 != 0 || !aligned(kpe_new, es) ||
      kpe_stride < kDRope || !aligned(page_table, 4) || !aligned(seq_lens, 4))
    return MLA_ERR_INVALID_ARG;
  AppendParams p{};
  p.c_new = c_new;
  p.kpe_new = kpe_new;
  p.c_stride = c_stride;
  p.kpe_stride = kpe_stride;
  p.token_start = token_start;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.global_seq_lens = a->global_seq_lens;
  p.kept = cache->kept;
  p.norm_weight = a->norm_weight;
  p.rope_table = a->rope_table;
  p.ckv = static_cast<uint8_t*>(ckv_cache);
  p.kpe = static_cast<uint8_t*>(kpe_cache);
  p.status = status;
  p.norm_eps = a->norm_eps;
  p.inv_descale = 1.f / a->kv_descale;
  p.num_tokens = num_tokens;
  p.B = B;
  p.per_row = num_tokens / B;
  p.rope_positions = a->rope_positions;
  p.interleaved = a->rope_interleaved;
  p.num_pages = cache->num_pages;
  p.page_shift = shift_of(cache);
  p.stride = cache->page_table_stride;
  p.cp_world = a->cp_world > 1 ? a->cp_world : 1;
  p.cp_rank = a->cp_world > 1 ? a->cp_rank : 0;
  p.cp_interleave = a->cp_interleave > 0 ? a->cp_interleave : 1;
  return cuda_status(launch_append(p, a->in_dtype == MLA_F32, cache->dtype == MLA_E4M3, stream));
}

mla_status_t mla_cache_workspace(const mla_cache_t* cache, int rows, size_t* workspace_bytes) {
  mla_status_t st = validate(cache);
  if (st != MLA_OK) return st;
  if (!workspace_bytes || rows < 0) return MLA_ERR_INVALID_ARG;
  if (rows > kMaxCacheRows) return MLA_ERR_UNSUPPORTED;
  *workspace_bytes = cache_ws(cache->num_pages, cache->page_table_stride, rows).total;
  return MLA_OK;
}

mla_status_t mla_cache_fork(const int32_t* page_table, const int32_t* seq_lens, int B, const int32_t* parents,
                            const int32_t* new_tokens, int N, const int32_t* ref_count, void* ckv_cache, void* kpe_cache,
                            const mla_cache_t* cache, int window_left, int sink_tokens, int32_t* page_table_out,
                            int32_t* seq_lens_out, int32_t* ref_count_out, void* workspace, size_t workspace_bytes,
                            uint32_t* status, cudaStream_t stream) {
  mla_status_t st = validate(cache);
  if (st != MLA_OK) return st;
  if (B < 0 || N < 0 || window_left < -1 || sink_tokens < 0) return MLA_ERR_INVALID_ARG;
  if (B > kMaxCacheRows || N > kMaxCacheRows || sink_tokens > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  const int W = cache->page_table_stride;
  // the pages all rows ask for, at most their tables' entries, are summed in 32 bits
  if ((long long)N * W > INT_MAX) return MLA_ERR_UNSUPPORTED;
  if (!ints_ok(page_table, B) || !ints_ok(seq_lens, B) || !ints_ok(parents, N) || !aligned(new_tokens, 4) ||
      !ints_ok(page_table_out, N) || !ints_ok(seq_lens_out, N) || !ints_ok(ref_count, 1) || !ints_ok(ref_count_out, 1) ||
      !aligned(status, 4) || !pools_ok(ckv_cache, kpe_cache) || !workspace || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  const size_t row = sizeof(int32_t) * (size_t)W, refs = sizeof(int32_t) * (size_t)cache->num_pages;
  const bool in_place = B > 0 && N > 0 && page_table == page_table_out;
  if (in_place ? seq_lens != seq_lens_out
               : overlap(page_table, row * B, page_table_out, row * N) ||
                     overlap(seq_lens, sizeof(int32_t) * (size_t)B, seq_lens_out, sizeof(int32_t) * (size_t)N))
    return MLA_ERR_INVALID_ARG;
  if (ref_count != ref_count_out && overlap(ref_count, refs, ref_count_out, refs)) return MLA_ERR_INVALID_ARG;
  const size_t kept = cache->kept ? sizeof(int32_t) * (size_t)N : 0;
  if (overlap(cache->kept, kept, page_table, row * B) || overlap(cache->kept, kept, page_table_out, row * N) ||
      overlap(cache->kept, kept, seq_lens_out, sizeof(int32_t) * (size_t)N) || overlap(cache->kept, kept, ref_count_out, refs))
    return MLA_ERR_INVALID_ARG;
  const int rows = std::max(B, N);
  if (workspace_bytes < cache_ws(cache->num_pages, W, rows).total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  ForkParams p{};
  p.table = page_table;
  p.lens = seq_lens;
  p.parents = parents;
  p.add = new_tokens;
  p.ref_in = ref_count;
  p.table_out = page_table_out;
  p.lens_out = seq_lens_out;
  p.ref = ref_count_out;
  p.kept = cache->kept;
  p.ckv = static_cast<uint8_t*>(ckv_cache);
  p.kpe = static_cast<uint8_t*>(kpe_cache);
  p.ws = static_cast<uint8_t*>(workspace);
  p.status = status;
  p.B = B;
  p.N = N;
  p.stride = W;
  p.page_shift = shift_of(cache);
  p.num_pages = cache->num_pages;
  p.es = elt_of(cache);
  p.window_left = window_left;
  p.sink_tokens = sink_tokens;
  p.ws_rows = rows;
  return cuda_status(launch_fork(p, stream));
}

mla_status_t mla_cache_compact(const int32_t* page_table, int B, const int32_t* ref_count, void* ckv_cache,
                               void* kpe_cache, const mla_cache_t* cache, int32_t* page_table_out, int32_t* ref_count_out,
                               int32_t* page_map, int32_t* num_used, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  mla_status_t st = validate(cache);
  if (st != MLA_OK) return st;
  if (B < 0) return MLA_ERR_INVALID_ARG;
  if (B > kMaxCacheRows) return MLA_ERR_UNSUPPORTED;
  if (!ints_ok(page_table, B) || !ints_ok(page_table_out, B) || !ints_ok(ref_count, 1) || !ints_ok(ref_count_out, 1) ||
      !ints_ok(page_map, 1) || !ints_ok(num_used, 1) || !pools_ok(ckv_cache, kpe_cache) || !workspace ||
      !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARG;
  const size_t table = sizeof(int32_t) * (size_t)cache->page_table_stride * (size_t)B;
  const size_t refs = sizeof(int32_t) * (size_t)cache->num_pages;
  if ((page_table != page_table_out && overlap(page_table, table, page_table_out, table)) ||
      (ref_count != ref_count_out && overlap(ref_count, refs, ref_count_out, refs)) ||
      overlap(page_map, refs, ref_count, refs) || overlap(page_map, refs, ref_count_out, refs) ||
      overlap(page_map, refs, page_table, table) || overlap(page_map, refs, page_table_out, table))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < cache_ws(cache->num_pages, cache->page_table_stride, B).total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  CompactParams p{};
  p.table = page_table;
  p.ref_in = ref_count;
  p.table_out = page_table_out;
  p.ref = ref_count_out;
  p.page_map = page_map;
  p.num_used = num_used;
  p.ckv = static_cast<uint8_t*>(ckv_cache);
  p.kpe = static_cast<uint8_t*>(kpe_cache);
  p.ws = static_cast<uint8_t*>(workspace);
  p.B = B;
  p.stride = cache->page_table_stride;
  p.page_shift = shift_of(cache);
  p.num_pages = cache->num_pages;
  p.es = elt_of(cache);
  p.ws_rows = B;
  return cuda_status(launch_compact(p, stream));
}

mla_status_t mla_cache_copy(const void* ckv_src, const void* kpe_src, int num_src_pages, void* ckv_cache, void* kpe_cache,
                            const int32_t* src_pages, const int32_t* dst_pages, int n, const mla_cache_t* cache,
                            uint32_t* status, cudaStream_t stream) {
  mla_status_t st = validate(cache);
  if (st != MLA_OK) return st;
  if (n < 0 || num_src_pages < 1 || !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (n == 0) return MLA_OK;
  if (!pools_ok(ckv_src, kpe_src) || !pools_ok(ckv_cache, kpe_cache) || !ints_ok(src_pages, n) || !ints_ok(dst_pages, n))
    return MLA_ERR_INVALID_ARG;
  CopyParams p{};
  p.ckv_src = static_cast<const uint8_t*>(ckv_src);
  p.kpe_src = static_cast<const uint8_t*>(kpe_src);
  p.ckv = static_cast<uint8_t*>(ckv_cache);
  p.kpe = static_cast<uint8_t*>(kpe_cache);
  p.src = src_pages;
  p.dst = dst_pages;
  p.status = status;
  p.n = n;
  p.src_pages = num_src_pages;
  p.dst_pages = cache->num_pages;
  p.page_shift = shift_of(cache);
  p.es = elt_of(cache);
  return cuda_status(launch_copy(p, stream));
}

mla_status_t mla_cache_status(const uint32_t* status, cudaStream_t stream) {
  if (!status || !aligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return MLA_ERR_CUDA;
  uint32_t w = 0;
  if (cudaMemcpy(&w, status, sizeof w, cudaMemcpyDeviceToHost) != cudaSuccess) return MLA_ERR_CUDA;
  if (w & (kErrBadPage | kErrBadLength | kErrBadRow)) return MLA_ERR_INVALID_ARG;
  return w & kErrNoPages ? MLA_ERR_NO_PAGES : MLA_OK;
}

}  // extern "C"
