// C ABI of the paged 4-bit cache and of the page operations: argument checks
// and dispatch (helpers of dca_api.cu, same translation unit).
#include "dca_kernels.cuh"
#include "kv4.cuh"

namespace dca {
namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

#define DCA_CHECK_INDEX(p)                                                                    \
  do {                                                                                        \
    if ((p) == nullptr || !aligned4(p))                                                       \
      return fail(DCA_ERR_INVALID_ARG, "%s: %s is null or not 4-byte aligned", fn, #p);       \
  } while (0)

dca_status_t check_kv4(const char* fn, int B, int T, int Hkv, int D, const int* block_table,
                       int max_blocks, int block_rows, int num_blocks) {
  dca_status_t st = check_heads(fn, B, 1, Hkv, Hkv, D);
  if (st != DCA_OK) return st;
  if (T < 0) return fail(DCA_ERR_INVALID_ARG, "%s: T=%d", fn, T);
  if (Hkv > 65535) return fail(DCA_ERR_UNSUPPORTED, "%s: Hkv=%d beyond the launch grid", fn, Hkv);
  if (B == 0 || T == 0) return DCA_OK;
  st = check_paged(fn, block_table, max_blocks, block_rows, num_blocks);
  if (st != DCA_OK) return st;
  DCA_CHECK_INDEX(block_table);
  return DCA_OK;
}

}  // namespace
}  // namespace dca

extern "C" {

size_t dca_kv4_tile_bytes(int D) {
  return D == 64 || D == 128 ? kv4::tile_bytes(D) : 0;
}

dca_status_t dca_kv4_append_paged(const void* k_new, const void* v_new, void* pool,
                                  const int* block_table, int max_blocks, int block_rows,
                                  int num_blocks, const int* cu_seqlens, const int* t0, int B,
                                  int T, int Hkv, int D, int s, int c, float base, void* stream) {
  const char* fn = "dca_kv4_append_paged";
  dca_status_t st = check_kv4(fn, B, T, Hkv, D, block_table, max_blocks, block_rows, num_blocks);
  if (st == DCA_OK) st = check_chunking(fn, s, c, base);
  if (st != DCA_OK) return st;
  if (B == 0 || T == 0) return DCA_OK;
  DCA_CHECK_PTR(k_new);
  DCA_CHECK_PTR(v_new);
  DCA_CHECK_PTR(pool);
  DCA_CHECK_INDEX(cu_seqlens);
  DCA_CHECK_INDEX(t0);
  cudaError_t e = launch_kv4_append(k_new, v_new, pool, block_table, max_blocks, block_rows,
                                    num_blocks, cu_seqlens, t0, B, T, Hkv, D, s, base,
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DCA_OK : cuda_fail(e, fn);
}

dca_status_t dca_kv4_read_paged(const void* pool, const int* block_table, int max_blocks,
                                int block_rows, int num_blocks, const int* cu_seqlens,
                                const int* t0, void* K, void* V, int B, int T, int Hkv, int D,
                                int out_rows, void* stream) {
  const char* fn = "dca_kv4_read_paged";
  dca_status_t st = check_kv4(fn, B, T, Hkv, D, block_table, max_blocks, block_rows, num_blocks);
  if (st != DCA_OK) return st;
  if (out_rows < 0) return fail(DCA_ERR_INVALID_ARG, "%s: out_rows=%d", fn, out_rows);
  if (B == 0 || T == 0) return DCA_OK;
  DCA_CHECK_PTR(pool);
  DCA_CHECK_INDEX(cu_seqlens);
  DCA_CHECK_INDEX(t0);
  DCA_CHECK_PTR(K);
  DCA_CHECK_PTR(V);
  cudaError_t e = launch_kv4_read(pool, block_table, max_blocks, block_rows, num_blocks,
                                  cu_seqlens, t0, K, V, B, T, Hkv, D, out_rows,
                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DCA_OK : cuda_fail(e, fn);
}

size_t dca_attn_decode_kv4_workspace(int B, int Hq, int Hkv, int D, int Tcap) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128) || Tcap < 1) return 0;
  if (!kv4_decode_fits(B, Hq, Hkv, D, Tcap)) return 0;
  return kv4_decode_workspace_bytes(B, Hq, Hkv, D, Tcap);
}

dca_status_t dca_attn_decode_kv4_paged(const void* q, const void* pool, const int* block_table,
                                       int max_blocks, int block_rows, int num_blocks,
                                       const int* t, void* O, float* LSE, int B, int Hq, int Hkv,
                                       int D, int s, int c, float base, float scale,
                                       void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "dca_attn_decode_kv4_paged";
  dca_status_t st = check_heads(fn, B, 1, Hq, Hkv, D);
  if (st == DCA_OK) st = check_chunking(fn, s, c, base);
  if (st == DCA_OK)
    st = check_kv4(fn, B, 1, Hkv, D, block_table, max_blocks, block_rows, num_blocks);
  if (st != DCA_OK) return st;
  if (B == 0) return DCA_OK;
  const long long cap = (long long)max_blocks * block_rows;
  if (!kv4_decode_fits(B, Hq, Hkv, D, cap))
    return fail(DCA_ERR_UNSUPPORTED, "%s: B=%d, Hq=%d and %lld rows beyond the launch grid", fn, B,
                Hq, cap);
  DCA_CHECK_PTR(q);
  DCA_CHECK_PTR(pool);
  DCA_CHECK_INDEX(t);
  DCA_CHECK_PTR(O);
  DCA_CHECK_INDEX(LSE);
  DCA_CHECK_PTR(workspace);
  const size_t need = kv4_decode_workspace_bytes(B, Hq, Hkv, D, cap);
  if (ws_bytes < need)
    return fail(DCA_ERR_WORKSPACE, "%s: workspace %zu bytes < required %zu", fn, ws_bytes, need);
  const float sc = scale != 0.f ? scale : 1.0f / sqrtf((float)D);
  cudaError_t e = launch_kv4_decode(q, pool, block_table, max_blocks, block_rows, num_blocks, t, O,
                                    LSE, B, Hq, Hkv, D, s, c, base, sc, workspace,
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DCA_OK : cuda_fail(e, fn);
}

}  // extern "C"

namespace dca {
namespace {

// Sizes, index arrays and pools shared by the page operations.
dca_status_t check_pages(const char* fn, const int* block_table, const int* refs,
                         const int* block_table_out, const int* refs_out, const int* info, int B,
                         int max_blocks, int num_blocks, int block_rows,
                         const dca_page_pool_t* pools, int n_pools, PoolList& list) {
  if (B < 0 || max_blocks < 1 || num_blocks < 1 || block_rows < 1)
    return fail(DCA_ERR_INVALID_ARG, "%s: B=%d max_blocks=%d num_blocks=%d block_rows=%d", fn, B,
                max_blocks, num_blocks, block_rows);
  if ((long long)B * max_blocks > (1ll << 30) || (long long)max_blocks * block_rows > (1ll << 30) ||
      num_blocks > (1 << 30))
    return fail(DCA_ERR_UNSUPPORTED, "%s: tables of more than 2^30 entries or rows", fn);
  if (B > 0) {
    DCA_CHECK_INDEX(block_table);
    DCA_CHECK_INDEX(block_table_out);
  }
  DCA_CHECK_INDEX(refs);
  DCA_CHECK_INDEX(refs_out);
  DCA_CHECK_INDEX(info);
  if (n_pools < 0 || n_pools > kMaxPools || (n_pools > 0 && pools == nullptr))
    return fail(DCA_ERR_INVALID_ARG, "%s: n_pools=%d (0 .. %d)", fn, n_pools, kMaxPools);
  list.n = n_pools;
  long long items = 0;
  for (int j = 0; j < n_pools; ++j) {
    const dca_page_pool_t& p = pools[j];
    if (p.base == nullptr || !aligned16(p.base))
      return fail(DCA_ERR_INVALID_ARG, "%s: pool %d is null or not 16-byte aligned", fn, j);
    if (p.outer < 1 || p.unit_rows < 1 || block_rows % p.unit_rows != 0 || p.unit_bytes == 0 ||
        p.unit_bytes % 16 != 0 || p.unit_bytes > (size_t(1) << 30))
      return fail(DCA_ERR_INVALID_ARG,
                  "%s: pool %d: outer=%d unit_rows=%d unit_bytes=%zu do not divide a page of %d "
                  "rows into 16-byte words", fn, j, p.outer, p.unit_rows, p.unit_bytes, block_rows);
    const long long part = (long long)(block_rows / p.unit_rows) * (long long)p.unit_bytes;
    if (part > (1ll << 40) || p.outer > (1 << 20) || (part >> 12) * p.outer > (1ll << 30))
      return fail(DCA_ERR_UNSUPPORTED, "%s: pool %d: a page of over 2^42 bytes", fn, j);
    items += ((part >> 14) + 1) * p.outer;
    if (items > (1ll << 30))
      return fail(DCA_ERR_UNSUPPORTED, "%s: a page of over 2^44 bytes in all pools", fn);
    list.p[j] = PoolDesc{static_cast<unsigned char*>(p.base), (long long)p.unit_bytes, p.outer,
                         p.unit_rows, 0, 0};
  }
  return DCA_OK;
}

}  // namespace
}  // namespace dca

extern "C" {

size_t dca_pages_workspace(int B, int max_blocks, int num_blocks) {
  if (B < 0 || max_blocks < 1 || num_blocks < 1) return 0;
  return pages_workspace_bytes(B, max_blocks, num_blocks);
}

dca_status_t dca_pages_remap(const int* src, const int* old_len, const int* new_len,
                             const int* block_table, const int* refs, int* block_table_out,
                             int* refs_out, int* info, int B, int max_blocks, int num_blocks,
                             int block_rows, const dca_page_pool_t* pools, int n_pools,
                             void* workspace, size_t ws_bytes, void* stream) {
  const char* fn = "dca_pages_remap";
  PoolList list;
  dca_status_t st = check_pages(fn, block_table, refs, block_table_out, refs_out, info, B,
                                max_blocks, num_blocks, block_rows, pools, n_pools, list);
  if (st != DCA_OK) return st;
  if (B > 0) {
    DCA_CHECK_INDEX(src);
    DCA_CHECK_INDEX(old_len);
    DCA_CHECK_INDEX(new_len);
  }
  DCA_CHECK_PTR(workspace);
  const size_t need = pages_workspace_bytes(B, max_blocks, num_blocks);
  if (ws_bytes < need)
    return fail(DCA_ERR_WORKSPACE, "%s: workspace %zu bytes < required %zu", fn, ws_bytes, need);
  cudaError_t e = launch_pages_remap(src, old_len, new_len, block_table, block_table_out, refs,
                                     refs_out, info, B, max_blocks, num_blocks, block_rows, list,
                                     workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DCA_OK : cuda_fail(e, fn);
}

dca_status_t dca_pages_compact(const int* len, const int* block_table, const int* refs,
                               int* block_table_out, int* refs_out, int* moved, int* info, int B,
                               int max_blocks, int num_blocks, int block_rows,
                               const dca_page_pool_t* pools, int n_pools, void* workspace,
                               size_t ws_bytes, void* stream) {
  const char* fn = "dca_pages_compact";
  PoolList list;
  dca_status_t st = check_pages(fn, block_table, refs, block_table_out, refs_out, info, B,
                                max_blocks, num_blocks, block_rows, pools, n_pools, list);
  if (st != DCA_OK) return st;
  if (B > 0) DCA_CHECK_INDEX(len);
  DCA_CHECK_INDEX(moved);
  DCA_CHECK_PTR(workspace);
  const size_t need = pages_workspace_bytes(B, max_blocks, num_blocks);
  if (ws_bytes < need)
    return fail(DCA_ERR_WORKSPACE, "%s: workspace %zu bytes < required %zu", fn, ws_bytes, need);
  cudaError_t e = launch_pages_compact(len, block_table, block_table_out, refs, refs_out, moved,
                                       info, B, max_blocks, num_blocks, block_rows, list,
                                       workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DCA_OK : cuda_fail(e, fn);
}

}  // extern "C"
