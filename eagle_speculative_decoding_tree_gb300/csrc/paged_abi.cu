// paged_abi.cu -- the extern "C" entry points of the paged KV cache: host-side argument checks, then the
// launches on the caller's stream (abi.cu has the others').
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "paged.h"

using namespace eagle;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int t) { return t == EAGLE_F32 || t == EAGLE_BF16; }

int check_write(const eagle_paged_desc* d) {
  if (!d || d->rows < 1) return EAGLE_ERR_INVALID_ARG;
  const int rc = check_paged_geometry(d->batch, d->n_kv_heads, d->head_dim, d->page_size, d->n_pages, d->max_pages);
  if (rc != EAGLE_OK) return rc;
  if (!dtype_ok(d->dtype) || static_cast<long long>(d->n_kv_heads) * d->rows > (1ll << 30)) return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

int check_commit(const eagle_paged_commit_desc* d) {
  if (!d || d->layers < 1 || d->rows < 1 || d->max_depth < 0 || d->feat_dim < 0) return EAGLE_ERR_INVALID_ARG;
  const int rc = check_paged_geometry(d->batch, d->n_kv_heads, d->head_dim, d->page_size, d->n_pages, d->max_pages);
  if (rc != EAGLE_OK) return rc;
  if (d->layers > kMaxLayers || d->rows > kMaxRows || d->max_depth >= kMaxRows || !dtype_ok(d->dtype) ||
      (d->feat_dim > 0 && !dtype_ok(d->feat_dtype)))
    return EAGLE_ERR_UNSUPPORTED;
  // (CTAs are counted in 32 bits: at most 2 vectors of 16 bytes a thread of 256 for every path row and head)
  const long long ctas = (static_cast<long long>(d->max_depth + 1) * d->n_kv_heads * 32 + 255) / 256 * d->batch * d->layers;
  return ctas > 0x7fffffffll ? EAGLE_ERR_UNSUPPORTED : EAGLE_OK;
}

int check_scores(int rows, int hq, int hkv, float scale, float cap, int window, int dtype) {
  if (rows < 1 || hq < 1 || hkv < 1 || !(scale > 0.f) || !isfinite(scale) || !(cap >= 0.f) || !isfinite(cap) ||
      window < 0)
    return EAGLE_ERR_INVALID_ARG;
  if (hq % hkv || rows > kMaxRows || !dtype_ok(dtype) || static_cast<long long>(rows) * hq > (1 << 20))
    return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

// The units that the kernels divide among themselves (128 keys of a row block of 16 or more) are counted in 32 bits.
bool units_ok(int batch, int heads, long long rows, int max_pages, int page_size) {
  const long long keys = static_cast<long long>(max_pages) * page_size / 128 + 2;
  return static_cast<long long>(batch) * heads * ((rows + 15) / 16) <= 0x7fffffffll / keys;
}

int check_attn(const eagle_paged_attn_desc* d) {
  if (!d) return EAGLE_ERR_INVALID_ARG;
  int rc = check_paged_geometry(d->batch, d->n_kv_heads, d->head_dim, d->page_size, d->n_pages, d->max_pages);
  if (rc == EAGLE_OK) rc = check_scores(d->rows, d->n_q_heads, d->n_kv_heads, d->scale, d->softcap, d->window, d->dtype);
  if (rc != EAGLE_OK) return rc;
  if ((d->precision != EAGLE_ATTN_PRECISE && d->precision != EAGLE_ATTN_FAST) ||
      (d->engine != EAGLE_ENGINE_AUTO && d->engine != EAGLE_ENGINE_MMA_SYNC))
    return EAGLE_ERR_INVALID_ARG;
  if (!dtype_ok(d->out_dtype) || (d->dtype == EAGLE_F32 && d->out_dtype != EAGLE_F32) ||
      static_cast<long long>(d->batch) * d->n_kv_heads > 65535 ||
      !units_ok(d->batch, d->n_kv_heads, static_cast<long long>(d->rows) * (d->n_q_heads / d->n_kv_heads), d->max_pages,
                d->page_size))
    return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

int check_weights(const eagle_paged_weights_desc* d) {
  if (!d || d->max_depth < 0) return EAGLE_ERR_INVALID_ARG;
  int rc = check_paged_geometry(d->batch, d->n_kv_heads, d->head_dim, d->page_size, d->n_pages, d->max_pages);
  if (rc == EAGLE_OK) rc = check_scores(d->rows, d->n_q_heads, d->n_kv_heads, d->scale, d->softcap, d->window, d->dtype);
  if (rc != EAGLE_OK) return rc;
  if (d->max_depth >= kMaxRows || static_cast<long long>(d->batch) * d->n_kv_heads > 65535 ||
      !units_ok(d->batch, d->n_kv_heads, 1, d->max_pages, d->page_size))
    return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

int check_evict(const eagle_paged_evict_desc* d) {
  if (!d || d->layers < 1 || d->budget < 1 || d->sink < 0 || d->recent < 0) return EAGLE_ERR_INVALID_ARG;
  const int rc = check_paged_geometry(d->batch, d->n_kv_heads, d->head_dim, d->page_size, d->n_pages, d->max_pages);
  if (rc != EAGLE_OK) return rc;
  if (d->limit < d->budget || d->sink > d->budget - d->recent ||
      static_cast<long long>(d->budget) > static_cast<long long>(d->max_pages) * d->page_size)
    return EAGLE_ERR_INVALID_ARG;
  const long long groups = static_cast<long long>(d->layers) * d->batch * d->n_kv_heads;
  if (d->layers > 128 || !dtype_ok(d->dtype) || groups > (1 << 24) ||
      groups * ((d->budget + 31ll) / 32) > 0x7fffffffll)
    return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

// The multiprocessors of the current device.
int sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    return 152;
  }
  return n;
}

}  // namespace

size_t eagle::paged_workspace_size(int which, const void* desc) {
  if (which == EAGLE_WS_PAGED_ATTN) {
    const eagle_paged_attn_desc* d = static_cast<const eagle_paged_attn_desc*>(desc);
    return check_attn(d) == EAGLE_OK ? paged_attn_ws(*d, sms()) : 0;
  }
  if (which == EAGLE_WS_PAGED_COMMIT) {
    const eagle_paged_commit_desc* d = static_cast<const eagle_paged_commit_desc*>(desc);
    return check_commit(d) == EAGLE_OK ? paged_commit_ws(*d) : 0;
  }
  if (which == EAGLE_WS_PAGED_EVICT) {
    const eagle_paged_evict_desc* d = static_cast<const eagle_paged_evict_desc*>(desc);
    return check_evict(d) == EAGLE_OK ? paged_evict_ws(*d) : 0;
  }
  return 0;
}

extern "C" {

int eagle_paged_write(const eagle_paged_desc* d, const void* k, const void* v, const int32_t* page_table,
                      const int32_t* start, const int32_t* count, void* k_pages, void* v_pages, uint32_t* status,
                      void* stream) {
  const int rc = check_write(d);
  if (rc != EAGLE_OK) return rc;
  if (!k || !v || !page_table || !start || !k_pages || !v_pages) return EAGLE_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(page_table, 4) ||
      !aligned(start, 4) || !aligned(count, 4) || !aligned(status, 4))
    return EAGLE_ERR_ALIGNMENT;
  return report_cuda_error(launch_paged_write(*d, k, v, page_table, start, count, k_pages, v_pages, status,
                                              static_cast<cudaStream_t>(stream)));
}

int eagle_paged_commit(const eagle_paged_commit_desc* d, void* const* k_pages_layers, void* const* v_pages_layers,
                       const void* const* tree_k_layers, const void* const* tree_v_layers,
                       const int32_t* page_table, const int32_t* n_acc, const int32_t* path, int32_t* seq_len,
                       int32_t* commit_pos, void* feat_pages, const void* tree_feat, uint32_t* status, void* ws,
                       size_t ws_bytes, void* stream) {
  const int rc = check_commit(d);
  if (rc != EAGLE_OK) return rc;
  if (!k_pages_layers || !v_pages_layers || !tree_k_layers || !tree_v_layers || !page_table || !n_acc || !path ||
      !seq_len || (d->feat_dim > 0 && (!feat_pages || !tree_feat)))
    return EAGLE_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(n_acc, 4) || !aligned(path, 4) || !aligned(seq_len, 4) ||
      !aligned(commit_pos, 4) || !aligned(status, 4) || !aligned(ws, 16))
    return EAGLE_ERR_ALIGNMENT;
  CommitArgs a;
  memset(&a, 0, sizeof a);
  for (int l = 0; l < d->layers; ++l) {
    a.k_cache[l] = k_pages_layers[l];
    a.v_cache[l] = v_pages_layers[l];
    a.tree_k[l] = tree_k_layers[l];
    a.tree_v[l] = tree_v_layers[l];
    if (!a.k_cache[l] || !a.v_cache[l] || !a.tree_k[l] || !a.tree_v[l]) return EAGLE_ERR_INVALID_ARG;
    if (!aligned(a.k_cache[l], 16) || !aligned(a.v_cache[l], 16) || !aligned(a.tree_k[l], 16) ||
        !aligned(a.tree_v[l], 16))
      return EAGLE_ERR_ALIGNMENT;
  }
  if (d->feat_dim > 0) {
    const size_t bytes = static_cast<size_t>(d->feat_dim) * (d->feat_dtype == EAGLE_F32 ? 4 : 2);
    const size_t need = bytes % 16 == 0 ? 16 : 2;
    if (!aligned(feat_pages, need) || !aligned(tree_feat, need)) return EAGLE_ERR_ALIGNMENT;
  }
  if (!ws || ws_bytes < paged_commit_ws(*d)) return EAGLE_ERR_WORKSPACE;
  return report_cuda_error(launch_paged_commit(*d, a, page_table, n_acc, path, seq_len, commit_pos,
                                               d->feat_dim > 0 ? feat_pages : nullptr, tree_feat, status, ws,
                                               static_cast<cudaStream_t>(stream)));
}

int eagle_paged_attn(const eagle_paged_attn_desc* d, const void* q, const void* k_pages, const void* v_pages,
                     const int32_t* page_table, const void* tree_k, const void* tree_v, const int32_t* seq_len,
                     const int32_t* n_nodes, const uint64_t* anc_mask, const float* slopes, void* out, float* lse,
                     uint32_t* status, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_attn(d);
  if (rc != EAGLE_OK) return rc;
  if (!q || !k_pages || !v_pages || !page_table || !seq_len || !out || (tree_k == nullptr) != (tree_v == nullptr) ||
      (tree_k == nullptr) != (anc_mask == nullptr))
    return EAGLE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(tree_k, 16) || !aligned(tree_v, 16) ||
      !aligned(out, 16) || !aligned(ws, 16) || !aligned(anc_mask, 8) || !aligned(page_table, 4) ||
      !aligned(seq_len, 4) || !aligned(n_nodes, 4) || !aligned(slopes, 4) || !aligned(lse, 4) || !aligned(status, 4))
    return EAGLE_ERR_ALIGNMENT;
  const int n = sms();
  if (!ws || ws_bytes < paged_attn_ws(*d, n)) return EAGLE_ERR_WORKSPACE;
  return report_cuda_error(launch_paged_attn(*d, q, k_pages, v_pages, page_table, tree_k, tree_v, seq_len, n_nodes,
                                             anc_mask, slopes, out, lse, status, ws, n,
                                             static_cast<cudaStream_t>(stream)));
}

int eagle_paged_weights(const eagle_paged_weights_desc* d, const void* q, const float* lse, const void* k_pages,
                        const int32_t* page_table, const int32_t* seq_len, const int32_t* n_acc, const int32_t* path,
                        const float* slopes, const float* prior, float* weights, uint32_t* status, void* stream) {
  const int rc = check_weights(d);
  if (rc != EAGLE_OK) return rc;
  if (!q || !lse || !k_pages || !page_table || !seq_len || !weights || (n_acc == nullptr) != (path == nullptr))
    return EAGLE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(seq_len, 4) ||
      !aligned(n_acc, 4) || !aligned(path, 4) || !aligned(slopes, 4) || !aligned(prior, 16) || !aligned(weights, 16) ||
      !aligned(status, 4))
    return EAGLE_ERR_ALIGNMENT;
  return report_cuda_error(launch_paged_weights(*d, q, lse, k_pages, page_table, seq_len, n_acc, path, slopes, prior,
                                                weights, status, sms(), static_cast<cudaStream_t>(stream)));
}

int eagle_paged_evict(const eagle_paged_evict_desc* d, void* const* k_pages_layers, void* const* v_pages_layers,
                      float* const* weights_layers, int32_t* page_table, int32_t* spare, int32_t* seq_len,
                      int32_t* kept, uint32_t* status, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_evict(d);
  if (rc != EAGLE_OK) return rc;
  if (!k_pages_layers || !v_pages_layers || !weights_layers || !page_table || !spare || !seq_len || !kept)
    return EAGLE_ERR_INVALID_ARG;
  if (!aligned(page_table, 4) || !aligned(spare, 4) || !aligned(seq_len, 4) || !aligned(kept, 4) ||
      !aligned(status, 4) || !aligned(ws, 16))
    return EAGLE_ERR_ALIGNMENT;
  PagedEvictArgs a;
  memset(&a, 0, sizeof a);
  for (int l = 0; l < d->layers; ++l) {
    a.k[l] = k_pages_layers[l];
    a.v[l] = v_pages_layers[l];
    a.w[l] = weights_layers[l];
    if (!a.k[l] || !a.v[l] || !a.w[l]) return EAGLE_ERR_INVALID_ARG;
    if (!aligned(a.k[l], 16) || !aligned(a.v[l], 16) || !aligned(a.w[l], 16)) return EAGLE_ERR_ALIGNMENT;
  }
  if (!ws || ws_bytes < paged_evict_ws(*d)) return EAGLE_ERR_WORKSPACE;
  return report_cuda_error(launch_paged_evict(*d, a, page_table, spare, seq_len, kept, status, ws,
                                              sms(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
