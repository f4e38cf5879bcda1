// paged.h -- launchers and plans of the paged KV cache (host side of paged_*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/eagle.h"
#include "launch.h"

namespace eagle {

// A cache row's place: page table and pool geometry.
struct PagedGeom {
  const int32_t* table;  // [B][max_pages]
  int n_pages, max_pages;
  int shift;             // log2 of the page size
  int Hkv;
  int capacity;          // max_pages << shift
};

inline int paged_shift(int page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

// The limits that every call on a paged cache shares: EAGLE_OK, or the error code.
inline int check_paged_geometry(int batch, int heads, int head_dim, int page_size, int n_pages, int max_pages) {
  if (batch < 1 || heads < 1 || head_dim < 1 || page_size < 1 || n_pages < 1 || max_pages < 1)
    return EAGLE_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || paged_shift(page_size) < 0 || batch > 65535 || heads > 1024 ||
      static_cast<long long>(max_pages) * page_size > (1ll << 31) - 256 ||
      static_cast<long long>(n_pages) * heads * page_size > (1ll << 31) - 256)
    return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

inline PagedGeom paged_geom(const int32_t* table, int n_pages, int max_pages, int page_size, int heads) {
  PagedGeom g;
  g.table = table;
  g.n_pages = n_pages;
  g.max_pages = max_pages;
  g.shift = paged_shift(page_size);
  g.Hkv = heads;
  g.capacity = max_pages << g.shift;
  return g;
}

// How a score is shaped (log2 units): t = raw * scale, capped, biased by the distance, cut off.
struct ScoreShape {
  float scale_log2;  // scale * log2 e (no cap)
  float cap_log2;    // cap * log2 e; 0: none
  float cap_x;       // scale / cap
  float cap_mul;     // 2 log2 e * scale / cap
  // where |raw| <= cap_small the capped score is raw (p[0] + p[1] raw^2 + .. + p[4] raw^8): tanh's Taylor polynomial,
  // off by less than 2.5e-7 of itself for arguments up to 0.35
  float cap_small, p[5];
  int window;        // 0: none
  const float* slopes;  // [Hq], NULL: none
};

inline ScoreShape score_shape(float scale, float cap, int window, const float* slopes) {
  const double log2e = 1.4426950408889634;
  ScoreShape s;
  s.scale_log2 = static_cast<float>(scale * log2e);
  s.cap_log2 = static_cast<float>(cap * log2e);
  s.cap_mul = cap > 0.f ? static_cast<float>(2.0 * log2e * scale / cap) : 0.f;
  const double x = cap > 0.f ? static_cast<double>(scale) / cap : 0.0;  // tanh's argument is raw x
  s.cap_x = static_cast<float>(x);
  s.cap_small = x > 0.0 ? static_cast<float>(0.35 / x) : 0.f;
  const double c[5] = {1.0, -1.0 / 3, 2.0 / 15, -17.0 / 315, 62.0 / 2835};
  double xx = scale * log2e;
  for (int i = 0; i < 5; ++i, xx *= x * x) s.p[i] = static_cast<float>(xx * c[i]);
  s.window = window;
  s.slopes = slopes;
  return s;
}

cudaError_t launch_paged_write(const eagle_paged_desc& d, const void* k, const void* v, const int32_t* table,
                               const int32_t* start, const int32_t* count, void* k_pages, void* v_pages,
                               uint32_t* status, cudaStream_t s);

size_t paged_commit_ws(const eagle_paged_commit_desc& d);
cudaError_t launch_paged_commit(const eagle_paged_commit_desc& d, const CommitArgs& a, const int32_t* table,
                                const int32_t* n_acc, const int32_t* path, int32_t* seq_len, int32_t* commit_pos,
                                void* feat_pages, const void* tree_feat, uint32_t* status, void* ws, cudaStream_t s);

struct PagedEvictArgs {
  void* k[128];
  void* v[128];
  float* w[128];
};
size_t paged_evict_ws(const eagle_paged_evict_desc& d);
cudaError_t launch_paged_evict(const eagle_paged_evict_desc& d, const PagedEvictArgs& a, int32_t* table,
                               int32_t* spare, int32_t* seq_len, int32_t* kept, uint32_t* status, void* ws,
                               int sms, cudaStream_t s);

cudaError_t launch_paged_weights(const eagle_paged_weights_desc& d, const void* q, const float* lse,
                                 const void* k_pages, const int32_t* table, const int32_t* seq_len,
                                 const int32_t* n_acc, const int32_t* path, const float* slopes, const float* prior,
                                 float* weights, uint32_t* status, int sms, cudaStream_t s);

// eagle_workspace_size of the paged entry points.
size_t paged_workspace_size(int which, const void* desc);

size_t paged_attn_ws(const eagle_paged_attn_desc& d, int sms);
cudaError_t launch_paged_attn(const eagle_paged_attn_desc& d, const void* q, const void* k_pages, const void* v_pages,
                              const int32_t* table, const void* tree_k, const void* tree_v, const int32_t* seq_len,
                              const int32_t* n_nodes, const uint64_t* anc_mask, const float* slopes, void* out,
                              float* lse, uint32_t* status, void* ws, int sms, cudaStream_t s);

}  // namespace eagle
