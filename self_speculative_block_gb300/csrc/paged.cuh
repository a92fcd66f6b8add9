// Host checks that the paged KV cache operators share.
#pragma once
#include "../../include/gocr.h"
#include "kernels.cuh"

namespace gocr {
namespace paged {

constexpr int MAX_REQUESTS = 4096;
constexpr int MAX_KEYS = 1 << 24;  // positions of a request: max_pages * page_size
constexpr int MAX_ROWS = 1 << 24;

inline bool page_size_ok(int ps) { return ps >= 16 && ps <= 256 && !(ps & (ps - 1)); }

inline int table_check(int n_req, int max_pages, int page_size, int n_pages) {
  if (!page_size_ok(page_size)) return op_fail(GOCR_EINVAL, "page size %d is not 16, 32, 64, 128 or 256", page_size);
  if (n_req < 0 || n_req > MAX_REQUESTS || max_pages < 1 || max_pages > MAX_KEYS / page_size || n_pages < 1 ||
      n_pages > 0x7fffffff / page_size)
    return op_fail(GOCR_EINVAL, "bad shape: %d requests of at most %d pages, %d pages of %d positions", n_req, max_pages,
                   n_pages, page_size);
  return GOCR_OK;
}

// A dimension of one entry has no stride to speak of; the others may nest in
// any order, each beyond the whole of the one inside it.
inline bool strides_ok(int64_t* st, const int64_t* n, int d) {
  int at[3], m = 0;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) st[i] = d;
    else if (st[i] < d || st[i] > (1ll << 32) || st[i] % 8) return false;
    else at[m++] = i;
  }
  for (int i = 1; i < m; ++i)  // by stride
    for (int j = i; j > 0 && st[at[j]] < st[at[j - 1]]; --j) {
      const int t = at[j];
      at[j] = at[j - 1];
      at[j - 1] = t;
    }
  for (int i = 1; i < m; ++i)
    if (st[at[i]] / n[at[i - 1]] < st[at[i - 1]]) return false;
  return true;
}

// Checks a cache and copies it, strides of single entries set.
inline int cache_check(const gocr_paged_kv* in, gocr_paged_kv* kv) {
  if (!in) return op_fail(GOCR_EINVAL, "null pointer");
  *kv = *in;
  if (!page_size_ok(kv->page_size))
    return op_fail(GOCR_EINVAL, "page size %d is not 16, 32, 64, 128 or 256", kv->page_size);
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024 || (kv->head_dim != 64 && kv->head_dim != 128) || kv->n_pages < 1 ||
      kv->n_pages > 0x7fffffff / kv->page_size)
    return op_fail(GOCR_EINVAL, "bad shape: a cache of %d pages of %d, %d heads of %d", kv->n_pages, kv->page_size,
                   kv->n_kv_heads, kv->head_dim);
  if (!kv->k || !kv->v) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)kv->k | (uintptr_t)kv->v) & 15) return op_fail(GOCR_EINVAL, "cache not 16-byte aligned");
  const int64_t n[3] = {kv->n_pages, kv->n_kv_heads, kv->page_size};
  if (!strides_ok(&kv->k_page, n, kv->head_dim) || !strides_ok(&kv->v_page, n, kv->head_dim))
    return op_fail(GOCR_EINVAL, "bad cache strides");
  return GOCR_OK;
}

inline bool pitch_ok(long long ld, int heads, int d) { return ld >= (long long)heads * d && ld % 8 == 0 && ld <= (1ll << 32); }

}  // namespace paged
}  // namespace gocr
