// Attention of requests' new rows over a paged KV cache.
//
//   o_i = sum_j exp(c q_i . k_j - lse_i) v_j,  lse_i = log sum_j exp(c q_i . k_j),  j the keys that row i reads
//
// A CTA owns a row and a q head, a warp every fourth key.
#include "attn_packed.cuh"
#include "paged.cuh"

using namespace gocr;
using namespace gocr::paged;

namespace {

struct PagedArgs {
  const bf16* q;
  gocr_paged_kv kv;
  const int *table, *cu, *kv_len;
  bf16* o;
  float* lse;
  long long ldq;
  int max_pages, n_req, T, Hq, G, draft, shift;
  float scale;
};

template <int D> __global__ void __launch_bounds__(128) attn_paged_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int r = -1, row0 = 0, n = 0;
  for (int i = 0; i < a.n_req; ++i) {
    const int c0 = min(max(a.cu[i], 0), a.T), c1 = min(max(a.cu[i + 1], 0), a.T);
    if (t >= c0 && t < c1) {
      r = i;
      row0 = c0;
      n = c1 - c0;
    }
  }
  if (r < 0) return;
  const int kv = min(a.kv_len[r], a.max_pages << a.shift);
  const int last = a.draft && t > row0 ? kv - 1 : kv - n + t - row0;
  const long long kh = (h / a.G) * a.kv.k_head, vh = (h / a.G) * a.kv.v_head;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[t * a.ldq + h * D + e * 32 + lane]) * a.scale;
  for (int j = warp; j <= last; j += 4) {
    const int page = a.table[(size_t)r * a.max_pages + (j >> a.shift)], off = j & ((1 << a.shift) - 1);
    const bool there = page >= 0 && page < a.kv.n_pages;
    const bf16* k = (const bf16*)a.kv.k + page * a.kv.k_page + kh + off * a.kv.k_token;
    const bf16* v = (const bf16*)a.kv.v + page * a.kv.v_page + vh + off * a.kv.v_token;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += there ? q[e] * __bfloat162float(k[e * 32 + lane]) : 0.f;
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float to = fmaxf(m, s), f = m == to ? 1.f : __expf(m - to),
                p = __expf(s - (to == -INFINITY ? 0.f : to));  // (NaN stays NaN)
    m = to;
    l = l * f + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + (there ? p * __bfloat162float(v[e * 32 + lane]) : 0.f);
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float f[4], sum = 0.f;
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == top ? 1.f : __expf(sm[w] - top);
    sum += f[w] * sl[w];
  }
  for (int c = threadIdx.x; c < D; c += 128) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w) x += f[w] * so[w][c];
    a.o[((size_t)t * a.Hq + h) * D + c] = __float2bfloat16_rn(sum == 0.f ? 0.f : x / sum);
  }
  if (threadIdx.x == 0) a.lse[(size_t)h * a.T + t] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

extern "C" size_t gocr_op_attention_paged_workspace(int T, int Hq, int Hkv, int d) {
  if (T < 0 || Hq < 1 || Hkv < 1 || d < 1) return 0;
  return 256;
}

extern "C" int gocr_op_attention_paged(const void* q, const gocr_paged_kv* cache, const int32_t* table, int max_pages,
                                       const int32_t* cu_rows, const int32_t* kv_len, int kind, void* o, float* lse,
                                       int n_req, int T, int Hq, long long ldq, float scale, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  gocr_paged_kv kv;
  if (int rc = cache_check(cache, &kv)) return rc;
  const int Hkv = kv.n_kv_heads, d = kv.head_dim;
  if (int rc = table_check(n_req, max_pages, kv.page_size, kv.n_pages)) return rc;
  if (kind != GOCR_FWD_AR && kind != GOCR_FWD_DRAFT && kind != GOCR_FWD_VERIFY) return op_fail(GOCR_EINVAL, "bad kind %d", kind);
  if (T < 0 || T > MAX_ROWS || Hq < 1 || Hq > 1024 || Hq % Hkv || Hq / Hkv > 64)
    return op_fail(GOCR_EINVAL, "bad shape: T=%d Hq=%d Hkv=%d", T, Hq, Hkv);
  if (!pitch_ok(ldq, Hq, d)) return op_fail(GOCR_EINVAL, "bad row pitch %lld", ldq);
  if (!(scale > 0.f) || scale > 1e30f) return op_fail(GOCR_EINVAL, "bad scale");
  if (!cu_rows || (n_req && (!table || !kv_len)) || (T && (!q || !o || !lse)) || !workspace) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)q | (uintptr_t)o | (uintptr_t)workspace) & 15) return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (((uintptr_t)table | (uintptr_t)cu_rows | (uintptr_t)kv_len | (uintptr_t)lse) & 3)
    return op_fail(GOCR_EINVAL, "array not 4-byte aligned");
  if (workspace_bytes < gocr_op_attention_paged_workspace(T, Hq, Hkv, d)) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T || !n_req) return GOCR_OK;
  int shift = 4;
  while ((1 << shift) < kv.page_size) ++shift;
  const PagedArgs a{(const bf16*)q, kv, table, cu_rows, kv_len, (bf16*)o, lse, ldq, max_pages, n_req, T, Hq, Hq / Hkv,
                   kind == GOCR_FWD_DRAFT, shift, scale};
  if (d == 128) attn_paged_kernel<128><<<dim3(T, Hq), 128, 0, s>>>(a);
  else attn_paged_kernel<64><<<dim3(T, Hq), 128, 0, s>>>(a);
  return op_launched("attention_paged");
}
