// Rotary embedding of a forward's q and k rows, and k and v into their pages.
//
//   y_i = c u_i - s u_(i+d/2),  y_(i+d/2) = c u_(i+d/2) + s u_i,  (c, s) = (cos, sin)(x theta^(-2i/d))
//
// A row's angles serve all of its heads, so a CTA takes a few rows, evaluates
// their cosines and sines once into shared memory, and its threads then take 8 + 8
// elements of a head each (both halves of the rotation), 16 bytes a load.  The angle
// in turns is x f_i mod 1 with f_i = theta^(-2i/d) / 2 pi as a 64-bit fraction:
// one integer product whose overflow drops the whole turns, exact to x 2^-54 or
// so (f_i comes from a double), where fp32 would lose 2^-24 of the whole angle.
#include "paged.cuh"

#include <cmath>

using namespace gocr;
using namespace gocr::paged;

namespace {

constexpr int THREADS = 256;
constexpr int MOST_ROWS = 8;  // rows of a CTA

struct WriteArgs {
  const bf16 *q, *k, *v;
  const int *pos, *slots;
  bf16* q_out;
  gocr_paged_kv kv;
  long long ldq, ldk, ldv;
  int T, Hq, rows, shift;
  unsigned long long freq[64];  // turns a position, 2^64 a turn
};

__device__ __forceinline__ float2 up2(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
__device__ __forceinline__ uint32_t down2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D> __global__ void __launch_bounds__(THREADS) kv_write_kernel(const __grid_constant__ WriteArgs a) {
  constexpr int H = D / 2, P = D / 16;  // pieces of 8 + 8 elements in a head
  __shared__ float2 cs[MOST_ROWS][H];
  const int t0 = blockIdx.x * a.rows, n = min(a.rows, a.T - t0), heads = a.Hq + 2 * a.kv.n_kv_heads;
  const unsigned n_slots = (unsigned)a.kv.n_pages << a.shift;
  for (int i = threadIdx.x; i < n * H; i += THREADS) {
    const unsigned long long turn = (unsigned long long)(long long)a.pos[t0 + i / H] * a.freq[i % H];
    float s, c;  // half turns in [-1, 1), to 2^-31
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
    cs[i / H][i % H] = make_float2(c, s);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * heads * P; i += THREADS) {
    const int p = i % P, h = i / P % heads, t = t0 + i / (P * heads);
    const unsigned slot = (unsigned)a.slots[t];
    if (slot >= n_slots) continue;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.kv.n_kv_heads;
    const int kh = h - a.Hq - (is_k ? 0 : a.kv.n_kv_heads);
    const bf16* src = is_q ? a.q + t * a.ldq + h * D : is_k ? a.k + t * a.ldk + kh * D : a.v + t * a.ldv + kh * D;
    const long long page = slot >> a.shift, off = slot & ((1u << a.shift) - 1);
    bf16* dst = is_q ? a.q_out + ((size_t)t * a.Hq + h) * D
                : is_k ? (bf16*)a.kv.k + page * a.kv.k_page + kh * a.kv.k_head + off * a.kv.k_token
                       : (bf16*)a.kv.v + page * a.kv.v_page + kh * a.kv.v_head + off * a.kv.v_token;
    uint4 lo = *reinterpret_cast<const uint4*>(src + p * 8), hi = *reinterpret_cast<const uint4*>(src + H + p * 8);
    if (is_q || is_k) {
      uint32_t *u = &lo.x, *w = &hi.x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = up2(u[e]), y = up2(w[e]);
        const float2 c0 = cs[t - t0][p * 8 + 2 * e], c1 = cs[t - t0][p * 8 + 2 * e + 1];
        u[e] = down2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
        w[e] = down2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
      }
    }
    *reinterpret_cast<uint4*>(dst + p * 8) = lo;
    *reinterpret_cast<uint4*>(dst + H + p * 8) = hi;
  }
}

}  // namespace

extern "C" int gocr_op_kv_write_paged(const void* q, const void* k, const void* v, const int32_t* pos,
                                      const int32_t* slots, void* q_out, const gocr_paged_kv* kv, int T, int Hq,
                                      long long ldq, long long ldk, long long ldv, float theta, void* stream) {
  WriteArgs a{};
  if (int rc = cache_check(kv, &a.kv)) return rc;
  const int Hkv = a.kv.n_kv_heads, d = a.kv.head_dim;
  if (T < 0 || T > MAX_ROWS || Hq < 1 || Hq > 1024 || Hq % Hkv)
    return op_fail(GOCR_EINVAL, "bad shape: T=%d Hq=%d Hkv=%d", T, Hq, Hkv);
  if (!pitch_ok(ldq, Hq, d) || !pitch_ok(ldk, Hkv, d) || !pitch_ok(ldv, Hkv, d))
    return op_fail(GOCR_EINVAL, "bad row pitch %lld, %lld, %lld", ldq, ldk, ldv);
  if (!(theta >= 1.f) || theta > 1e30f) return op_fail(GOCR_EINVAL, "bad theta");
  if (T && (!q || !k || !v || !pos || !slots || !q_out)) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) & 15)
    return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (((uintptr_t)pos | (uintptr_t)slots) & 3) return op_fail(GOCR_EINVAL, "pos or slots not 4-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T) return GOCR_OK;
  a.q = (const bf16*)q;
  a.k = (const bf16*)k;
  a.v = (const bf16*)v;
  a.pos = pos;
  a.slots = slots;
  a.q_out = (bf16*)q_out;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.T = T;
  a.Hq = Hq;
  while ((1 << a.shift) < a.kv.page_size) ++a.shift;
  for (int i = 0; i < d / 2; ++i)  // at most 1 / 2 pi of a turn
    a.freq[i] = (unsigned long long)std::ldexp(std::pow((double)theta, -2.0 * i / d) / 6.283185307179586476925, 64);
  a.rows = 1;
  const int grid = (T + a.rows - 1) / a.rows;
  if (d == 128) kv_write_kernel<128><<<grid, THREADS, 0, s>>>(a);
  else kv_write_kernel<64><<<grid, THREADS, 0, s>>>(a);
  return op_launched("kv_write_paged");
}
