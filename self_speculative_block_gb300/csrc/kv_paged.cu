// Rotary embedding of a forward's q and k rows, and k and v into their pages.
//
//   y_i = c u_i - s u_(i+d/2),  y_(i+d/2) = c u_(i+d/2) + s u_i,  (c, s) = (cos, sin)(x theta^(-2i/d))
//
// A row's angles serve all of its heads, so a CTA takes a few rows and evaluates
// their cosines and sines once into shared memory, while its threads' loads are under
// way: a thread takes 8 + 8 elements of a head (both halves of the rotation), 16 bytes a
// load, two such pieces at a time.  The angle in turns is x f_i mod 1 with f_i =
// theta^(-2i/d) / 2 pi as a 64-bit fraction: one integer product whose overflow
// drops the whole turns, where fp32 would lose 2^-24 of the whole angle.  f_i comes from
// doubles, to 2^-50 of its value and so to x 2^-52.6 turns; the top 32 bits of the product
// lose 2^-32 and their conversion to fp32 2^-26 more: 2^-25.7 turns up to position 2^24.
//
// Bound by HBM: 13,655 rows of 12 + 2 x 4 heads of 128 (140 MB) 28.7 us, 4.9 TB/s
// (torch's copy of 70 MB takes 47), of heads of 64 11.5; without the angles the same.  Two
// pieces a batch and 256 threads: four pieces 30.5, 128 or 512 threads 28.4 to 31,
// streaming loads and stores 28.3; a row a CTA 36.  528 rows take 3.5 us (heads of
// 64: 2.5), 64 2.1.
#include "paged.cuh"
#include "tc.cuh"

#include <cmath>

using namespace gocr;
using namespace gocr::paged;

namespace {

constexpr int THREADS = 256, BATCH = 2;
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
  constexpr int H = D / 2, P = D / 16, STEP = THREADS / P;  // pieces of a head; heads a step
  __shared__ __align__(16) float2 cs[MOST_ROWS][H];
  __shared__ unsigned slot_of[MOST_ROWS];
  const int t0 = blockIdx.x * a.rows, n = min(a.rows, a.T - t0), Hq = a.Hq, Hkv = a.kv.n_kv_heads, heads = Hq + 2 * Hkv;
  const unsigned n_slots = (unsigned)a.kv.n_pages << a.shift;
  const int p = threadIdx.x % P;
  tc::grid_dep_launch();  // the next kernel's beginning overlaps this one, this one's the last one's
  tc::grid_dep_wait();
  int row = 0, h = threadIdx.x / P;
  for (bool first = true;; first = false) {
    uint4 lo[BATCH], hi[BATCH];
    int rows[BATCH], hs[BATCH];
#pragma unroll
    for (int e = 0; e < BATCH; ++e) {
      while (h >= heads) {
        h -= heads;
        ++row;
      }
      rows[e] = row;
      hs[e] = h;
      if (row < n) {
        const long long t = t0 + row;
        const bf16* src = (h < Hq ? a.q + t * a.ldq + h * D : h < Hq + Hkv ? a.k + t * a.ldk + (h - Hq) * D
                                                                           : a.v + t * a.ldv + (h - Hq - Hkv) * D) + p * 8;
        lo[e] = *reinterpret_cast<const uint4*>(src);
        hi[e] = *reinterpret_cast<const uint4*>(src + H);
      }
      h += STEP;
    }
    if (first) {
      for (int i = threadIdx.x; i < n * H; i += THREADS) {
        const unsigned long long turn = (unsigned long long)(long long)a.pos[t0 + i / H] * a.freq[i % H];
        float s, c;  // half turns in [-1, 1), to 2^-31
        sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
        cs[i / H][i % H] = make_float2(c, s);
      }
      if (threadIdx.x < n) slot_of[threadIdx.x] = (unsigned)a.slots[t0 + threadIdx.x];
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < BATCH; ++e) {
      const int r = rows[e], hh = hs[e];
      if (r >= n) return;  // (rows do not decrease)
      const unsigned slot = slot_of[r];
      if (slot >= n_slots) continue;
      if (hh < Hq + Hkv) {
        uint32_t *u = &lo[e].x, *w = &hi[e].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = up2(u[i]), y = up2(w[i]);
          const float4 c = *reinterpret_cast<const float4*>(&cs[r][p * 8 + 2 * i]);
          u[i] = down2(x.x * c.x - y.x * c.y, x.y * c.z - y.y * c.w);
          w[i] = down2(y.x * c.x + x.x * c.y, y.y * c.z + x.y * c.w);
        }
      }
      const long long page = slot >> a.shift, off = slot & ((1u << a.shift) - 1);
      bf16* dst = (hh < Hq ? a.q_out + ((size_t)(t0 + r) * Hq + hh) * D
                   : hh < Hq + Hkv ? (bf16*)a.kv.k + page * a.kv.k_page + (hh - Hq) * a.kv.k_head + off * a.kv.k_token
                                   : (bf16*)a.kv.v + page * a.kv.v_page + (hh - Hq - Hkv) * a.kv.v_head + off * a.kv.v_token) + p * 8;
      *reinterpret_cast<uint4*>(dst) = lo[e];
      *reinterpret_cast<uint4*>(dst + H) = hi[e];
    }
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
  // theta^(-2i/d) as the product of its powers of two in i (relative 2^-50); at most 1 / 2 pi of a turn
  double power[64] = {0x1p64 / 6.283185307179586476925};
  for (int bit = 1; bit < d / 2; bit *= 2) {
    const double f = std::pow((double)theta, -2.0 * bit / d);
    for (int i = 0; i < bit; ++i) power[bit + i] = power[i] * f;
  }
  for (int i = 0; i < d / 2; ++i) a.freq[i] = (unsigned long long)power[i];
  // rows that a CTA's threads take in one batch; fewer where that leaves SMs without a CTA
  const int fit = THREADS * BATCH / ((Hq + 2 * Hkv) * (d / 16)), spread = (T + 2 * SM_COUNT - 1) / (2 * SM_COUNT);
  a.rows = fit < spread ? fit : spread;
  a.rows = a.rows < 1 ? 1 : a.rows > MOST_ROWS ? MOST_ROWS : a.rows;
  const int grid = (T + a.rows - 1) / a.rows;
  if (d == 128) launch_k(kv_write_kernel<128>, dim3(grid), dim3(THREADS), 0, s, true, a);
  else launch_k(kv_write_kernel<64>, dim3(grid), dim3(THREADS), 0, s, true, a);
  return op_launched("kv_write_paged");
}
