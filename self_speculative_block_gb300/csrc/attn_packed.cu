// Causal attention over packed sequences with grouped heads, forward.
//
//   S_ij = c q_i . k_j (j <= i),  lse_i = log sum_j exp S_ij,  o_i = sum_j exp(S_ij - lse_i) v_j
//
// One CTA per (256 query rows of a sequence, q head): two tiles of 128 rows
// share the K/V ring that a TMA warp fills.  Both products run on tcgen05: S =
// Q K^T (128 x 128 x D) into tensor memory, P (bf16) back into tensor memory
// over S, O += P V with P read from there and V N-major as it lies.  A softmax
// thread owns a row: its 128 scores come from its own tensor memory lane, so
// the running maximum and sum need no exchange.  While one tile's softmax
// runs, the tensor cores work for the other.  O stays in tensor memory and is
// rescaled only when a row's maximum grows by more than 2^8 over the one its
// exponentials refer to (the sum and O use the same reference, so nothing is
// lost; P is at most 2^8).  P is rounded to bf16 (relative 2^-8) since the
// tensor cores take it so; scores, maxima, sums and O are fp32.  No partial
// results leave the CTA: a row's bits depend on its own sequence only.
#include "../../include/gocr.h"
#include "attn_packed.cuh"

using namespace gocr;
using namespace gocr::packed;

namespace {

constexpr int QT = 256;        // query rows of a CTA
// Two softmax groups of four warps, and a group with the TMA and the MMA warp.
// A softmax thread holds a row's 128 scores: its group takes 208 registers a
// thread of the 168 x 384 that the block is launched with, the third 88.
constexpr int THREADS = 384;
constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;
static_assert(2 * SOFTMAX_REGS + OTHER_REGS <= 3 * 168, "registers of the block at launch");
constexpr float GROW = 8.f;    // log2 of the growth of a row's maximum that rescales O

static __device__ int g_error;  // DevErr of a wait that gave up

struct FwdArgs {
  const int* cu;
  bf16* o;
  float* lse;
  int n_seq, T, Hq, Hkv;
  float scale;
};

template <int D> struct Fwd {
  static constexpr int SLOTS = D == 128 ? 4 : 8;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TILE_BYTES<D>;
  static constexpr int OFF_BAR = OFF_KV + SLOTS * TILE_BYTES<D>;
  static constexpr int SMEM = OFF_BAR + 256 + 1024;
  static constexpr uint32_t O_COL = 256;  // S0, S1 at 0, 128; O0, O1 behind them
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_packed_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const FwdArgs a) {
  using F = Fwd<D>;
  constexpr int SLOTS = F::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + F::OFF_BAR);
  uint64_t* full = q_full + 1;
  uint64_t* empty = full + SLOTS;
  uint64_t* s_full = empty + SLOTS;  // [2]
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* o_full = p_full + 2;     // [2]
  uint64_t* v_tail = o_full + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(v_tail + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int head = blockIdx.x % a.Hq;
  const Block blk = find_block<true>(a.cu, a.n_seq, a.T, QT, blockIdx.x / a.Hq);  // each warp for itself
  if (blk.len == 0) return;
  const int kvh = head / (a.Hq / a.Hkv);
  // key blocks of the two tiles: up to the diagonal, and within the sequence
  const int left = blk.len - blk.at;
  const int n0 = blk.at / 128 + 1;
  const int n1 = left > 128 ? n0 + 1 : 0;
  const int n = n1 ? n1 : n0;
  const int tail = blk.len - (n - 1) * 128;  // rows of the last key block within the sequence, if < 128

  if (tid == 0) {
    tc::mbar_init(q_full, 1);
    for (int s = 0; s < SLOTS; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 1);
    }
    for (int j = 0; j < 2; ++j) {
      tc::mbar_init(s_full + j, 1);
      tc::mbar_init(p_full + j, 4);
      tc::mbar_init(o_full + j, 1);
    }
    tc::mbar_init(v_tail, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (warp == 9) tc::tmem_alloc(holder, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *holder;
  bool ok = true;

  if (warp >= 8) {
    fewer_registers<OTHER_REGS>();
    if (warp == 8) {
    // K(0), V(0), K(1), V(1), ... through the ring
    if (lane == 0) {
      tc::mbar_expect_tx(q_full, (n1 ? 2 : 1) * TILE_BYTES<D>);
      load_tile<D>(sm + F::OFF_Q, &mq, head, blk.row0 + blk.at, q_full);
      if (n1) load_tile<D>(sm + F::OFF_Q + TILE_BYTES<D>, &mq, head, blk.row0 + blk.at + 128, q_full);
      int slot = 0, ph = 0;
      for (int i = 0; i < 2 * n; ++i) {
        if (!(ok = tc::mbar_wait_ns(empty + slot, ph ^ 1))) break;
        tc::mbar_expect_tx(full + slot, TILE_BYTES<D>);
        load_tile<D>(sm + F::OFF_KV + slot * TILE_BYTES<D>, i & 1 ? &mv : &mk, kvh, blk.row0 + (i >> 1) * 128, full + slot);
        if (++slot == SLOTS) { slot = 0; ph ^= 1; }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (ok && tail < 128) {  // the last V tile: nothing behind the sequence
      const int i = 2 * n - 1, slot = i % SLOTS;
      ok = __all_sync(0xffffffffu, tc::mbar_wait_ns(full + slot, (i / SLOTS) & 1));
      zero_rows<D>(sm + F::OFF_KV + slot * TILE_BYTES<D>, tail);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(v_tail);
    }
    } else if (warp == 9) {
    if (lane == 0) {
      constexpr uint32_t idesc_s = tc::idesc_bf16(128, 128);
      constexpr uint32_t idesc_o = tc::idesc_bf16(128, D) | tc::IDESC_B_MN;
      const uint32_t q = tc::smem_u32(sm + F::OFF_Q), kv = tc::smem_u32(sm + F::OFF_KV);
      auto tile_of = [&](int i) { return kv + (i % SLOTS) * TILE_BYTES<D>; };
      auto wait_full = [&](int i) {
        const bool w = tc::mbar_wait_ns(full + i % SLOTS, (i / SLOTS) & 1);
        tc::fence_after_sync();
        return w;
      };
      auto scores = [&](int j, int it) {
        const uint32_t k = tile_of(2 * it);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc::mma_bf16(tmem + j * 128, desc_k(q + j * TILE_BYTES<D>, ks), desc_k(k, ks), idesc_s, ks > 0 ? 1u : 0u);
        tc::mma_commit(s_full + j);
      };
      ok = tc::mbar_wait_ns(q_full, 0) && wait_full(0);
      if (ok) {
        scores(0, 0);
        if (n1) scores(1, 0);
        tc::mma_commit(empty);
      }
      for (int it = 0; it < n && ok; ++it) {
        if (!(ok = wait_full(2 * it + 1))) break;
        if (it == n - 1 && tail < 128) {
          if (!(ok = tc::mbar_wait_ns(v_tail, 0))) break;
          tc::fence_after_sync();
        }
        const uint32_t v = tile_of(2 * it + 1);
        const bool more = it + 1 < n;
        bool have_k = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int nj = j ? n1 : n0;
          if (it >= nj) continue;
          if (!(ok = tc::mbar_wait_ns(p_full + j, it & 1))) break;
          tc::fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_bf16_ta(tmem + F::O_COL + j * D, tmem + j * 128 + ks * 8, desc_n(v, ks), idesc_o,
                            it > 0 || ks > 0 ? 1u : 0u);
          if (it + 1 < nj) {
            if (!have_k && !(ok = wait_full(2 * it + 2))) break;
            have_k = true;
            scores(j, it + 1);
          } else {
            tc::mma_commit(o_full + j);
          }
        }
        if (!ok) break;
        tc::mma_commit(empty + (2 * it + 1) % SLOTS);
        if (more) tc::mma_commit(empty + (2 * it + 2) % SLOTS);
      }
    }
    }
  } else {
    more_registers<SOFTMAX_REGS>();
    const int j = warp >> 2;
    const int nj = j ? n1 : n0;
    const int row = blk.at + j * 128 + (warp & 3) * 32 + lane;  // within the sequence
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + j * 128 + lanes, to = tmem + F::O_COL + j * D + lanes;
    const float sl2 = a.scale * LOG2E;
    float ref = 0.f, ref2 = 0.f, l = 0.f;  // the exponentials' reference, also times sl2; their sum
    for (int it = 0; it < nj; ++it) {
      if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait_ns(s_full + j, it & 1)))) break;
      tc::fence_after_sync();
      uint32_t u[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_ld32_nowait(ts + c * 32, u + c * 32);
      tc::tmem_wait_ld();
      if (it + 1 == nj) {  // the diagonal block; it holds the end of the sequence, too
        const int see = min(row, blk.len - 1) - it * 128;
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i > see) u[i] = 0xff800000u;  // -infinity
      }
      float m4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) m4[e] = fmaxf(__uint_as_float(u[e]), __uint_as_float(u[e + 4]));
#pragma unroll
      for (int i = 8; i < 128; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(fmaxf(m4[e], __uint_as_float(u[i + e])), __uint_as_float(u[i + e + 4]));
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      if (it == 0) {
        ref = mx == -INFINITY ? 0.f : mx;
        ref2 = ref * sl2;
      } else {
        const bool grow = (mx - ref) * sl2 > GROW;
        if (__any_sync(0xffffffffu, grow)) {
          // S(it) was issued after P V(it - 1): O is complete
          const float to_new = grow ? mx : ref;
          const float f = ex2(ref2 - to_new * sl2);
          ref = to_new;
          ref2 = ref * sl2;
          l *= f;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t w[32];
            tc::tmem_ld32_nowait(to + c, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
            tc::tmem_st32(to + c, w);
          }
        }
      }
      const F2 scale2 = f2(sl2, sl2), ref22 = f2(-ref2, -ref2);
      F2 s4[4] = {f2(l, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < 128; i += 2) {
        float x, y;
        split(fma2(f2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), scale2, ref22), x, y);
        x = ex2(x);
        y = ex2(y);
        s4[(i >> 1) & 3] = add2(s4[(i >> 1) & 3], f2(x, y));
        u[i / 2] = pack2(x, y);
      }
      {
        float x, y;
        split(add2(add2(s4[0], s4[1]), add2(s4[2], s4[3])), x, y);
        l = x + y;
      }
      tc::tmem_st32(ts, u);
      tc::tmem_st32(ts + 32, u + 32);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_full + j);
    }
    if (nj && ok) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait_ns(o_full + j, 0));
      tc::fence_after_sync();
      const float inv = 1.f / l;
      const size_t t = (size_t)blk.row0 + row;
      bf16* dst = a.o + (t * a.Hq + head) * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t w[32];
        tc::tmem_ld32_nowait(to + c, w);
        tc::tmem_wait_ld();
        if (ok && row < blk.len)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = pack2(__uint_as_float(w[g * 8 + 2 * e]) * inv, __uint_as_float(w[g * 8 + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + c + g * 8) = make_uint4(h[0], h[1], h[2], h[3]);
          }
      }
      if (ok && row < blk.len) a.lse[(size_t)head * a.T + t] = (ref2 + log2f(l)) * LN2;
    }
  }
  if (!ok) atomicCAS(&g_error, 0, (int)DERR_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D> int forward(const CUtensorMap* m, const FwdArgs& a, cudaStream_t s) {
  using F = Fwd<D>;
  if (!kernel_smem_at_least(reinterpret_cast<const void*>(&attn_packed_kernel<D>), F::SMEM))
    return op_fail(GOCR_ECUDA, "kernel configuration rejected");
  attn_packed_kernel<D><<<(unsigned)(max_blocks(a.n_seq, a.T, QT) * a.Hq), THREADS, F::SMEM, s>>>(m[0], m[1], m[2], a);
  return op_launched("attention_packed");
}

}  // namespace

namespace gocr {
cudaError_t take_attn_packed_error(int* out) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_error, sizeof(int));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_error, &zero, sizeof(int));
  return e;
}

int attn_packed_check(int n_seq, int T, int Hq, int Hkv, int d, long long ldq, long long ldk, long long ldv,
                      float scale) {
  if (n_seq < 0 || n_seq > (1 << 20) || T < 0 || T > (1 << 24) || Hkv < 1 || Hq < 1 || Hq % Hkv || Hq > 1024 ||
      (d != 64 && d != 128) || max_blocks(n_seq, T, 128) * (Hq + Hkv) > 0x7fffffffLL)
    return op_fail(GOCR_EINVAL, "bad shape: %d sequences, T=%d Hq=%d Hkv=%d d=%d", n_seq, T, Hq, Hkv, d);
  const long long most = 1ll << 32;  // row pitch: 2^33 bytes, within a TMA stride
  if (ldq < (long long)Hq * d || ldk < (long long)Hkv * d || ldv < (long long)Hkv * d || (ldq | ldk | ldv) % 8 ||
      ldq > most || ldk > most || ldv > most)
    return op_fail(GOCR_EINVAL, "bad row pitch %lld, %lld, %lld", ldq, ldk, ldv);
  if (!(scale > 0.f) || scale > 1e30f) return op_fail(GOCR_EINVAL, "bad scale");
  return GOCR_OK;
}
}  // namespace gocr

extern "C" int gocr_op_attention_packed(const void* q, const void* k, const void* v, void* o, float* lse,
                                        const int32_t* cu_seqlens, int n_seq, int T, int Hq, int Hkv, int d,
                                        long long ldq, long long ldk, long long ldv, float scale, void* stream) {
  if (int rc = attn_packed_check(n_seq, T, Hq, Hkv, d, ldq, ldk, ldv, scale)) return rc;
  if (!cu_seqlens || (T && (!q || !k || !v || !o || !lse))) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o) & 15) return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T || !n_seq) return GOCR_OK;
  CUtensorMap m[3];
  if (!map_rows(&m[0], q, T, Hq, d, ldq) || !map_rows(&m[1], k, T, Hkv, d, ldk) || !map_rows(&m[2], v, T, Hkv, d, ldv))
    return op_fail(GOCR_ECUDA, "a TMA descriptor was rejected");
  const FwdArgs a{cu_seqlens, (bf16*)o, lse, n_seq, T, Hq, Hkv, scale};
  return d == 128 ? forward<128>(m, a, s) : forward<64>(m, a, s);
}
