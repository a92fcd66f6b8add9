// Shared parts of the packed-sequence attention kernels (forward in
// attn_packed.cu, backward in attn_packed_bwd.cu).
//
// Rows of several sequences lie one after the other: sequence s is rows
// cu[s] .. cu[s + 1] - 1 of q, k, v and o.  Row i of a sequence reads rows
// 0 .. i of the same sequence.  q head h reads k/v head h / (Hq / Hkv).
#pragma once
#include "kernels.cuh"
#include "tc.cuh"

#include <cuda.h>

namespace gocr {
namespace packed {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Two fp32 operations an instruction.
struct F2 { unsigned long long v; };
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct Block {
  int row0;   // first row of the sequence
  int len;    // its rows
  int at;     // first row (within the sequence) of this block of `size` rows
};

// Where a search for a block may begin: a sequence, and the blocks before it.
struct Cursor { int seq = 0, before = 0; };

// The b-th block of `size` rows over all sequences, a sequence's last block
// first (its rows read the most keys); one warp, all lanes get the answer.  len = 0: there is no such block.  Whatever cu holds,
// the rows stay within 0 .. T - 1.  A lane takes PER sequences at a time, whose
// loads go out together, and a later search goes on where this one ended: with
// 2,000 sequences of 64 a lane for each one and a fresh start took more time
// than the attention (PER = 8 and going on: 2,400 -> 513 us).  A CTA that has one
// block only cannot go on: the backward call's take theirs from a table.
template <int PER>
__device__ __forceinline__ Block find_block(const int* cu, int n_seq, int T, int size, int b, Cursor& from) {
  const int lane = threadIdx.x & 31;
  Block r{0, 0, 0};
  if (b < from.before) from = Cursor{};
  while (from.seq < n_seq) {
    const int s = from.seq + lane * PER;
    int c[PER + 1], sum = 0;
#pragma unroll
    for (int i = 0; i <= PER; ++i) c[i] = min(max(cu[min(s + i, n_seq)], 0), T);
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += (max(c[i + 1] - c[i], 0) + size - 1) / size;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, from.before + inc > b);
    if (past) {
      int at = b - (from.before + inc - sum);  // among this lane's blocks
      bool open = true;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int len = max(c[i + 1] - c[i], 0), n = (len + size - 1) / size;
        if (open && at < n) {
          r.row0 = c[i];
          r.len = len;
          r.at = (n - 1 - at) * size;
          open = false;
        }
        at -= n;
      }
      const int src = __ffs(past) - 1;
      r.row0 = __shfl_sync(0xffffffffu, r.row0, src);
      r.len = __shfl_sync(0xffffffffu, r.len, src);
      r.at = __shfl_sync(0xffffffffu, r.at, src);
      return r;
    }
    from.before += __shfl_sync(0xffffffffu, inc, 31);
    from.seq += 32 * PER;
  }
  return r;
}

// The blocks of `size` rows of all sequences, in order, as (row0, len, at), and
// len = 0 for what is left of `n` entries.  One CTA of 256 threads.
__device__ __forceinline__ void block_table(const int* cu, int n_seq, int T, int size, int4* table, int n) {
  constexpr int PER = 8;
  __shared__ int sums[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int before = 0;  // blocks of the steps before
  for (int s0 = 0; s0 < n_seq; s0 += 256 * PER) {
    const int s = s0 + tid * PER;
    int c[PER + 1], sum = 0;
#pragma unroll
    for (int i = 0; i <= PER; ++i) c[i] = min(max(cu[min(s + i, n_seq)], 0), T);
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += (max(c[i + 1] - c[i], 0) + size - 1) / size;
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int at = before + inc - sum;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += sums[w];
      before += sums[w];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int len = max(c[i + 1] - c[i], 0);
      for (int r = 0; r < len && at < n; r += size) table[at++] = make_int4(c[i], len, r, 0);
    }
  }
  for (int i = before + tid; i < n; i += 256) table[i] = make_int4(0, 0, 0, 0);
}

// Most blocks of `size` rows that n_seq sequences of T rows in all can have.
inline long long max_blocks(int n_seq, int T, int size) {
  const int m = n_seq < T ? n_seq : T;  // sequences that are not empty
  return (long long)m + (T - m) / size;
}

// A tile of 128 rows x D bf16 in shared memory: D / 64 boxes of 128 rows x 128
// bytes, swizzled, as TMA writes them.
template <int D> constexpr int TILE_BYTES = 128 * D * 2;
constexpr int BOX_BYTES = 128 * 128;

template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const void* map, int head, int row, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(dst + c * BOX_BYTES, map, c * 64, head, row, bar);
}

// Rows n .. 127 of a tile become zero: they belong to another sequence or to
// nobody and may hold anything, and a product that runs over rows would carry
// their NaN or infinity into this sequence.  One warp.
template <int D> __device__ __forceinline__ void zero_rows(uint8_t* tile, int n) {
  const int lane = threadIdx.x & 31;
  for (int i = n * 8 + lane; i < 128 * 8; i += 32)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) *reinterpret_cast<uint4*>(tile + c * BOX_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
}

// Products over tiles of 128 rows, issued by one elected lane.
//   mma_rows   dst[128, N] = X Y^T over D: both tiles K-major; N = 64: rows 64
//              half .. of Y's, N = 128: all of them
//   mma_add    dst[128, D] (+)= P Y over rows 64 half .. of Y's, N-major: P
//              (bf16, two a column) from tensor memory
// first: dst is overwritten.
constexpr int HALF_ROWS = 64 * 128;  // bytes of 64 rows in a box
template <int D, int N = 64> __device__ __forceinline__ void mma_rows(uint32_t dst, uint32_t x, uint32_t y, int half) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, N);
  const uint64_t xd = tc::sdesc_sw128(x), yd = tc::sdesc_sw128(y + half * HALF_ROWS);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t step = ((ks >> 2) * BOX_BYTES + (ks & 3) * 32) >> 4;
    tc::mma_bf16(dst, xd + step, yd + step, idesc, ks > 0 ? 1u : 0u);
  }
}
template <int D> __device__ __forceinline__ void mma_add(uint32_t dst, uint32_t p, uint32_t y, int half, bool first) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, D) | tc::IDESC_B_MN;
  const uint64_t yd = tc::sdesc_sw128_mn(y + half * HALF_ROWS, BOX_BYTES);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) tc::mma_bf16_ta(dst, p + ks * 8, yd + (ks * 2048 >> 4), idesc, !first || ks > 0 ? 1u : 0u);
}

// 3-D TMA map over [T, heads, D] bf16 rows `ld` elements apart: boxes of 64
// columns x 1 head x 128 rows.
inline bool map_rows(CUtensorMap* m, const void* p, int T, int heads, int D, long long ld) {
  const unsigned long long dims[3] = {(unsigned long long)D, (unsigned long long)heads, (unsigned long long)T};
  const unsigned long long st[2] = {(unsigned long long)D * 2, (unsigned long long)ld * 2};
  const unsigned box[3] = {64, 1, 128};
  return encode_tmap(m, p, false, 3, dims, st, box);
}

}  // namespace packed
}  // namespace gocr
