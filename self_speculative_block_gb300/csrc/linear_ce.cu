// Softmax cross entropy of a linear head over a large vocabulary, without the
// logits ever being stored, and its gradient.
//
//   z_tv = x_t . w_v      lse_t = log sum_v exp z_tv      loss_t = lse_t - z_t,y(t)
//   g_tv = (exp(z_tv - lse_t) - [v = y(t)]) dloss_t        dx = g W      dw = g^T x
//
// All of it is matrix products on tcgen05: 2 T V H operations forward, 6 T V H
// backward (z again, dx, dw).  One persistent kernel shape serves the three
// products: a CTA per SM walks 128 x 256 output tiles, a TMA warp keeps a ring
// of 64-deep stages full, one thread issues the MMAs into one of two tensor
// memory accumulators, and four warps (one row a thread) run the epilogue of
// the other:
//   STATS  (z) the row's maximum, sum of exponentials over the tile's 256
//          columns, and the label's z: 8 bytes per row and tile leave the SM.
//          A second kernel joins them in tile order;
//   GRAD   (z) g in bf16, stored to the piece of the vocabulary in the
//          workspace;
//   PROD   dx += g W (fp32, each tile owned by one CTA, or by one CTA per
//          slice of the contraction in a slab of its own) and dw = g^T x (bf16)
//          of the piece, both read g as it lies: rows for dx (K-major), columns
//          for dw (M-major), W and x N-major, so nothing is transposed.
// The vocabulary goes by in pieces whose g fits the workspace (and L2); the
// tiles of both products of a piece share one launch, the longer ones first.
// g is rounded to bf16 (relative 2^-8) because the tensor cores take it so;
// every sum is in fp32.  Nothing is added by atomics across CTAs, so the same
// inputs give the same bits.
#include "../../include/gocr.h"
#include "kernels.cuh"
#include "tc.cuh"

#include <cuda.h>

using namespace gocr;

namespace {

constexpr int TM = 128, TN = 256, TK = 64;
constexpr int STAGES = 4;
constexpr int A_BYTES = TM * TK * 2, B_BYTES = TN * TK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX = 64 * 128;            // one box of 64 rows x 64 columns
constexpr int STORE_BYTES = 32 * 128;    // one epilogue box: 32 rows x 128 bytes
constexpr int OFF_STORE = STAGES * STAGE_BYTES;
constexpr int OFF_BAR = OFF_STORE + 4 * 2 * STORE_BYTES;
constexpr int SMEM = OFF_BAR + 256 + 1024;
static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
constexpr int THREADS = 192;  // TMA warp, MMA warp, four epilogue warps
constexpr float LOG2E = 1.4426950408889634f;

enum Kind { STATS, GRAD, PROD };

static __device__ int g_error;  // DevErr of a wait that gave up

struct Maps {
  CUtensorMap a0, b0;   // STATS, GRAD: x, w.  PROD: g (rows), w (N-major)
  CUtensorMap a1, b1;   // PROD: g (columns), x (N-major)
  CUtensorMap out0;     // GRAD: g.  PROD: the dx slabs
  CUtensorMap out1;     // PROD: dw
};

struct Args {
  int T, H, V;
  int v0, vc;           // GRAD, PROD: the piece of the vocabulary
  const int* labels;
  const float* lse;
  const float* dloss;
  float2* part;         // STATS: [T][vocabulary tiles] (maximum, sum)
  float* zlab;          // STATS: [T] z of the label
  int m_tiles, n_tiles;               // STATS, GRAD, and dx
  int splits, split_k, slab_rows;     // dx: slices of the contraction, in K steps
  int add;                            // dx: add to the slab (a later piece)
  int m_tiles1;                       // dw
  int tiles0, tiles;                  // tiles of the first product, of both
};

struct Tile {
  int prod;             // PROD: 0 dx, 1 dw
  int m0, n0, k0, ks;   // first row, column, K step; K steps
  int nb;               // 64-column blocks of B
  int row_out;          // dx: first row in the slabs
};

template <int KIND> __device__ __forceinline__ Tile tile_of(const Args& a, int i) {
  Tile t;
  t.prod = 0; t.k0 = 0; t.row_out = 0; t.nb = TN / 64;
  if (KIND != PROD) {
    // rows fastest: the CTAs of a wave share a few tiles of w
    t.m0 = (i % a.m_tiles) * TM;
    t.n0 = (i / a.m_tiles) * TN;
    t.ks = (a.H + TK - 1) / TK;
    return t;
  }
  if (i < a.tiles0) {
    const int s = i % a.splits, r = i / a.splits;
    const int steps = (a.vc + TK - 1) / TK;
    t.m0 = (r / a.n_tiles) * TM;
    t.n0 = (r % a.n_tiles) * TN;
    t.k0 = s * a.split_k;
    t.ks = max(0, min(a.split_k, steps - t.k0));
    t.row_out = s * a.slab_rows + t.m0;
  } else {
    i -= a.tiles0;
    t.prod = 1;
    t.m0 = (i / a.n_tiles) * TM;
    t.n0 = (i % a.n_tiles) * TN;
    t.ks = (a.T + TK - 1) / TK;
  }
  t.nb = min(TN / 64, (a.H - t.n0 + 63) / 64);
  return t;
}

__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Byte offset of 16-byte chunk c of row r in a 32-row swizzled box.
__device__ __forceinline__ uint32_t box_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

template <int KIND>
__global__ void __launch_bounds__(THREADS, 1) linear_ce_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;  // [2]
  uint64_t* acc_free = acc_full + 2;    // [2]
  uint32_t* holder = reinterpret_cast<uint32_t*>(acc_free + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(acc_full + b, 1);
      tc::mbar_init(acc_free + b, 4);
    }
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) tc::tmem_alloc(holder, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *holder;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int st = 0, ph = 0;
      for (int i = blockIdx.x; i < a.tiles && ok; i += gridDim.x) {
        const Tile t = tile_of<KIND>(a, i);
        const uint32_t bytes = A_BYTES + t.nb * BOX;
        for (int k = 0; k < t.ks; ++k) {
          if (!(ok = tc::mbar_wait_ns(empty + st, ph ^ 1))) break;
          uint8_t* sa = sm + st * STAGE_BYTES;
          uint8_t* sb = sa + A_BYTES;
          const int kk = (t.k0 + k) * TK;
          tc::mbar_expect_tx(full + st, bytes);
          if (KIND != PROD) {
            tc::tma_load_2d(sa, &maps.a0, kk, t.m0, full + st);
            tc::tma_load_2d(sb, &maps.b0, kk, a.v0 + t.n0, full + st);
          } else if (t.prod == 0) {
            tc::tma_load_2d(sa, &maps.a0, kk, t.m0, full + st);
            for (int b = 0; b < t.nb; ++b) tc::tma_load_2d(sb + b * BOX, &maps.b0, t.n0 + b * 64, a.v0 + kk, full + st);
          } else {
            tc::tma_load_2d(sa, &maps.a1, t.m0, kk, full + st);
            tc::tma_load_2d(sa + BOX, &maps.a1, t.m0 + 64, kk, full + st);
            for (int b = 0; b < t.nb; ++b) tc::tma_load_2d(sb + b * BOX, &maps.b1, t.n0 + b * 64, kk, full + st);
          }
          if (++st == STAGES) { st = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0, ph = 0, acc = 0, aph = 0;
      for (int i = blockIdx.x; i < a.tiles && ok; i += gridDim.x) {
        const Tile t = tile_of<KIND>(a, i);
        if (!(ok = tc::mbar_wait_ns(acc_free + acc, aph ^ 1))) break;
        tc::fence_after_sync();
        const uint32_t d = tmem + acc * TN;
        uint32_t idesc = tc::idesc_bf16(TM, t.nb * 64);
        if (KIND == PROD) idesc |= tc::IDESC_B_MN | (t.prod ? tc::IDESC_A_MN : 0u);
        for (int k = 0; k < t.ks; ++k) {
          if (!(ok = tc::mbar_wait_ns(full + st, ph))) break;
          tc::fence_after_sync();
          const uint32_t sa = tc::smem_u32(sm + st * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
          for (int j = 0; j < TK / 16; ++j) {
            const uint64_t ad = KIND == PROD && t.prod ? tc::sdesc_sw128_mn(sa + j * 2048, BOX) : tc::sdesc_sw128(sa + j * 32);
            const uint64_t bd = KIND == PROD ? tc::sdesc_sw128_mn(sb + j * 2048, BOX) : tc::sdesc_sw128(sb + j * 32);
            tc::mma_bf16(d, ad, bd, idesc, k > 0 || j > 0 ? 1u : 0u);
          }
          tc::mma_commit(empty + st);
          if (++st == STAGES) { st = 0; ph ^= 1; }
        }
        if (!ok) break;
        tc::mma_commit(acc_full + acc);
        acc ^= 1;
        if (acc == 0) aph ^= 1;
      }
    }
  } else {
    const int q = warp & 3;  // the tensor memory lanes this warp may read: 32 q ..
    uint8_t* box = sm + OFF_STORE + q * 2 * STORE_BYTES;
    int acc = 0, aph = 0, buf = 0;
    for (int i = blockIdx.x; i < a.tiles; i += gridDim.x) {
      const Tile t = tile_of<KIND>(a, i);
      // one verdict a warp: its lanes leave the loop together
      if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait_ns(acc_full + acc, aph)))) break;
      tc::fence_after_sync();
      const uint32_t src = tmem + acc * TN + ((uint32_t)(q * 32) << 16);
      const int row = t.m0 + q * 32 + lane;
      if (KIND == STATS) {
        const bool in = row < a.T;
        const int label = in ? a.labels[row] : -1;
        float m = -INFINITY, s = 0.f;
        for (int c = 0; c < TN; c += 32) {
          const int col = t.n0 + c;
          if (col >= a.V) break;
          float v[32];
          tc::tmem_ld32(src + c, v);
          if (col + 32 > a.V) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col + j >= a.V) v[j] = -INFINITY;
          }
          float mc = v[0];
#pragma unroll
          for (int j = 1; j < 32; ++j) mc = fmaxf(mc, v[j]);
          const float mn = fmaxf(m, mc);
          const float ref = mn == -INFINITY ? 0.f : mn * LOG2E;
          float e0 = 0.f, e1 = 0.f;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            e0 += exp2f(fmaf(v[j], LOG2E, -ref));
            e1 += exp2f(fmaf(v[j + 1], LOG2E, -ref));
          }
          s = fmaf(s, m == -INFINITY ? 0.f : exp2f(fmaf(m, LOG2E, -ref)), e0 + e1);
          m = mn;
          const unsigned at = (unsigned)(label - col);
          if (__any_sync(0xffffffffu, at < 32u)) {
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z = at == (unsigned)j ? v[j] : z;
            if (at < 32u && label < a.V) a.zlab[row] = z;
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(acc_free + acc);
        if (in) a.part[(size_t)row * a.n_tiles + t.n0 / TN] = make_float2(m, s);
      } else if (KIND == GRAD) {
        int label = -1;
        float f = 0.f, ref = 0.f;
        if (row < a.T) {
          label = a.labels[row];
          if ((unsigned)label < (unsigned)a.V) {
            f = a.dloss[row];
            ref = a.lse[row] * LOG2E;
          } else {
            label = -1;
          }
        }
        const int col0 = a.v0 + t.n0;
        const bool has = label >= 0;
        for (int c = 0; c < TN; c += 64) {
          if (t.n0 + c >= a.vc) break;
          if (lane == 0) bulk_wait_read1();
          __syncwarp();
          uint8_t* bx = box + buf * STORE_BYTES;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            tc::tmem_ld32(src + c + h * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = has ? f * exp2f(fmaf(v[j], LOG2E, -ref)) : 0.f;
            const unsigned at = (unsigned)(label - (col0 + c + h * 32));
            if (__any_sync(0xffffffffu, has && at < 32u)) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (has && at == (unsigned)j) v[j] -= f;
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(v[g * 8 + 2 * e], v[g * 8 + 2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t*>(&p);
              }
              *reinterpret_cast<uint4*>(bx + box_at(lane, h * 4 + g)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (t.m0 + q * 32 < a.T) tc::tma_store_2d(&maps.out0, bx, t.n0 + c, t.m0 + q * 32);
            tc::bulk_commit();
          }
          buf ^= 1;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(acc_free + acc);
      } else {
        const int step = t.prod ? 64 : 32;  // columns of one box
        for (int c = 0; c < t.nb * 64 && t.n0 + c < a.H; c += step) {
          if (lane == 0) bulk_wait_read1();
          __syncwarp();
          uint8_t* bx = box + buf * STORE_BYTES;
          if (t.prod == 0) {
            float v[32];
            tc::tmem_ld32(src + c, v);
#pragma unroll
            for (int g = 0; g < 8; ++g)
              *reinterpret_cast<float4*>(bx + box_at(lane, g)) =
                  t.ks > 0 ? make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[32];
              tc::tmem_ld32(src + c + h * 32, v);
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const __nv_bfloat162 p = __floats2bfloat162_rn(v[g * 8 + 2 * e], v[g * 8 + 2 * e + 1]);
                  w[e] = *reinterpret_cast<const uint32_t*>(&p);
                }
                *reinterpret_cast<uint4*>(bx + box_at(lane, h * 4 + g)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (t.prod) {
              if (a.v0 + t.m0 + q * 32 < a.V) tc::tma_store_2d(&maps.out1, bx, t.n0 + c, a.v0 + t.m0 + q * 32);
            } else if (a.add) {
              tc::tma_add_2d(&maps.out0, bx, t.n0 + c, t.row_out + q * 32);
            } else {
              tc::tma_store_2d(&maps.out0, bx, t.n0 + c, t.row_out + q * 32);
            }
            tc::bulk_commit();
          }
          buf ^= 1;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(acc_free + acc);
      }
      acc ^= 1;
      if (acc == 0) aph ^= 1;
    }
    if (lane == 0) bulk_wait_all();
  }
  if (!ok) atomicCAS(&g_error, 0, (int)DERR_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// One warp per row: the tiles' (maximum, sum) in a fixed order.
__global__ void __launch_bounds__(256) linear_ce_join_kernel(const float2* part, const float* zlab, const int* labels,
                                                             float* loss, float* lse, int T, int V, int n_tiles) {
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= T) return;
  const float2* p = part + (size_t)t * n_tiles;
  float m = -INFINITY;
  for (int i = lane; i < n_tiles; i += 32) m = fmaxf(m, p[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.f;
  for (int i = lane; i < n_tiles; i += 32) {
    const float2 v = p[i];
    s += v.x == m ? v.y : v.y * expf(v.x - m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
    const float l = m + logf(s);
    lse[t] = l;
    loss[t] = (unsigned)labels[t] < (unsigned)V ? l - zlab[t] : 0.f;
  }
}

// dx = the sum of the slabs, in slab order.
__global__ void __launch_bounds__(256) linear_ce_dx_kernel(const float* slabs, bf16* dx, int T, int H, int splits,
                                                           size_t slab) {
  const size_t n = (size_t)T * H / 8, step = (size_t)gridDim.x * 256;
  for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < n; i += step) {
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
    for (int s = 0; s < splits; ++s) {
      const float4* p = reinterpret_cast<const float4*>(slabs + s * slab + i * 8);
      const float4 x = p[0], y = p[1];
      u.x += x.x; u.y += x.y; u.z += x.z; u.w += x.w;
      w.x += y.x; w.y += y.y; w.z += y.z; w.w += y.w;
    }
    const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(u.x, u.y), __floats2bfloat162_rn(u.z, u.w),
                                 __floats2bfloat162_rn(w.x, w.y), __floats2bfloat162_rn(w.z, w.w)};
    reinterpret_cast<uint4*>(dx)[i] = *reinterpret_cast<const uint4*>(h);
  }
}

inline int cdiv(int a, int b) { return (a + b - 1) / b; }
inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// bf16 [rows, cols] with `ld` elements a row, boxes of 64 columns x box_rows
bool map2(CUtensorMap* m, const void* p, int rows, int cols, size_t ld, int box_rows) {
  const unsigned long long dims[2] = {(unsigned long long)cols, (unsigned long long)rows}, st[1] = {ld * 2};
  const unsigned box[2] = {64, (unsigned)box_rows};
  return encode_tmap(m, p, false, 2, dims, st, box);
}

// Columns of one piece's g: G_BYTES of workspace, so that a piece is read back
// from L2, but at least MIN_PIECE columns, which keep the contraction of dx and
// the tiles of dw long enough to fill the SMs.
constexpr size_t G_BYTES = 64u << 20;
constexpr int MIN_PIECE = 4096;

struct Plan2 {
  int piece, splits, slab_rows;
  size_t off_slab, bytes;
};

Plan2 backward_plan(int T, int V, int H) {
  Plan2 p;
  const int v_all = cdiv(V, TN) * TN;
  long long c = (long long)(G_BYTES / 2 / (T < 1 ? 1 : T)) / TN * TN;
  if (c < MIN_PIECE) c = MIN_PIECE;
  p.piece = c < v_all ? (int)c : v_all;
  // few tiles of dx: slices of the contraction, at least 512 deep, so that
  // dx alone has a tile for every SM
  const int tiles = cdiv(T < 1 ? 1 : T, TM) * cdiv(H, TN);
  int s = cdiv(SM_COUNT, tiles);
  if (s > p.piece / 512) s = p.piece / 512;
  if (s > 32) s = 32;
  p.splits = s < 1 ? 1 : s;
  p.slab_rows = cdiv(T, TM) * TM;
  p.off_slab = up256((size_t)T * p.piece * 2);
  p.bytes = p.off_slab + (size_t)p.splits * p.slab_rows * H * 4 + 256;
  return p;
}

int check_shape(int T, int V, int H) {
  if (T < 0 || T > (1 << 24) || V < 1 || V > (1 << 24) || H < 8 || H % 8 || H > (1 << 16))
    return op_fail(GOCR_EINVAL, "bad shape T=%d V=%d H=%d", T, V, H);
  return GOCR_OK;
}

template <int KIND> int launch(const Maps& m, const Args& a, cudaStream_t s) {
  if (!kernel_smem_at_least(reinterpret_cast<const void*>(&linear_ce_kernel<KIND>), SMEM))
    return op_fail(GOCR_ECUDA, "kernel configuration rejected");
  linear_ce_kernel<KIND><<<a.tiles < SM_COUNT ? a.tiles : SM_COUNT, THREADS, SMEM, s>>>(m, a);
  return op_launched("linear_ce");
}

int bad_map() { return op_fail(GOCR_ECUDA, "a TMA descriptor was rejected"); }

}  // namespace

namespace gocr {
cudaError_t take_linear_ce_error(int* out) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_error, sizeof(int));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_error, &zero, sizeof(int));
  return e;
}
}  // namespace gocr

extern "C" {

size_t gocr_op_linear_ce_workspace(int T, int V) {
  if (T < 0 || V < 1) return 0;
  return up256((size_t)T * cdiv(V, TN) * 8) + up256((size_t)T * 4) + 256;
}

int gocr_op_linear_ce(const void* x, const void* w, const int32_t* labels, float* loss, float* lse, int T, int V,
                      int H, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_shape(T, V, H)) return rc;
  if (!w || !workspace || (T && (!x || !labels || !loss || !lse))) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)workspace) & 15) return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (workspace_bytes < gocr_op_linear_ce_workspace(T, V)) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T) return GOCR_OK;
  Maps m{};
  Args a{};
  a.T = T; a.H = H; a.V = V;
  a.labels = labels;
  a.m_tiles = cdiv(T, TM); a.n_tiles = cdiv(V, TN);
  a.tiles = a.m_tiles * a.n_tiles;
  a.part = (float2*)workspace;
  a.zlab = (float*)((char*)workspace + up256((size_t)T * a.n_tiles * 8));
  if (!map2(&m.a0, x, T, H, H, TM) || !map2(&m.b0, w, V, H, H, TN)) return bad_map();
  if (int rc = launch<STATS>(m, a, s)) return rc;
  linear_ce_join_kernel<<<cdiv(T, 8), 256, 0, s>>>(a.part, a.zlab, labels, loss, lse, T, V, a.n_tiles);
  return op_launched("linear_ce join");
}

size_t gocr_op_linear_ce_backward_workspace(int T, int V, int H) {
  if (T < 0 || V < 1 || H < 1) return 0;
  return backward_plan(T, V, H).bytes;
}

int gocr_op_linear_ce_backward(const float* dloss, const void* x, const void* w, const int32_t* labels,
                               const float* lse, void* dx, void* dw, int T, int V, int H, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (int rc = check_shape(T, V, H)) return rc;
  if (!w || !dw || !workspace || (T && (!dloss || !x || !labels || !lse || !dx)))
    return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)dx | (uintptr_t)dw | (uintptr_t)workspace) & 15)
    return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  const Plan2 p = backward_plan(T, V, H);
  if (workspace_bytes < p.bytes) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T) {
    if (cudaMemsetAsync(dw, 0, (size_t)V * H * 2, s) != cudaSuccess) return op_fail(GOCR_ECUDA, "cudaMemsetAsync failed");
    return GOCR_OK;
  }
  float* slabs = (float*)((char*)workspace + p.off_slab);
  Maps z{}, pr{};
  if (!map2(&z.a0, x, T, H, H, TM) || !map2(&z.b0, w, V, H, H, TN) || !map2(&pr.b0, w, V, H, H, 64) ||
      !map2(&pr.b1, x, T, H, H, 64) || !map2(&pr.out1, dw, V, H, H, 32))
    return bad_map();
  {
    const unsigned long long dims[2] = {(unsigned long long)H, (unsigned long long)p.splits * p.slab_rows},
                             st[1] = {(unsigned long long)H * 4};
    const unsigned box[2] = {32, 32};
    if (!encode_tmap(&pr.out0, slabs, true, 2, dims, st, box)) return bad_map();
  }
  for (int v0 = 0; v0 < V; v0 += p.piece) {
    Args a{};
    a.T = T; a.H = H; a.V = V;
    a.labels = labels; a.lse = lse; a.dloss = dloss;
    a.v0 = v0; a.vc = V - v0 < p.piece ? V - v0 : p.piece;
    if (!map2(&z.out0, workspace, T, a.vc, p.piece, 32) || !map2(&pr.a0, workspace, T, a.vc, p.piece, TM) ||
        !map2(&pr.a1, workspace, T, a.vc, p.piece, 64))
      return bad_map();
    a.m_tiles = cdiv(T, TM); a.n_tiles = cdiv(a.vc, TN);
    a.tiles = a.m_tiles * a.n_tiles;
    if (int rc = launch<GRAD>(z, a, s)) return rc;
    a.n_tiles = cdiv(H, TN);
    a.m_tiles1 = cdiv(a.vc, TM);
    a.splits = p.splits;
    a.split_k = cdiv(cdiv(a.vc, TK), p.splits);
    a.slab_rows = p.slab_rows;
    a.add = v0 > 0;
    a.tiles0 = a.m_tiles * a.n_tiles * a.splits;
    a.tiles = a.tiles0 + a.m_tiles1 * a.n_tiles;
    if (int rc = launch<PROD>(pr, a, s)) return rc;
  }
  const size_t vecs = (size_t)T * H / 8;
  const unsigned blocks = (unsigned)(vecs / 256 + 1 < 8u * SM_COUNT ? vecs / 256 + 1 : 8u * SM_COUNT);
  linear_ce_dx_kernel<<<blocks, 256, 0, s>>>(slabs, (bf16*)dx, T, H, p.splits, (size_t)p.slab_rows * H);
  return op_launched("linear_ce dx");
}

}  // extern "C"
