// Token embedding and its gradient, for training and scoring.
//
//   y_t  = s * row(id_t)      row: E[id], the [M] row for id = -1, else zero
//   dE_v = s * sum of dy_t over id_t = v;  d[M] likewise
//
// Memory bounds the forward call, which reads the distinct rows and writes T rows
// (10,240 rows of 1,536 bf16: 9.3 us, 5.5 TB/s), and the backward call up to a few
// ten thousand positions: it reads T rows of dy and writes the dense V x H
// gradient, which is most of its bytes.  Of more positions the sort takes over, which
// has 8 SMs whatever T is (1,048,576 of 65,536 x 512: 0.6 of 0.93 ms; each CTA that
// writes zeros then reads all ids, too).  The sum of a row runs over the token's positions in increasing
// order, in pieces that follow from ids alone, in fp32 and without atomics, so
// the gradient's bits are the same on every call.
//
// Backward, three launches (times: 10,240 positions, a third [M], 65,536 x 1,536
// bf16):
//   sort  a cluster of SORT_CTAS CTAs sorts the positions by token: a stable
//         radix sort, digits of at most 9 bits, counts exchanged over
//         distributed shared memory.  17 us of latencies on 8 SMs, so the next
//         launch starts beside it;
//   sum   the launch's first CTAs write the zeros of the rows that no position
//         names, by bulk copies, and wait for nothing.  The others wait for the
//         sort; then a CTA takes PIECE sorted positions.  A run of equal tokens
//         is summed and written by the piece in which it begins, unless it is
//         longer than LONG: each piece then leaves an fp32 partial row of it.
//         37 us for 232 MB, 6.2 TB/s;
//   join  one CTA per (long run, 128 columns) adds up the partial rows, eight
//         warps a share each: 12 us, one dependent read after the other.
// With the zeros in the sort's launch the sum came after both: 72 us the two
// directions together, 67 now.  Half the zeros beside the join: no gain.
// A frequent token ([M] above all) is one long run, so no CTA ever walks more
// than PIECE + LONG rows of dy.
#include "../../include/gocr.h"
#include "kernels.cuh"
#include "tc.cuh"

#include <algorithm>
#include <cooperative_groups.h>

using namespace gocr;
namespace cg = cooperative_groups;

namespace {

constexpr int SORT_CTAS = 8;
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_DIGITS = 512;
// Sorted positions of a sum CTA.  Few positions want many CTAs; of many, pieces
// of 128 leave an eighth of the partial rows, which one CTA per 128 columns of a
// run joins (262,144 positions, 30 % [M], of 65,536 x 1,536: 519 -> 373 us).
constexpr int PIECE_FEW = 16, PIECE_MANY = 128, MANY = 1 << 15;
constexpr int LONG = 16;
inline int piece_of(int T) { return T > MANY ? PIECE_MANY : PIECE_FEW; }
constexpr int FILL_BYTES = 16384;  // one bulk copy of zeros
constexpr int FILL_ROWS = 32768;   // most table rows of a CTA that writes zeros

// 16 bytes of a row in fp32
template <typename T> struct Vec;
template <> struct Vec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(bf16* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(256) embed_rows_kernel(const T* __restrict__ embed, const T* __restrict__ mask,
                                                         const int* __restrict__ ids, T* __restrict__ y, int rows,
                                                         int H, int V, float scale) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x & 31;
  const long long nw = (long long)gridDim.x * 8;
  for (long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); t < rows; t += nw) {
    const int id = ids[t];
    const T* src = (unsigned)id < (unsigned)V ? embed + (size_t)id * H : (id == TOK_MASK ? mask : nullptr);
    T* dst = y + (size_t)t * H;
#pragma unroll 4
    for (int c = lane * N; c < H; c += 32 * N) {
      float v[N];
      if (src) {
        Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + c), v);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= scale;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
      }
      Vec<T>::store(dst + c, v);
    }
  }
}

// Sort key of a position: its token, V for [M], V + 1 for a row without a
// gradient (an id outside the table, or [M] when no [M] gradient is wanted).
__device__ __forceinline__ int key_of(int id, int V, bool mask) {
  return (unsigned)id < (unsigned)V ? id : (id == TOK_MASK && mask ? V : V + 1);
}

struct SortArgs {
  const int* ids;
  int* key[2];   // [T] sorted keys; the last pass's output is key[1]
  int* pos[2];   // [T] positions in that order
  int T, V, mask, passes, digit_bits;
  int* n_long;   // zeroed: the long runs that the sum kernel lists
};

__global__ void __launch_bounds__(SORT_THREADS) embed_sort_kernel(SortArgs a) {
  __shared__ int cnt[SORT_WARPS][MAX_DIGITS];  // keys of (warp, digit), then the warp's next place
  __shared__ int cta_cnt[MAX_DIGITS];
  __shared__ int scan[MAX_DIGITS];
  if (threadIdx.x == 0) tc::grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_long = 0;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = 1 << a.digit_bits;
  // warp w of CTA c owns the positions [(16 c + w) share, + share): the order
  // of (CTA, warp, position) is the order of the positions
  const int share = ((a.T + SORT_CTAS * SORT_WARPS - 1) / (SORT_CTAS * SORT_WARPS) + 31) & ~31;
  const long long lo_ = (long long)(rank * SORT_WARPS + warp) * share;
  const int lo = lo_ < a.T ? (int)lo_ : a.T;
  const int hi = lo_ + share < a.T ? (int)(lo_ + share) : a.T;
  const unsigned below = (1u << lane) - 1u;
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.digit_bits;
    // the output of pass p is buffer (passes - p) & 1, so that the last one is 1
    const int* kin = a.key[(a.passes - p + 1) & 1];
    const int* pin = a.pos[(a.passes - p + 1) & 1];
    int* kout = a.key[(a.passes - p) & 1];
    int* pout = a.pos[(a.passes - p) & 1];
    for (int d = lane; d < D; d += 32) cnt[warp][d] = 0;
    __syncwarp();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < hi;
      const int k = in ? (p == 0 ? key_of(a.ids[i], a.V, a.mask) : __ldcg(kin + i)) : 0;
      const int dg = in ? (k >> shift) & (D - 1) : D;
      const unsigned same = __match_any_sync(0xffffffffu, dg);
      if (in && (same & below) == 0) cnt[warp][dg] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    for (int d = tid; d < D; d += SORT_THREADS) {  // before warp w in this CTA
      int s = 0;
      for (int w = 0; w < SORT_WARPS; ++w) {
        const int c = cnt[w][d];
        cnt[w][d] = s;
        s += c;
      }
      cta_cnt[d] = s;
    }
    cluster.sync();
    int before = 0, total = 0;  // digit tid: keys of the CTAs before this one, of all CTAs
    if (tid < D)
      for (int c = 0; c < SORT_CTAS; ++c) {
        const int v = *cluster.map_shared_rank(&cta_cnt[tid], c);
        if (c < rank) before += v;
        total += v;
      }
    scan[tid] = tid < D ? total : 0;  // SORT_THREADS = MAX_DIGITS
    __syncthreads();
    for (int o = 1; o < MAX_DIGITS; o <<= 1) {
      const int v = tid >= o ? scan[tid - o] : 0;
      __syncthreads();
      scan[tid] += v;
      __syncthreads();
    }
    if (tid < D) {
      const int base = scan[tid] - total + before;
      for (int w = 0; w < SORT_WARPS; ++w) cnt[w][tid] += base;
    }
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < hi;
      const int k = in ? (p == 0 ? key_of(a.ids[i], a.V, a.mask) : __ldcg(kin + i)) : 0;
      const int at = in ? (p == 0 ? i : __ldcg(pin + i)) : 0;
      const int dg = in ? (k >> shift) & (D - 1) : D;
      const unsigned same = __match_any_sync(0xffffffffu, dg);
      const int mine = __popc(same & below);
      int place = 0;
      if (in) place = cnt[warp][dg] + mine;
      __syncwarp();
      if (in && mine == 0) cnt[warp][dg] += __popc(same);
      __syncwarp();
      if (in) {
        kout[place] = k;
        pout[place] = at;
      }
    }
    __threadfence();
    cluster.sync();  // the pass's output, and every read of cta_cnt, is complete
  }
}

struct SumArgs {
  const void* dy;
  const int* ids;
  const int* key;
  const int* pos;
  void* d_embed;
  void* d_mask;
  float* part;   // [pieces][2][H] of long runs: the one that comes into the piece, the one that begins in it
  int* n_long;
  int* run;      // [n_long] the pieces in which a long run begins
  int T, H, V;
  float scale;
  int fill, fill_rows;  // the sum launch's CTAs that write zeros, table rows of each
  int pieces;
};

template <typename T>
__device__ __forceinline__ T* grad_row(const SumArgs& a, int key) {
  return key < a.V ? reinterpret_cast<T*>(a.d_embed) + (size_t)key * a.H : reinterpret_cast<T*>(a.d_mask);
}

// n bytes of zeros (a multiple of 16) at d.
__device__ __forceinline__ void fill_zero(uint8_t* d, size_t n, uint32_t zeros) {
  for (size_t i = 0; i < n; i += FILL_BYTES) {
    const uint32_t b = (uint32_t)(n - i < FILL_BYTES ? n - i : FILL_BYTES);
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(d + i), "r"(zeros), "r"(b) : "memory");
  }
}

// Zeros for the rows of the table's share blockIdx.x that no position names, and with
// share 0 for the [M] row if none names it.  Nothing here waits for the sort: the CTA
// notes the named rows of its share from the positions' tokens themselves.
template <typename T>
__device__ __forceinline__ void fill_unnamed(const SumArgs& a) {
  __shared__ __align__(16) uint4 zeros[FILL_BYTES / 16];
  __shared__ unsigned named[FILL_ROWS / 32];
  __shared__ int mask_named;
  const int row0 = blockIdx.x * a.fill_rows, rows = min(a.fill_rows, a.V - row0);
  for (int i = threadIdx.x; i < FILL_BYTES / 16; i += blockDim.x) zeros[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += blockDim.x) named[i] = 0;
  if (threadIdx.x == 0) mask_named = 0;
  tc::fence_proxy_async_smem();
  __syncthreads();
  auto note = [&](int id) {
    const unsigned r = (unsigned)id - (unsigned)row0;
    if (r < (unsigned)rows) atomicOr(&named[r >> 5], 1u << (r & 31));
    if (id == TOK_MASK) mask_named = 1;
  };
  // four tokens a load, between the first 16-byte boundary and the last
  const int head = min(a.T, (int)((16 - ((uintptr_t)a.ids & 15)) & 15) / 4), quads = (a.T - head) / 4;
  const int4* q = reinterpret_cast<const int4*>(a.ids + head);
#pragma unroll 8
  for (int i = threadIdx.x; i < quads; i += blockDim.x) {
    const int4 v = q[i];
    note(v.x);
    note(v.y);
    note(v.z);
    note(v.w);
  }
  for (int i = threadIdx.x; i < a.T - 4 * quads; i += blockDim.x) note(a.ids[i < head ? i : 4 * quads + i]);
  __syncthreads();
  const size_t row_bytes = (size_t)a.H * sizeof(T);
  const uint32_t z = tc::smem_u32(zeros);
  uint8_t* d = reinterpret_cast<uint8_t*>(a.d_embed) + (size_t)row0 * row_bytes;
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += blockDim.x) {
    unsigned left = ~named[i];
    if (rows - 32 * i < 32) left &= (1u << (rows - 32 * i)) - 1u;
    while (left) {  // a run of unnamed rows
      const int at = __ffs(left) - 1, len = __ffs(~(left >> at)) ? __ffs(~(left >> at)) - 1 : 32;
      fill_zero(d + (size_t)(32 * i + at) * row_bytes, len * row_bytes, z);
      left &= len < 32 ? ~(((1u << len) - 1u) << at) : 0u;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.d_mask && !mask_named)
    fill_zero(reinterpret_cast<uint8_t*>(a.d_mask), row_bytes, z);
  tc::bulk_commit();
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Rows of dy fetched at a time by a thread.
constexpr int BATCH = 8;

template <typename T, int PIECE>
__global__ void __launch_bounds__(256) embed_sum_kernel(SumArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int WIN = LONG + PIECE + LONG;  // positions b - LONG .. b + PIECE + LONG - 1
  __shared__ int keys[WIN + 1];             // and the next one
  __shared__ int poss[PIECE + LONG];        // of positions b ..
  __shared__ int edge[4];  // the runs of the piece's first and last position: first position, and past the last
  if (threadIdx.x == 0) tc::grid_dep_launch();
  if (blockIdx.x < a.fill) return fill_unnamed<T>(a);
  const int piece = (blockIdx.x - a.fill) % a.pieces, part = (blockIdx.x - a.fill) / a.pieces;
  if (threadIdx.x < 4) edge[threadIdx.x] = threadIdx.x & 1 ? PIECE + LONG + 1 : -LONG;
  tc::grid_dep_wait();
  const int b = piece * PIECE, n = min(PIECE, a.T - b);
  for (int i = threadIdx.x; i < WIN + 1; i += blockDim.x) {
    const int at = b - LONG + i;
    keys[i] = at >= 0 && at < a.T ? a.key[at] : -1;
    if (i < PIECE + LONG) poss[i] = b + i < a.T ? a.pos[b + i] : 0;
  }
  __syncthreads();
  const int* k0 = keys + LONG;  // k0[i]: position b + i
  for (int i0 = (threadIdx.x & ~31) - LONG + 1; i0 <= PIECE + LONG; i0 += blockDim.x) {
    const int i = i0 + (threadIdx.x & 31);
    const bool start = i <= PIECE + LONG && k0[i] != k0[i - 1];
    const int far = 1 << 20;
    const int s0 = __reduce_max_sync(0xffffffffu, start && i <= 0 ? i : -far);
    const int e0 = __reduce_min_sync(0xffffffffu, start && i > 0 ? i : far);
    const int s1 = __reduce_max_sync(0xffffffffu, start && i < n ? i : -far);
    const int e1 = __reduce_min_sync(0xffffffffu, start && i >= n ? i : far);
    if ((threadIdx.x & 31) == 0) {
      atomicMax(&edge[0], s0);
      atomicMin(&edge[1], e0);
      atomicMax(&edge[2], s1);
      atomicMin(&edge[3], e1);
    }
  }
  __syncthreads();
  // A run is long when it has more than LONG positions; the window shows that
  // much of it, so every piece that it touches comes to the same verdict.
  const bool comes = k0[-1] == k0[0], in = comes && edge[1] - edge[0] > LONG;
  const int first = comes ? min(edge[1], n) : 0;  // the first run that begins in the piece
  int end = n;  // the last run that begins here is summed to its end, unless it is long
  if (first < n && edge[3] > n) {
    if (edge[3] - edge[2] <= LONG) end = edge[3];
    else if (part == 0 && threadIdx.x == 0 && k0[n - 1] <= a.V) a.run[atomicAdd(a.n_long, 1)] = piece;
  }
  const int c = (part * blockDim.x + threadIdx.x) * N;
  if (c >= a.H) return;
  const T* dy = reinterpret_cast<const T*>(a.dy) + c;
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  for (int i0 = in ? 0 : first; i0 < end; i0 += BATCH) {
    uint4 v[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      if (i0 + u < end && k0[i0 + u] <= a.V) v[u] = *reinterpret_cast<const uint4*>(dy + (size_t)poss[i0 + u] * a.H);
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int i = i0 + u;
      if (i >= end) break;
      const int k = k0[i];
      if (k > a.V) return;  // rows without a gradient come last
      float x[N];
      Vec<T>::unpack(v[u], x);
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] += x[j];
      const bool goes_on = k0[i + 1] == k;
      if (goes_on && i + 1 < end) continue;
      const bool comes_in = in && i < n && k == k0[-1];
      if (comes_in || goes_on) {
        float* p = a.part + ((size_t)piece * 2 + (comes_in ? 0 : 1)) * a.H + c;
#pragma unroll
        for (int j = 0; j < N; j += 4) *reinterpret_cast<float4*>(p + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] *= a.scale;
        Vec<T>::store(grad_row<T>(a, k) + c, acc);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = 0.f;
    }
  }
}

// The long runs: warp w adds the w-th eighth of a run's partial rows, four
// columns a lane, and warp 0 the eight sums.
template <typename T, int PIECE>
__global__ void __launch_bounds__(256) embed_join_kernel(SumArgs a) {
  __shared__ float4 sums[8][32];
  __shared__ int s_last;
  tc::grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pieces = a.pieces, n = *a.n_long;
  const int c = blockIdx.y * 128 + lane * 4;
  for (int r = blockIdx.x; r < n; r += gridDim.x) {
    const int first = a.run[r];
    const int k = a.key[(first + 1) * PIECE - 1];
    if (threadIdx.x == 0) s_last = pieces - 1;
    __syncthreads();
    // the run ends in the first piece whose next position is not its own
    for (int j0 = first + 1; j0 < pieces; j0 += 1024) {
      int at = pieces;
#pragma unroll
      for (int u = 3; u >= 0; --u) {
        const int j = j0 + u * 256 + threadIdx.x;
        if (j < pieces - 1 && a.key[(j + 1) * PIECE] != k) at = j;
      }
      if (at < pieces) atomicMin(&s_last, at);
      if (__syncthreads_or(at < pieces)) break;
    }
    const int m = s_last - first, share = (m + 8) / 8;  // m + 1 partial rows
    const int lo = warp * share, hi = min(lo + share, m + 1);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.H) {
#pragma unroll 8
      for (int j = lo; j < hi; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(a.part + ((size_t)(first + j) * 2 + (j == 0 ? 1 : 0)) * a.H + c);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.H) {
      for (int w = 1; w < 8; ++w) {
        const float4 v = sums[w][lane];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      T* d = grad_row<T>(a, k) + c;
      d[0] = from_f32<T>(s.x * a.scale);
      d[1] = from_f32<T>(s.y * a.scale);
      d[2] = from_f32<T>(s.z * a.scale);
      d[3] = from_f32<T>(s.w * a.scale);
    }
    __syncthreads();
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t sort_bytes(int T) { return 4 * up256((size_t)T * 4); }

int check_shape(int dtype, int T, int H, int V) {
  if (dtype != GOCR_DTYPE_F32 && dtype != GOCR_DTYPE_BF16) return op_fail(GOCR_EINVAL, "bad dtype");
  if (T < 0 || T > (1 << 28) || H < 8 || H % 8 || H > (1 << 20) || V < 1 || V > (1 << 28))
    return op_fail(GOCR_EINVAL, "bad shape T=%d H=%d V=%d", T, H, V);
  return GOCR_OK;
}

template <typename T, int PIECE>
int embed_backward(const SortArgs& so, SumArgs su, cudaStream_t s) {
  if (su.T) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(SORT_CTAS);
    cfg.blockDim = dim3(SORT_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = SORT_CTAS;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, embed_sort_kernel, so);
    if (int rc = op_launched("embedding sort")) return rc;
  }
  // two CTAs per SM write the zeros, fewer for a small table, more for one
  // whose shares would be longer than FILL_ROWS
  const size_t bytes = (size_t)su.V * su.H * sizeof(T);
  const int want = (int)std::min<size_t>((bytes + FILL_BYTES - 1) / FILL_BYTES, 2 * SM_COUNT);
  su.fill_rows = std::min(FILL_ROWS, (su.V + want - 1) / want);
  su.fill = (su.V + su.fill_rows - 1) / su.fill_rows;
  su.pieces = (su.T + PIECE - 1) / PIECE;
  const int vecs = su.H / Vec<T>::N;
  const int th = std::max(128, std::min(256, (vecs + 31) / 32 * 32));
  const unsigned parts = (unsigned)((vecs + th - 1) / th);
  launch_k(embed_sum_kernel<T, PIECE>, dim3(su.fill + su.pieces * parts), dim3(th), 0, s, su.T > 0, su);
  if (int rc = op_launched("embedding sum")) return rc;
  if (su.T > LONG) {
    launch_k(embed_join_kernel<T, PIECE>, dim3(std::min(su.T / LONG, 64), (su.H + 127) / 128), dim3(256), 0, s, true, su);
    return op_launched("embedding join");
  }
  return GOCR_OK;
}

}  // namespace

extern "C" {

int gocr_op_embed(int dtype, const void* embed, const void* mask_embed, const int32_t* ids, void* y, int T, int H,
                  int V, float scale, void* stream) {
  if (int rc = check_shape(dtype, T, H, V)) return rc;
  if (!embed || (T && (!ids || !y))) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)embed | (uintptr_t)mask_embed | (uintptr_t)y) & 15)
    return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if ((uintptr_t)ids & 3) return op_fail(GOCR_EINVAL, "ids not 4-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T) return GOCR_OK;
  const int grid = T <= 8 * 8 * SM_COUNT ? (T + 7) / 8 : 8 * SM_COUNT;
  if (dtype == GOCR_DTYPE_BF16)
    embed_rows_kernel<bf16><<<grid, 256, 0, s>>>((const bf16*)embed, (const bf16*)mask_embed, ids, (bf16*)y, T, H, V, scale);
  else
    embed_rows_kernel<float><<<grid, 256, 0, s>>>((const float*)embed, (const float*)mask_embed, ids, (float*)y, T, H, V, scale);
  return op_launched("embedding");
}

size_t gocr_op_embed_backward_workspace(int T, int H) {
  if (T < 0 || H < 1) return 0;
  size_t pieces = ((size_t)T + piece_of(T) - 1) / piece_of(T);
  if (T > MANY) pieces = std::max<size_t>(pieces, MANY / PIECE_FEW);  // enough for fewer positions, too
  return sort_bytes(T) + pieces * 2 * H * 4 + up256(pieces * 4 + 4) + 256;
}

int gocr_op_embed_backward(int dtype, const void* dy, const int32_t* ids, void* d_embed, void* d_mask, int T, int H,
                           int V, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_shape(dtype, T, H, V)) return rc;
  if (!d_embed || !workspace || (T && (!dy || !ids))) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)dy | (uintptr_t)d_embed | (uintptr_t)d_mask | (uintptr_t)workspace) & 15)
    return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if ((uintptr_t)ids & 3) return op_fail(GOCR_EINVAL, "ids not 4-byte aligned");
  if (workspace_bytes < gocr_op_embed_backward_workspace(T, H)) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  SortArgs so{};
  char* ws = (char*)workspace;
  const size_t arr = up256((size_t)T * 4);
  so.ids = ids;
  for (int i = 0; i < 2; ++i) {
    so.key[i] = (int*)(ws + i * arr);
    so.pos[i] = (int*)(ws + (2 + i) * arr);
  }
  so.T = T; so.V = V; so.mask = d_mask != nullptr;
  int bits = 1;
  while ((1ll << bits) < (long long)V + 2) ++bits;
  so.passes = (bits + 8) / 9;
  so.digit_bits = (bits + so.passes - 1) / so.passes;
  float* part = (float*)(ws + 4 * arr);
  int* n_long = (int*)(part + (size_t)((T + piece_of(T) - 1) / piece_of(T)) * 2 * H);
  so.n_long = n_long;
  SumArgs su{dy, ids, so.key[1], so.pos[1], d_embed, d_mask, part, n_long, n_long + 1, T, H, V, scale, 0, 0, 0};
  if (piece_of(T) == PIECE_MANY)
    return dtype == GOCR_DTYPE_BF16 ? embed_backward<bf16, PIECE_MANY>(so, su, s) : embed_backward<float, PIECE_MANY>(so, su, s);
  return dtype == GOCR_DTYPE_BF16 ? embed_backward<bf16, PIECE_FEW>(so, su, s) : embed_backward<float, PIECE_FEW>(so, su, s);
}

}  // extern "C"
