// Softmax cross entropy of a linear head over a large vocabulary, without the
// logits ever being stored, and its gradient.
//
//   z_tv = x_t . w_v      lse_t = log sum_v exp z_tv      loss_t = lse_t - z_t,y(t)
//   g_tv = (exp(z_tv - lse_t) - [v = y(t)]) dloss_t        dx = g W      dw = g^T x
//   (g is kept divided by a unit that the rows' weights share: weight_unit)
//
// All of it is matrix products on tcgen05: 2 T V H operations forward, 6 T V H
// backward (z again, dx, dw).  One persistent kernel shape serves the three
// products: a pair of CTAs walks 256 x 256 output tiles (128 rows a CTA; each
// CTA stages its rows of A and half the columns of B, so a byte of shared
// memory feeds twice the operations of a single CTA's tile), a TMA warp keeps
// a ring of 64-deep stages full, one thread of the pair issues the MMAs into
// one of two tensor memory accumulators, and four warps a CTA (one row a
// thread) run the epilogue of the other:
//   STATS  (z) the row's maximum and sum of exponentials over the tile's
//          columns (256 or fewer) without the label's: 8 bytes per row and tile
//          leave the SM.
//          A second kernel joins them in tile order with the label's z, which
//          it computes in fp32, and takes the loss as log(1 + exp(lse of the
//          others - z of the label)): a confident row's small loss keeps its
//          precision, where lse - z would cancel;
//   GRAD   (z) g in bf16, stored to the piece of the vocabulary in the
//          workspace.  The label's exp(z - lse) - 1 is expm1(-loss) where the
//          forward call's loss is given: of a confident row the difference of
//          two rounded logits of tens has no right digit left (losses of
//          1e-6 to 1e-5: dx off by 0.9 of its norm);
//   PROD   dx += g W (fp32 slabs) and dw = g^T x (bf16) of the piece, x from a
//          copy that is zero in the rows without a target; both read
//          g as it lies: rows for dx (K-major), columns for dw (M-major), W and
//          x N-major, so nothing is transposed.
// The vocabulary goes by in pieces of 64 MB of g, but of no fewer than 4,096
// columns: of a small vocabulary all of g is there at once.  In PROD every
// pair gets the same number of K steps: its share of the dw tiles, which are
// not split, and a range of the dx tiles' steps, which may end inside a tile;
// the parts of a tile go to slabs of their own that a last kernel adds up in
// order.  g is rounded to bf16 (relative 2^-8) because the tensor cores take
// it so; every sum is in fp32.  Nothing is added by atomics across CTAs in an
// order that could change, so the same inputs give the same bits.
//
// What bounds it: with many rows the tensor pipe, and with seconds of it the
// card's power.  2,047 rows x 65,536 x 1,536 forward take 237 us (1.74 PFLOP/s,
// the pipe busy 93 % of STATS); 4,096 rows with the gradient 2,012 to 2,070 us (1.59
// to 1.64 PFLOP/s of the four products' operations, where cuBLAS sustains 1.73).  33
// rows forward take 40 us, 35 of them reading w's 201 MB (5.8 TB/s) and 4 the
// join.  193 rows x 8,191 x 512 with the gradient take 52 us, five launches of 7
// to 18 us and the host's calls.
#include "../../include/gocr.h"
#include "kernels.cuh"
#include "tc.cuh"

#include <cuda.h>

using namespace gocr;

namespace {

constexpr int TM = 256, TN = 256, TK = 64;  // of a pair
constexpr int RM = TM / 2, RN = TN / 2;     // rows of A and columns of B that one CTA stages
constexpr int A_BYTES = RM * TK * 2, B_BYTES = RN * TK * 2;
constexpr int RING = 6 * (A_BYTES + B_BYTES);
constexpr int MAX_STAGES = 16;
constexpr int PAIRS = SM_COUNT / 2;
constexpr int BOX = 64 * 128;            // one box of 64 rows x 64 columns
constexpr int STORE_BYTES = 32 * 128;    // one epilogue box: 32 rows x 128 bytes
constexpr int OFF_STORE = RING;
constexpr int OFF_BAR = OFF_STORE + 4 * 2 * STORE_BYTES;
constexpr int OFF_UNIT = OFF_BAR + 384;  // weight_unit's eight words, behind the barriers
constexpr int SMEM = OFF_BAR + 512 + 1024;
static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
static_assert((2 * MAX_STAGES + 5) * 8 + 4 <= OFF_UNIT - OFF_BAR, "room for the barriers");
constexpr int THREADS = 192;  // TMA warp, MMA warp, four epilogue warps
constexpr float LOG2E = 1.4426950408889634f;

enum Kind { STATS, GRAD, PROD };

static __device__ unsigned g_gave_up;  // threads whose wait gave up, ever

struct Maps {
  CUtensorMap a0, b0;   // STATS, GRAD: x, w.  PROD: g (rows), w (N-major)
  CUtensorMap a1, b1;   // PROD: g (columns), x of the rows with a target (N-major)
  CUtensorMap out0;     // GRAD: g.  PROD: the dx slabs
  CUtensorMap out1;     // PROD: dw
};

// How PROD's work is dealt to the pairs.  Pairs 0 .. c - 1 take one dw tile
// more than the others; the dx steps (tiles in order, `steps` each) are cut
// into ranges of q_hi steps for those pairs and q_lo for the others.
struct Deal {
  int c, q_hi, q_lo;
  int steps, tiles;        // dx: K steps of a tile, tiles
  __host__ __device__ int begin(int p) const {
    const int s = p < c ? p * q_hi : c * q_hi + (p - c) * q_lo;
    return s < steps * tiles ? s : steps * tiles;
  }
  __host__ __device__ int pair_of(int s) const { return s < c * q_hi ? s / q_hi : c + (s - c * q_hi) / q_lo; }
  // parts of dx tile t, and which of them pair p has
  __host__ __device__ int parts(int t) const { return pair_of((t + 1) * steps - 1) - pair_of(t * steps) + 1; }
  __host__ __device__ int part(int t, int p) const { return p - pair_of(t * steps); }
};

struct Args {
  int T, H, V;
  int v0, vc;           // GRAD, PROD: the piece of the vocabulary
  const int* labels;
  const float* lse;
  const float* loss;    // GRAD: the forward call's, or null
  const float* dloss;
  const uint4* x;       // GRAD of the first piece: x, and
  uint4* x_targets;     // where copy_targets puts it
  float* unit;          // GRAD of the first piece writes it (weight_unit), the later launches read it
  float2* part;         // STATS: [T][vocabulary tiles] (maximum, sum)
  int m_tiles, n_tiles; // STATS, GRAD; n_tiles also of PROD
  int tn;               // STATS, GRAD: columns of a tile
  int stages;           // of the ring
  int a_rows;           // rows of A that a CTA stages at most: 128, or fewer for few rows
  int tiles;            // STATS, GRAD: all; PROD: dw
  Deal deal, before;    // PROD: this piece's, the earlier pieces' (tiles = 0: this is the first)
  int slab_rows;
};

struct Tile {
  int prod;             // PROD: 0 dx, 1 dw
  int m0, n0, k0, ks;   // first row, column, K step; K steps
  int cols;             // columns of B: 256, or fewer
  int row_out, add;     // dx: first row in the slabs; add to them
};

// The pair's i-th tile; false past the last one.
template <int KIND> __device__ __forceinline__ bool tile_of(const Args& a, int pair, int i, Tile& t) {
  t.prod = 0; t.k0 = 0; t.row_out = 0; t.add = 0;
  if (KIND != PROD) {
    // rows fastest: the pairs of a wave share a few tiles of w
    const int x = pair + i * PAIRS;
    if (x >= a.tiles) return false;
    t.m0 = (x % a.m_tiles) * TM;
    t.n0 = (x / a.m_tiles) * a.tn;
    t.ks = (a.H + TK - 1) / TK;
    t.cols = a.tn;
    return true;
  }
  const Deal& d = a.deal;
  const int b = d.begin(pair), e = d.begin(pair + 1);
  const int first = b / d.steps;
  const int n_dx = e > b ? (e - 1) / d.steps - first + 1 : 0;
  if (i < n_dx) {
    const int x = first + i;
    const int lo = max(b, x * d.steps), hi = min(e, (x + 1) * d.steps);
    const int part = d.part(x, pair);
    t.m0 = (x / a.n_tiles) * TM;
    t.n0 = (x % a.n_tiles) * TN;
    t.k0 = lo - x * d.steps;
    t.ks = hi - lo;
    t.row_out = part * a.slab_rows + t.m0;
    t.add = a.before.tiles && part < a.before.parts(x);
  } else {
    const int x = pair + (i - n_dx) * PAIRS;
    if (x >= a.tiles) return false;
    t.prod = 1;
    t.m0 = (x / a.n_tiles) * TM;
    t.n0 = (x % a.n_tiles) * TN;
    t.ks = (a.T + TK - 1) / TK;
  }
  t.cols = a.H - t.n0 <= RN ? RN : TN;
  return true;
}

__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Byte offset of 16-byte chunk c of row r in a 32-row swizzled box.
__device__ __forceinline__ uint32_t box_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// The factor that g is divided by and its sums get back in fp32.  A stream's rows
// have one weight in a mean, and the label's g is nearly all of it: rounded to
// bf16 with the weight in it, that would be the same relative error of the whole
// stream, up to 2^-8, which does not average out of dx and dw.  With the streams of a
// joint loss there are two weights (powers of two aside).  So the unit is the one,
// up to a power of two in [1, 2), in which the smallest mantissa among the targets'
// weights is a / 128 with a whole number a, and of those a the one that brings the
// largest mantissa nearest to 8 bits, too: means over 2,000 to 4,000 and 600 to
// 2,000 rows keep a common error of 4e-5 on average instead of 1.6e-3.  One weight:
// a = 128 and no error.  Further weights between the two are rounded as they come.
// The 128 threads of the epilogue warps, while the first tile's products run; all
// get the answer.
__device__ __forceinline__ float weight_unit(const float* dloss, const int* labels, int T, int V, unsigned* tmp) {
  constexpr int PER = 8;
  const int me = threadIdx.x - 64, lane = threadIdx.x & 31;
  unsigned lo = 0x00800000u, hi = 0;  // mantissa bits
  for (int t0 = 0; t0 < T; t0 += 128 * PER) {
    float f[PER];
    int label[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int t = t0 + u * 128 + me;
      f[u] = t < T ? fabsf(dloss[t]) : 0.f;
      label[u] = t < T ? labels[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if ((unsigned)label[u] < (unsigned)V && f[u] >= 1.1754943508e-38f && f[u] <= 3.4028234664e38f) {
        lo = min(lo, __float_as_uint(f[u]) & 0x007fffffu);
        hi = max(hi, __float_as_uint(f[u]) & 0x007fffffu);
      }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    tmp[me >> 5] = lo;
    tmp[4 + (me >> 5)] = hi;
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");
  for (int w = 0; w < 4; ++w) {
    lo = min(lo, tmp[w]);
    hi = max(hi, tmp[4 + w]);
  }
  if (lo > hi) return 1.f;  // no target with a weight
  const float m = __uint_as_float(lo | 0x3f800000u);
  if (lo == hi) return m;
  const float ratio = __uint_as_float(hi | 0x3f800000u) / m;  // 1 .. 2
  unsigned least = 0xffffffffu;
  int a = 0;
  for (int i = 0; i < 4; ++i) {
    const int k = 128 + lane * 4 + i;
    const float y = k * ratio, r = y < 256.f ? rintf(y) : 2.f * rintf(0.5f * y);
    const unsigned e = __float_as_uint(fabsf(r - y) / y);
    if (e < least) { least = e; a = k; }
  }
  const unsigned e = __reduce_min_sync(0xffffffffu, least);
  a = (int)__reduce_min_sync(0xffffffffu, least == e ? (unsigned)a : 256u);
  const float u = m * 128.f / a;
  return u < 1.f ? 2.f * u : u;
}

// x with zeros in the rows without a target, for dw = g^T x: their g is zero, but
// nobody need have written their x, and zero times NaN is NaN.  The MMA warps of
// the odd CTAs, which have nothing else to do, while the first piece's g is made;
// w of n warps, COPY vectors a lane in flight.
__device__ __forceinline__ void copy_targets(const Args& a, int w, int n) {
  constexpr int COPY = 16;
  const int lane = threadIdx.x & 31, vecs = a.H / 8, parts = (vecs + 31) / 32;
  const long long total = (long long)a.T * parts;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (long long i0 = (long long)w * COPY; i0 < total; i0 += (long long)n * COPY) {
    const int row0 = (int)(i0 / parts), part0 = (int)(i0 % parts);
    uint4 v[COPY];
    int label[COPY];
    int row = row0, part = part0;
#pragma unroll
    for (int u = 0; u < COPY; ++u) {
      const int c = part * 32 + lane;
      const bool in = row < a.T && c < vecs;
      v[u] = in ? a.x[(size_t)row * vecs + c] : zero;
      label[u] = in ? a.labels[row] : -1;
      if (++part == parts) { part = 0; ++row; }
    }
    row = row0;
    part = part0;
#pragma unroll
    for (int u = 0; u < COPY; ++u) {
      const int c = part * 32 + lane;
      if (row < a.T && c < vecs) a.x_targets[(size_t)row * vecs + c] = (unsigned)label[u] < (unsigned)a.V ? v[u] : zero;
      if (++part == parts) { part = 0; ++row; }
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");  // PROD reads it by TMA
}

template <int KIND>
__global__ void __launch_bounds__(THREADS, 1) linear_ce_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + OFF_BAR);  // the even CTA's: both CTAs' loads of a stage
  uint64_t* empty = full + MAX_STAGES;  // each CTA's: the stage has been read
  uint64_t* acc_full = empty + MAX_STAGES;  // [2], each CTA's
  uint64_t* acc_free = acc_full + 2;    // [2], the even CTA's: the epilogue warps of both
  uint64_t* drained = acc_free + 2;     // each CTA's: the products, at the MMA warp's end
  uint32_t* holder = reinterpret_cast<uint32_t*>(drained + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
  const int a_bytes = a.a_rows * 128;
  const int stage_bytes = a_bytes + (KIND != PROD ? a.tn / 2 * 128 : B_BYTES);

  if (tid == 0) {
    tc::grid_dep_launch();
    for (int s = 0; s < a.stages; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(acc_full + b, 1);
      tc::mbar_init(acc_free + b, 8);
    }
    tc::mbar_init(drained, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) tc::tmem_alloc_pair(holder, 512);
  tc::fence_before_sync();
  __syncthreads();
  __syncwarp();
  tc::cluster_arrive_release();  // barriers of both CTAs are initialised
  tc::cluster_wait_acquire();
  tc::fence_after_sync();
  // all 512 columns, which start at 0: a constant keeps the MMAs' operands in uniform registers
  constexpr uint32_t tmem = 0;
  tc::grid_dep_wait();
  bool ok = true;
  Tile t;

  if (warp == 0) {
    int st = 0, ph = 0, loads = 0;
    for (int i = 0; ok && tile_of<KIND>(a, pair, i, t); ++i) {
      // few rows: the odd CTA has none; what its part of A then holds only
      // reaches accumulator rows that nobody reads
      const bool with_a = KIND == PROD || a.a_rows == RM || rank == 0;
      const uint32_t bytes = t.cols * 128 + (KIND == PROD || a.a_rows == RM ? 2 * A_BYTES : a_bytes);
      const int m = t.m0 + rank * RM, n = t.n0 + rank * (t.cols / 2);
      for (int k = 0; k < t.ks; ++k) {
        if (!(ok = tc::mbar_wait_warp(empty + st, ph ^ 1))) break;
        uint8_t* sa = sm + st * stage_bytes;
        uint8_t* sb = sa + a_bytes;
        const int kk = (t.k0 + k) * TK;
        const uint32_t bar = tc::mapa(tc::smem_u32(full + st), 0);
        if (tc::elect_one()) {
          if (rank == 0) tc::mbar_expect_tx(full + st, bytes);
          if (KIND != PROD) {
            if (with_a) tc::tma_load_2d_pair(sa, &maps.a0, kk, m, bar);
            tc::tma_load_2d_pair(sb, &maps.b0, kk, a.v0 + n, bar);
          } else {
            if (t.prod == 0) {
              tc::tma_load_2d_pair(sa, &maps.a0, kk, m, bar);
            } else {
              tc::tma_load_2d_pair(sa, &maps.a1, m, kk, bar);
              tc::tma_load_2d_pair(sa + BOX, &maps.a1, m + 64, kk, bar);
            }
            const CUtensorMap* mb = t.prod ? &maps.b1 : &maps.b0;
            const int row = t.prod ? kk : a.v0 + kk;
            tc::tma_load_2d_pair(sb, mb, n, row, bar);
            if (t.cols > RN) tc::tma_load_2d_pair(sb + BOX, mb, n + 64, row, bar);
          }
        }
        __syncwarp();
        ++loads;
        if (++st == a.stages) { st = 0; ph ^= 1; }
      }
    }
    // the even CTA's barriers count both CTAs' loads, and the odd one does not leave before it
    if (rank == 0) ok = tc::ring_landed(full, a.stages, loads) && ok;
  } else if (warp == 1 && rank == 1) {
    if (KIND == GRAD && a.v0 == 0) copy_targets(a, pair, gridDim.x / 2);
  } else if (warp == 1) {
    int st = 0, ph = 0, acc = 0, aph = 0;
    for (int i = 0; ok && tile_of<KIND>(a, pair, i, t); ++i) {
      if (!(ok = tc::mbar_wait_warp(acc_free + acc, aph ^ 1))) break;
      tc::fence_after_sync();
      const uint32_t d = tmem + acc * TN;
      uint32_t idesc = tc::idesc_bf16(TM, t.cols);
      if (KIND == PROD) idesc |= tc::IDESC_B_MN | (t.prod ? tc::IDESC_A_MN : 0u);
      for (int k = 0; k < t.ks; ++k) {
        if (!(ok = tc::mbar_wait_warp(full + st, ph))) break;
        tc::fence_after_sync();
        const uint32_t sa = tc::smem_u32(sm + st * stage_bytes), sb = sa + a_bytes;
        if (tc::elect_one()) {
          // a step of 16 along K: 32 bytes of a K-major tile, 16 rows of an M- or N-major one
          const bool a_mn = KIND == PROD && t.prod;
          const uint64_t ad = a_mn ? tc::sdesc_sw128_mn(sa, BOX) : tc::sdesc_sw128(sa);
          const uint64_t bd = KIND == PROD ? tc::sdesc_sw128_mn(sb, BOX) : tc::sdesc_sw128(sb);
          const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (KIND == PROD ? 2048 : 32) >> 4;
#pragma unroll
          for (int j = 0; j < TK / 16; ++j) tc::mma_bf16_pair(d, ad + j * a_step, bd + j * b_step, idesc, k > 0 || j > 0 ? 1u : 0u);
          tc::mma_commit_pair(empty + st);
          if (k + 1 == t.ks) tc::mma_commit_pair(acc_full + acc);
        }
        __syncwarp();
        if (++st == a.stages) { st = 0; ph ^= 1; }
      }
      acc ^= 1;
      if (acc == 0) aph ^= 1;
    }
    ok = tc::mma_drain_pair(drained) && ok;
  } else {
    const int q = warp & 3;  // the tensor memory lanes this warp may read: 32 q ..
    uint8_t* box = sm + OFF_STORE + q * 2 * STORE_BYTES;
    int acc = 0, aph = 0, buf = 0;
    float unit = 1.f;
    if (KIND == GRAD && a.v0 == 0) {
      unit = weight_unit(a.dloss, a.labels, a.T, a.V, reinterpret_cast<unsigned*>(sm + OFF_UNIT));
      if (blockIdx.x == 0 && tid == 64) *a.unit = unit;
    } else if (KIND != STATS) {
      unit = *a.unit;
    }
    for (int i = 0; tile_of<KIND>(a, pair, i, t); ++i) {
      const int row0 = t.m0 + rank * RM + q * 32;  // the warp's first row
      const int row = row0 + lane;
      // GRAD: the row's weight without the unit, its lse, and its label's g;
      // before the wait, so that the loads cost nothing
      int label = -1;
      float f = 0.f, lse = 0.f, own = 0.f;
      if (KIND == GRAD && row < a.T) {
        const float d = a.dloss[row], e = a.lse[row], l = a.loss ? a.loss[row] : 0.f;
        label = a.labels[row];
        if ((unsigned)label < (unsigned)a.V) {
          f = d / unit;
          lse = e;
          own = f * expm1f(-l);
        } else {
          label = -1;
        }
      }
      const uint32_t mask = label >= 0 ? 0xffffffffu : 0u;  // whatever z holds in a row without a target
      const float ref = lse * LOG2E;
      if (!(ok = tc::mbar_wait_warp(acc_full + acc, aph))) break;
      tc::fence_after_sync();
      const uint32_t src = tmem + acc * TN + ((uint32_t)(q * 32) << 16);
      const uint32_t freed = tc::mapa(tc::smem_u32(acc_free + acc), 0);
      if (KIND == STATS) {
        const bool in = row < a.T;
        const int label = in ? a.labels[row] : -1;
        float m = -INFINITY, s = 0.f;
        for (int c = 0; c < a.tn; c += 32) {
          const int col = t.n0 + c;
          if (col >= a.V) break;
          float v[32];
          tc::tmem_ld32(src + c, v);
          if (col + 32 > a.V) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col + j >= a.V) v[j] = -INFINITY;
          }
          const unsigned at = (unsigned)label - (unsigned)col;
          if (__any_sync(0xffffffffu, at < 32u)) {  // the label's column is the join kernel's
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = at == (unsigned)j ? -INFINITY : v[j];
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
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(freed);
        if (in) a.part[(size_t)row * a.n_tiles + t.n0 / a.tn] = make_float2(m, s);
      } else if (KIND == GRAD) {
        const int col0 = a.v0 + t.n0;
        for (int c = 0; c < a.tn; c += 64) {
          if (t.n0 + c >= a.vc) break;
          if (lane == 0) bulk_wait_read1();
          __syncwarp();
          uint8_t* bx = box + buf * STORE_BYTES;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            tc::tmem_ld32(src + c + h * 32, v);
            // the epilogue is nearly as long as the products: with exp2f's care for
            // subnormal results, and a select per element, a launch took 65 us, not 57
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = f * tc::ex2(fmaf(v[j], LOG2E, -ref));
            const unsigned at = (unsigned)(label - (col0 + c + h * 32));
            if (__any_sync(0xffffffffu, at < 32u)) {
              float g = own;
              if (!a.loss) {  // the difference, but a share is not above one
#pragma unroll
                for (int j = 0; j < 32; ++j) g = at == (unsigned)j ? v[j] - f : g;
                if ((__float_as_int(g) ^ __float_as_int(f)) >= 0 && g == g) g = 0.f;
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = at == (unsigned)j ? g : v[j];
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(v[g * 8 + 2 * e], v[g * 8 + 2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t*>(&p) & mask;
              }
              *reinterpret_cast<uint4*>(bx + box_at(lane, h * 4 + g)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < a.T) tc::tma_store_2d(&maps.out0, bx, t.n0 + c, row0);
            tc::bulk_commit();
          }
          buf ^= 1;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(freed);
      } else {
        const int step = t.prod ? 64 : 32;  // columns of one box
        for (int c = 0; c < TN && t.n0 + c < a.H; c += step) {
          if (lane == 0) bulk_wait_read1();
          __syncwarp();
          uint8_t* bx = box + buf * STORE_BYTES;
          if (t.prod == 0) {
            float v[32];
            tc::tmem_ld32(src + c, v);
#pragma unroll
            for (int g = 0; g < 8; ++g)
              *reinterpret_cast<float4*>(bx + box_at(lane, g)) =
                  make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
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
                  const __nv_bfloat162 p = __floats2bfloat162_rn(v[g * 8 + 2 * e] * unit, v[g * 8 + 2 * e + 1] * unit);
                  w[e] = *reinterpret_cast<const uint32_t*>(&p);
                }
                *reinterpret_cast<uint4*>(bx + box_at(lane, h * 4 + g)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int out = t.row_out + rank * RM + q * 32;
            if (t.prod) {
              if (a.v0 + row0 < a.V) tc::tma_store_2d(&maps.out1, bx, t.n0 + c, a.v0 + row0);
            } else if (t.add) {
              tc::tma_add_2d(&maps.out0, bx, t.n0 + c, out);
            } else {
              tc::tma_store_2d(&maps.out0, bx, t.n0 + c, out);
            }
            tc::bulk_commit();
          }
          buf ^= 1;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster(freed);
      }
      acc ^= 1;
      if (acc == 0) aph ^= 1;
    }
    if (lane == 0) bulk_wait_all();
  }
  if (!ok) atomicAdd(&g_gave_up, 1u);
  tc::fence_before_sync();
  __syncthreads();
  __syncwarp();
  tc::cluster_arrive_release();  // the other CTA still reads this one's shared memory and barriers
  tc::cluster_wait_acquire();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 512);
  }
}

// Sum or maximum over the 128 threads of a CTA, in a fixed order.
template <bool MAX> __device__ __forceinline__ float cta_reduce(float v, float* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  return MAX ? fmaxf(fmaxf(tmp[0], tmp[1]), fmaxf(tmp[2], tmp[3])) : (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
}

// One CTA per row: the tiles' (maximum, sum) of the columns that are not the
// label, in a fixed order, and the label's z = x . w in fp32.  Latency: 4.5 us
// for 33 rows, 6 for 2,047.
__global__ void __launch_bounds__(128) linear_ce_join_kernel(const float2* part, const bf16* x, const bf16* w,
                                                             const int* labels, float* loss, float* lse, int V, int H,
                                                             int n_tiles) {
  __shared__ float tmp[3][4];
  const int t = blockIdx.x, tid = threadIdx.x;
  tc::grid_dep_wait();
  const int label = labels[t];
  const bool has = (unsigned)label < (unsigned)V;
  const float2* p = part + (size_t)t * n_tiles;
  float m = -INFINITY;
  for (int i = tid; i < n_tiles; i += 128) m = fmaxf(m, p[i].x);
  float z = 0.f;
  if (has) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + (size_t)t * H);
    const uint4* wr = reinterpret_cast<const uint4*>(w + (size_t)label * H);
    for (int i = tid; i < H / 8; i += 128) {
      const uint4 u = xr[i], v = wr[i];
      const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z = fmaf(__uint_as_float(us[e] << 16), __uint_as_float(vs[e] << 16), z);
        z = fmaf(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(vs[e] & 0xffff0000u), z);
      }
    }
  }
  m = cta_reduce<true>(m, tmp[0]);
  float s = 0.f;
  for (int i = tid; i < n_tiles; i += 128) {
    const float2 v = p[i];
    s += v.x == m ? v.y : v.y * expf(v.x - m);
  }
  s = cta_reduce<false>(s, tmp[1]);
  z = cta_reduce<false>(z, tmp[2]);
  if (tid == 0) {
    const float others = m + logf(s);  // -infinity when the label is the only column
    float l = 0.f, all = others;
    if (has) {
      const float d = others - z;      // loss = log(1 + exp(d))
      l = (d > 0.f ? d : 0.f) + log1pf(expf(-fabsf(d)));
      if (d != d) l = d;               // a NaN (or infinite) logit
      all = d > 0.f ? others + log1pf(expf(-d)) : z + l;
    }
    lse[t] = all;
    loss[t] = l;
  }
}

// dx = the sum of the tile's parts, in slab order: memory-bound, 13 us for 4,096
// rows x 1,536.
__global__ void __launch_bounds__(256) linear_ce_dx_kernel(const float* slabs, bf16* dx, int T, int H, int n_tiles,
                                                           size_t slab, Deal last, Deal before, const float* unit_at) {
  tc::grid_dep_wait();
  const float unit = *unit_at;
  const size_t n = (size_t)T * H / 8, step = (size_t)gridDim.x * 256;
  for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < n; i += step) {
    const int row = (int)(i * 8 / H), col = (int)(i * 8 % H);
    const int tile = row / TM * n_tiles + col / TN;
    int parts = last.parts(tile);
    if (before.tiles) parts = max(parts, before.parts(tile));
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
    for (int s = 0; s < parts; ++s) {
      const float4* p = reinterpret_cast<const float4*>(slabs + s * slab + i * 8);
      const float4 x = p[0], y = p[1];
      u.x += x.x; u.y += x.y; u.z += x.z; u.w += x.w;
      w.x += y.x; w.y += y.y; w.z += y.z; w.w += y.w;
    }
    const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(u.x * unit, u.y * unit), __floats2bfloat162_rn(u.z * unit, u.w * unit),
                                 __floats2bfloat162_rn(w.x * unit, w.y * unit), __floats2bfloat162_rn(w.z * unit, w.w * unit)};
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

// Columns of one piece's g: G_BYTES of workspace, but at least MIN_PIECE
// columns, which keep the contraction of dx and the tiles of dw long enough to
// fill the SMs.  At 64 MB g is still in L2 when it is read; 32, 48, 128, 256 and
// 512 MB were slower (4,096 rows x 65,536 x 1,536).
constexpr size_t G_BYTES = 64u << 20;
constexpr int MIN_PIECE = 4096;
// A dw tile's epilogue in K steps, for the balance between the pairs.
constexpr int DW_EXTRA = 4;
constexpr int MAX_PARTS = 32;

struct BackwardPlan {
  int piece, slabs, slab_rows;
  Deal full, last;         // of the pieces before the last (tiles = 0: none), of the last
  size_t off_slab, off_x, bytes;
};

Deal deal_of(int T, int vc, int H) {
  Deal d;
  const int nt = cdiv(H, TN);
  d.steps = cdiv(vc, TK);
  d.tiles = cdiv(T, TM) * nt;
  const long long dx = (long long)d.steps * d.tiles;
  const int dw = cdiv(vc, TM) * nt, cost = cdiv(T, TK) + DW_EXTRA;
  const int lo = dw / PAIRS;
  d.c = dw % PAIRS;
  const long long each = (dx + (long long)dw * cost + PAIRS - 1) / PAIRS;
  // no more than MAX_PARTS - 1 ranges to a tile, so that its parts fit the slabs
  const int least = cdiv(d.steps, MAX_PARTS - 2);
  long long q_hi = each - (lo + 1LL) * cost, q_lo = each - (long long)lo * cost;
  if (q_lo < least) q_lo = least;
  if (q_hi < least) q_hi = 0;
  const long long rest = dx - d.c * q_hi;  // what the others take, whatever the first took
  if (q_lo * (PAIRS - d.c) < rest) q_lo = (rest + PAIRS - d.c - 1) / (PAIRS - d.c);
  d.q_hi = (int)q_hi;
  d.q_lo = (int)q_lo;
  return d;
}

// Ranges of at least q steps cut a tile into at most this many parts.
int most_parts(const Deal& d) {
  const int q = d.c && d.q_hi && d.q_hi < d.q_lo ? d.q_hi : d.q_lo;
  return cdiv(d.steps - 1, q) + 1;
}

BackwardPlan backward_plan(int T, int V, int H) {
  BackwardPlan p;
  const int v_all = cdiv(V, TN) * TN;
  long long c = (long long)(G_BYTES / 2 / (T < 1 ? 1 : T)) / TN * TN;
  if (c < MIN_PIECE) c = MIN_PIECE;
  p.piece = c < v_all ? (int)c : v_all;
  const int n = cdiv(V, p.piece), rows = T < 1 ? 1 : T;
  p.last = deal_of(rows, V - (n - 1) * p.piece, H);
  p.full = deal_of(rows, p.piece, H);
  if (n == 1) p.full.tiles = 0;
  p.slabs = most_parts(p.last);
  if (n > 1 && most_parts(p.full) > p.slabs) p.slabs = most_parts(p.full);
  p.slab_rows = cdiv(rows, TM) * TM;
  p.off_slab = up256((size_t)T * p.piece * 2);
  p.off_x = p.off_slab + up256((size_t)p.slabs * p.slab_rows * H * 4);
  p.bytes = p.off_x + up256((size_t)T * H * 2) + 256;  // the unit comes last
  return p;
}

int check_shape(int T, int V, int H) {
  if (T < 0 || T > (1 << 22) || V < 1 || V > (1 << 22) || H < 8 || H % 8 || H > (1 << 15))
    return op_fail(GOCR_EINVAL, "bad shape T=%d V=%d H=%d", T, V, H);
  return GOCR_OK;
}

// Columns of a tile of the z products, a multiple of `step`: as many as 256
// would take rounds of the pairs, but no more than fill them (33 rows x 65,536 x
// 1,536: 256 tiles of 256 columns are four rounds of 76 pairs, the last a third
// full; with 224 all four are full).  At least 128: an MMA of 128 columns takes
// nearly the time of one of 256.
int z_columns(int T, int vc, int step) {
  const int m = cdiv(T < 1 ? 1 : T, TM);
  const long long rounds = ((long long)m * cdiv(vc, TN) + PAIRS - 1) / PAIRS;
  const int n = (int)(rounds * PAIRS / m);  // tiles a row of tiles may have
  const int c = cdiv(cdiv(vc, n), step) * step;
  return c < RN ? RN : c;
}
constexpr int STATS_STEP = 32, GRAD_STEP = 64;  // columns that an epilogue step takes

// Few rows: only those that there are are staged, so that the ring holds more
// of w, whose reading bounds the call.
void set_ring(Args& a, bool z) {
  a.a_rows = z && a.T < RM ? cdiv(a.T, 8) * 8 : RM;
  const int stage = a.a_rows * 128 + (z ? a.tn / 2 * 128 : B_BYTES);
  const int n = RING / stage;
  a.stages = n < MAX_STAGES ? n : MAX_STAGES;
}

template <int KIND> int launch(const Maps& m, const Args& a, int pairs, cudaStream_t s) {
  if (!kernel_smem_at_least(reinterpret_cast<const void*>(&linear_ce_kernel<KIND>), SMEM))
    return op_fail(GOCR_ECUDA, "kernel configuration rejected");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (pairs < PAIRS ? pairs : PAIRS));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, linear_ce_kernel<KIND>, m, a);
  return op_launched("linear_ce");
}

int bad_map() { return op_fail(GOCR_ECUDA, "a TMA descriptor was rejected"); }

}  // namespace

namespace gocr {
cudaError_t linear_ce_gave_up(unsigned* out, cudaStream_t s) {
  return cudaMemcpyFromSymbolAsync(out, g_gave_up, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
}
}  // namespace gocr

extern "C" {

size_t gocr_op_linear_ce_workspace(int T, int V) {
  if (T < 0 || V < 1) return 0;
  // a bound that grows with T (T x tiles need not): tiles have RN columns at
  // least, and there are at most PAIRS / (row tiles) more of them than of TN
  const size_t narrow = (size_t)T * cdiv(V, RN), wide = (size_t)T * cdiv(V, TN) + TM * PAIRS;
  return up256((narrow < wide ? narrow : wide) * 8) + 256;
}

int gocr_op_linear_ce(const void* x, const void* w, const int32_t* labels, float* loss, float* lse, int T, int V,
                      int H, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_shape(T, V, H)) return rc;
  if (!w || !workspace || (T && (!x || !labels || !loss || !lse))) return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)workspace) & 15) return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (((uintptr_t)labels | (uintptr_t)loss | (uintptr_t)lse) & 3)
    return op_fail(GOCR_EINVAL, "labels, loss or lse not 4-byte aligned");
  if (workspace_bytes < gocr_op_linear_ce_workspace(T, V)) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T) return GOCR_OK;
  Maps m{};
  Args a{};
  a.T = T; a.H = H; a.V = V;
  a.labels = labels;
  a.tn = z_columns(T, V, STATS_STEP);
  set_ring(a, true);
  a.m_tiles = cdiv(T, TM); a.n_tiles = cdiv(V, a.tn);
  a.tiles = a.m_tiles * a.n_tiles;
  a.part = (float2*)workspace;
  if (!map2(&m.a0, x, T, H, H, a.a_rows) || !map2(&m.b0, w, V, H, H, a.tn / 2)) return bad_map();
  if (int rc = launch<STATS>(m, a, a.tiles, s)) return rc;
  launch_k(linear_ce_join_kernel, dim3(T), dim3(128), 0, s, true, (const float2*)a.part, (const bf16*)x, (const bf16*)w, labels,
           loss, lse, V, H, a.n_tiles);
  return op_launched("linear_ce join");
}

size_t gocr_op_linear_ce_backward_workspace(int T, int V, int H) {
  if (T < 0 || V < 1 || H < 1) return 0;
  return backward_plan(T, V, H).bytes;
}

int gocr_op_linear_ce_backward_with_loss(const float* dloss, const void* x, const void* w, const int32_t* labels,
                                         const float* loss, const float* lse, void* dx, void* dw, int T, int V, int H,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_shape(T, V, H)) return rc;
  if (!w || !dw || !workspace || (T && (!dloss || !x || !labels || !lse || !dx)))
    return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)x | (uintptr_t)w | (uintptr_t)dx | (uintptr_t)dw | (uintptr_t)workspace) & 15)
    return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (((uintptr_t)dloss | (uintptr_t)labels | (uintptr_t)loss | (uintptr_t)lse) & 3)
    return op_fail(GOCR_EINVAL, "dloss, labels, loss or lse not 4-byte aligned");
  const BackwardPlan p = backward_plan(T, V, H);
  if (workspace_bytes < p.bytes) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T) {
    if (cudaMemsetAsync(dw, 0, (size_t)V * H * 2, s) != cudaSuccess) return op_fail(GOCR_ECUDA, "cudaMemsetAsync failed");
    return GOCR_OK;
  }
  float* slabs = (float*)((char*)workspace + p.off_slab);
  void* x_targets = (char*)workspace + p.off_x;
  float* unit = (float*)((char*)workspace + p.bytes - 256);
  Maps z{}, pr{};
  Args common{};
  common.T = T; common.H = H; common.V = V;
  common.labels = labels; common.lse = lse; common.loss = loss; common.dloss = dloss; common.unit = unit;
  common.x = (const uint4*)x; common.x_targets = (uint4*)x_targets;
  common.tn = z_columns(T, p.piece, GRAD_STEP);
  set_ring(common, true);
  if (!map2(&z.a0, x, T, H, H, common.a_rows) || !map2(&z.b0, w, V, H, H, common.tn / 2) || !map2(&pr.b0, w, V, H, H, 64) ||
      !map2(&pr.b1, x_targets, T, H, H, 64) || !map2(&pr.out1, dw, V, H, H, 32))
    return bad_map();
  {
    const unsigned long long dims[2] = {(unsigned long long)H, (unsigned long long)p.slabs * p.slab_rows},
                             st[1] = {(unsigned long long)H * 4};
    const unsigned box[2] = {32, 32};
    if (!encode_tmap(&pr.out0, slabs, true, 2, dims, st, box)) return bad_map();
  }
  for (int v0 = 0; v0 < V; v0 += p.piece) {
    Args a = common;
    a.v0 = v0; a.vc = V - v0 < p.piece ? V - v0 : p.piece;
    if (!map2(&z.out0, workspace, T, a.vc, p.piece, 32) || !map2(&pr.a0, workspace, T, a.vc, p.piece, RM) ||
        !map2(&pr.a1, workspace, T, a.vc, p.piece, 64))
      return bad_map();
    a.m_tiles = cdiv(T, TM); a.n_tiles = cdiv(a.vc, a.tn);
    a.tiles = a.m_tiles * a.n_tiles;
    if (int rc = launch<GRAD>(z, a, a.tiles, s)) return rc;
    set_ring(a, false);
    a.n_tiles = cdiv(H, TN);
    a.tiles = cdiv(a.vc, TM) * a.n_tiles;
    a.deal = v0 + p.piece < V ? p.full : p.last;
    a.before = p.full;
    if (v0 == 0) a.before.tiles = 0;
    a.slab_rows = p.slab_rows;
    if (int rc = launch<PROD>(pr, a, PAIRS, s)) return rc;
  }
  const size_t vecs = (size_t)T * H / 8;
  const unsigned blocks = (unsigned)(vecs / 256 + 1 < 8u * SM_COUNT ? vecs / 256 + 1 : 8u * SM_COUNT);
  launch_k(linear_ce_dx_kernel, dim3(blocks), dim3(256), 0, s, true, (const float*)slabs, (bf16*)dx, T, H, cdiv(H, TN),
           (size_t)p.slab_rows * H, p.last, p.full, (const float*)common.unit);
  return op_launched("linear_ce dx");
}

int gocr_op_linear_ce_backward(const float* dloss, const void* x, const void* w, const int32_t* labels,
                               const float* lse, void* dx, void* dw, int T, int V, int H, void* workspace,
                               size_t workspace_bytes, void* stream) {
  return gocr_op_linear_ce_backward_with_loss(dloss, x, w, labels, nullptr, lse, dx, dw, T, V, H, workspace,
                                              workspace_bytes, stream);
}

}  // extern "C"
