// Causal attention over packed sequences with grouped heads, backward.
//
//   P_ij = exp(c q_i . k_j - lse_i)      delta_i = do_i . o_i
//   dP_ij = do_i . v_j                   dS_ij = P_ij (dP_ij - delta_i)
//   dv_j = sum_i P_ij do_i               dk_j = c sum_i dS_ij q_i      dq_i = c sum_j dS_ij k_j
//
// dk and dv also sum over the q heads of the group.  Two launches: delta with a
// table of the blocks, then one of two kinds of CTA: for dk and dv one per (128 keys, k/v head), which
// walks the q heads and the query blocks that see the keys; for dq one per (128
// query rows, q head), which walks the keys.  S and dP are computed by both,
// seven products of 128 x 128 x D a block pair instead of five; in return every
// sum has one owner: no atomics, no fp32 dq in memory, and the same bits on
// every call.  The longest CTAs come first and the short dq ones fill up.
//
// All products run on tcgen05 with fp32 accumulators in tensor memory.  A dk/dv
// CTA works on the transposed blocks (a lane is a key): P^T and dS^T (bf16,
// relative 2^-8, as the tensor cores take them) go back to tensor memory over
// the scores they came from and are the A operands of dV += P^T dO and dK +=
// dS^T Q; dO and Q serve as they lie, K-major for S^T and dP^T and N-major
// here.  A dq CTA has lanes of query rows and dQ += dS K.  Two groups of four
// warps do the elementwise work, 64 columns of a block to a thread; it overlaps
// the products: P^T with dK and dP^T, dS^T with dV and the next S^T.
//
// What bounds it: 12 heads of 128, one sequence of 8,192 takes 505 us: 1.43
// PFLOP/s of the seven products that run, 1.02 of the five that the formulas
// need, the tensor pipe busy 61 % of the time.  A block pair's chain (S, P, dS,
// sums) is longer than its products, and there is room for one pair at a time
// (dV, dK, S^T and dP^T fill all 512 columns of tensor memory).  15 sequences of
// 95 to 1,203 take 109 us (heads of 64: 441 us for the long one), 46 at the long one's rate; the rest goes to blocks on
// the diagonal, ragged ones, and CTAs that start and finish.  Measured slower:
// groups that run ahead of one another on products of 64 columns (541 to 667 us
// for the long one), one MMA warp (541).
//
// delta from o takes o's rounding to bf16 into every dS of the row.  That
// matters where a row sees few keys (o is then large), so for the first 32 rows
// of a sequence delta is sum_j P_ij dP_ij instead, in fp32.
#include "../../include/gocr.h"
#include "attn_packed.cuh"

using namespace gocr;
using namespace gocr::packed;

namespace {

// Eight elementwise warps, a TMA warp, and two MMA warps: a warp's waits cost
// 100 cycles and more behind its own queue of MMAs, which then run dry unless
// the other warp has some.
constexpr int THREADS = 352;
constexpr int EW = 4;         // warps of an elementwise group
// Seven tiles of D = 128 (dynamic shared memory starts at a multiple of 1,024,
// checked in the kernel: there is no room for slack), -lse and -delta of two
// query blocks, barriers.
constexpr int ROW_OFF = 7 * 128 * 128 * 2;
constexpr int BAR_OFF = ROW_OFF + 2 * 2 * 128 * 4;
constexpr int SMEM = BAR_OFF + 256;
static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");

// A role that gives up has waited for two seconds since the last copy or product that
// it issued, so none is under way when its CTA leaves; the last of a role that does
// not give up are what the others wait for.  Asking the barriers once more at the
// roles' ends, as the forward kernel does, slowed the loops here by 1.4 % (one
// sequence of 8,192: 505 -> 512 us).
static __device__ unsigned g_gave_up;  // threads whose wait gave up, ever
static __device__ unsigned g_unaligned;  // CTAs whose shared memory did not begin at a multiple of 1,024

constexpr int FLAT = 4;  // 16-byte pieces of o and of do in flight a thread
constexpr int FEW = 32;  // rows at the start of a sequence with delta from P and dP

struct BwdArgs {
  const int* cu;
  const float* lse;
  const float* delta; const float* first;  // first: of the first FEW rows of a sequence
  bf16* dq; bf16* dk; bf16* dv;
  const int4* table;  // the blocks of 128 rows
  int n_seq, T, Hq, Hkv;
  float scale;
};

struct DeltaArgs {
  const bf16* q; const bf16* k; const bf16* v; const bf16* o; const bf16* d_o;
  long long ldq, ldk, ldv;
  const int* cu;
  const float* lse;
  float* delta; float* first;
  int4* table; int blocks;  // the table of blocks and its entries
  int n_seq, T, Hq, Hkv;
  float scale;
};

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y, float s) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), s);
    s = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), s);
  }
  return s;
}

// The table of blocks, by the first CTA, and delta, by two kinds of CTA.  n_seq x
// Hq take the first 32 rows of a sequence for a q head, with its rows of q, k, v
// and do in shared memory and lanes of keys; the others take o and do as they lie
// (of every row, which costs less than finding out which they are), D / 8 lanes to
// a (row, head).  8,192 rows x 12 heads: 13 us, 101 MB half of which the forward call
// left in L2; with 15 sequences 15 us, the first rows' chains beside it.
template <int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const DeltaArgs a) {
  constexpr int L = D / 8, LD = L + 1;  // 16-byte pieces of a row; row pitch in shared memory
  __shared__ uint4 t[4][FEW][LD];       // q, k, do, v
  if (threadIdx.x == 0) tc::grid_dep_launch();
  if (blockIdx.x == 0) return block_table(a.cu, a.n_seq, a.T, 128, a.table, a.blocks);
  const int b = blockIdx.x - 1;
  const int firsts = a.n_seq * a.Hq;
  if (b >= firsts) {
    const long long i0 = (long long)(b - firsts) * (256 * FLAT) + threadIdx.x;  // of a piece of o
    const long long n = (long long)a.T * a.Hq * L;
    const uint4 z = make_uint4(0, 0, 0, 0);
    uint4 x[FLAT], y[FLAT];
#pragma unroll
    for (int u = 0; u < FLAT; ++u) {
      const long long i = i0 + u * 256;
      x[u] = i < n ? reinterpret_cast<const uint4*>(a.o)[i] : z;
      y[u] = i < n ? reinterpret_cast<const uint4*>(a.d_o)[i] : z;
    }
#pragma unroll
    for (int u = 0; u < FLAT; ++u) {
      const long long i = i0 + u * 256;
      float s = dot8(x[u], y[u], 0.f);
#pragma unroll
      for (int m = L / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
      const int r = (int)(i / L);
      if (i < n && i % L == 0) a.delta[(size_t)(r % a.Hq) * a.T + r / a.Hq] = s;
    }
    return;
  }
  const int head = b % a.Hq, seq = b / a.Hq;
  const int lo = min(max(a.cu[seq], 0), a.T), n = min(FEW, min(a.cu[seq + 1], a.T) - lo);
  if (n <= 0) return;
  const size_t row0 = lo;
  float* out = a.first + (size_t)head * a.T + row0;
  const int kvh = head / (a.Hq / a.Hkv);
  for (int i = threadIdx.x; i < FEW * L; i += 256) {
    const int r = i / L, l = i % L;
    const size_t row = row0 + r;
    const uint4 z = make_uint4(0, 0, 0, 0);
    t[0][r][l] = r < n ? reinterpret_cast<const uint4*>(a.q + row * a.ldq + head * D)[l] : z;
    t[1][r][l] = r < n ? reinterpret_cast<const uint4*>(a.k + row * a.ldk + kvh * D)[l] : z;
    t[2][r][l] = r < n ? reinterpret_cast<const uint4*>(a.d_o)[(row * a.Hq + head) * L + l] : z;
    t[3][r][l] = r < n ? reinterpret_cast<const uint4*>(a.v + row * a.ldv + kvh * D)[l] : z;
  }
  __syncthreads();
  const int key = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < n; r += 8) {
    float s = 0.f, dp = 0.f;
#pragma unroll 4
    for (int l = 0; l < L; ++l) {
      s = dot8(t[0][r][l], t[1][key][l], s);
      dp = dot8(t[2][r][l], t[3][key][l], dp);
    }
    float x = key <= r ? tc::ex2((s * a.scale - a.lse[(size_t)head * a.T + row0 + r]) * LOG2E) * dp : 0.f;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (key == 0) out[r] = x;
  }
}

// The 32 columns of an accumulator row, times f, as bf16 to dst (16-byte aligned).
__device__ __forceinline__ void store32(uint32_t taddr, float f, bf16* dst, bool in) {
  uint32_t w[32];
  tc::tmem_ld32_nowait(taddr, w);
  tc::tmem_wait_ld();
  if (in)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = pack2(__uint_as_float(w[g * 8 + 2 * e]) * f, __uint_as_float(w[g * 8 + 2 * e + 1]) * f);
      *reinterpret_cast<uint4*>(dst + g * 8) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// ---------------------------------------------------------------- dk, dv

template <int D> struct DkvGeo {
  static constexpr int TILE = TILE_BYTES<D>;
  static constexpr int OFF_K = 0, OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;    // [3]: S^T(it + 1) runs while dK(it - 1) still needs its Q
  static constexpr int OFF_DO = 5 * TILE;   // [2]
};

template <int D>
__device__ void dkv_cta(uint8_t* sm, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                        const CUtensorMap& mdo, const BwdArgs& a, const Block& blk, int kvh) {
  using G = DkvGeo<D>;
  float* rows = reinterpret_cast<float*>(sm + ROW_OFF);  // [2 stages][-lse log2 e, -delta][128]
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + BAR_OFF);
  uint64_t* q_full = kv_full + 1;    // [3]
  uint64_t* q_empty = q_full + 3;    // [3]
  uint64_t* do_full = q_empty + 3;   // [2]
  uint64_t* do_empty = do_full + 2;  // [2]
  uint64_t* row_full = do_empty + 2; // [2] lse and delta of the stage; ragged tiles zeroed
  uint64_t* row_free = row_full + 2; // [2] their readers are done
  uint64_t* s_full = row_free + 2;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_full = dp_full + 1;    // [2 groups]
  uint64_t* ds_full = p_full + 2;    // [2]
  uint64_t* done = ds_full + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(done + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int group = a.Hq / a.Hkv;
  const int kb = blk.at / 128, nqb = (blk.len + 127) / 128;
  const int per = nqb - kb;         // query blocks of a head that see these keys
  const int n = group * per;
  const int tail = blk.len - (nqb - 1) * 128;  // rows of the last query block within the sequence
  // group 1 has the second 64 rows of a query block, if the sequence has them
  auto both = [&](int it) { return it % per + 1 < per || tail > 64; };

  if (tid == 0) {
    tc::mbar_init(kv_full, 1);
    for (int s = 0; s < 3; ++s) {
      tc::mbar_init(q_full + s, 1);
      tc::mbar_init(q_empty + s, 2);   // both MMA warps read Q and dO
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(do_full + s, 1);
      tc::mbar_init(do_empty + s, 2);
      tc::mbar_init(row_full + s, 1);
      tc::mbar_init(row_free + s, 2 * EW);
    }
    tc::mbar_init(s_full, 1);
    tc::mbar_init(dp_full, 1);
    for (int g = 0; g < 2; ++g) {
      tc::mbar_init(p_full + g, EW);
      tc::mbar_init(ds_full + g, EW);
    }
    tc::mbar_init(done, 2);
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (warp == 9) tc::tmem_alloc(holder, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // all 512 columns, which start at 0: a constant keeps the MMAs' operands in uniform registers
  constexpr uint32_t tmem = 0;
  constexpr uint32_t DP = 128, DV = 256, DK = 256 + D;  // S^T at 0
  bool ok = true;

  if (warp == 8) {
    if (lane == 0) {
      tc::mbar_expect_tx(kv_full, 2 * G::TILE);
      load_tile<D>(sm + G::OFF_K, &mk, kvh, blk.row0 + blk.at, kv_full);
      load_tile<D>(sm + G::OFF_V, &mv, kvh, blk.row0 + blk.at, kv_full);
    }
    for (int it = 0; it < n; ++it) {
      const int st = it & 1, ph = (it >> 1) & 1;
      const int head = kvh * group + it / per, at = (kb + it % per) * 128;
      const bool ragged = at + 128 > blk.len;
      const int qs = it % 3, qp = it / 3 & 1;
      uint8_t* q = sm + G::OFF_Q + qs * G::TILE;
      uint8_t* d_o = sm + G::OFF_DO + st * G::TILE;
      if (!(ok = tc::mbar_wait_warp(q_empty + qs, qp ^ 1))) break;
      if (tc::elect_one()) {
        tc::mbar_expect_tx(q_full + qs, G::TILE);
        load_tile<D>(q, &mq, head, blk.row0 + at, q_full + qs);
      }
      __syncwarp();
      if (!(ok = tc::mbar_wait_warp(do_empty + st, ph ^ 1))) break;
      if (tc::elect_one()) {
        tc::mbar_expect_tx(do_full + st, G::TILE);
        load_tile<D>(d_o, &mdo, head, blk.row0 + at, do_full + st);
      }
      __syncwarp();
      // the stage's rows were last read for the block two back
      if (it > 1 && !(ok = tc::mbar_wait_warp(row_free + st, ph ^ 1))) break;
      float* lse = rows + st * 256;
      for (int i = lane; i < 128; i += 32) {
        const bool in = at + i < blk.len;
        const size_t src = (size_t)head * a.T + blk.row0 + at + i;
        lse[i] = in ? a.lse[src] * -LOG2E : 0.f;
        lse[128 + i] = in ? -(at + i < FEW ? a.first : a.delta)[src] : 0.f;
      }
      if (ragged) {
        ok = tc::mbar_wait_warp(q_full + qs, qp) && tc::mbar_wait_warp(do_full + st, ph);
        if (!ok) break;
        zero_rows<D>(q, tail);
        zero_rows<D>(d_o, tail);
        tc::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(row_full + st);
    }
  } else if (warp >= 9) {
    // warp 9: S^T and dV, warp 10: dP^T and dK
    const bool ds = warp == 10;
    const uint32_t kv = tc::smem_u32(sm + (ds ? G::OFF_V : G::OFF_K));    // A of the blocks
    const uint32_t bx = tc::smem_u32(sm + (ds ? G::OFF_DO : G::OFF_Q));   // their B
    const uint32_t by = tc::smem_u32(sm + (ds ? G::OFF_Q : G::OFF_DO));   // B of the sums
    uint64_t* bx_full = ds ? do_full : q_full;
    uint64_t* by_full = ds ? q_full : do_full;
    uint64_t* bx_empty = ds ? do_empty : q_empty;
    uint64_t* by_empty = ds ? q_empty : do_empty;
    uint64_t* out_full = ds ? dp_full : s_full;
    uint64_t* in_full = ds ? ds_full : p_full;
    const int bx_n = ds ? 2 : 3, by_n = ds ? 3 : 2;  // stages
    const uint32_t blocks = ds ? DP : 0, sum = ds ? DK : DV;
    auto wait = [&](uint64_t* bar, int ph) {
      const bool w = tc::mbar_wait_warp(bar, ph);
      tc::fence_after_sync();
      return w;
    };
    auto product = [&](int st, bool two) {
      if (two) mma_rows<D, 128>(tmem + blocks, kv, bx + st * G::TILE, 0);
      else mma_rows<D, 64>(tmem + blocks, kv, bx + st * G::TILE, 0);
      tc::mma_commit(out_full);
    };
    ok = wait(kv_full, 0) && wait(bx_full, 0);
    if (ok && tc::elect_one()) {
      product(0, both(0));
      tc::mma_commit(bx_empty);
    }
    __syncwarp();
    int x = 0, xp = 0, y = 0, yp = 0;  // stage and phase of the block's B of both kinds
    for (int it = 0; it < n && ok; ++it) {
      const bool more = it + 1 < n, two = both(it);
      if (!(ok = wait(by_full + y, yp))) break;
      if (++x == bx_n) { x = 0; xp ^= 1; }  // of the next block
      if (more && !(ok = wait(bx_full + x, xp))) break;
      if (!(ok = wait(in_full, it & 1))) break;
      if (tc::elect_one()) mma_add<D>(tmem + sum, tmem + blocks, by + y * G::TILE, 0, it == 0);
      __syncwarp();
      if (!(ok = wait(in_full + 1, it & 1))) break;
      if (tc::elect_one()) {
        if (two) mma_add<D>(tmem + sum, tmem + blocks + 64, by + y * G::TILE, 1, false);
        tc::mma_commit(by_empty + y);
        if (more) product(x, both(it + 1));
        tc::mma_commit(more ? bx_empty + x : done);
      }
      __syncwarp();
      if (++y == by_n) { y = 0; yp ^= 1; }
    }
  } else {
    const int half = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int key = blk.at + (warp & 3) * 32 + lane;  // within the sequence
    const uint32_t ts = tmem + lanes + half * 64, tp = ts + DP;
    const F2 scale2 = f2(a.scale * LOG2E, a.scale * LOG2E);
    for (int it = 0; it < n; ++it) {
      if (half && !both(it)) {
        // nothing to do, but in step: a barrier tells only neighbouring phases apart
        if (!(ok = tc::mbar_wait_warp(s_full, it & 1))) break;
        if (lane == 0) tc::mbar_arrive(p_full + 1);
        if (!(ok = tc::mbar_wait_warp(dp_full, it & 1))) break;
        if (lane == 0) {
          tc::mbar_arrive(ds_full + 1);
          tc::mbar_arrive(row_free + (it & 1));
        }
        continue;
      }
      const int st = it & 1;
      const int at = (kb + it % per) * 128 + half * 64;  // first query row of this thread's columns
      const float4* lse = reinterpret_cast<const float4*>(rows + st * 256 + half * 64);
      const float4* del = lse + 32;
      ok = tc::mbar_wait_ns(row_full + st, (it >> 1) & 1) && tc::mbar_wait_ns(s_full, it & 1);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc::fence_after_sync();
      // query column i is visible from `lo` on (causal) and below `hi` (the end of the sequence)
      const int lo = key - at, hi = blk.len - at;
      const bool cut = at < blk.at + 128 || hi < 64;  // uniform
      float p[64];
      {
        uint32_t u[64];
        tc::tmem_ld32_nowait(ts, u);
        tc::tmem_ld32_nowait(ts + 32, u + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 r = lse[i / 4];  // -lse, in units of log2
          float x, y;
          split(fma2(f2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), scale2, f2(r.x, r.y)), x, y);
          p[i] = tc::ex2(x);
          p[i + 1] = tc::ex2(y);
          split(fma2(f2(__uint_as_float(u[i + 2]), __uint_as_float(u[i + 3])), scale2, f2(r.z, r.w)), x, y);
          p[i + 2] = tc::ex2(x);
          p[i + 3] = tc::ex2(y);
        }
        if (cut)
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i < lo || i >= hi) p[i] = 0.f;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pack2(p[2 * i], p[2 * i + 1]);
        tc::tmem_st32(ts, w);
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(p_full + half);
      if (!(ok = tc::mbar_wait_warp(dp_full, it & 1))) break;
      tc::fence_after_sync();
      {
        uint32_t u[64];
        tc::tmem_ld32_nowait(tp, u);
        tc::tmem_ld32_nowait(tp + 32, u + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float4 r = del[i / 4];  // -delta
          split(mul2(f2(p[i], p[i + 1]), add2(f2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), f2(r.x, r.y))), p[i], p[i + 1]);
          split(mul2(f2(p[i + 2], p[i + 3]), add2(f2(__uint_as_float(u[i + 2]), __uint_as_float(u[i + 3])), f2(r.z, r.w))), p[i + 2],
                p[i + 3]);
        }
        if (cut)
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i < lo || i >= hi) p[i] = 0.f;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = pack2(p[2 * i], p[2 * i + 1]);
        tc::tmem_st32(tp, w);
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(ds_full + half);
        tc::mbar_arrive(row_free + st);
      }
    }
    if (ok) {
      ok = tc::mbar_wait_warp(done, 0);
      tc::fence_after_sync();
      const bool in = ok && key < blk.len;
      const size_t at = ((size_t)(blk.row0 + key) * a.Hkv + kvh) * D + half * (D / 2);
      const uint32_t tv = tmem + lanes + DV + half * (D / 2), tk = tmem + lanes + DK + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        store32(tv + c, 1.f, a.dv + at + c, in);
        store32(tk + c, a.scale, a.dk + at + c, in);
      }
    }
  }
  if (!ok) atomicAdd(&g_gave_up, 1u);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- dq

template <int D> struct DqGeo {
  static constexpr int TILE = TILE_BYTES<D>;
  static constexpr int OFF_Q = 0, OFF_DO = TILE;
  static constexpr int OFF_K = 2 * TILE;  // [3]: S(it + 1) runs while dQ(it) still needs K(it)
  static constexpr int OFF_V = 5 * TILE;  // [2]
};

template <int D>
__device__ void dq_cta(uint8_t* sm, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const CUtensorMap& mdo, const BwdArgs& a, const Block& blk, int head) {
  using G = DqGeo<D>;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + BAR_OFF);
  uint64_t* k_full = q_full + 1;    // [3]
  uint64_t* k_empty = k_full + 3;   // [3]
  uint64_t* v_full = k_empty + 3;   // [2]
  uint64_t* v_empty = v_full + 2;   // [2]
  uint64_t* k_tail = v_empty + 2;
  uint64_t* s_full = k_tail + 1;    // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_free = dp_full + 1;  // both groups
  // [2 groups][2 score buffers]: a group may finish a block and the next one while
  // the other group holds up the warp that waits for both, but not a third
  uint64_t* ds_full = dp_free + 1;
  uint64_t* done = ds_full + 4;
  uint32_t* holder = reinterpret_cast<uint32_t*>(done + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int kvh = head / (a.Hq / a.Hkv);
  const int n = blk.at / 128 + 1;
  const int tail = blk.len - blk.at;  // rows of the last key block within the sequence, if < 128
  // group 1 has the second 64 keys of a block, if the sequence has them
  auto both = [&](int it) { return it + 1 < n || tail > 64; };

  if (tid == 0) {
    tc::mbar_init(q_full, 1);
    for (int s = 0; s < 3; ++s) {
      tc::mbar_init(k_full + s, 1);
      tc::mbar_init(k_empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(v_full + s, 1);
      tc::mbar_init(v_empty + s, 1);
      tc::mbar_init(s_full + s, 1);
      tc::mbar_init(ds_full + s, EW);
      tc::mbar_init(ds_full + 2 + s, EW);
    }
    tc::mbar_init(k_tail, 1);
    tc::mbar_init(dp_full, 1);
    tc::mbar_init(dp_free, 2 * EW);
    tc::mbar_init(done, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (warp == 9) tc::tmem_alloc(holder, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // all 512 columns, which start at 0: a constant keeps the MMAs' operands in uniform registers
  constexpr uint32_t tmem = 0;
  constexpr uint32_t DP = 256, DQ = 384;  // S at 0 and 128
  bool ok = true;

  if (warp == 8) {
    if (tc::elect_one()) {
      tc::mbar_expect_tx(q_full, 2 * G::TILE);
      load_tile<D>(sm + G::OFF_Q, &mq, head, blk.row0 + blk.at, q_full);
      load_tile<D>(sm + G::OFF_DO, &mdo, head, blk.row0 + blk.at, q_full);
    }
    __syncwarp();
    for (int it = 0; it < n; ++it) {
      const int st = it & 1, ph = (it >> 1) & 1, ks = it % 3;
      if (!(ok = tc::mbar_wait_warp(k_empty + ks, (it / 3 & 1) ^ 1))) break;
      if (tc::elect_one()) {
        tc::mbar_expect_tx(k_full + ks, G::TILE);
        load_tile<D>(sm + G::OFF_K + ks * G::TILE, &mk, kvh, blk.row0 + it * 128, k_full + ks);
      }
      __syncwarp();
      if (!(ok = tc::mbar_wait_warp(v_empty + st, ph ^ 1))) break;
      if (tc::elect_one()) {
        tc::mbar_expect_tx(v_full + st, G::TILE);
        load_tile<D>(sm + G::OFF_V + st * G::TILE, &mv, kvh, blk.row0 + it * 128, v_full + st);
      }
      __syncwarp();
    }
    if (ok && tail < 128) {  // nothing behind the sequence in dQ += dS K
      const int ks = (n - 1) % 3;
      ok = tc::mbar_wait_warp(k_full + ks, (n - 1) / 3 & 1);
      zero_rows<D>(sm + G::OFF_K + ks * G::TILE, tail);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(k_tail);
    }
  } else if (warp >= 9) {
    const uint32_t q = tc::smem_u32(sm + G::OFF_Q), d_o = tc::smem_u32(sm + G::OFF_DO);
    const uint32_t k = tc::smem_u32(sm + G::OFF_K), v = tc::smem_u32(sm + G::OFF_V);
    auto wait = [&](uint64_t* bar, int ph) {
      const bool w = tc::mbar_wait_warp(bar, ph);
      tc::fence_after_sync();
      return w;
    };
    ok = wait(q_full, 0);
    if (warp == 9) {  // S and dQ
      ok = ok && wait(k_full, 0);
      if (ok && tc::elect_one()) {
        mma_rows<D, 128>(tmem, q, k, 0);
        tc::mma_commit(s_full);
      }
      __syncwarp();
      for (int it = 0; it < n && ok; ++it) {
        const int st = it & 1, nx = (it + 1) & 1, ks0 = it % 3, ks1 = (it + 1) % 3;
        const bool more = it + 1 < n;
        if (more) {
          // the other score buffer: its dS was consumed by dQ(it - 1), issued before
          if (!(ok = wait(k_full + ks1, (it + 1) / 3 & 1))) break;
          if (tc::elect_one()) {
            mma_rows<D, 128>(tmem + nx * 128, q, k + ks1 * G::TILE, 0);
            tc::mma_commit(s_full + nx);
          }
          __syncwarp();
        } else if (tail < 128 && !(ok = wait(k_tail, 0))) {
          break;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bool has = g == 0 || both(it);
          if (has && !(ok = wait(ds_full + 2 * g + st, (it >> 1) & 1))) break;
          if (tc::elect_one()) {
            if (has) mma_add<D>(tmem + DQ, tmem + st * 128 + g * 64, k + ks0 * G::TILE, g, it == 0 && g == 0);
            if (g == 1) tc::mma_commit(more ? k_empty + ks0 : done);
          }
          __syncwarp();
        }
      }
    } else {  // dP
      for (int it = 0; it < n && ok; ++it) {
        const int st = it & 1;
        if (!(ok = wait(v_full + st, (it >> 1) & 1))) break;
        if (it > 0 && !(ok = wait(dp_free, (it - 1) & 1))) break;
        if (tc::elect_one()) {
          if (both(it)) mma_rows<D, 128>(tmem + DP, d_o, v + st * G::TILE, 0);
          else mma_rows<D, 64>(tmem + DP, d_o, v + st * G::TILE, 0);
          tc::mma_commit(dp_full);
          tc::mma_commit(v_empty + st);
        }
        __syncwarp();
      }
    }
  } else {
    const int half = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int row = blk.at + (warp & 3) * 32 + lane;  // within the sequence
    const bool in = row < blk.len;
    const size_t t = (size_t)blk.row0 + row;
    const float lse = in ? a.lse[(size_t)head * a.T + t] * -LOG2E : 0.f;
    const float del = in ? -(row < FEW ? a.first : a.delta)[(size_t)head * a.T + t] : 0.f;
    const F2 scale2 = f2(a.scale * LOG2E, a.scale * LOG2E), lse2 = f2(lse, lse);
    const uint32_t tp = tmem + lanes + DP + half * 64;
    for (int it = 0; it < n; ++it) {
      if (half && !both(it)) break;  // the last block
      const int st = it & 1;
      const uint32_t ts = tmem + lanes + st * 128 + half * 64;
      if (!(ok = tc::mbar_wait_warp(s_full + st, (it >> 1) & 1))) break;
      tc::fence_after_sync();
      float p[64];
      {
        uint32_t u[64];
        tc::tmem_ld32_nowait(ts, u);
        tc::tmem_ld32_nowait(ts + 32, u + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float x, y;
          split(fma2(f2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), scale2, lse2), x, y);
          p[i] = tc::ex2(x);
          p[i + 1] = tc::ex2(y);
        }
      }
      if (!(ok = tc::mbar_wait_warp(dp_full, it & 1))) break;
      tc::fence_after_sync();
      {
        uint32_t u[64];
        tc::tmem_ld32_nowait(tp, u);
        tc::tmem_ld32_nowait(tp + 32, u + 32);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(dp_free);
        // the diagonal block holds the end of the sequence, too: it lies past every row
        const int see = it + 1 == n ? min(row, blk.len - 1) - it * 128 - half * 64 : 64;
#pragma unroll
        for (int i = 0; i < 64; i += 2)
          split(mul2(f2(p[i], p[i + 1]), add2(f2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), f2(del, del))), p[i], p[i + 1]);
        if (it + 1 == n)
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i > see) p[i] = 0.f;
      }
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = pack2(p[2 * i], p[2 * i + 1]);
      tc::tmem_st32(ts, w);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(ds_full + 2 * half + st);
    }
    if (ok) {
      ok = tc::mbar_wait_warp(done, 0);
      tc::fence_after_sync();
      const uint32_t tq = tmem + lanes + DQ + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) store32(tq + c, a.scale, a.dq + (t * a.Hq + head) * D + half * (D / 2) + c, ok && in);
    }
  }
  if (!ok) atomicAdd(&g_gave_up, 1u);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_packed_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                           const BwdArgs a, int n_dkv) {
  extern __shared__ __align__(1024) uint8_t sm[];
  tc::grid_dep_wait();
  if (tc::smem_u32(sm) & 1023u) {  // every thread sees the same
    if (threadIdx.x == 0) atomicAdd(&g_unaligned, 1u);
    return;
  }
  // The blocks come from a table: with a search from the first sequence on in every
  // CTA, 40,000 sequences of 5 took 78 ms, with the table 8.2 (10,000: 6.4 and 2.0; 256
  // of 64: 0.35 and 0.33; 15 long ones the same).  A dk/dv CTA takes the first keys first,
  // which the most rows read, a dq CTA the last rows, which read the most keys.
  int b = blockIdx.x;
  const bool dkv = b < n_dkv;
  if (!dkv) b -= n_dkv;
  const int4 e = a.table[b / (dkv ? a.Hkv : a.Hq)];
  Block blk{e.x, e.y, e.z};
  if (!blk.len) return;
  if (dkv) {
    dkv_cta<D>(sm, mq, mk, mv, mdo, a, blk, b % a.Hkv);
  } else {
    blk.at = (blk.len - 1) / 128 * 128 - blk.at;
    dq_cta<D>(sm, mq, mk, mv, mdo, a, blk, b % a.Hq);
  }
}

template <int D>
int backward(const CUtensorMap* m, const BwdArgs& a, const DeltaArgs& da, cudaStream_t s) {
  if (!kernel_smem_at_least(reinterpret_cast<const void*>(&attn_packed_bwd_kernel<D>), SMEM))
    return op_fail(GOCR_ECUDA, "kernel configuration rejected");
  const long long firsts = (long long)a.n_seq * a.Hq, threads = (long long)a.T * a.Hq * (D / 8);
  launch_k(attn_delta_kernel<D>, dim3((unsigned)(1 + firsts + (threads + 256 * FLAT - 1) / (256 * FLAT))), dim3(256), 0, s,
           false, da);
  if (int rc = op_launched("attention_packed delta")) return rc;
  const long long blocks = da.blocks;
  launch_k(attn_packed_bwd_kernel<D>, dim3((unsigned)(blocks * (a.Hkv + a.Hq))), dim3(THREADS), SMEM, s, true, m[0], m[1],
           m[2], m[3], a, (int)(blocks * a.Hkv));
  return op_launched("attention_packed backward");
}

}  // namespace

namespace gocr {
cudaError_t attn_packed_bwd_gave_up(unsigned* out, cudaStream_t s) {
  return cudaMemcpyFromSymbolAsync(out, g_gave_up, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
}
cudaError_t attn_packed_bwd_unaligned(unsigned* out, cudaStream_t s) {
  return cudaMemcpyFromSymbolAsync(out, g_unaligned, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
}
}  // namespace gocr

static size_t table_at(int T, int Hq) { return ((size_t)T * Hq * 8 + 255) & ~(size_t)255; }

extern "C" {

size_t gocr_op_attention_packed_backward_workspace(int T, int Hq) {
  if (T < 0 || Hq < 1) return 0;
  // delta and that of the first rows, and the table: no more than T blocks have a row
  return table_at(T, Hq) + (size_t)T * sizeof(int4) + 256;
}

int gocr_op_attention_packed_backward(const void* d_o, const void* q, const void* k, const void* v, const void* o,
                                      const float* lse, const int32_t* cu_seqlens, void* dq, void* dk, void* dv,
                                      int n_seq, int T, int Hq, int Hkv, int d, long long ldq, long long ldk,
                                      long long ldv, float scale, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (int rc = attn_packed_check(n_seq, T, Hq, Hkv, d, ldq, ldk, ldv, scale)) return rc;
  if (!cu_seqlens || !workspace || (T && (!d_o || !q || !k || !v || !o || !lse || !dq || !dk || !dv)))
    return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)d_o | (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o | (uintptr_t)dq | (uintptr_t)dk |
       (uintptr_t)dv | (uintptr_t)workspace) & 15)
    return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (((uintptr_t)lse | (uintptr_t)cu_seqlens) & 3) return op_fail(GOCR_EINVAL, "lse or cu_seqlens not 4-byte aligned");
  if (workspace_bytes < gocr_op_attention_packed_backward_workspace(T, Hq)) return op_fail(GOCR_ECAPACITY, "workspace too small");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T || !n_seq) return GOCR_OK;
  CUtensorMap m[4];
  if (!map_rows(&m[0], q, T, Hq, d, ldq) || !map_rows(&m[1], k, T, Hkv, d, ldk) || !map_rows(&m[2], v, T, Hkv, d, ldv) ||
      !map_rows(&m[3], d_o, T, Hq, d, (long long)Hq * d))
    return op_fail(GOCR_ECUDA, "a TMA descriptor was rejected");
  float* delta = (float*)workspace;
  float* first = delta + (size_t)T * Hq;
  int4* table = (int4*)((char*)workspace + table_at(T, Hq));
  const BwdArgs a{cu_seqlens, lse, delta, first, (bf16*)dq, (bf16*)dk, (bf16*)dv, table, n_seq, T, Hq, Hkv, scale};
  const DeltaArgs da{(const bf16*)q, (const bf16*)k, (const bf16*)v, (const bf16*)o, (const bf16*)d_o, ldq, ldk, ldv,
                     cu_seqlens, lse, delta, first, table, (int)max_blocks(n_seq, T, 128), n_seq, T, Hq, Hkv, scale};
  return d == 128 ? backward<128>(m, a, da, s) : backward<64>(m, a, da, s);
}

}  // extern "C"
