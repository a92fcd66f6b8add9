// Causal attention over packed sequences with grouped heads, forward.
//
//   S_ij = c q_i . k_j (j <= i),  lse_i = log sum_j exp S_ij,  o_i = sum_j exp(S_ij - lse_i) v_j
//
// A work item is 256 query rows of a sequence and a q head: two tiles of 128
// rows share the K/V ring that a TMA warp fills.  Keys go by in blocks of 64.
// Both products run on tcgen05: S = Q K^T (128 x 64 x D) into one of two
// buffers a tile in tensor memory, P (bf16) back into tensor memory over S, O
// += P V with P read from there and V N-major as it lies.  A softmax thread owns
// a row: its 64 scores come from its own tensor memory lane, so the running
// maximum and sum need no exchange.
//
// What bounds it: the products of a tile with 64 keys take 646 cycles of the
// tensor pipe (score MMAs of 64 columns read A again for half the columns: 49
// cycles instead of 32), its softmax 620 of four warps, and the chain scores,
// softmax, P V is as long as both.  128 keys of both tiles pass in 3,270 cycles,
// 2,586 of them products.  (The tensor pipe's counter takes such a score MMA for 32
// cycles: by it 63 % of this loop is busy, and 47 % of a launch of one long sequence,
// with its items' first and last blocks, the halves that the diagonal masks, and the
// SMs without an item at the end.)  With one score buffer a tile and blocks of 128 keys
// the tiles waited for one another; with two buffers a tile's next scores are
// ready when its softmax is.  Each tile has an MMA warp, because a warp's wait
// on a barrier costs 100 cycles and more behind its own queue of MMAs, a time
// that the other warp's MMAs fill.  12 heads of 128: one sequence of 8,192 in
// 176 us (1.17 PFLOP/s), 16 prompts of 25 to 1,200 in 45 (heads of 64: 143 and 35),
// 18 regions of 1 to 140 in 17, where a launch's fixed chain (sequence search, loads, one block, store)
// is most of it.  Measured slower: part of the exponentials as polynomials on
// the FMA pipe, P given over in halves, sixteen softmax warps (two threads a
// row), one MMA warp, score MMAs of 128 columns with 208 registers a thread.
//
// O stays in tensor memory and is rescaled only when a row's maximum grows by
// more than 2^8 over the one its exponentials refer to (the sum and O use the
// same reference, so nothing is lost; P is at most 2^8).  P is rounded to bf16
// (relative 2^-8) since the tensor cores take it so; scores, maxima, sums and O
// are fp32.  No partial results leave the CTA: a row's bits depend on its own
// sequence only.
//
// The grid has a CTA per work item, but a running CTA takes over the items of
// those that have not started (cluster launch control), so barriers and tensor
// memory are set up once per SM and the next item's Q, K and V are on their way
// while the last one's output is written.  A warp takes the next item when the
// last loads of this one have been issued.
#include "../../include/gocr.h"
#include "attn_packed.cuh"

using namespace gocr;
using namespace gocr::packed;

namespace {

constexpr int QT = 256;        // query rows of a work item
// Eight softmax warps (two tiles x four lane quarters), then the TMA warp, an
// MMA warp a tile and the work warp.
constexpr int SW = 8, THREADS = (SW + 4) * 32;
constexpr float GROW = 8.f;    // log2 of the growth of a row's maximum that rescales O

static __device__ unsigned g_gave_up;  // threads whose wait gave up, ever

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
  static constexpr int OFF_WORK = OFF_KV + SLOTS * TILE_BYTES<D>;  // int4 [2], and the launch control's answer
  static constexpr int OFF_BAR = OFF_WORK + 64;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t O_COL = 256;  // S [2 tiles][2 buffers] of 64 columns; O [2 tiles] of D behind them
};

// One work item, as every warp sees it.
struct Item {
  Block blk;
  int head;
  int n0, n1, n;  // K/V tiles of the two query tiles: up to the diagonal, and within the sequence
  int tail;       // rows of the last K/V tile within the sequence, if < 128
  __device__ explicit Item(int4 w) : blk{w.x, w.y, w.z}, head(w.w) {
    n0 = blk.at / 128 + 1;
    n1 = blk.len - blk.at > 128 ? n0 + 1 : 0;
    n = n1 ? n1 : n0;
    tail = blk.len - (n - 1) * 128;
  }
  // blocks of 64 keys of query tile j; the last K/V tile's second may lie behind the sequence
  __device__ int blocks(int j) const {
    const int nj = j ? n1 : n0;
    return 2 * nj - (nj == n && tail <= 64);
  }
};

// The warp's next item from the ring of two; false past the last one.
__device__ __forceinline__ bool next_item(const int4* work, uint64_t* work_full, uint64_t* work_free, int i, int4& w,
                                          bool& ok) {
  const int s = i & 1;
  if (!(ok = tc::mbar_wait_warp(work_full + s, (i >> 1) & 1))) return false;
  w = work[s];
  // as uniform values, for the loops and operands that follow from them
  w.x = __shfl_sync(0xffffffffu, w.x, 0);
  w.y = __shfl_sync(0xffffffffu, w.y, 0);
  w.z = __shfl_sync(0xffffffffu, w.z, 0);
  w.w = __shfl_sync(0xffffffffu, w.w, 0);
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(work_free + s);
  return w.y > 0;
}

// Asks for a CTA of this launch that has not started, and its index if it now
// will not start, else -1 (then no further ask is allowed).  One warp.
__device__ __forceinline__ void ask_cta(void* answer, uint64_t* bar) {
  if ((threadIdx.x & 31) == 0) {
    tc::fence_proxy_async_smem();
    tc::mbar_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(tc::smem_u32(answer)), "r"(tc::smem_u32(bar)) : "memory");
  }
  __syncwarp();
}
__device__ __forceinline__ int taken_cta(const void* answer, uint64_t* bar, int turn, bool& ok) {
  if (!(ok = tc::mbar_wait_warp(bar, turn & 1))) return -1;
  uint32_t yes, x;  // every lane reads the answer; lane 0's counts
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(yes), "=r"(x) : "r"(tc::smem_u32(answer)) : "memory");
  return __shfl_sync(0xffffffffu, yes ? (int)x : -1, 0);
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_packed_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const FwdArgs a) {
  using F = Fwd<D>;
  constexpr int SLOTS = F::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + F::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* full = q_empty + 1;
  uint64_t* empty = full + SLOTS;
  uint64_t* s_full = empty + SLOTS;  // [2 tiles][2 buffers]
  uint64_t* p_full = s_full + 4;     // [2 tiles][2 buffers]
  uint64_t* o_full = p_full + 4;     // [2] a block's P V is complete
  uint64_t* o_done = o_full + 2;     // [2] the item's last one is
  // ragged V tiles, one barrier a slot: a slot's next load waits for this one's
  // use, so no barrier is ever two phases ahead of the warp that waits on it
  uint64_t* v_tail = o_done + 2;         // [SLOTS] the rows behind the sequence are zero
  uint64_t* work_full = v_tail + SLOTS;  // [2]
  uint64_t* work_free = work_full + 2;  // [2]
  uint64_t* taken = work_free + 2;
  uint64_t* issued = taken + 1;            // the item's loads are on their way
  uint64_t* drained = issued + 1;          // [2] an MMA warp's products, at its end
  uint32_t* holder = reinterpret_cast<uint32_t*>(drained + 2);
  int4* work = reinterpret_cast<int4*>(sm + F::OFF_WORK);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    tc::mbar_init(q_full, 1);
    tc::mbar_init(q_empty, 2);
    for (int s = 0; s < SLOTS; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 2);
      tc::mbar_init(v_tail + s, 1);
    }
    for (int j = 0; j < 4; ++j) {
      tc::mbar_init(s_full + j, 1);
      tc::mbar_init(p_full + j, SW / 2);
    }
    for (int j = 0; j < 2; ++j) {
      tc::mbar_init(o_full + j, 1);
      tc::mbar_init(o_done + j, 1);
      tc::mbar_init(drained + j, 1);
      tc::mbar_init(work_full + j, 1);
      tc::mbar_init(work_free + j, SW + 3);
    }
    tc::mbar_init(taken, 1);
    tc::mbar_init(issued, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  if (warp == SW + 1) tc::tmem_alloc(holder, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // all 512 columns, which start at 0: a constant keeps the MMAs' operands in uniform registers
  constexpr uint32_t tmem = 0;
  bool ok = true;
  int4 w;

  if (warp >= SW) {
    if (warp == SW) {
      // K(0), V(0), K(1), V(1), ... through the ring, Q behind the item's K(0)
      int slot = 0, ph = 0, loads = 0, q_loads = 0;
      for (int i = 0; next_item(work, work_full, work_free, i, w, ok); ++i) {
        const Item t(w);
        const int kvh = t.head / (a.Hq / a.Hkv);
        for (int x = 0; x < 2 * t.n; ++x) {
          if (!(ok = tc::mbar_wait_warp(empty + slot, ph ^ 1))) break;
          if (tc::elect_one()) {
            tc::mbar_expect_tx(full + slot, TILE_BYTES<D>);
            load_tile<D>(sm + F::OFF_KV + slot * TILE_BYTES<D>, x & 1 ? &mv : &mk, kvh, t.blk.row0 + (x >> 1) * 128, full + slot);
          }
          __syncwarp();
          ++loads;
          if (++slot == SLOTS) { slot = 0; ph ^= 1; }
          if (x == 0) {
            if (!(ok = tc::mbar_wait_warp(q_empty, (i & 1) ^ 1))) break;
            if (tc::elect_one()) {
              tc::mbar_expect_tx(q_full, (t.n1 ? 2 : 1) * TILE_BYTES<D>);
              load_tile<D>(sm + F::OFF_Q, &mq, t.head, t.blk.row0 + t.blk.at, q_full);
              if (t.n1) load_tile<D>(sm + F::OFF_Q + TILE_BYTES<D>, &mq, t.head, t.blk.row0 + t.blk.at + 128, q_full);
            }
            __syncwarp();
            ++q_loads;
          }
        }
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive(issued);
      }
      ok = tc::ring_landed(full, SLOTS, loads) && tc::ring_landed(q_full, 1, q_loads) && ok;
    } else if (warp < SW + 3) {
      const int j = warp - (SW + 1);  // the tile
      const uint32_t q = tc::smem_u32(sm + F::OFF_Q + j * TILE_BYTES<D>), kv = tc::smem_u32(sm + F::OFF_KV);
      const uint32_t s_col = tmem + j * 128, o_col = tmem + F::O_COL + j * D;
      int ring = 0;           // ring position of the item's K(0)
      unsigned tails = 0;     // parity of each slot's ragged tiles so far
      int turn[2] = {0, 0};   // blocks of each buffer so far
      auto wait = [&](uint64_t* bar, int ph) {
        const bool r = tc::mbar_wait_warp(bar, ph & 1);
        tc::fence_after_sync();
        return r;
      };
      for (int i = 0; next_item(work, work_full, work_free, i, w, ok); ++i) {
        const Item t(w);
        const int nb = t.blocks(j), most = max(t.blocks(0), t.blocks(1));
        auto wait_full = [&](int x) { return wait(full + (ring + x) % SLOTS, (ring + x) / SLOTS); };
        auto tile_of = [&](int x) { return kv + ((ring + x) % SLOTS) * TILE_BYTES<D>; };
        // both MMA warps give a K/V tile back, whether they used it or not
        // (but not before it is there: its barrier is in an older phase)
        auto release = [&](int x) { tc::mma_commit(empty + (ring + x) % SLOTS); };
        auto scores = [&](int b) {
          mma_rows<D>(s_col + (b & 1) * 64, q, tile_of(2 * (b >> 1)), b & 1);
          tc::mma_commit(s_full + j * 2 + (b & 1));
        };
        // after the scores of block b: the K tile, and at last Q
        auto release_k = [&](int b) {
          if ((b & 1) || b + 1 == most) release(2 * (b >> 1));
          if (b + 1 == most) tc::mma_commit(q_empty);
        };
        if (!(ok = wait(q_full, i) && wait_full(0))) break;
        if (tc::elect_one()) {
          // over P of the last item, whose products were issued before
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (b < nb) scores(b);
            if (b < most) release_k(b);
          }
        }
        __syncwarp();
        for (int b = 0; b < most; ++b) {
          if (!(b & 1)) {
            if (!(ok = wait_full(b + 1))) break;                  // V tile b / 2
            if (b + 2 < most && !(ok = wait_full(b + 2))) break;  // K tile b / 2 + 1
            if (b + 2 >= most && t.tail < 128) {
              const int slot = (ring + b + 1) % SLOTS;
              if (!(ok = wait(v_tail + slot, tails >> slot))) break;
              tails ^= 1u << slot;
            }
          }
          if (b < nb && !(ok = wait(p_full + j * 2 + (b & 1), turn[b & 1]++))) break;
          if (tc::elect_one()) {
            if (b < nb) {
              mma_add<D>(o_col, s_col + (b & 1) * 64, tile_of(2 * (b >> 1) + 1), b & 1, b == 0);
              tc::mma_commit(o_full + j);
              if (b + 1 == nb) tc::mma_commit(o_done + j);
            }
            if (b + 2 < nb) scores(b + 2);
            if ((b & 1) || b + 1 == most) release(2 * (b >> 1) + 1);
            if (b + 2 < most) release_k(b + 2);
          }
          __syncwarp();
        }
        if (!ok) break;
        ring += 2 * t.n;
      }
      ok = tc::mma_drain(drained + j) && ok;
    } else {
      // the items: this CTA's own, then those of CTAs that have not started;
      // and the last V tile of a ragged item: nothing behind the sequence
      int id = blockIdx.x, asks = 0, takes = 0, ring = 0;
      Cursor cursor;
      for (int i = 0; ok; ++i) {
        const int s = i & 1;
        Block blk{0, 0, 0};
        while (id >= 0 && ok) {
          blk = a.n_seq <= 32 ? find_block<1>(a.cu, a.n_seq, a.T, QT, id / a.Hq, cursor)
                              : find_block<8>(a.cu, a.n_seq, a.T, QT, id / a.Hq, cursor);
          if (blk.len) break;
          ask_cta(work + 2, taken);
          ++asks;
          id = taken_cta(work + 2, taken, takes++, ok);
        }
        const bool more = id >= 0;
        if (!ok || !(ok = tc::mbar_wait_warp(work_free + s, ((i >> 1) & 1) ^ 1))) break;
        w = make_int4(blk.row0, more ? blk.len : 0, blk.at, more ? id % a.Hq : 0);
        if (lane == 0) {
          work[s] = w;
          tc::mbar_arrive(work_full + s);
        }
        if (!more) break;
        // no earlier: an item in hand here is one that no idle SM can take
        if (!(ok = tc::mbar_wait_warp(issued, i & 1))) break;
        ask_cta(work + 2, taken);
        ++asks;
        const Item t(w);
        if (t.tail < 128) {
          const int x = ring + 2 * t.n - 1, slot = x % SLOTS;
          if (!(ok = tc::mbar_wait_warp(full + slot, (x / SLOTS) & 1))) break;
          zero_rows<D>(sm + F::OFF_KV + slot * TILE_BYTES<D>, t.tail);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(v_tail + slot);
        }
        ring += 2 * t.n;
        id = taken_cta(work + 2, taken, takes++, ok);
      }
      if (asks > takes) {  // gave up with a question under way
        bool answered;
        taken_cta(work + 2, taken, takes, answered);
      }
    }
  } else {
    const int j = warp >> 2, r = (warp & 3) * 32 + lane;  // tile, row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + F::O_COL + j * D + lanes;
    const float sl2 = a.scale * LOG2E;
    int turn[2] = {0, 0}, outs = 0, done = 0;  // blocks of each buffer, of the tile, and items so far
    for (int i = 0; ok && next_item(work, work_full, work_free, i, w, ok); ++i) {
      const Item t(w);
      const int nj = j ? t.n1 : t.n0, nb = t.blocks(j);
      if (!nj) continue;
      const int row = t.blk.at + j * 128 + r;  // within the sequence
      const int see = min(row, t.blk.len - 1); // the last key that the row sees
      float ref = 0.f, ref2 = 0.f, l = 0.f;    // the exponentials' reference, also times sl2; their sum
      for (int b = 0; b < nb; ++b, ++outs) {
        const uint32_t ts = tmem + j * 128 + (b & 1) * 64 + lanes;
        if (!(ok = tc::mbar_wait_warp(s_full + j * 2 + (b & 1), (b & 1 ? turn[1]++ : turn[0]++) & 1))) break;
        tc::fence_after_sync();
        uint32_t u[64];
        tc::tmem_ld32_nowait(ts, u);
        tc::tmem_ld32_nowait(ts + 32, u + 32);
        tc::tmem_wait_ld();
        if (b >= 2 * nj - 2) {  // the diagonal's K/V tile; it holds the end of the sequence, too
          const int last = see - b * 64;
#pragma unroll
          for (int x = 0; x < 64; ++x)
            if (x > last) u[x] = 0xff800000u;  // -infinity
        }
        float m4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(__uint_as_float(u[e]), __uint_as_float(u[e + 4]));
#pragma unroll
        for (int x = 8; x < 64; x += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = fmaxf(fmaxf(m4[e], __uint_as_float(u[x + e])), __uint_as_float(u[x + e + 4]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        if (b == 0) {
          ref = mx == -INFINITY ? 0.f : mx;
          ref2 = __fmul_rn(ref, sl2);
        } else {
          const bool grow = (mx - ref) * sl2 > GROW;
          if (__any_sync(0xffffffffu, grow)) {
            // the last block's P V; these scores vouch for the one before it, and
            // the next one waits for this block's P, so the parity is unambiguous
            if (!(ok = tc::mbar_wait_warp(o_full + j, (outs - 1) & 1))) break;
            tc::fence_after_sync();
            // a row whose reference stays, beside one whose grows (which may be of the
            // next sequence), keeps its bits: the products are rounded by themselves,
            // not in a fused multiply-add, so that its factor is 2^0
            const float to_new = grow ? mx : ref, to_new2 = __fmul_rn(to_new, sl2);
            const float f = tc::ex2(ref2 - to_new2);
            ref = to_new;
            ref2 = to_new2;
            l *= f;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t x[32];
              tc::tmem_ld32_nowait(to + c, x);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
              tc::tmem_st32(to + c, x);
            }
          }
        }
        const F2 scale2 = f2(sl2, sl2), ref22 = f2(-ref2, -ref2);
        F2 s4[4] = {f2(l, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          float p, q;
          split(fma2(f2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])), scale2, ref22), p, q);
          p = tc::ex2(p);
          q = tc::ex2(q);
          s4[x & 3] = add2(s4[x & 3], f2(p, q));
          u[x] = pack2(p, q);
        }
        tc::tmem_st32(ts, u);
        float p, q;
        split(add2(add2(s4[0], s4[1]), add2(s4[2], s4[3])), p, q);
        l = p + q;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + j * 2 + (b & 1));
      }
      if (!ok || !(ok = tc::mbar_wait_warp(o_done + j, done++ & 1))) break;
      tc::fence_after_sync();
      const float inv = 1.f / l;
      const size_t tok = (size_t)t.blk.row0 + row;
      bf16* dst = a.o + (tok * a.Hq + t.head) * D;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t x[32];
        tc::tmem_ld32_nowait(to + c, x);
        tc::tmem_wait_ld();
        if (row < t.blk.len)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              h[e] = pack2(__uint_as_float(x[g * 8 + 2 * e]) * inv, __uint_as_float(x[g * 8 + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + c + g * 8) = make_uint4(h[0], h[1], h[2], h[3]);
          }
      }
      if (row < t.blk.len) a.lse[(size_t)t.head * a.T + tok] = (ref2 + log2f(l)) * LN2;
      tc::fence_before_sync();  // O has been read before the next item's P V, which waits for its P
    }
  }
  if (!ok) atomicAdd(&g_gave_up, 1u);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == SW + 1) {
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
cudaError_t attn_packed_gave_up(unsigned* out, cudaStream_t s) {
  return cudaMemcpyFromSymbolAsync(out, g_gave_up, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
}

int attn_packed_check(int n_seq, int T, int Hq, int Hkv, int d, long long ldq, long long ldk, long long ldv,
                      float scale) {
  if (n_seq < 0 || n_seq > (1 << 20) || T < 0 || T > (1 << 24) || Hkv < 1 || Hq < 1 || Hq % Hkv || Hq > 1024 ||
      (d != 64 && d != 128))
    return op_fail(GOCR_EINVAL, "bad shape: %d sequences, T=%d Hq=%d Hkv=%d d=%d", n_seq, T, Hq, Hkv, d);
  if (((long long)n_seq + T) * (Hq + Hkv) > 0x7fffffffLL)  // CTAs of a launch
    return op_fail(GOCR_EINVAL, "bad shape: (%d sequences + T=%d) x (Hq=%d + Hkv=%d) is above 2^31 - 1", n_seq, T, Hq, Hkv);
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
  if (((uintptr_t)lse | (uintptr_t)cu_seqlens) & 3) return op_fail(GOCR_EINVAL, "lse or cu_seqlens not 4-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T || !n_seq) return GOCR_OK;
  CUtensorMap m[3];
  if (!map_rows(&m[0], q, T, Hq, d, ldq) || !map_rows(&m[1], k, T, Hkv, d, ldk) || !map_rows(&m[2], v, T, Hkv, d, ldv))
    return op_fail(GOCR_ECUDA, "a TMA descriptor was rejected");
  const FwdArgs a{cu_seqlens, (bf16*)o, lse, n_seq, T, Hq, Hkv, scale};
  return d == 128 ? forward<128>(m, a, s) : forward<64>(m, a, s);
}
