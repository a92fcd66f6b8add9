// Attention of requests' new rows over a paged KV cache.
//
//   S_ij = c q_i . k_j,  lse_i = log sum_j exp S_ij,  o_i = sum_j exp(S_ij - lse_i) v_j,  j = 0 .. the last key row i reads
//
// A unit of work is a request, a kv head and up to two tiles of query rows; a
// tile holds 128 / G tokens with the G q heads that share the kv head, so a
// window's rows read their keys once.  All units' key tiles (of 128 keys) lie on
// one axis, which is cut into equal pieces, one a CTA: a single token's long
// context spreads over the device, and chunks of prompts leave no last wave.  A
// unit that a cut divides leaves its parts (O, maximum, sum, in fp32) in the workspace, and
// a second launch joins them in order; the others are finished in place.
//
// Inside, a CTA runs as the packed-sequence kernel does: a TMA warp fills a ring
// of K and V tiles (a box a page), an MMA warp a softmax group issues S = Q K^T (128 x
// 64 x D, two score buffers a group in tensor memory) and O += P V with P read from
// tensor memory, and a softmax thread owns a row.  With two query tiles each group has
// one; with one, each has half of its keys, and they join in tensor memory.
// Rows, tiles and keys that do not exist cost their products but no exponentials:
// with one token a product of 128 rows takes less time than its keys do from HBM.
//
// What bounds it (12 q and 4 kv heads of 128, pages of 16, times on the device):
//   few rows: HBM.  256 single tokens of 1,000 to 4,000 keys 182 us (6.1 TB/s, 90 % of a
//     copy's rate), 64 of 256 to 8,192 51 (4.8 TB/s: 7 us before the first keys are there, 4 for
//     the join), a window of 33 behind 131,105 keys 56, one token over 1,097 keys 12;
//   many rows: the tensor pipe.  A prompt of 16,384 rows 513 us (1.61 PFLOP/s, 85 % of
//     the library's product), two last chunks of 2,048 rows over 8,192 keys 133 (1.35);
//     128 keys of two query tiles pass in 3,000 cycles, 2,590 of them products;
//   heads of 64: the chain of a block of 64 keys (scores, maximum, exponentials, P V), as long
//     as with heads of 128 for half the products: the prompt 435 us, two chunks 108, with the
//     tensor pipe 37 % active, the special-function pipe 37 %, the issue slots 46 %;
//   short requests: the chain of an item (Q, scores, softmax, P V, store), 3 us each:
//     1,000 tokens of 16 to 400 keys 84 us.
// The roles' code has to stay in the instruction cache: with waits of twenty sites,
// rescaling and eight boxes a load unrolled, three and a half times as much of it, two chunks'
// call took 207 us (176 with the waits and the loads rolled up).  A part costs 0.5 KB a row, written and read: the
// join of the two chunks' 302 parts is 15 us of 133, where cuts at unit boundaries only
// would leave two thirds of the SMs idle in the second round of their 200 units.
//
// P is rounded to bf16 for its product, which runs at the tensor pipe's full rate so (tf32 would
// halve it, and V would have to be widened first); its sum is taken
// before the rounding, in fp32, as are scores, statistics and the parts.  Against 64 bits o is
// off by 0.0021 to 0.0024 of its norm; the rounding of o alone makes 0.0017.
#include "attn_packed.cuh"
#include "paged.cuh"

#include <numeric>
#include <type_traits>

using namespace gocr;
using namespace gocr::packed;
using namespace gocr::paged;

namespace {

constexpr int KT = 128;        // keys of a tile
constexpr int GRID = SM_COUNT; // pieces of the work; parts depend on it, so it is a constant
// Eight softmax warps (two tiles x four lane quarters), then the TMA warp, an
// MMA warp a tile and the work warp.
constexpr int SW = 8, THREADS = (SW + 4) * 32;
constexpr float GROW = 8.f;    // log2 of the growth of a row's maximum that rescales O

static __device__ unsigned g_gave_up;  // threads whose wait gave up, ever

// A unit that its CTA began and did not finish.
struct Split {
  unsigned after;  // where the next CTA's piece begins, within the unit
  unsigned work, piece;
  int row0, n, kv, tok0, head, two, pad[3];
};

struct PagedArgs {
  const int *table, *cu, *kv_len;
  bf16* o;
  float* lse;
  float4* part;   // [2 GRID][D / 4][rows]
  float2* stat;   // [2 GRID][rows]: reference (times scale log2 e) and sum of the exponentials
  Split* split;   // [GRID], n = 0: none
  int* tasks;     // [GRID], of their joins
  int max_pages, n_pages, n_req, T, Hq, Hkv, G, toks, draft, shift, rows;
  int k_page, k_head, k_units, v_page, v_head, v_units;  // page and head strides of the maps' last dimension, and its size
  float scale;
};

// A tile of K or V in shared memory: 16 groups of 8 keys, in each the D / 64
// swizzled 8 x 128-byte atoms of its columns.  So a page's keys are whole groups, and one
// TMA box brings all columns of a page.
template <int D> constexpr int GROUP = 8 * D * 2;  // bytes of a group
// dst[128, 64] = Q K^T over D: rows 64 half .. of K's tile; Q's as load_tile leaves it.
template <int D> __device__ __forceinline__ void mma_scores(uint32_t dst, uint32_t q, uint32_t k, int half) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, 64);
  const uint64_t qd = tc::sdesc_sw128(q), kd = tc::sdesc_sw128(k + half * 8 * GROUP<D>, GROUP<D>);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    tc::mma_bf16(dst, qd + (((ks >> 2) * BOX_BYTES + (ks & 3) * 32) >> 4), kd + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4),
                 idesc, ks > 0 ? 1u : 0u);
}
// dst[128, D] (+)= P V over rows 64 half .. of V's tile, P from tensor memory.
template <int D> __device__ __forceinline__ void mma_values(uint32_t dst, uint32_t p, uint32_t v, int half, bool first) {
  constexpr uint32_t idesc = tc::idesc_bf16(128, D) | tc::IDESC_B_MN;
  const uint64_t vd = tc::sdesc_sw128_mn(v + half * 8 * GROUP<D>, 1024, GROUP<D>);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    tc::mma_bf16_ta(dst, p + ks * 8, vd + (ks * 2 * GROUP<D> >> 4), idesc, !first || ks > 0 ? 1u : 0u);
}
// Keys n .. 127 of a tile become zero: they are nobody's and may hold anything.  One warp.
template <int D> __device__ __forceinline__ void zero_keys(uint8_t* tile, int n) {
#pragma unroll 1
  for (int i = n * 8 + (threadIdx.x & 31); i < KT * 8; i += 32)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      *reinterpret_cast<uint4*>(tile + (i >> 6) * GROUP<D> + c * 1024 + (i & 63) * 16) = make_uint4(0, 0, 0, 0);
}

template <int D> struct Lay {
  static constexpr int SLOTS = D == 128 ? 4 : 8;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * TILE_BYTES<D>;
  static constexpr int OFF_WORK = OFF_KV + SLOTS * TILE_BYTES<D>;  // int4 [2][3]
  static constexpr int OFF_BAR = OFF_WORK + 96;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t O_COL = 256;  // S [2 tiles][2 buffers] of 64 columns; O [2 tiles] of D behind them
};

struct Req {
  int row0, n, kv;
};
__device__ __forceinline__ Req request(const PagedArgs& a, int r) {
  const int c0 = min(max(a.cu[r], 0), a.T), c1 = min(max(a.cu[r + 1], 0), a.T);
  return Req{c0, max(c1 - c0, 0), min(max(a.kv_len[r], 0), a.max_pages << a.shift)};
}
// The last key that token i reads; negative: none.
__device__ __forceinline__ int last_key(const PagedArgs& a, const Req& q, int i) {
  return a.draft && i > 0 ? q.kv - 1 : q.kv - q.n + i;
}
// Work of a unit, the two query tiles from token i on: 5 a key tile (3,000 cycles) and 16
// for its beginning and end where both hold tokens (a prompt of 8,192 rows takes 154.6 us
// with 16 for the ends, 159.9 with 10); 4 and 2 where one does, whose keys' way from HBM hides
// most of the ends (2,480 cycles a tile; 64 single tokens take 50.7 us with 2, 53.1 with 10).
// Weighed with heads of 128; with heads of 64 the same: other ends, or 6 a key tile of two query
// tiles, change two chunks (108.1 us), a prompt of 16,384 (437) and 64 tokens (33.9) by 1 % at
// most, and 10 for single tiles' ends takes draft windows from 16.9 to 16.1 and chunks to 109.4.
__device__ __forceinline__ bool two_tiles(const PagedArgs& a, const Req& q, int i) { return q.n - i > a.toks; }
__device__ __forceinline__ int key_tiles(const PagedArgs& a, const Req& q, int i) {
  const int last = i < q.n ? last_key(a, q, min(i + 2 * a.toks, q.n) - 1) : -1;
  return last < 0 ? 0 : last / KT + 1;
}
__device__ __forceinline__ unsigned work_of(const PagedArgs& a, const Req& q, int i) {
  const unsigned n = key_tiles(a, q, i);
  return n ? (two_tiles(a, q, i) ? 16 + 5 * n : 2 + 4 * n) : 0;
}
// The key tiles of a unit that lie before its work x.
__device__ __forceinline__ int tile_at(unsigned x, bool two) {
  return two ? (max(x, 16u) - 12) / 5 : (max(x, 2u) + 1) / 4;
}

// The join of a unit: its parts (pieces that may hold a tile of it), the warps that
// share a task's parts (each takes two or more), and its tasks of JOIN_WARPS warps.
constexpr int JOIN_CTAS = 4 * SM_COUNT, JOIN_WARPS = 8;
__device__ __forceinline__ int parts_of(const Split& s) { return 2 + (int)((s.work - s.after - 1) / s.piece); }
__device__ __forceinline__ int share_of(int parts) { return parts >= 16 ? 8 : parts >= 8 ? 4 : parts >= 4 ? 2 : 1; }
__device__ __forceinline__ int rows_of(const PagedArgs& a, const Split& s) { return min(s.n - s.tok0, 2 * a.toks) * a.G; }
template <int D> __device__ __forceinline__ int tasks_of(const PagedArgs& a, const Split& s) {
  const int each = 32 * JOIN_WARPS / share_of(parts_of(s));
  return s.n ? (rows_of(a, s) * (D / 8) + each - 1) / each : 0;
}

// One work item, as every warp sees it.
struct Item {
  Req q;
  int tok0, head, k0, k1, part, req;
  __device__ Item(const int4* w)
      : q{w[0].x, w[0].y, w[0].z}, tok0(w[0].w), head(w[1].x), k0(w[1].y), k1(w[1].z), part(w[1].w), req(w[2].x) {}
  // tokens of query tile j
  __device__ int tokens(const PagedArgs& a, int j) const { return min(max(q.n - tok0 - j * a.toks, 0), a.toks); }
  // With one query tile, both softmax groups (each with its MMA warp) take it: group 0 the
  // first 64 keys of each key tile, group 1 the others, and they join at the end.
  __device__ bool one(const PagedArgs& a) const { return q.n - tok0 <= a.toks; }
  // blocks of 64 keys of group j within the item
  __device__ int blocks(const PagedArgs& a, int j) const {
    const bool both = one(a);
    const int end = min(q.n, tok0 + (both || j == 0 ? a.toks : 2 * a.toks)), last = last_key(a, q, end - 1);
    const int all = last < 0 ? 0 : max(min(2 * k1, last / 64 + 1) - 2 * k0, 0);
    return both ? (all + 1 - j) >> 1 : all;
  }
  // keys of the item's last tile that exist
  __device__ int tail() const { return min(q.kv - (k1 - 1) * KT, KT); }
};

// tc::mbar_wait_warp in few instructions: the roles' loops together have to stay in
// the instruction cache (with twenty waits of the longer form a chunk's call takes 6 % more).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  uint32_t t0 = 0, t;  // low words: a wait of two seconds ends before they come round
  bool there;
#pragma unroll 1
  do {
#pragma unroll 1
    for (int i = 0; i < 64 && !(there = tc::mbar_try_wait(bar, parity)); ++i) {}
    if (there) break;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
    if (!t0) t0 = t | 1;
  } while (t - t0 + 1 < (uint32_t)tc::WAIT_NS);
  return __all_sync(0xffffffffu, there);
}

// The warp's next item from the ring of two; false past the last one.
__device__ __forceinline__ bool next_item(const int4* work, uint64_t* work_full, uint64_t* work_free, int i, int4* w,
                                          bool& ok) {
  const int s = i & 1;
  if (!(ok = wait_warp(work_full + s, (i >> 1) & 1))) return false;
#pragma unroll
  for (int e = 0; e < 3; ++e) {
    w[e] = work[s * 3 + e];
    // as uniform values, for the loops and operands that follow from them
    w[e].x = __shfl_sync(0xffffffffu, w[e].x, 0);
    w[e].y = __shfl_sync(0xffffffffu, w[e].y, 0);
    w[e].z = __shfl_sync(0xffffffffu, w[e].z, 0);
    w[e].w = __shfl_sync(0xffffffffu, w[e].w, 0);
  }
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(work_free + s);
  return w[0].y > 0;
}

// The pages of a request as the last coordinates of the K and V maps: 32 a warp in
// hand and the next 32 on their way.
struct Pages {
  const int* row;
  int n, at, next, k, v;
  __device__ int entry(int i) const { return i < n ? row[i] : -1; }
  __device__ void take(const PagedArgs& a, int head, int page) {
    const bool there = page >= 0 && page < a.n_pages;  // behind a map's end TMA reads zeros
    k = there ? page * a.k_page + head * a.k_head : a.k_units;
    v = there ? page * a.v_page + head * a.v_head : a.v_units;
  }
  __device__ Pages(const PagedArgs& a, const Item& t)
      : row(a.table + (size_t)t.req * a.max_pages), n((t.q.kv + (1 << a.shift) - 1) >> a.shift), at((t.k0 * KT) >> a.shift) {
    const int lane = threadIdx.x & 31, first = entry(at + lane);
    next = entry(at + 32 + lane);
    take(a, t.head, first);
  }
  // Before the pages of a tile, i and behind, are asked for; 32 is a multiple of a tile's pages.
  __device__ void reach(const PagedArgs& a, int head, int i) {
    if (i < at + 32) return;
    at += 32;
    take(a, head, next);
    next = entry(at + 32 + (threadIdx.x & 31));
  }
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ PagedArgs a) {
  using F = Lay<D>;
  constexpr int SLOTS = F::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) unsigned sums[SW + 4];
  __shared__ unsigned start_at;            // where this CTA's piece begins within its first request,
  __shared__ int start_req, start_of[3];   // and that request
  __shared__ float2 chain[2][128];         // of a tile whose keys both softmax groups share: reference and sum
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
  uint64_t* v_tail = o_done + 2;         // [SLOTS] the rows behind the request's keys are zero
  uint64_t* work_full = v_tail + SLOTS;  // [2]
  uint64_t* work_free = work_full + 2;   // [2]
  uint64_t* issued = work_free + 2;      // [2] an item's loads are on their way
  uint64_t* drained = issued + 2;        // [2] an MMA warp's products, at its end
  uint64_t* met = drained + 2;           // [4] the two warps that own the same 32 rows of a tile
  uint32_t* holder = reinterpret_cast<uint32_t*>(met + 4);
  int4* work = reinterpret_cast<int4*>(sm + F::OFF_WORK);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // as a uniform value, for what follows from it

  if (warp == SW && lane == 0) {
    tc::prefetch_tmap(&mk);
    tc::prefetch_tmap(&mv);
    tc::prefetch_tmap(&mq);
    tc::mbar_init(q_full, 1);
    tc::mbar_init(q_empty, 2);
#pragma unroll 1
    for (int s = 0; s < SLOTS; ++s) {
      tc::mbar_init(full + s, 1);
      tc::mbar_init(empty + s, 2);
      tc::mbar_init(v_tail + s, 1);
    }
    for (int j = 0; j < 4; ++j) {
      tc::mbar_init(met + j, 2);
      tc::mbar_init(s_full + j, 1);
      tc::mbar_init(p_full + j, SW / 2);
    }
    for (int j = 0; j < 2; ++j) {
      tc::mbar_init(o_full + j, 1);
      tc::mbar_init(o_done + j, 1);
      tc::mbar_init(issued + j, 1);
      tc::mbar_init(drained + j, 1);
      tc::mbar_init(work_full + j, 1);
      tc::mbar_init(work_free + j, SW + 3);
    }
    tc::fence_mbar_init();
    start_req = a.n_req;
  }
  __syncwarp();
  if (warp == SW + 1) tc::tmem_alloc(holder, 512);
  tc::grid_dep_wait();  // so far nothing that an earlier kernel may write was read

  // All requests' work: its sum, and where this CTA's piece begins.
  const int per = (a.n_req + THREADS - 1) / THREADS, r0 = min(tid * per, a.n_req), r1 = min(r0 + per, a.n_req);
  auto sum_of = [&](const Req& q) {
    unsigned sum = 0;
#pragma unroll 1
    for (int i = 0; i < q.n; i += 2 * a.toks) sum += work_of(a, q, i);
    return sum * a.Hkv;
  };
  Req q0{0, 0, 0};  // the thread's first request
  unsigned first = 0, mine = 0;
  bool without = false;  // a request has rows without keys
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const Req q = request(a, r);
    const unsigned sum = sum_of(q);
    if (r == r0) {
      q0 = q;
      first = sum;
    }
    mine += sum;
    without |= q.n > q.kv;
  }
  unsigned inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sums[warp] = inc;
  tc::fence_before_sync();
  without = __syncthreads_or(without);
  tc::fence_after_sync();
  unsigned before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < SW + 4; ++w) {
    const unsigned v = sums[w];
    if (w < warp) before += v;
    total += v;
  }
  const unsigned piece = (total + GRID - 1) / GRID, x0 = min(piece * blockIdx.x, total), x1 = x0 + min(piece, total - x0);
  if (before <= x0 && x0 < before + mine) {
    int r = r0;
#pragma unroll 1
    while (x0 >= before + first && r + 1 < r1) {
      before += first;
      q0 = request(a, ++r);
      first = sum_of(q0);
    }
    start_req = r;
    start_of[0] = q0.row0;
    start_of[1] = q0.n;
    start_of[2] = q0.kv;
    start_at = x0 - before;
  }
  if (without) {
    // Rows without keys, in requests with more rows than keys: a warp finds the requests among its
    // own and writes a share of each one's rows, so that all CTAs' warps write a request together.
    // (A refused prompt of 16,384 rows beside 64 tokens: 85 us, 56 without it; with its rows in one CTA 2,770.)
#pragma unroll 1
    for (int at = warp * 32; at < a.n_req; at += THREADS) {
      const Req q = at + lane < a.n_req ? request(a, at + lane) : Req{0, 0, 0};
      const int none = q.kv == 0 ? q.n : a.draft ? min(1, q.n - q.kv) : q.n - q.kv;
#pragma unroll 1
      for (unsigned some = __ballot_sync(0xffffffffu, none > 0); some; some &= some - 1) {
        const int l = __ffs(some) - 1, row0 = __shfl_sync(0xffffffffu, q.row0, l), n = __shfl_sync(0xffffffffu, none, l);
        const unsigned first = (blockIdx.x + at + l) % GRID * 32 + lane, rows = (unsigned)n * a.Hq;
        uint4* o = reinterpret_cast<uint4*>(a.o + (size_t)row0 * a.Hq * D);
#pragma unroll 1
        for (size_t i = first; i < (size_t)rows * (D / 8); i += GRID * 32) o[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (unsigned i = first; i < rows; i += GRID * 32) a.lse[(size_t)(i / n) * a.T + row0 + i % n] = -INFINITY;
      }
    }
  }
  __syncthreads();
  // all 512 columns, which start at 0: a constant keeps the MMAs' operands in uniform registers
  constexpr uint32_t tmem = 0;
  bool ok = true;
  int4 w[3];

  if (warp >= SW) {
    if (warp == SW) {
      // K(0), V(0), K(1), V(1), ... through the ring, Q behind the item's K(0)
      int slot = 0, ph = 0, loads = 0, q_loads = 0;
      const int shift = min(a.shift, 7);  // log2 of the keys of a page that a tile holds
      for (int i = 0; next_item(work, work_full, work_free, i, w, ok); ++i) {
        const Item t(w);
        Pages pages(a, t);
#pragma unroll 1
        for (int x = t.k0; ok && x < t.k1; ++x) {
          const int key0 = x * KT, boxes = (min(t.q.kv - key0, KT) + (1 << shift) - 1) >> shift;
          const int page = key0 >> a.shift, group = (key0 & ((1 << a.shift) - 1)) >> 3;
          pages.reach(a, t.head, page);
          // a lane has a page, and loads its keys (a loop over the pages in one lane, which first gets
          // each page from the lane that has it, takes 5 % more of two chunks' call)
          const int b = (lane - (page - pages.at)) & 31;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (!(ok = wait_warp(empty + slot, ph ^ 1))) break;
            if (tc::elect_one()) tc::mbar_expect_tx(full + slot, boxes << shift + (D == 128 ? 8 : 7));
            __syncwarp();
            if (b < boxes)
              tc::tma_load_5d(sm + F::OFF_KV + slot * TILE_BYTES<D> + (b << shift) * D * 2, v ? &mv : &mk, 0, 0, 0, group,
                              v ? pages.v : pages.k, full + slot);
            __syncwarp();
            ++loads;
            if (++slot == SLOTS) { slot = 0; ph ^= 1; }
            if (x == t.k0 && v == 0) {
              if (!(ok = wait_warp(q_empty, (i & 1) ^ 1))) break;
              const int tiles = t.tokens(a, 1) ? 2 : 1;
              if (tc::elect_one()) {
                tc::mbar_expect_tx(q_full, tiles * a.toks * a.G * D * 2);
#pragma unroll 1
                for (int j = 0; j < tiles; ++j)
#pragma unroll
                  for (int c = 0; c < D / 64; ++c)
                    tc::tma_load_3d(sm + F::OFF_Q + j * TILE_BYTES<D> + c * BOX_BYTES, &mq, c * 64, t.head * a.G,
                                    t.q.row0 + t.tok0 + j * a.toks, q_full);
              }
              __syncwarp();
              ++q_loads;
            }
          }
        }
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive(issued + (i & 1));
      }
      // a copy that lands after its CTA has left would do so in the shared memory of the next
      bool landed = !q_loads || wait_warp(q_full, (q_loads - 1) & 1);
#pragma unroll 1
      for (int s = 0; s < SLOTS && s < loads; ++s) landed = landed && wait_warp(full + s, ((loads - 1 - s) / SLOTS) & 1);
      ok = landed && ok;
    } else if (warp < SW + 3) {
      const int j = warp - (SW + 1);  // the softmax group
      const uint32_t q = tc::smem_u32(sm + F::OFF_Q), kv = tc::smem_u32(sm + F::OFF_KV);
      const uint32_t s_col = tmem + j * 128, o_col = tmem + F::O_COL + j * D;
      int ring = 0;           // ring position of the item's K(0)
      unsigned tails = 0;     // parity of each slot's ragged tiles so far
      unsigned turns = 0;     // parity of each buffer's blocks so far
      auto wait = [&](uint64_t* bar, int ph) {
        const bool r = wait_warp(bar, ph & 1);
        tc::fence_after_sync();
        return r;
      };
      for (int i = 0; next_item(work, work_full, work_free, i, w, ok); ++i) {
        const Item t(w);
        // the item's loop, once for one query tile and once for two: an instruction more between a
        // block's P and its products is time in which the tensor pipe waits
        auto products = [&](auto lone) {
          constexpr bool one = decltype(lone)::value;
          const int nb = t.blocks(a, j), most = one ? t.k1 - t.k0 : max(t.blocks(a, 0), t.blocks(a, 1)), tail = t.tail();
          auto wait_full = [&](int x) { return wait(full + (ring + x) % SLOTS, (ring + x) / SLOTS); };
          auto tile_of = [&](int x) { return kv + ((ring + x) % SLOTS) * TILE_BYTES<D>; };
          // the K/V tile of the group's block b, and which 64 keys of it
          auto at = [&](int b) { return one ? b : b >> 1; };
          auto half = [&](int b) { return one ? j : b & 1; };
          auto opens = [&](int b) { return one || !(b & 1); };
          auto closes = [&](int b) { return one || (b & 1) || b + 1 == most; };
          // both MMA warps give a K/V tile back, whether they used it or not
          // (but not before it is there: its barrier is in an older phase)
          auto release = [&](int x) { tc::mma_commit(empty + (ring + x) % SLOTS); };
          auto scores = [&](int b) {
            if (b >= nb) return;
            mma_scores<D>(s_col + (b & 1) * 64, q + (one ? 0 : j * TILE_BYTES<D>), tile_of(2 * at(b)), half(b));
            tc::mma_commit(s_full + j * 2 + (b & 1));
          };
          // after the scores of block b: the K tile, and at last Q
          auto release_k = [&](int b) {
            if (closes(b)) release(2 * at(b));
            if (b + 1 == most) tc::mma_commit(q_empty);
          };
          auto values = [&](int b) {
            if (b >= nb) return;
            mma_values<D>(o_col, s_col + (b & 1) * 64, tile_of(2 * at(b) + 1), half(b), b == 0);
            tc::mma_commit(o_full + j);
            if (b + 1 == nb) tc::mma_commit(o_done + j);
          };
          auto release_v = [&](int b) {
            if (closes(b)) release(2 * at(b) + 1);
          };
          if (!(ok = wait(q_full, i))) return;
          // block -2, -1: scores only (over P of the last item, whose products were issued before)
#pragma unroll 1
          for (int b = -2; b < most; ++b) {
            if (b >= 0 && opens(b)) {
              const int v = 2 * at(b) + 1;
              if (!(ok = wait_full(v))) break;
              if (at(b) + 1 == t.k1 - t.k0 && tail < KT) {
                const int slot = (ring + v) % SLOTS;
                if (!(ok = wait(v_tail + slot, tails >> slot))) break;
                tails ^= 1u << slot;
              }
            }
            // Two tiles: the next K tile is there by now, and is not waited for between P and
            // its product.  One: it may be on its way still, and the V tile's slot does not wait for it.
            const bool more = b + 2 < most;
            if (more && (b < 0 || !one) && opens(b + 2) && !(ok = wait_full(2 * at(b + 2)))) break;
            if (b >= 0 && b < nb) {
              if (!(ok = wait(p_full + j * 2 + (b & 1), turns >> (b & 1)))) break;
              turns ^= 1u << (b & 1);
            }
            if (tc::elect_one()) {
              if (b >= 0) values(b);
              if (more && (b < 0 || !one)) scores(b + 2);
              if (b >= 0) release_v(b);
              if (more && (b < 0 || !one)) release_k(b + 2);
            }
            __syncwarp();
            if (more && b >= 0 && one) {
              if (!(ok = wait_full(2 * at(b + 2)))) break;
              if (tc::elect_one()) {
                scores(b + 2);
                release_k(b + 2);
              }
              __syncwarp();
            }
          }
        };
        if (t.one(a)) products(std::true_type{});
        else products(std::false_type{});
        if (!ok) break;
        ring += 2 * (t.k1 - t.k0);
      }
      if (tc::elect_one()) tc::mma_commit(drained + j);
      __syncwarp();
      ok = wait_warp(drained + j, 0) && ok;
    } else {
      // The piece's items; and the last V tile of a ragged item: nothing behind the request's keys.
      int r = start_req, h = 0, i = 0, items = 0, ring = 0;
      unsigned at = 0, left = r < a.n_req ? x1 - x0 : 0;  // within the unit; of the piece
      Req q{0, 0, 0};
      Split split{};
      if (left > 0) {
        // (row ranges that overlap may be more work than 32 bits count: whatever the sums
        // say then, rows and heads stay within the arrays)
        q = Req{start_of[0], min(start_of[1], a.T - start_of[0]), start_of[2]};
        at = start_at;
        if (q.n <= 2 * a.toks) {
          const unsigned one = max(work_of(a, q, 0), 1u);
          h = at / one;
          at -= h * one;
        } else {
          // 32 units at a time: the sum of a head's, then the unit
          unsigned sum = 0;
#pragma unroll 1
          for (int b = 0; b < q.n; b += 64 * a.toks) sum += __reduce_add_sync(0xffffffffu, work_of(a, q, b + lane * 2 * a.toks));
          h = at / max(sum, 1u);
          at -= h * sum;
#pragma unroll 1
          for (bool found = false; !found && i < q.n;) {
            const unsigned v = work_of(a, q, i + lane * 2 * a.toks);
            unsigned upto = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
              if (lane >= o) upto += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > at);
            found = past != 0;
            const int l = found ? __ffs(past) - 1 : 31;
            at -= __shfl_sync(0xffffffffu, found ? upto - v : upto, l);
            i += (found ? l : 32) * 2 * a.toks;
          }
        }
        if ((unsigned)h >= (unsigned)a.Hkv) left = 0;
      }
      auto advance = [&] {  // to the next unit
        at = 0;
        i += 2 * a.toks;
        if (i < q.n) return;
        i = 0;
        if (++h < a.Hkv) return;
        h = 0;
        if (left > 0 && ++r < a.n_req) q = request(a, r);
        else left = 0;
      };
      int tail = KT, tail_at = 0;  // of the item before
#pragma unroll 1
      while (ok) {
        int k0 = 0, k1 = 0, part = -1;
#pragma unroll 1
        while (left > 0) {  // the next unit's piece; a cut may leave no whole tile of it
          const unsigned all = work_of(a, q, i);
          if (at < all) {
            const bool two = two_tiles(a, q, i);
            const unsigned end = at + min(left, all - at);
            const int tiles = key_tiles(a, q, i);
            k0 = tile_at(at, two);
            k1 = tile_at(end, two);
            part = k0 == 0 && k1 == tiles ? -1 : 2 * (int)blockIdx.x + (k0 == 0);
            if (k0 == 0 && 0 < k1 && k1 < tiles) split = Split{end, all, piece, q.row0, q.n, q.kv, i, h, two, {}};
            left -= end - at;
            if (k0 < k1) break;
          }
          advance();
        }
        const int s = items & 1;
        if (!(ok = wait_warp(work_free + s, ((items >> 1) & 1) ^ 1))) break;
        if (lane == 0) {
          work[s * 3] = make_int4(q.row0, k0 < k1 ? q.n : 0, q.kv, i);
          work[s * 3 + 1] = make_int4(h, k0, k1, part);
          work[s * 3 + 2] = make_int4(r, 0, 0, 0);
          tc::mbar_arrive(work_full + s);
        }
        ++items;
        // The item before, whose tail the next one's loads need not wait for.  Once its
        // loads are issued the slot's barrier is in their phase or the one before;
        // of the barriers that say so, two in turn, none is asked two phases late.
        if (items > 1 && !(ok = wait_warp(issued + (items & 1), ((items - 2) >> 1) & 1))) break;
        if (tail < KT) {
          const int slot = tail_at % SLOTS;
          if (!(ok = wait_warp(full + slot, (tail_at / SLOTS) & 1))) break;
          zero_keys<D>(sm + F::OFF_KV + slot * TILE_BYTES<D>, tail);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(v_tail + slot);
        }
        if (k0 >= k1) break;
        ring += 2 * (k1 - k0);
        tail = min(q.kv - (k1 - 1) * KT, KT);
        tail_at = ring - 1;
        advance();
      }
      if (lane == 0) {
        a.split[blockIdx.x] = split;
        a.tasks[blockIdx.x] = split.n ? tasks_of<D>(a, split) : 0;
      }
    }
  } else {
    const int j = warp >> 2, r = (warp & 3) * 32 + lane;  // group, row of its tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + F::O_COL + j * D + lanes;
    const float sl2 = a.scale * LOG2E;
    const int tok_of = r / a.G, head_of = r % a.G;
    unsigned turns = 0;  // parity of each buffer's blocks so far
    int outs = 0, done = 0, meets = 0;  // the group's blocks, items and meetings so far
    auto meet = [&] {  // with the other group's warp of these rows
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(met + (warp & 3));
      const bool there = wait_warp(met + (warp & 3), meets++ & 1);
      tc::fence_after_sync();
      return there;
    };
    for (int i = 0; ok && next_item(work, work_full, work_free, i, w, ok); ++i) {
      const Item t(w);
      const bool one = t.one(a);
      const int tile = one ? 0 : j, n = t.tokens(a, tile), nb = t.blocks(a, j), row = tile * a.toks * a.G + r;
      const bool mine = tok_of < n, any = (warp & 3) * 32 < n * a.G;  // the thread's row, the warp's
      if (!nb && !one) {
        if (t.part >= 0 && mine) a.stat[(size_t)t.part * a.rows + row] = make_float2(0.f, 0.f);
        continue;
      }
      const int first = t.tok0 + tile * a.toks, tok = first + tok_of;
      const int see = last_key(a, t.q, tok), least = last_key(a, t.q, first);
      float ref = 0.f, ref2 = 0.f, l = 0.f;    // the exponentials' reference, also times sl2; their sum
#pragma unroll 1
      for (int b = 0; b < nb; ++b, ++outs) {
        const uint32_t ts = tmem + j * 128 + (b & 1) * 64 + lanes;
        if (!(ok = wait_warp(s_full + j * 2 + (b & 1), turns >> (b & 1) & 1))) break;
        turns ^= 1u << (b & 1);
        tc::fence_after_sync();
        if (any) {
          uint32_t u[64];
          tc::tmem_ld32_nowait(ts, u);
          tc::tmem_ld32_nowait(ts + 32, u + 32);
          tc::tmem_wait_ld();
          const int key0 = (2 * t.k0 + (one ? 2 * b + j : b)) * 64;
          if (key0 + 63 > least) {  // some row does not read all of these keys
            const int last = see - key0;
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
            const bool grow = mine && (mx - ref) * sl2 > GROW;
            if (__any_sync(0xffffffffu, grow)) {
              // the last block's P V; these scores vouch for the one before it, and
              // the next one waits for this block's P, so the parity is unambiguous
              if (!(ok = wait_warp(o_full + j, (outs - 1) & 1))) break;
              tc::fence_after_sync();
              // a row whose reference stays, beside one whose grows (which may be of the
              // next request), keeps its bits: the products are rounded by themselves,
              // not in a fused multiply-add, so that its factor is 2^0
              const float to_new = grow ? mx : ref, to_new2 = __fmul_rn(to_new, sl2);
              const float f = tc::ex2(ref2 - to_new2);
              ref = to_new;
              ref2 = to_new2;
              l *= f;
#pragma unroll 1
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
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(p_full + j * 2 + (b & 1));
      }
      if (!ok || (nb && !(ok = wait_warp(o_done + j, done++ & 1)))) break;
      tc::fence_after_sync();
      if (!any) continue;
      // The row's O (its columns c0 .. c1 - 1 in this thread), sum and reference.  A tile
      // that both groups took: the two warps of these rows tell one another theirs, and each
      // joins half of the columns from both groups' O, which lie in the same lanes.
      int c0 = 0, c1 = D;
      float own = 1.f, other = 0.f;
      if (one) {
        chain[j][r] = make_float2(ref2, l);
        if (!(ok = meet())) break;
        const float2 x = chain[j ^ 1][r];
        const float top = l == 0.f ? x.x : x.y == 0.f ? ref2 : fmaxf(ref2, x.x);
        own = l == 0.f ? 0.f : tc::ex2(ref2 - top);
        other = x.y == 0.f ? 0.f : tc::ex2(x.x - top);
        l = j ? other * x.y + own * l : own * l + other * x.y;  // in one order
        ref2 = top;
        c0 = j * (D / 2);
        c1 = c0 + D / 2;
      }
      const float inv = t.part >= 0 ? 1.f : 1.f / l;
      const size_t at = (size_t)t.q.row0 + tok, head = t.head * a.G + head_of;
      const bool out = mine && (t.part >= 0 || see >= 0);
      float4* part = a.part + (size_t)max(t.part, 0) * (D / 4) * a.rows + row;
      bf16* dst = a.o + (at * a.Hq + head) * D;
#pragma unroll 1
      for (int x0 = c0; x0 < c1; x0 += 32) {  // (unrolled, a call of few keys would wait for its instructions)
        uint32_t x[32];
        tc::tmem_ld32_nowait(to + x0, x);
        if (one) {
          uint32_t y[32];
          tc::tmem_ld32_nowait(to + (j ? -D : D) + x0, y);
          tc::tmem_wait_ld();
          // (a group none of whose keys the row reads has nothing there)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float u = own == 0.f ? 0.f : own * __uint_as_float(x[e]);
            const float v = other == 0.f ? 0.f : other * __uint_as_float(y[e]);
            x[e] = __float_as_uint(u + v);
          }
        } else {
          tc::tmem_wait_ld();
        }
        if (out) {
          if (t.part >= 0) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              part[(size_t)(x0 / 4 + g) * a.rows] = make_float4(__uint_as_float(x[4 * g]), __uint_as_float(x[4 * g + 1]),
                                                                __uint_as_float(x[4 * g + 2]), __uint_as_float(x[4 * g + 3]));
          } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack2(__uint_as_float(x[g * 8 + 2 * e]) * inv, __uint_as_float(x[g * 8 + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + x0 + g * 8) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
      }
      if (out && c0 == 0) {
        if (t.part >= 0) a.stat[(size_t)t.part * a.rows + row] = make_float2(ref2, l);
        else a.lse[head * a.T + at] = (ref2 + log2f(l)) * LN2;
      }
      if (one && !(ok = meet())) break;  // the other group's next P V waits for its own warps only
      tc::fence_before_sync();  // O has been read before the next item's P V, which waits for its P
    }
  }
  tc::grid_dep_launch();  // the join's CTAs start as SMs fall free, and wait for this grid's end
  if (!ok) atomicAdd(&g_gave_up, 1u);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == SW + 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the units that cuts divide: the part of the CTA that began
// the unit, then the first one of each CTA behind it.  A task is some columns (eight a
// thread) of a unit's rows; warps share a task's parts where there are many.  A
// thread has BATCH parts' loads in flight: 4 for short calls, which wait for one
// chain of loads (one token 11.5 us with 4, 12.1 with 2), and 2 for long ones, whose
// parts want the loads of four CTAs an SM (two chunks of 2,048 rows 133.2 us with 2,
// 136.7 with 4).
template <int D, int BATCH>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 8 / BATCH) attn_paged_join_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ int ends[256 + 1];  // tasks of the units before
  __shared__ float sums[JOIN_WARPS][10][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  static_assert(GRID <= 256, "a thread takes a split");
  // Long calls read the counts first and a task's split later: 608 CTAs that read all
  // splits wait for one another's cache lines (16 draft windows 21.4 us, 19.8 so); short
  // ones would wait for one load more (64 tokens 51.3 us, 50.8 so).
  constexpr bool AHEAD = BATCH == 4;
  __shared__ Split splits[AHEAD ? GRID : 1];
  int count = 0;
  if (tid < GRID) {
    if constexpr (AHEAD) {
      const Split s = a.split[tid];
      splits[tid] = s;
      if (s.n) count = tasks_of<D>(a, s);
    } else {
      count = a.tasks[tid];
    }
  }
  __shared__ int warp_sums[JOIN_WARPS];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, count, o);
    if (lane >= o) count += v;
  }
  if (lane == 31) warp_sums[warp] = count;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < JOIN_WARPS; ++v) count += v < warp ? warp_sums[v] : 0;
  ends[tid + 1] = count;
  if (tid == 0) ends[0] = 0;
  __syncthreads();
  for (int task = blockIdx.x; task < ends[GRID]; task += JOIN_CTAS) {
    int c = 0;
#pragma unroll 1
    for (int step = 128; step; step >>= 1)
      if (c + step < GRID && ends[c + step] <= task) c += step;
    const Split s = AHEAD ? splits[AHEAD ? c : 0] : a.split[c];
    const int n = parts_of(s), share = share_of(n), g = warp % share, rows = rows_of(a, s);
    const int id = (task - ends[c]) * (32 * JOIN_WARPS / share) + warp / share * 32 + lane, row = id % rows, c8 = id / rows;
    const Req q{s.row0, s.n, s.kv};
    const int tok = s.tok0 + row / a.G;
    const bool out = c8 < D / 8 && last_key(a, q, tok) >= 0;
    float top = -INFINITY, sum = 0.f, acc[8] = {};
    if (out) {
#pragma unroll 1
      for (int p0 = g; p0 < n; p0 += BATCH * share) {
        float2 st[BATCH];
        float4 x[BATCH], y[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const int p = p0 + e * share;
          // (a piece may hold none of the unit's tiles)
          const unsigned from = s.after + (p - 1) * s.piece, to = from + min(s.piece, s.work - from);
          const bool there = p < n && c + p < GRID && (p == 0 || tile_at(from, s.two) < tile_at(to, s.two));
          const size_t at = p == 0 ? 2 * c + 1 : 2 * (c + p);
          st[e] = there ? a.stat[at * a.rows + row] : make_float2(0.f, 0.f);
          const float4* src = a.part + (at * (D / 4) + 2 * c8) * a.rows + row;
          x[e] = y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (there) {
            x[e] = src[0];
            y[e] = src[a.rows];
          }
        }
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          if (st[e].y == 0.f) continue;  // none of the part's keys is the row's: it holds nothing
          const float to = fmaxf(top, st[e].x), f = tc::ex2(st[e].x - to), k = top == -INFINITY ? 0.f : tc::ex2(top - to);
          top = to;
          sum = sum * k + f * st[e].y;
          const float v[8] = {x[e].x, x[e].y, x[e].z, x[e].w, y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = acc[i] * k + f * v[i];
        }
      }
    }
    if (share > 1) {
      __syncthreads();
      sums[warp][8][lane] = sum;
      sums[warp][9][lane] = top;
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[warp][i][lane] = acc[i];
      __syncthreads();
      if (g == 0)
#pragma unroll 1
        for (int w = 1; w < share; ++w) {
          const float l = sums[warp + w][8][lane], m = sums[warp + w][9][lane];
          if (l == 0.f) continue;
          const float to = fmaxf(top, m), f = tc::ex2(m - to), k = top == -INFINITY ? 0.f : tc::ex2(top - to);
          top = to;
          sum = sum * k + f * l;
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = acc[i] * k + f * sums[warp + w][i][lane];
        }
    }
    if (out && g == 0) {
      const float inv = 1.f / sum;
      const size_t at = (size_t)s.row0 + tok, head = s.head * a.G + row % a.G;
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = pack2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      *reinterpret_cast<uint4*>(a.o + (at * a.Hq + head) * D + c8 * 8) = make_uint4(h[0], h[1], h[2], h[3]);
      if (c8 == 0) a.lse[head * a.T + at] = (top + log2f(sum)) * LN2;
    }
  }
}

// Rows of a part: two tiles of tokens, or all there are.
inline int part_rows(int T, int G) {
  const int toks = 2 * (128 / G);
  return (toks < T ? toks : T > 0 ? T : 1) * G;
}
inline size_t part_bytes(int rows, int d) { return ((size_t)2 * GRID * rows * d * 4 + 255) / 256 * 256; }
inline size_t stat_bytes(int rows) { return ((size_t)2 * GRID * rows * 8 + 255) / 256 * 256; }

template <int D> int attend(const CUtensorMap* m, const PagedArgs& a, cudaStream_t s) {
  using F = Lay<D>;
  if (!kernel_smem_at_least(reinterpret_cast<const void*>(&attn_paged_kernel<D>), F::SMEM))
    return op_fail(GOCR_ECUDA, "kernel configuration rejected");
  launch_k(attn_paged_kernel<D>, dim3(GRID), dim3(THREADS), F::SMEM, s, true, m[0], m[1], m[2], a);
  if (int rc = op_launched("attention_paged")) return rc;
  launch_k(a.T < 8 * a.toks ? attn_paged_join_kernel<D, 4> : attn_paged_join_kernel<D, 2>, dim3(JOIN_CTAS),
           dim3(JOIN_WARPS * 32), 0, s, true, a);
  return op_launched("attention_paged's join");
}

// K or V as TMA sees it: a box is all columns of the keys of a page that a tile
// holds, in groups of 8.  A box's page and head share one dimension, whose stride is the
// largest that both strides are multiples of.
struct PageMap {
  const void* p;
  int64_t token, unit, page, head, units;  // strides in elements; page and head strides in units, and units in all
  PageMap(const void* p, const int64_t* st, const gocr_paged_kv& kv)
      : p(p), token(st[2]), unit(std::gcd(st[0], st[1])), page(st[0] / unit), head(st[1] / unit),
        units((kv.n_pages - 1) * page + (kv.n_kv_heads - 1) * head + 1) {}
  bool encode(CUtensorMap* m, const gocr_paged_kv& kv) const {
    const unsigned long long dims[5] = {64, 8, (unsigned long long)kv.head_dim / 64, (unsigned long long)kv.page_size / 8,
                                        (unsigned long long)units};
    const unsigned long long strides[4] = {(unsigned long long)token * 2, 128, (unsigned long long)token * 16,
                                           (unsigned long long)unit * 2};
    const unsigned box[5] = {64, 8, (unsigned)kv.head_dim / 64, (unsigned)(kv.page_size < KT ? kv.page_size : KT) / 8, 1};
    return encode_tmap(m, p, false, 5, dims, strides, box);
  }
};

// The same over q: boxes of 64 columns x the G heads of a kv head x the tokens of a tile.
bool map_queries(CUtensorMap* m, const void* p, int T, int Hq, int G, int D, long long ld) {
  const unsigned long long dims[3] = {(unsigned long long)D, (unsigned long long)Hq, (unsigned long long)T};
  const unsigned long long st[2] = {(unsigned long long)D * 2, (unsigned long long)ld * 2};
  const unsigned box[3] = {64, (unsigned)G, (unsigned)(128 / G)};
  return encode_tmap(m, p, false, 3, dims, st, box);
}

}  // namespace

namespace gocr {
cudaError_t attn_paged_gave_up(unsigned* out, cudaStream_t s) {
  return cudaMemcpyFromSymbolAsync(out, g_gave_up, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, s);
}
}  // namespace gocr

extern "C" size_t gocr_op_attention_paged_workspace(int T, int Hq, int Hkv, int d) {
  if (T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 64 || d < 1) return 0;
  const int rows = part_rows(T, Hq / Hkv);
  return part_bytes(rows, d) + stat_bytes(rows) + GRID * (sizeof(Split) + sizeof(int));
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
  if (T < 0 || T > MAX_ROWS || Hq < 1 || Hq > 1024 || Hq % Hkv || Hq / Hkv > 64 || (long long)T * Hq > 0x7fffffffLL)
    return op_fail(GOCR_EINVAL, "bad shape: T=%d Hq=%d Hkv=%d", T, Hq, Hkv);
  if (!pitch_ok(ldq, Hq, d)) return op_fail(GOCR_EINVAL, "bad row pitch %lld", ldq);
  if (!(scale > 0.f) || scale > 1e30f) return op_fail(GOCR_EINVAL, "bad scale");
  if (!cu_rows || (n_req && (!table || !kv_len)) || (T && (!q || !o || !lse)) || !workspace)
    return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)q | (uintptr_t)o | (uintptr_t)workspace) & 15) return op_fail(GOCR_EINVAL, "operand not 16-byte aligned");
  if (((uintptr_t)table | (uintptr_t)cu_rows | (uintptr_t)kv_len | (uintptr_t)lse) & 3)
    return op_fail(GOCR_EINVAL, "array not 4-byte aligned");
  if (workspace_bytes < gocr_op_attention_paged_workspace(T, Hq, Hkv, d)) return op_fail(GOCR_ECAPACITY, "workspace too small");
  const int G = Hq / Hkv, rows = part_rows(T, G);
  // the work of a call, at most 5 a key tile and 16 for each unit, is counted in 32 bits
  const long long units = (T / (2 * (128 / G)) + (long long)(T < n_req ? T : n_req)) * Hkv;
  if (units * (((long long)max_pages * kv.page_size - 1) / KT + 5) > 1 << 29)
    return op_fail(GOCR_EINVAL, "bad shape: T=%d rows of %d requests over %d pages of %d", T, n_req, max_pages, kv.page_size);
  const PageMap km(kv.k, &kv.k_page, kv), vm(kv.v, &kv.v_page, kv);
  if (km.units > 0x7fffffff || vm.units > 0x7fffffff)
    return op_fail(GOCR_EINVAL, "bad cache strides: %d pages whose strides have no common unit", kv.n_pages);
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  if (!T || !n_req) return GOCR_OK;
  CUtensorMap m[3];
  if (!map_queries(&m[0], q, T, Hq, G, d, ldq) || !km.encode(&m[1], kv) || !vm.encode(&m[2], kv))
    return op_fail(GOCR_ECUDA, "a TMA descriptor was rejected");
  int shift = 4;
  while ((1 << shift) < kv.page_size) ++shift;
  uint8_t* ws = (uint8_t*)workspace;
  const PagedArgs a{table, cu_rows, kv_len, (bf16*)o, lse, (float4*)ws, (float2*)(ws + part_bytes(rows, d)),
                    (Split*)(ws + part_bytes(rows, d) + stat_bytes(rows)),
                    (int*)(ws + part_bytes(rows, d) + stat_bytes(rows) + GRID * sizeof(Split)), max_pages, kv.n_pages, n_req, T, Hq, Hkv, G,
                    128 / G, kind == GOCR_FWD_DRAFT, shift, rows, (int)km.page, (int)km.head, (int)km.units, (int)vm.page,
                    (int)vm.head, (int)vm.units, scale};
  return d == 128 ? attend<128>(m, a, s) : attend<64>(m, a, s);
}
