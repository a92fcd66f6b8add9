// Block tables, positions and slots of the next forward, from request lengths.
//
//   have = ceil(held / ps), want = ceil(end / ps); back = max(have - want, 0), need = max(want - have, 0)
//   F = sum of back, S = n_free + F: page f given back -> stack[S - 1 - f], page k needed <- stack[S - 1 - k]
//
// Every output is a function of the inputs: a page that one request gives back
// and another takes in the same call is read from the first one's table row, not
// from the stack, and the stack is read below *n_free and written at and above it.
// So CTAs need not wait for one another: each scans all lengths (three prefix sums, kept
// in shared memory) and does its share of the rows, of the pages taken and of
// those given back, finding the request of each by bisection.  A call is a chain of
// loads, scans and bisections, whatever it moves: 16 windows of 33 rows 3.4 us, 64
// prompts of 1,537 4.4, 1,000 requests of which a third shrink or end 6.7.
#include "paged.cuh"
#include "tc.cuh"

using namespace gocr;
using namespace gocr::paged;

namespace {

constexpr int THREADS = 256;
constexpr size_t STATIC_SMEM = THREADS / 32 * sizeof(int);  // the scans' sums of warps
constexpr int MOST = (1 << 30) - 1;  // sums end here: above every count that can be served, and 2 * MOST fits an int

struct StepArgs {
  const int *held, *start, *end, *n_free;
  int *table, *free_pages, *n_free_out, *held_out, *kv_len, *cu_rows, *pos, *slots;
  int n_req, max_pages, shift, n_pages, T;
};

__device__ __forceinline__ int add(int a, int b) { return min(a + b, MOST); }

// Exclusive sum over the CTA's threads of v (sums end at MOST), and the total.
__device__ __forceinline__ int scan(int v, int* sums, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = add(inc, x);
  }
  if (lane == 31) sums[warp] = inc;
  const int up = __shfl_up_sync(0xffffffffu, inc, 1);
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before = add(before, sums[w]);
    total = add(total, sums[w]);
  }
  __syncthreads();
  return lane ? add(before, up) : before;
}

// The last r < n with a[r] <= x; a does not decrease and a[0] <= x.
__device__ __forceinline__ int find(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m;
    else hi = m;
  }
  return lo;
}

__global__ void __launch_bounds__(THREADS) page_step_kernel(const StepArgs a) {
  extern __shared__ int sh[];
  __shared__ int sums[THREADS / 32];
  const int R = a.n_req, tid = threadIdx.x, cap = a.max_pages << a.shift, round = (1 << a.shift) - 1;
  tc::grid_dep_launch();  // the next kernel's beginning overlaps this one, this one's the last one's
  tc::grid_dep_wait();
  int *rows = sh, *need = sh + R + 1, *back = need + R + 1;  // sums over the requests before
  const int per = (R + THREADS - 1) / THREADS, r0 = min(tid * per, R), r1 = min(r0 + per, R);
  auto sane = [&](int h, int s, int e) { return 0 <= s && s <= h && s <= e && h <= cap && e <= cap; };

  int sum = 0, total;
  for (int r = r0; r < r1; ++r) {
    const int s = a.start[r], e = a.end[r];
    const int n = sane(a.held[r], s, e) ? e - s : 0;
    rows[r + 1] = n;
    sum = add(sum, n);
  }
  int at = scan(sum, sums, total);
  int n_need = 0, n_back = 0;
  for (int r = r0; r < r1; ++r) {
    at = add(at, rows[r + 1]);
    rows[r + 1] = at;  // rows behind T are nobody's: a request that has some is refused
    const int h = a.held[r], e = a.end[r];
    const int d = sane(h, a.start[r], e) && at <= a.T ? ((e + round) >> a.shift) - ((h + round) >> a.shift) : 0;
    need[r + 1] = max(d, 0);
    back[r + 1] = max(-d, 0);
    n_need = add(n_need, max(d, 0));
    n_back = add(n_back, max(-d, 0));
  }
  int F, all;
  n_need = scan(n_need, sums, all);
  n_back = scan(n_back, sums, F);
  for (int r = r0; r < r1; ++r) {
    need[r + 1] = n_need = add(n_need, need[r + 1]);
    back[r + 1] = n_back = add(n_back, back[r + 1]);
  }
  if (tid == 0) rows[0] = need[0] = back[0] = 0;
  __syncthreads();

  const int nf = min(max(*a.n_free, 0), a.n_pages), S = min(nf + F, a.n_pages);
  // whether request r gets what it asks for: needs up to and with its own that there are pages for
  auto served = [&](int r) {
    return rows[r + 1] <= a.T && sane(a.held[r], a.start[r], a.end[r]) && (need[r + 1] == need[r] || need[r + 1] <= S);
  };
  // page f given back
  auto given = [&](int f) {
    const int r = find(back, R, f);
    return a.table[(size_t)r * a.max_pages + ((a.end[r] + round) >> a.shift) + f - back[r]];
  };
  // page k needed
  auto taken = [&](int k) {
    const int i = S - 1 - k;
    return i >= nf ? given(S - 1 - i) : a.free_pages[i];
  };
  const int step = gridDim.x * THREADS, first = blockIdx.x * THREADS + tid;
  // needs that are served: up to the first request whose need is not
  int takes = min(all, S);
  if (takes > 0 && all > S) takes = need[find(need, R + 1, S)];
  for (int t = first; t < a.T; t += step) {
    int x = -1, slot = -1;
    if (t < rows[R]) {
      const int r = find(rows, R, t);
      if (served(r)) {
        x = a.start[r] + t - rows[r];
        const int i = x >> a.shift, have = (a.held[r] + round) >> a.shift;
        const int page = i < have ? a.table[(size_t)r * a.max_pages + i] : taken(need[r] + i - have);
        if (page >= 0 && page < a.n_pages) slot = (page << a.shift) + (x & round);
      }
    }
    a.pos[t] = x;
    a.slots[t] = slot;
  }
  for (int k = first; k < takes; k += step) {
    const int r = find(need, R, k);
    a.table[(size_t)r * a.max_pages + ((a.held[r] + round) >> a.shift) + k - need[r]] = taken(k);
  }
  for (int f = first; f < S - nf; f += step) a.free_pages[S - 1 - f] = given(f);
  for (int r = first; r <= R; r += step) {
    a.cu_rows[r] = min(rows[r], a.T);
    if (r == R) break;
    const bool ok = served(r);
    a.held_out[r] = ok ? a.end[r] : a.held[r];
    a.kv_len[r] = ok ? a.end[r] : 0;
  }
  if (first == 0) *a.n_free_out = S - takes;
}

}  // namespace

extern "C" int gocr_op_page_step(const int32_t* held, const int32_t* start, const int32_t* end, int n_req,
                                 int32_t* table, int max_pages, int page_size, int32_t* free_pages, int n_pages,
                                 const int32_t* n_free, int32_t* n_free_out, int32_t* held_out, int32_t* kv_len,
                                 int32_t* cu_rows, int32_t* pos, int32_t* slots, int T, void* stream) {
  if (int rc = table_check(n_req, max_pages, page_size, n_pages)) return rc;
  if (T < 0 || T > MAX_ROWS) return op_fail(GOCR_EINVAL, "bad shape: T=%d", T);
  if (!free_pages || !n_free || !n_free_out || !cu_rows ||
      (n_req && (!held || !start || !end || !table || !held_out || !kv_len)) || (T && (!pos || !slots)))
    return op_fail(GOCR_EINVAL, "null pointer");
  if (((uintptr_t)held | (uintptr_t)start | (uintptr_t)end | (uintptr_t)table | (uintptr_t)free_pages | (uintptr_t)n_free |
       (uintptr_t)n_free_out | (uintptr_t)held_out | (uintptr_t)kv_len | (uintptr_t)cu_rows | (uintptr_t)pos |
       (uintptr_t)slots) & 3)
    return op_fail(GOCR_EINVAL, "array not 4-byte aligned");
  cudaStream_t s = (cudaStream_t)stream;
  if (int rc = op_stream_check(s)) return rc;
  int shift = 4;
  while ((1 << shift) < page_size) ++shift;
  const StepArgs a{held, start, end, n_free, table, free_pages, n_free_out, held_out, kv_len, cu_rows, pos, slots,
                   n_req, max_pages, shift, n_pages, T};
  // up to two CTAs an SM; where there are fewer rows than pages to hand over, 16 pages a request
  const long long work = T > 16 * n_req ? T : 16ll * n_req;
  const int grid = (int)((work + THREADS - 1) / THREADS < 2 * SM_COUNT ? (work + THREADS - 1) / THREADS : 2 * SM_COUNT);
  const size_t smem = 3 * (size_t)(n_req + 1) * sizeof(int);
  // (the default limit of 48 KB counts the kernel's own 32 bytes, too)
  if (smem + STATIC_SMEM > 48 * 1024 && !kernel_smem_at_least(reinterpret_cast<const void*>(&page_step_kernel), smem))
    return op_fail(GOCR_ECUDA, "kernel configuration rejected");
  launch_k(page_step_kernel, dim3(grid > 0 ? grid : 1), dim3(THREADS), smem, s, true, a);
  return op_launched("page_step");
}
