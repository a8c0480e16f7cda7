// nq_kv_plan.cu — block tables and slots of a step's tokens from request lengths.
//
// Request b holds c_b tokens and gains n_b.  With pages of P tokens it has
// ceil(c_b / P) pages and needs ceil((c_b + n_b) / P); the difference is taken
// from the free list in request order, so its first entry is the exclusive
// sum of the differences before it.  Token i of request b has position c_b + i
// and slot page(position / P) * P + position % P.
//
// One launch: every CTA scans the requests' lengths itself (both sums at once)
// into shared memory, then takes its share of the tokens and of the new table
// entries, finding their request by bisection.  The sums stay at 2^32 - 1 once
// they get there, so that they never fall and lengths that do not fit are cut
// like any others.  A slot in a
// page that this very call allocates is read from the free list, never from
// the table, so the CTAs need no order among themselves.  A second launch that
// reads the finished sums would cost more than the repeated scan: the step is
// bound by latency (two dependent loads, a scan, a store) at the usual sizes.
#include "nq_device.cuh"
#include "nq_kv.h"

namespace nq {

namespace {

// Sums of tokens and pages.
struct Sums {
  uint32_t tokens, pages;
};
__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b) { return a + b < a ? 0xffffffffu : a + b; }
__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {add_up(a.tokens, b.tokens), add_up(a.pages, b.pages)}; }
__device__ __forceinline__ Sums shift_up(Sums a, int lanes) {
  return {__shfl_up_sync(kFull, a.tokens, lanes), __shfl_up_sync(kFull, a.pages, lanes)};
}
__device__ __forceinline__ Sums from_lane(Sums a, int lane) {
  return {__shfl_sync(kFull, a.tokens, lane), __shfl_sync(kFull, a.pages, lane)};
}

struct Request {
  int32_t cached, tokens, have, pages;  // tokens that get a row, pages held, pages gained
};

__device__ __forceinline__ Request request_of(const KvPlanArgs& a, int b, bool* bad) {
  int64_t c = a.cached[b], n = a.added[b];
  if (c < 0 || n < 0) *bad = true;
  c = c < 0 ? 0 : c;
  n = n < 0 ? 0 : n;
  const int64_t room = int64_t(a.width) << a.log_page;  // tokens a table row can address
  if (c + n > room) *bad = true;
  const int P1 = (1 << a.log_page) - 1;
  const int64_t have = min((c + P1) >> a.log_page, int64_t(a.width));
  const int64_t need = min((c + n + P1) >> a.log_page, int64_t(a.width));
  return {int32_t(c), int32_t(n), int32_t(have), int32_t(need - have)};
}

// Most pages that one call lays out.
constexpr uint32_t kMostPages = 0x7fffffffu;

// Largest i in [0, n) with s[i] <= x, for s[0] <= x and s not decreasing.
__device__ __forceinline__ int last_not_above(const int32_t* s, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kKvPlanThreads) plan_kernel(const KvPlanArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* first_token = smem;           // [B + 1]
  int32_t* first_page = smem + a.B + 1;  // [B + 1]
  int32_t* cached = first_page + a.B + 1;  // [B]
  __shared__ Sums warp_sum[kKvPlanThreads / 32];
  constexpr int kItems = 4;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;

  griddep_wait();
  griddep_launch_dependents();
  const int32_t head = a.free_head[0];
  bool bad = head < 0;
  Sums carry = {0, 0};
  for (int base = 0; base < a.B; base += kKvPlanThreads * kItems) {
    Sums item[kItems], sum = {0, 0};
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int b = base + tid * kItems + i;
      item[i] = {0, 0};
      if (b < a.B) {
        const Request r = request_of(a, b, &bad);
        item[i] = {uint32_t(r.tokens), uint32_t(r.pages)};
        cached[b] = r.cached;
      }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) sum = sum + item[i];
    auto scan = [&](Sums x, int lanes) {
#pragma unroll
      for (int o = 1; o < lanes; o <<= 1) {
        const Sums up = shift_up(x, o);
        if (lane >= o) x = x + up;
      }
      return x;
    };
    const Sums incl = scan(sum, 32), left = shift_up(incl, 1);  // `left`: of the lanes before
    if (base) __syncthreads();  // warp_sum of the previous pass has been read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    // Over the warps in every warp again (a loop over their sums took 0.3 us more).
    constexpr int kWarps = kKvPlanThreads / 32;
    const Sums warps = scan(lane < kWarps ? warp_sum[lane] : Sums{0, 0}, kWarps);
    const Sums all = carry + from_lane(warps, kWarps - 1), warps_before = from_lane(warps, warp - 1);
    Sums before = warp > 0 ? carry + warps_before : carry;
    if (lane > 0) before = before + left;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int b = base + tid * kItems + i;
      if (b < a.B) {
        first_token[b] = int32_t(min(before.tokens, uint32_t(a.T)));
        first_page[b] = int32_t(min(before.pages, kMostPages));
      }
      before = before + item[i];
    }
    carry = all;
  }
  const int32_t pages = int32_t(min(carry.pages, kMostPages));
  if (carry.tokens > uint32_t(a.T) || int64_t(head) + carry.pages > a.n_free) bad = true;
  if (tid == 0) {
    first_token[a.B] = int32_t(min(carry.tokens, uint32_t(a.T)));
    first_page[a.B] = pages;
  }
  __syncthreads();
  if (blockIdx.x == 0 && bad) atomicOr(a.err, kErrPlan);

  const int step = int(gridDim.x) * kKvPlanThreads, me = int(blockIdx.x) * kKvPlanThreads + tid;
  auto fresh = [&](int64_t i) {  // i-th page that this call takes; -1 past the list's end
    const int64_t at = head + i;
    return at >= 0 && at < a.n_free ? a.free_pages[at] : -1;
  };
  auto held = [&](int b) {  // pages that request b holds
    return int(min((int64_t(cached[b]) + (1 << a.log_page) - 1) >> a.log_page, int64_t(a.width)));
  };
  for (int b = me; b <= a.B; b += step) {
    a.cu_q[b] = first_token[b];
    if (b < a.B) {
      bool unused = false;
      const Request r = request_of(a, b, &unused);
      a.kv_lens[b] = int32_t(min(int64_t(r.cached) + r.tokens, int64_t(a.width) << a.log_page));
    } else {
      *a.free_head_out = max(head, int32_t(min(int64_t(head) + pages, int64_t(a.n_free))));
    }
  }
  for (int64_t f = me; f < pages; f += step) {  // 64 bits: the step behind the last one may pass 2^31
    const int b = last_not_above(first_page, a.B, int32_t(f));
    const int64_t column = held(b) + f - first_page[b];
    if (column < a.width) a.table[b * a.ld_table + column] = fresh(f);  // always, unless pages were cut
  }
  const int32_t mask = (1 << a.log_page) - 1;
  for (int64_t t = me; t < a.T; t += step) {
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < first_token[a.B]) {
      const int b = last_not_above(first_token, a.B, int32_t(t));
      const int64_t at = int64_t(cached[b]) + (t - first_token[b]);
      const int64_t p = at >> a.log_page;
      pos = int32_t(min(at, int64_t(0x7fffffff)));
      if (p < a.width) {
        const int have = held(b);
        const int32_t page = p < have ? a.table[b * a.ld_table + p] : fresh(int64_t(first_page[b]) + (p - have));
        if (page >= 0) slot = (int64_t(page) << a.log_page) + (at & mask);
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

}  // namespace

const void* kv_plan_kernel() { return reinterpret_cast<const void*>(&plan_kernel); }

}  // namespace nq
