// nq_kv_plan.cu — block tables and slots of a step's tokens from request lengths.
//
// Request b holds c_b tokens and gains n_b.  With pages of P tokens it has
// ceil(c_b / P) pages and needs ceil((c_b + n_b) / P); the difference is taken
// from the free list in request order, so its first entry is the exclusive
// sum of the differences before it.  Token i of request b has position c_b + i
// and slot page(position / P) * P + position % P.
//
// One launch: every CTA scans the requests' lengths itself (both sums at once,
// packed in 64 bits) into shared memory, then takes its share of the tokens and
// of the new table entries, finding their request by bisection.  A slot in a
// page that this very call allocates is read from the free list, never from
// the table, so the CTAs need no order among themselves.  A second launch that
// reads the finished sums would cost more than the repeated scan: the step is
// bound by latency (two dependent loads, a scan, a store) at the usual sizes.
#include "nq_device.cuh"
#include "nq_kv.h"

namespace nq {

namespace {

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
  __shared__ uint64_t warp_sum[kKvPlanThreads / 32];
  constexpr int kItems = 4;
  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;

  griddep_wait();
  griddep_launch_dependents();
  const int32_t head = a.free_head[0];
  bool bad = head < 0;
  uint64_t carry = 0;  // tokens in the high half, pages in the low half
  for (int base = 0; base < a.B; base += kKvPlanThreads * kItems) {
    uint64_t item[kItems], sum = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int b = base + tid * kItems + i;
      item[i] = 0;
      if (b < a.B) {
        const Request r = request_of(a, b, &bad);
        item[i] = (uint64_t(uint32_t(r.tokens)) << 32) | uint32_t(r.pages);
        cached[b] = r.cached;
      }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) sum += item[i];
    uint64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    if (base) __syncthreads();  // warp_sum of the previous pass has been read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint64_t before = carry;
    uint64_t all = carry;
    for (int w = 0; w < kKvPlanThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    before += incl - sum;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int b = base + tid * kItems + i;
      if (b < a.B) {
        first_token[b] = int32_t(min(uint32_t(before >> 32), uint32_t(a.T)));
        first_page[b] = int32_t(uint32_t(before));
      }
      const uint64_t after = before + item[i];
      bad |= after < before || uint32_t(after) < uint32_t(before);  // more than 2^32 tokens or pages
      before = after;
    }
    carry = all;
  }
  const uint32_t tokens = uint32_t(carry >> 32);
  const int32_t pages = int32_t(uint32_t(carry));
  if (tokens > uint32_t(a.T) || int64_t(head) + uint32_t(pages) > a.n_free) bad = true;
  if (tid == 0) {
    first_token[a.B] = int32_t(min(tokens, uint32_t(a.T)));
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
      *a.free_head_out = head + pages;
    }
  }
  for (int f = me; f < pages; f += step) {
    const int b = last_not_above(first_page, a.B, f);
    const int64_t column = int64_t(held(b)) + f - first_page[b];
    if (column < a.width) a.table[b * a.ld_table + column] = fresh(f);  // always, unless the sums ran over
  }
  const int32_t mask = (1 << a.log_page) - 1;
  for (int t = me; t < a.T; t += step) {
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < first_token[a.B]) {
      const int b = last_not_above(first_token, a.B, t);
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
