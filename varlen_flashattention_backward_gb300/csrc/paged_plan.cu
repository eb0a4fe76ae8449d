// Block tables and slot maps from request lengths (fa_paged_plan).

#include "paged.h"

namespace fav {
namespace {

constexpr int kThreads = 1024;
constexpr int kPerThread = 2;   // requests per thread: kThreads * kPerThread = the largest batch

struct Sums {
  int64_t rows, need, give;
};

// What one request asks for, from its length and delta alone.
struct Ask {
  int64_t rows;      // packed rows
  int have, target;  // pages held, length wanted
  bool sound, grow, in_row;
};

__device__ __forceinline__ int pages_of(int64_t len, int page_size) {
  return int((len + page_size - 1) / page_size);
}

__device__ __forceinline__ Ask ask_of(const PlanParams &p, int len, int delta) {
  Ask a;
  const int64_t most = int64_t(p.max_pages) * p.page_size;
  a.rows = delta > 0 ? delta : 0;
  a.sound = len >= 0 && len <= most;
  a.grow = a.sound && delta > 0;
  int64_t target = int64_t(len) + delta;
  if (target < 0) target = 0;
  a.in_row = target <= most;
  a.target = int(a.in_row ? target : 0);
  a.have = a.sound ? pages_of(len, p.page_size) : 0;
  return a;
}

// Exclusive block-wide prefix of v over the threads; `total` gets the sum.
__device__ int64_t block_prefix(int64_t v, int64_t *buf, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t w = buf[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    buf[lane] = w;
  }
  __syncthreads();
  total = buf[31];
  const int64_t before = (warp ? buf[warp - 1] : 0) + x - v;
  __syncthreads();
  return before;
}

__device__ __forceinline__ int ring_at(const PlanParams &p, int64_t i) {
  return int(i >= p.num_pages ? i - p.num_pages : i);
}

// One CTA.  Phase 1: three block-wide prefix sums over the requests (rows,
// pages taken, pages given).  Phase 2: pages and slots, flat over all of
// them.  Phase 3: lengths and pool, which may be the inputs.
__global__ void __launch_bounds__(kThreads) plan_kernel(PlanParams p) {
  __shared__ int64_t buf[32];
  __shared__ int64_t s_row[kThreads * kPerThread + 1];   // first packed row of each request
  __shared__ int s_off[kThreads * kPerThread];           // first page taken or given
  __shared__ int s_len[kThreads * kPerThread];
  __shared__ uint8_t s_kind[kThreads * kPerThread];      // 1: granted, 2: shrinks
  const int tid = threadIdx.x;
  int err = 0;

  int len[kPerThread], delta[kPerThread];
  Ask a[kPerThread];
  int64_t rows = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    len[i] = b < p.batch ? p.lens[b] : 0;
    delta[i] = b < p.batch ? p.delta[b] : 0;
    a[i] = ask_of(p, len[i], delta[i]);
    rows += a[i].rows;
    if (!a[i].sound) err |= FA_PAGED_BAD_LENGTH;
    if (a[i].grow && !a[i].in_row) err |= FA_PAGED_ROW_FULL;
  }
  const int64_t head = p.state[0], count = p.state[1];
  int64_t total_rows, total_need, total_give;
  int64_t row = block_prefix(rows, buf, total_rows);

  int need[kPerThread], give[kPerThread];
  bool ask[kPerThread];
  int64_t needs = 0, gives = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    s_row[b] = row;
    row += a[i].rows;
    ask[i] = a[i].grow && a[i].in_row && row <= p.max_tokens;
    if (a[i].grow && a[i].in_row && !ask[i]) err |= FA_PAGED_ROWS;
    const int want = pages_of(a[i].target, p.page_size);
    need[i] = ask[i] ? want - a[i].have : 0;
    give[i] = a[i].sound && delta[i] < 0 ? a[i].have - want : 0;
    needs += need[i];
    gives += give[i];
  }
  if (tid == kThreads - 1) s_row[kThreads * kPerThread] = row;
  int64_t off_need = block_prefix(needs, buf, total_need);
  int64_t off_give = block_prefix(gives, buf, total_give);
  // Granted requests are a prefix of those that need pages, so their pages
  // start where the sum over all before them says.
  int64_t granted_pages = 0;
  bool granted[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    granted[i] = ask[i] && (need[i] == 0 || off_need + need[i] <= count);
    if (ask[i] && !granted[i]) err |= FA_PAGED_EXHAUSTED;
    if (granted[i]) granted_pages += need[i];
    s_off[b] = int(granted[i] ? off_need : off_give);
    s_len[b] = len[i];
    s_kind[b] = granted[i] ? 1 : (a[i].sound && delta[i] < 0) ? 2 : 0;
    off_need += need[i];
    off_give += give[i];
  }
  int64_t taken;
  block_prefix(granted_pages, buf, taken);
  // With room for all of them behind the end, the pages given back land on no
  // entry that this call takes.
  const bool whole = head >= 0 && head < p.num_pages && count >= 0 && count <= p.num_pages &&
                     count + total_give <= p.num_pages;
  if (!whole) err |= FA_PAGED_BAD_POOL;
  // Row starts of requests behind the batch equal the total, which s_row[batch]
  // then holds.
  for (int b = tid; b <= p.batch; b += kThreads) p.cu[b] = s_row[b];

  if (whole) {
    const int warp = tid >> 5, lane = tid & 31;
    for (int b = warp; b < p.batch; b += kThreads / 32) {
      const int kind = s_kind[b];
      if (kind == 0) continue;
      const int64_t d = p.delta[b], l = s_len[b];
      const int64_t target = l + d < 0 ? 0 : l + d;
      const int have = pages_of(l, p.page_size), want = pages_of(target, p.page_size);
      int32_t *tab = p.table + b * p.table_stride;
      if (kind == 1) {
        for (int i = lane; i < want - have; i += 32)
          tab[have + i] = p.ring[ring_at(p, head + s_off[b] + i)];
      } else {
        const int64_t base = (head + count) % p.num_pages;
        for (int i = lane; i < have - want; i += 32)
          p.ring[ring_at(p, base + s_off[b] + i)] = tab[want + i];
      }
    }
  }
  __syncthreads();

  for (int64_t t = tid; t < p.max_tokens; t += kThreads) {
    int64_t slot = -1;
    if (whole && t < total_rows) {
      int lo = 0, hi = p.batch - 1;   // the request with s_row[b] <= t < s_row[b + 1]
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_row[mid] <= t) lo = mid; else hi = mid - 1;
      }
      if (s_kind[lo] == 1) {
        const int pos = int(s_len[lo] + t - s_row[lo]);
        const int page = p.table[lo * p.table_stride + pos / p.page_size];
        if (page >= 0 && page < p.num_pages)
          slot = int64_t(page) * p.page_size + pos % p.page_size;
        else
          err |= FA_PAGED_BAD_PAGE;
      }
    }
    p.slots[t] = slot;
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    if (b < p.batch) p.lens_out[b] = whole && s_kind[b] ? a[i].target : len[i];
  }
  if (tid == 0) {
    p.state_out[0] = whole ? (head + taken) % p.num_pages : head;
    p.state_out[1] = whole ? count - taken + total_give : count;
  }
  if (err && p.error) atomicOr(p.error, err);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams &p, cudaStream_t s) {
  plan_kernel<<<1, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fav
