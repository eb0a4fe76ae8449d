// Block tables and slot maps from request lengths (fa_paged_plan).

#include "paged.h"

namespace fav {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPer = 4;                        // requests per thread
constexpr int kMaxRequests = kThreads * kMaxPer;  // the largest batch

// Exclusive prefixes of N values over the CTA's threads; `total` gets the sums.
// `buf` is not written again before the next barrier.
template <int N>
__device__ __forceinline__ void block_prefix(int64_t (&v)[N], int64_t (*buf)[kWarps],
                                             int64_t (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = v[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t y = __shfl_up_sync(kFull, x[k], o);
      if (lane >= o) x[k] += y;
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (lane == 31) buf[k][warp] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = x[k] - v[k];
    total[k] = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int64_t w = buf[k][i];
      if (i < warp) v[k] += w;
      total[k] += w;
    }
  }
}

// What the flat loops read of each request.
struct Requests {
  int row[kMaxRequests + 1];   // first packed row
  int need[kMaxRequests];      // pages taken before it (up to the last granted)
  int give[kMaxRequests + 1];  // pages given back before it
  int len[kMaxRequests];
  int have[kMaxRequests];      // pages held
  uint8_t granted[kMaxRequests];
};

// The request with first[b] <= i < first[b + 1].
__device__ __forceinline__ int owner_of(const int *first, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int wrap(int64_t i, int n) { return int(i >= n ? i - n : i); }

// Phase 1: prefix sums over the requests, of rows, then of pages taken and
// given back.  Phase 2, over the packed rows and the moved pages, a warp
// taking a run of them: one binary search at its start, then a walk.  The
// pages that a request takes are read from the ring, not from the table, so
// that nothing in phase 2 depends on anything else in it.  Phase 3: lengths
// and pool, which may be updated in place.
//
// A small call is one CTA that does all three.  A large one spreads phase 2
// over many CTAs, each of which does phase 1 for itself, and leaves phase 3 to
// one more CTA, launched as their dependent: it does its phase 1 beside them
// and writes when they are done.
//
// Bound by latency: a chain of four dependent accesses (lengths, two prefix sums
// with a barrier each, the entry of ring or table, the slot) and the launch.  A
// step of 256 requests takes 6.0 us; 256 requests of which half take prompts of up to
// 4096 tokens and a fifth end (400000 slots) 9.8 us.  Their bytes would take less than
// 0.01 and 0.5 us.
enum : int { kFill = 1, kCommit = 2 };

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const __grid_constant__ PlanParams p) {
  __shared__ int64_t buf[3][kWarps];
  __shared__ Requests s;
  __shared__ int s_taken;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x;
  const bool first_cta = (p.phases & kFill) && blockIdx.x == 0;
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int64_t most = int64_t(p.max_pages) * p.page_size;
  if (tid == 0) s_taken = 0;
  int err = 0;

  int len[kMaxPer], delta[kMaxPer];
  const int64_t head = p.state[0], count = p.state[1];
  int64_t rows[1] = {0};
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int b = tid * per + i;
    const bool in = i < per && b < p.batch;
    len[i] = in ? p.lens[b] : 0;
    delta[i] = in ? p.delta[b] : 0;
    rows[0] += max(delta[i], 0);
  }
  int64_t sums[1], moved_sums[2];
  block_prefix(rows, &buf[0], sums);
  int64_t row = rows[0];
  const int64_t total_rows = sums[0];

  int need[kMaxPer], give[kMaxPer], target[kMaxPer], have[kMaxPer];
  bool ask[kMaxPer];
  int64_t first_row[kMaxPer], moved[2] = {0, 0};   // pages needed, given back
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const bool sound = len[i] >= 0 && len[i] <= most;
    const int64_t want_len = max(int64_t(len[i]) + delta[i], int64_t(0));
    const bool in_row = want_len <= most;
    first_row[i] = row;
    row += max(delta[i], 0);
    const bool grows = sound && delta[i] > 0 && in_row;
    ask[i] = grows && row <= p.max_tokens;
    if (!sound) err |= FA_PAGED_BAD_LENGTH;
    if (sound && delta[i] > 0 && !in_row) err |= FA_PAGED_ROW_FULL;
    if (grows && !ask[i]) err |= FA_PAGED_ROWS;
    have[i] = sound ? (len[i] + p.page_size - 1) / p.page_size : 0;
    target[i] = in_row ? int(want_len) : 0;
    const int want = (target[i] + p.page_size - 1) / p.page_size;
    need[i] = ask[i] ? want - have[i] : 0;
    give[i] = sound && delta[i] < 0 ? have[i] - want : 0;
    moved[0] += need[i];
    moved[1] += give[i];
  }
  block_prefix(moved, &buf[1], moved_sums);
  int64_t off_need = moved[0], off_give = moved[1];
  const int64_t total_give = moved_sums[1];
  // With room for all of them behind the end, the pages given back land on no
  // entry that this call takes.
  const bool whole = head >= 0 && head < p.num_pages && count >= 0 && count <= p.num_pages &&
                     count + total_give <= p.num_pages;
  if (!whole) err |= FA_PAGED_BAD_POOL;
  bool granted[kMaxPer];
  int64_t granted_upto = 0;
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int b = tid * per + i;
    const bool in = i < per && b < p.batch;
    // Of the requests that need pages a prefix is granted, so the sum over all
    // before a granted one is the sum over the granted ones.
    granted[i] = ask[i] && (need[i] == 0 || off_need + need[i] <= count);
    if (ask[i] && !granted[i]) err |= FA_PAGED_EXHAUSTED;
    if (granted[i] && need[i] > 0) granted_upto = off_need + need[i];
    if (in) {
      s.row[b] = int(min(first_row[i], p.max_tokens));
      s.need[b] = int(min(off_need, max(count, int64_t(0))));
      s.give[b] = int(min(off_give, int64_t(p.num_pages)));
      s.len[b] = len[i];
      s.have[b] = have[i];
      s.granted[b] = granted[i] && whole;
      if (first_cta) p.cu[b] = first_row[i];
    }
    off_need += need[i];
    off_give += give[i];
  }
  if (granted_upto > 0) atomicMax(&s_taken, int(granted_upto));
  if (tid == 0) {
    s.row[p.batch] = int(min(total_rows, p.max_tokens));
    s.give[p.batch] = whole ? int(total_give) : 0;
    if (first_cta) p.cu[p.batch] = total_rows;
  }
  __syncthreads();
  const int taken = s_taken, given = s.give[p.batch];

  const int lane = tid & 31;
  const int warps = int(gridDim.x) * kWarps, warp = int(blockIdx.x) * kWarps + (tid >> 5);
  const auto page_of_new = [&](int b, int k) {   // the k-th page that request b takes
    return p.ring[wrap(head + s.need[b] + k, p.num_pages)];
  };

  // Slots, in runs of whole 32s per warp.
  if (p.phases & kFill) {
    const int64_t run = ((p.max_tokens + warps - 1) / warps + 31) / 32 * 32;
    const int64_t end = min(run * (warp + 1), p.max_tokens);
    const int used = s.row[p.batch];
    int64_t t = run * warp + lane;
    int b = t < used ? owner_of(s.row, p.batch, int(t)) : p.batch - 1;
#pragma unroll 2
    for (; t < end; t += 32) {
      int64_t slot = -1;
      if (t < used) {
        while (b + 1 < p.batch && s.row[b + 1] <= t) ++b;
        if (s.granted[b]) {
          const int pos = s.len[b] + int(t) - s.row[b];
          const int idx = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
          const int page = idx < s.have[b] ? p.table[b * p.table_stride + idx]
                                           : page_of_new(b, idx - s.have[b]);
          if (page >= 0 && page < p.num_pages)
            slot = int64_t(page) * p.page_size + (pos - idx * p.page_size);
          else
            err |= FA_PAGED_BAD_PAGE;
        }
      }
      p.slots[t] = slot;
    }
  }
  // Pages taken, then pages given back, as one list.
  if (whole && (p.phases & kFill)) {
    const int64_t items = int64_t(taken) + given;
    const int64_t run = ((items + warps - 1) / warps + 31) / 32 * 32;
    const int64_t end = min(run * (warp + 1), items);
    const int64_t tail = wrap(head + count, p.num_pages);
    int bt = -1, bg = -1;
#pragma unroll 2
    for (int64_t at = run * warp + lane; at < end; at += 32) {
      if (at < taken) {
        const int i = int(at);
        if (bt < 0) bt = owner_of(s.need, p.batch, i);
        while (bt + 1 < p.batch && s.need[bt + 1] <= i) ++bt;
        const int k = i - s.need[bt];
        p.table[bt * p.table_stride + s.have[bt] + k] = page_of_new(bt, k);
      } else {
        const int i = int(at - taken);
        if (bg < 0) bg = owner_of(s.give, p.batch, i);
        while (bg + 1 < p.batch && s.give[bg + 1] <= i) ++bg;
        // It gives back its last pages.
        const int left = s.have[bg] - (s.give[bg + 1] - s.give[bg]);
        p.ring[wrap(tail + i, p.num_pages)] =
            p.table[bg * p.table_stride + left + (i - s.give[bg])];
      }
    }
  }
  if (p.phases & kCommit) {
    if (!(p.phases & kFill)) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int i = 0; i < kMaxPer; ++i) {
      const int b = tid * per + i;
      const bool shrinks = delta[i] < 0 && len[i] >= 0 && len[i] <= most;
      const bool moved = whole && (granted[i] || shrinks);
      if (i < per && b < p.batch) p.lens_out[b] = moved ? target[i] : len[i];
    }
    if (tid == 0) {
      p.state_out[0] = whole ? (head + taken) % p.num_pages : head;
      p.state_out[1] = whole ? count - taken + given : count;
    }
  }
  if (err && p.error && (p.phases & kFill)) atomicOr(p.error, err);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams &p0, cudaStream_t s) {
  PlanParams p = p0;
  // Items of work that the host can see: rows, and the pages that requests may
  // give back.  One CTA where each thread has at most one request and two rows: one
  // new token each for 64, 256, 512 requests takes it 5.8, 6.0, 6.4 us, many CTAs 6.0,
  // 6.4, 6.8 and a second launch, but 600 requests take 8.2 and 6.8, and 64 requests of
  // 16, 64, 500 new tokens 7.3, 9.7, 28 and 7.2, 7.5, 8.0.  The bound on pages is for the
  // step that ends all requests at once (256 that give back 8192, 32768 pages: 11.5, 27
  // us and 6.2, 7.4); a usual one gives back few.
  const int64_t items = p.max_tokens + int64_t(p.batch) * p.max_pages;
  p.phases = kFill | kCommit;
  if (p.batch <= kThreads && p.max_tokens <= 2 * kThreads && items <= 32768) {
    plan_kernel<<<1, kThreads, 0, s>>>(p);
    return cudaGetLastError();
  }
  p.phases = kFill;
  const int64_t ctas = (items + 4 * kThreads - 1) / (4 * kThreads);
  plan_kernel<<<unsigned(ctas < 152 ? ctas : 152), kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  p.phases = kCommit;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, p);
}

}  // namespace fav
