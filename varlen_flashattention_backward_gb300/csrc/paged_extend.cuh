// Attention of a chunk of new tokens per request over the paged cache
// (fa_paged_extend): the parts that its kernels share.  S_ij = scale q_i . k_j,
// P = exp(S - max), y_i = sum_j P_ij v_j / sum_j P_ij over the keys that row i sees.
#pragma once

#include <math_constants.h>

#include "common.cuh"
#include "paged.h"
#include "sm103.cuh"

namespace fav {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Division of the work
//
// The query heads of one key head stand side by side: packed row r of a request and
// key head is token r / group, head r % group of the group.  BR packed rows are a
// block, which is worked off against the tiles of BN keys that any of its rows sees.
// The blocks, request by request, head by head, each weighing its tiles plus
// kSwitch (what it costs to begin one), form a line that is cut into equal spans, one
// per CTA.  A CTA's share of a block is a segment.  A segment with all of its
// block's tiles writes y itself; of the others a CTA has at most two: the first,
// where the block began in an earlier CTA (slot 0), and the last (slot 1).  Their
// unscaled results go to the workspace, and extend_join adds up each block's parts,
// in order.  All of it follows from the lengths alone, which are on the device, so
// every CTA measures the line for itself.
// ---------------------------------------------------------------------------
// (kSwitch 2: prompts 817 -> 796 us, a step of single tokens and chunks 236 -> 256.)
constexpr int kSwitch = 1;
// Units of a request that rules the call out: more than 2^28 / 64 blocks of 2^30 / 32 tiles
// have, and 2048 times as many still fit.
constexpr int64_t kTooMany = int64_t(1) << 49;

struct Request {
  int start, n;   // rows of q
  int len;        // keys
};

__device__ __forceinline__ Request request_of(const ExtendParams &p, int b, int &err) {
  Request r;
  const int64_t c0 = p.cu[b], c1 = p.cu[b + 1];
  const int64_t start = min(max(c0, int64_t(0)), int64_t(p.tokens));
  const int64_t end = min(max(c1, start), int64_t(p.tokens));
  if (start != c0 || end != c1) err |= FA_PAGED_ROWS;
  r.start = int(start);
  r.n = int(end - start);
  const int most = p.max_pages * p.page_size, len = p.lens[b];
  if (len < 0 || len > most) err |= FA_PAGED_BAD_LENGTH;
  r.len = min(max(len, 0), most);
  return r;
}

// Keys [lo, hi) that token t of the request sees.  (|pos| < 2^30 and the window's
// bounds are clamped to [-2^30, 2^30 - 1]: 32 bits do.)
__device__ __forceinline__ void keys_of(const ExtendParams &p, const Request &r, int t, int &lo, int &hi) {
  const int pos = r.len - r.n + t;
  lo = min(max(pos - p.pre, 0), r.len);
  hi = min(max(pos + p.next + 1, 0), r.len);
}

// What the line is cut by: block i of a request, of `rows` packed rows in all.
struct Block {
  int row0, rows;      // its packed rows
  int tile0, tiles;    // the keys' tiles that any of them may see
};

template <int BR, int BN>
__device__ __forceinline__ Block block_of(const ExtendParams &p, const Request &r, int i) {
  Block k;
  k.row0 = i * BR;
  k.rows = min(BR, r.n * p.group - k.row0);
  int lo, hi, unused;
  keys_of(p, r, k.row0 / p.group, lo, unused);
  keys_of(p, r, (k.row0 + k.rows - 1) / p.group, unused, hi);
  k.tile0 = lo / BN;
  k.tiles = hi > lo ? (hi + BN - 1) / BN - k.tile0 : 0;
  return k;
}

template <int BR>
__device__ __forceinline__ int blocks_of(const ExtendParams &p, const Request &r) {
  return (r.n * p.group + BR - 1) / BR;
}

// A place on the line.
struct Place {
  int b, h, i;        // request, key head, block
  int64_t off;        // units into the block
  int64_t at;         // units from the line's beginning
  int64_t left;       // units to the end of the CTA's span
  int before;         // blocks of the requests before b, per key head
  Request r;          // b's
};

struct Line {
  int64_t span;       // units per CTA
  int64_t units;      // in all
};

// Scratch of measure(), per CTA.
struct Measure {
  int64_t upto[kMaxBatch + 1];   // units of one key head before each request
  int blocks[kMaxBatch + 1];     // blocks before each request
  int64_t sum64[32];
  int sum32[32];
  Request request[kMaxBatch];
};

// Measures the line and finds the CTA's place on it; all threads of the CTA.  False:
// there is nothing for it.
template <int BR, int BN, int THREADS>
__device__ bool measure(const ExtendParams &p, Measure &m, Line &line, Place &at) {
  constexpr int kWarps = THREADS / 32;
  constexpr int kLanes = 8;      // that share a request's blocks
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int err = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.batch; b0 += THREADS / kLanes) {
    const int b = b0 + tid / kLanes;
    int64_t units = 0;
    int n = 0;
    if (b < p.batch) {
      const bool descends = p.cu[b + 1] < p.cu[b];
      const Request r = request_of(p, b, err);
      if (tid % kLanes == 0) m.request[b] = r;
      n = blocks_of<BR>(p, r);
#pragma unroll 1
      for (int i = tid % kLanes; i < n; i += kLanes) units += block_of<BR, BN>(p, r, i).tiles + kSwitch;
      if (descends) units = tid % kLanes == 0 ? kTooMany : 0;
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) units += __shfl_xor_sync(kFull, units, o);
    if (b < p.batch && tid % kLanes == 0) {
      m.upto[b + 1] = units;
      m.blocks[b + 1] = n;
    }
  }
  if (err && blockIdx.x == 0 && p.error) atomicOr(p.error, err);
  __syncthreads();
  // Prefix sums: each thread a run of requests, each warp, all warps.  (Blocks of requests
  // whose bounds descend need not fit 32 bits; they are not used.)
  const int per = (p.batch + THREADS - 1) / THREADS;
  int64_t own = 0, own_blocks = 0;
#pragma unroll 1
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b < p.batch) {
      own += m.upto[b + 1];
      own_blocks += m.blocks[b + 1];
    }
  }
  int64_t x = own, y = own_blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, x, o), v = __shfl_up_sync(kFull, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  __syncthreads();
  if (lane == 31) {
    m.sum64[warp] = x;
    m.sum32[warp] = int(min(y, int64_t(1) << 30));
  }
  __syncthreads();
  int64_t before = x - own, before_blocks = y - own_blocks, all = 0;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      before += m.sum64[w];
      before_blocks += m.sum32[w];
    }
    all += m.sum64[w];
  }
#pragma unroll 1
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b < p.batch) {
      before += m.upto[b + 1];
      before_blocks += m.blocks[b + 1];
      m.upto[b + 1] = before;
      m.blocks[b + 1] = int(min(before_blocks, int64_t(1) << 30));
    }
  }
  if (tid == 0) {
    m.upto[0] = 0;
    m.blocks[0] = 0;
  }
  __syncthreads();
  // Requests whose bounds descend could share rows: nothing is done then.  (Ascending ones
  // have rows of their own, so that no more blocks come together than the workspace has
  // flags for.)
  line.units = all >= kTooMany ? 0 : all * p.n_kv;
  line.span = max((line.units + gridDim.x - 1) / gridDim.x, int64_t(p.least_span));
  at.at = line.span * blockIdx.x;
  at.left = min(line.span, line.units - at.at);
  if (at.left <= 0) return false;
  // The request: the last one with upto * n_kv <= at, that has units.
  int lo = 0, hi = p.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (m.upto[mid] * p.n_kv <= at.at) lo = mid; else hi = mid - 1;
  }
  at.b = lo;
  at.before = m.blocks[lo];
  const int64_t each = max(m.upto[lo + 1] - m.upto[lo], int64_t(1));
  const int64_t in = at.at - m.upto[lo] * p.n_kv;
  at.h = int(in / each);
  int64_t rest = in - at.h * each;
  // The block: each warp by itself, 32 at a time.
  const Request r = m.request[lo];
  at.r = r;
  const int n = blocks_of<BR>(p, r);
  at.i = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int64_t units = i < n ? block_of<BR, BN>(p, r, i).tiles + kSwitch : 0;
    int64_t upto = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += u;
    }
    const uint32_t beyond = __ballot_sync(kFull, i < n && upto > rest);
    if (beyond) {
      const int k = __ffs(beyond) - 1;
      at.i = i0 + k;
      rest -= __shfl_sync(kFull, upto - units, k);
      break;
    }
    rest -= __shfl_sync(kFull, upto, 31);
  }
  at.off = rest;
  return true;
}

// A CTA's share of a block.
struct Segment {
  Request r;
  Block k;
  int b, h, i;
  int t0, t1;      // its tiles, counted from the block's first
  int item;        // number of (request, key head, block)
  int slot;        // 0 or 1: a part; -1: the whole block
};

// Workspace: a record per CTA, two slots of partial results each, and one word of flags
// for 32 rows of each block.
struct Record {
  int32_t has[2];          // which slots were written
  int32_t cut;             // the last block goes on in the next CTA
  int32_t last;            // ... up to this one
  int32_t b, h, i;
  Request r;
  int32_t flagged;         // some row of the blocks that it finished is to be looked at
  int32_t item0, items;    // those blocks, and others beside them
  int32_t odd;             // a tile had a key with a bad page
  int32_t pad[2];
};
static_assert(sizeof(Record) == kExtendRecord, "records");

template <int BR>
__device__ __forceinline__ float *part_of(const ExtendParams &p, int cta, int slot) {
  return p.parts + int64_t(2 * cta + slot) * BR * (p.d + 3);
}

// Walks a span, segment by segment.  Used by one warp (or one thread) of a CTA.
template <int BR, int BN>
struct Walk {
  Place at;
  Line line;
  Request r;
  int blocks;
  Record rec;
  int err;
  bool ended;      // the block was the last segment's, to its end

  __device__ __forceinline__ void begin(const ExtendParams &p, const Line &l, const Place &place, bool any) {
    line = l;
    at = place;
    rec = Record{};
    err = 0;
    ended = false;
    if (!any) {
      at.left = 0;
      return;
    }
    r = at.r;
    blocks = blocks_of<BR>(p, r);
  }

  // To the block behind the last one.
  __device__ __forceinline__ void advance(const ExtendParams &p) {
    ended = false;
    at.off = 0;
    if (++at.i < blocks) return;
    at.i = 0;
    if (++at.h < p.n_kv) return;
    at.h = 0;
    do {
      at.before += blocks;
      if (++at.b >= p.batch) return;
      r = request_of(p, at.b, err);
      blocks = blocks_of<BR>(p, r);
    } while (blocks == 0);
  }

  // False at the end.
  __device__ __forceinline__ bool next(const ExtendParams &p, Segment &s) {
    while (at.left > 0) {
      if (ended) advance(p);
      if (at.b >= p.batch) break;
      const Block k = block_of<BR, BN>(p, r, at.i);
      const int64_t units = k.tiles + kSwitch;
      const int64_t take = min(at.left, units - at.off);
      s.r = r;
      s.k = k;
      s.b = at.b;
      s.h = at.h;
      s.i = at.i;
      s.t0 = int(max(at.off - kSwitch, int64_t(0)));
      s.t1 = int(max(at.off + take - kSwitch, int64_t(0)));
      s.item = at.before * p.n_kv + at.h * blocks + at.i;
      const bool whole = s.t0 == 0 && s.t1 == k.tiles;
      const bool begins = at.off == 0, ends = at.off + take == units;
      s.slot = whole ? -1 : begins ? 1 : 0;
      if (begins && !ends) {
        rec.cut = 1;
        rec.last = int((at.at + units - 1) / line.span);
        rec.b = at.b;
        rec.h = at.h;
        rec.i = at.i;
        rec.r = r;
      }
      at.at += take;
      at.left -= take;
      at.off += take;
      ended = ends;
      if (rec.items == 0) rec.item0 = s.item;
      rec.items = s.item - rec.item0 + 1;
      if (whole ? begins || s.t1 > 0 : s.t1 > s.t0) {
        if (!whole) rec.has[s.slot] = 1;
        return true;
      }
    }
    return false;
  }
};

// ---------------------------------------------------------------------------
// Rows whose result is not finite, computed once more
//
// Products of whole tiles multiply weights of 0 with the values in masked places,
// which gives NaN where those are not finite.  Nothing is checked on the way there: a row
// that comes out finite met no such value.  For one that does not, a warp looks
// at the masked places that its block's tiles held, and where one of them is not finite
// computes the row again from the keys that it sees; its statistics, of which masked
// scores are no part, stand.  (Without one, the row sees a value that is not finite itself, or
// large ones whose sum passes fp32's range, and stays; but it becomes 0 where all of its
// scores are -inf.)
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ const T *cached(const ExtendParams &p, const void *cache, int b, int h, int key) {
  const int at = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
  const int page = p.table[b * p.table_stride + at];
  if (page < 0 || page >= p.num_pages) return nullptr;
  return static_cast<const T *>(cache) + page * p.page_stride + (key - at * p.page_size) * p.token_stride +
         h * p.head_stride;
}

__device__ __forceinline__ void write_stats(const ExtendParams &p, int64_t row, float top, float total) {
  if (p.smax == nullptr) return;
  float4 *m = reinterpret_cast<float4 *>(p.smax + row * 8), *l = reinterpret_cast<float4 *>(p.ssum + row * 8);
  const float4 a = make_float4(top, top, top, top), z = make_float4(total, total, total, total);
  if (p.stat_chunks) {
    m[0] = m[1] = a;
    l[0] = l[1] = z;
    return;
  }
  for (int i = 0; i < 8; ++i) {
    p.smax[row * 8 + i] = top;
    p.ssum[row * 8 + i] = total;
  }
}

template <typename T, int D, int BR, int BN>
__device__ __noinline__ void mend_row(const ExtendParams &p, int b, int h, int i, int row) {
  constexpr int PL = D / 32;
  const int lane = threadIdx.x & 31;
  int err = 0;
  const Request r = request_of(p, b, err);
  const Block k = block_of<BR, BN>(p, r, i);
  if (row >= k.rows) return;      // (flags that a call whose wait ran out has not written)
  const int packed = k.row0 + row, t = packed / p.group, n = h * p.group + packed % p.group;
  int lo, hi;
  keys_of(p, r, t, lo, hi);
  if (hi < lo) hi = lo;
  // The masked places of the block's tiles.
  const int first = k.tile0 * BN, end = min((k.tile0 + k.tiles) * BN, r.len);
  bool found = false;
  for (int j = first; j < end; ++j) {
    if (j >= lo && j < hi) {
      j = hi - 1;
      continue;
    }
    const T *v = cached<T>(p, p.vc, b, h, j);
    if (v == nullptr) continue;
#pragma unroll
    for (int e = 0; e < PL; ++e) found |= !isfinite(to_f<T>(v[lane + 32 * e]));
  }
  found = __any_sync(kFull, found);
  const T *q = static_cast<const T *>(p.q) + (r.start + t) * p.q_stride + int64_t(n) * D;
  float qd[PL], o[PL];
#pragma unroll
  for (int e = 0; e < PL; ++e) {
    qd[e] = to_f<T>(q[lane + 32 * e]) * p.sign;
    o[e] = 0.f;
  }
  float top = -CUDART_INF_F, total = 0.f;
  for (int j = lo; j < hi; ++j) {
    const T *kr = cached<T>(p, p.kc, b, h, j), *vr = cached<T>(p, p.vc, b, h, j);
    if (kr == nullptr) continue;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < PL; ++e) s = fmaf(qd[e], to_f<T>(kr[lane + 32 * e]), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kFull, s, x);
    s *= p.scale_log2;
    const float m = fmaxf(top, s), ref = m == -CUDART_INF_F ? 0.f : m;
    const float f = exp2f(top - ref), w = exp2f(s - ref + p.bias);   // (as large as in the first place)
    top = m;
    total = total * f + w;
    bool lost = true;
#pragma unroll
    for (int e = 0; e < PL; ++e) {
      o[e] = o[e] * f + w * to_f<T>(vr[lane + 32 * e]);
      lost &= isnan(o[e]);
    }
    if (total == 0.f) continue;
    if (!found) return;
    if (__all_sync(kFull, lost)) break;    // whatever follows
  }
  T *y = static_cast<T *>(p.y) + (r.start + t) * p.y_stride + int64_t(n) * D;
  const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int e = 0; e < PL; ++e) y[lane + 32 * e] = from_f<T>(total == 0.f ? 0.f : o[e] * inv);
}

// The request of an item and how many blocks a key head of it has; `item` is counted from
// the request's first then.  By a whole warp, 32 requests at a time; b = -1 where there
// is none (flags that a call whose wait ran out has not written).
template <int BR>
__device__ __noinline__ int2 find_request(const ExtendParams &p, int &item) {
  const int lane = threadIdx.x & 31;
  int err = 0;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int blocks = b0 + lane < p.batch ? blocks_of<BR>(p, request_of(p, b0 + lane, err)) : 0;
    int upto = blocks * p.n_kv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += u;
    }
    const uint32_t beyond = __ballot_sync(kFull, upto > item);
    const int k = beyond ? __ffs(beyond) - 1 : 31, n = __shfl_sync(kFull, blocks, k);
    item -= __shfl_sync(kFull, upto, k) - (beyond ? n * p.n_kv : 0);
    if (beyond) return make_int2(b0 + k, n);
  }
  return make_int2(-1, 0);
}

// Reports the bad pages of request b that any of its rows sees; by a warp, where a tile had
// some (looked for key by key in the loaders, 2 to 10% of calls whose keys come in pieces):
// tiles begin in front of a window and end behind it.  (Windows of neighbouring rows
// lie one key apart, so that together they leave no gap; where they are empty, what lies
// between two of them is nobody's.)
__device__ __noinline__ void report_pages(const ExtendParams &p, int b) {
  int lo, hi, unused, err = 0;
  const Request r = request_of(p, b, err);
  keys_of(p, r, 0, lo, unused);
  keys_of(p, r, r.n - 1, unused, hi);
  if (r.n == 0 || p.pre + p.next < 0 || lo >= hi) return;
  bool bad = false;
  for (int i = lo / p.page_size + (threadIdx.x & 31); i <= (hi - 1) / p.page_size; i += 32) {
    const int page = p.table[b * p.table_stride + i];
    bad |= page < 0 || page >= p.num_pages;
  }
  if (bad && p.error) atomicOr(p.error, FA_PAGED_BAD_PAGE);
}

// ---------------------------------------------------------------------------
// Adds the parts of the blocks that were cut, mends rows and reports bad pages.  CTA
// (x, y) takes 32 rows of the block that begins last in span x; a warp takes D / 8
// columns, a lane a row.  Bound by latency, of the record, then of the parts, which lie in the L2: two are
// on the way at a time (20 parts a block: 13 us of a call of 42; four on the way take as
// long there, and 10 us more in cross attention).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <typename T, int D, int BR, int BN>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) extend_join(const __grid_constant__ ExtendParams p) {
  constexpr int C = D / kJoinWarps;
  __shared__ float s_y[32][D + 1];
  __shared__ uint32_t s_bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_bad = 0;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Record *records = reinterpret_cast<const Record *>(p.records);
  const Record rec = records[blockIdx.x];
  const int row0 = blockIdx.y * 32, row = row0 + lane;
  if (rec.cut) {
    const Request r = rec.r;
    const Block k = block_of<BR, BN>(p, r, rec.i);
    if (row0 < k.rows) {
      float mx = -CUDART_INF_F, top = -CUDART_INF_F, sum = 0.f, acc[C];
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] = 0.f;
      bool some = false;
      for (int x0 = blockIdx.x; x0 <= rec.last; x0 += 32) {
        // Which of the next 32 CTAs have a part.
        const int mine = x0 + lane;
        uint32_t has =
            __ballot_sync(kFull, mine <= rec.last && records[mine].has[mine == int(blockIdx.x) ? 1 : 0]);
        some |= has != 0;
        while (has) {
          constexpr int U = 2;
          float m[U], l[U], t[U], o[U][C];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int j = __ffs(has) - 1;
            has &= has - 1;
            m[u] = t[u] = -CUDART_INF_F;
            l[u] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) o[u][c] = 0.f;
            if (j < 0) continue;
            const float *src = part_of<BR>(p, x0 + j, x0 + j == int(blockIdx.x) ? 1 : 0) + row;
            m[u] = src[D * BR];
            l[u] = src[(D + 1) * BR];
            t[u] = src[(D + 2) * BR];
#pragma unroll
            for (int c = 0; c < C; ++c) o[u][c] = src[(warp * C + c) * BR];
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            top = fmaxf(top, t[u]);
            const float mn = fmaxf(mx, m[u]), ref = mn == -CUDART_INF_F ? 0.f : mn;
            const float f = exp2f(mx - ref), f2 = exp2f(m[u] - ref);
            mx = mn;
            sum = sum * f + l[u] * f2;
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = acc[c] * f + o[u][c] * f2;
          }
        }
      }
      if (some) {            // (none: one CTA had all of its tiles after all)
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          bad |= !isfinite(acc[c]);
          s_y[lane][warp * C + c] = acc[c] * inv;
        }
        const int packed = k.row0 + row;
        if (warp == 0 && row < k.rows)
          write_stats(p, int64_t(r.start + packed / p.group) * p.n + rec.h * p.group + packed % p.group,
                      top * kLn2, sum * exp2f((mx == -CUDART_INF_F ? 0.f : mx - top) - p.bias));
        const uint32_t bads = __ballot_sync(kFull, bad && row < k.rows);
        __syncthreads();
        if (lane == 0 && bads) atomicOr(&s_bad, bads);
        __syncthreads();
        for (int w = warp; w < min(32, k.rows - row0); w += kJoinWarps) {
          const int pr = k.row0 + row0 + w, t = pr / p.group, n = rec.h * p.group + pr % p.group;
          T *y = static_cast<T *>(p.y) + (r.start + t) * p.y_stride + int64_t(n) * D;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) y[lane + 32 * e] = from_f<T>(s_y[w][lane + 32 * e]);
          if ((s_bad >> w) & 1) {
            __syncwarp();
            mend_row<T, D, BR, BN>(p, rec.b, rec.h, rec.i, row0 + w);
          }
        }
      }
    }
  }
  if (!(rec.flagged | rec.odd)) return;
  const int turn = blockIdx.y * kJoinWarps + warp, turns = gridDim.y * kJoinWarps;
  if (rec.odd) {
    int first = rec.item0, last = rec.item0 + rec.items - 1;
    const int b0 = find_request<BR>(p, first).x, b1 = find_request<BR>(p, last).x;
    for (int b = max(b0, 0) + turn; b <= b1; b += turns) report_pages(p, b);
  }
  if (!rec.flagged) return;
  // The flags of the blocks that were not cut.  Every warp of the span looks at all of
  // them and takes its turn of the rows: where a cache is full of such values, all rows are
  // flagged (8192 tokens of 8 heads behind 20000, D 64, one column of NaN: 12.5 s with one
  // warp at work, 0.5 s so; every column: 1.5 ms).
  const int words = rec.items * (BR / 32), words0 = rec.item0 * (BR / 32);
  int at_turn = 0;       // of the next flagged row
  for (int w0 = 0; w0 < words; w0 += 32) {
    const uint32_t mine = w0 + lane < words ? p.flags[int64_t(words0) + w0 + lane] : 0u;
    uint32_t some = __ballot_sync(kFull, mine != 0);
    while (some) {
      const int at = __ffs(some) - 1;
      some &= some - 1;
      uint32_t bits = __shfl_sync(kFull, mine, at);
      int item = (words0 + w0 + at) / (BR / 32);
      int2 found = make_int2(-1, 0);
      const int group = (words0 + w0 + at) % (BR / 32);
      for (; bits; bits &= bits - 1) {
        const bool own = at_turn == turn;
        if (++at_turn == turns) at_turn = 0;
        if (!own) continue;
        if (found.x < 0) found = find_request<BR>(p, item);
        if (found.x < 0) break;
        mend_row<T, D, BR, BN>(p, found.x, item / found.y, item % found.y, group * 32 + __ffs(bits) - 1);
      }
    }
  }
}

// The join, as the main kernel's dependent, so that its launch overlaps that one's run.
template <typename T, int D, int BR, int BN>
cudaError_t launch_join(const ExtendParams &p, int ctas, cudaStream_t s) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const int64_t rows = int64_t(p.tokens) * p.group;      // no block has more
  cfg.gridDim = dim3(unsigned(ctas), unsigned(rows < BR ? (rows + 31) / 32 : BR / 32));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, extend_join<T, D, BR, BN>, p);
}

#define FAV_EXTEND_BY_DIM(FN)             \
  switch (p.d) {                          \
    case 32: return FN<32>(p, ctas, s);   \
    case 64: return FN<64>(p, ctas, s);   \
    case 96: return FN<96>(p, ctas, s);   \
    case 128: return FN<128>(p, ctas, s); \
    case 192: return FN<192>(p, ctas, s); \
  }                                       \
  return cudaErrorInvalidValue

}  // namespace
}  // namespace fav
