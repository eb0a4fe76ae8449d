// Attention of one new token per request over the paged cache
// (fa_paged_decode): S_j = scale q . k_j, P = exp(S - max), y = P V / sum P.
// Included by one translation unit per type.
#pragma once

#include <cuda.h>
#include <math_constants.h>

#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "sm103.cuh"

namespace fav {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kFull = 0xffffffffu;
// Beginning a segment costs a warp about as much as this many blocks of keys (0, 1, 2
// and 4 measure alike but where requests are short: 61 of up to 1024 keys 18.2 us
// with 0, 15.1 with 1).
constexpr int kSwitchBlocks = 1;
// Most CTAs of a cluster that shares a segment, and blocks for each team of it (16
// requests of 512 keys, 8 key heads: 8.9 us so, 11.7 by ranges; one of 8000 keys 14.6
// and 12.5).
constexpr int kMaxDirect = 8;
constexpr int kDirectBlocks = 8;

// ---------------------------------------------------------------------------
// Division of the work
//
// A segment is one request, one key head and up to R of its query heads; its
// keys are cut into blocks of KB (at least one, which may hold no key).  The
// segments, each weighing its blocks plus kSwitchBlocks, form a line that is
// cut into ranges of equal weight, one per team of TW warps of the grid (a team
// shares its blocks; each of its warps has its own R / TW query heads).  Weights
// count in units of 2^unit_shift blocks, which the host chooses so that 32 bits hold
// the line's length whatever the lengths; the shift is 0 up to a product of
// segments and longest length, in blocks, of 2^31.
//
// A team's share of a segment is a part.  A part that is a whole segment
// writes y from the warps' registers.  Of the others a team has at most two,
// its first (slot 0, where it does not begin its segment) and its last (slot 1,
// where it does), which go to the range's slots in the workspace.  join_kernel
// adds the parts of a segment, in order.
//
// Where there are few segments and none can be long (decode_plan), a segment gets
// a cluster of CTAs instead: its blocks are dealt to their teams, whose parts are
// added in shared memory, and the CTAs' sums through distributed shared memory.
// That saves finding the ranges, the workspace and the second kernel.
// ---------------------------------------------------------------------------
struct Span {
  int lo, hi;        // keys [lo, hi) that the query sees
  int blk0;          // first block (absolute)
  int blocks;
};

template <int KB>
__device__ __forceinline__ Span span_of(const DecodeParams &p, int len) {
  Span s;
  const int most = p.max_pages * p.page_size;
  len = len < 0 ? 0 : len > most ? most : len;
  s.hi = len;
  const int lo = len - 1 - p.pre;
  s.lo = lo < 0 ? 0 : lo > len ? len : lo;
  s.blk0 = s.lo / KB;
  s.blocks = s.hi > s.lo ? (s.hi + KB - 1) / KB - s.blk0 : 1;
  return s;
}

__device__ __forceinline__ int units_of(const DecodeParams &p, int blocks) {
  return (blocks + kSwitchBlocks + (1 << p.unit_shift) - 1) >> p.unit_shift;
}

// The line: its ranges' lengths (the first `rest` are one longer than `each`).
struct Line {
  int each, rest;
  __device__ __forceinline__ int start(int range) const {
    return range * each + min(range, rest);
  }
  __device__ __forceinline__ int range_of(int unit) const {
    const int longer = rest * (each + 1);
    return unit < longer ? unit / (each + 1) : rest + (unit - longer) / each;
  }
};

// A place on it: a segment, and how far inside.
struct Place {
  int b, seg;        // request, segment inside it
  int off;           // units into the segment
  int units;         // of each of the request's segments
};

// The length that request b holds.  A kernel of this file may be on the GPU while
// the one before it still writes lengths, tables and rows, so none of them is read
// through the read-only path, which asks for memory that nobody writes as long as the
// reader lives: the main kernel reads them by plain loads behind its wait, and the
// join, which looks at lengths ahead of its own wait (the main kernel, behind its, let
// it start), at the L2, where that kernel's wait has seen them arrive.
template <bool kAhead = false>
__device__ __forceinline__ int length_of(const DecodeParams &p, int b) {
  if constexpr (kAhead) {
    int len;
    asm("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(len) : "l"(p.lens + b));   // any time will do
    return len;
  } else {
    return p.lens[b];
  }
}

// The units of each of request b's segments, 0 behind the last request.
template <int KB, bool kAhead>
__device__ __forceinline__ int units_at(const DecodeParams &p, int b, bool &bad) {
  if (b >= p.batch) return 0;
  const int len = length_of<kAhead>(p, b);
  bad |= len < 0 || len > p.max_pages * p.page_size;
  return units_of(p, span_of<KB>(p, len).blocks);
}

// Measures the line and finds unit `start(range) - before` on it.  Every warp
// of the main kernel works it out for itself from all lengths: that costs less than
// meeting other warps would.  Lane i sums up requests 32 i .. 32 i + 31 (and
// those 1024 further on), then the warp looks at the 32 that hold the unit.
// False: nothing is there.  (The indexes are held in bounds for the sake of
// lengths that change during the call, which is an error of the caller's.)
template <int KB, bool kAhead>
__device__ __forceinline__ bool find(const DecodeParams &p, int segs, int range, int before,
                                     Line &line, Place &at) {
  const int lane = threadIdx.x & 31;
  const int rows = (p.batch + 31) >> 5;            // at most 64
  int sum[2] = {0, 0};
  int units = 0;
  bool bad = false;
#pragma unroll 8
  for (int i = 0; i < rows; ++i) {
    units = units_at<KB, kAhead>(p, i * 32 + lane, bad);
    const int all = __reduce_add_sync(kFull, units);
    if (lane == (i & 31)) sum[i >> 5] = all;
  }
  if (bad && range == 0 && p.error) atomicOr(p.error, FA_PAGED_BAD_LENGTH);
  int upto[2] = {sum[0], sum[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, upto[0], o), y = __shfl_up_sync(kFull, upto[1], o);
    if (lane >= o) {
      upto[0] += x;
      upto[1] += y;
    }
  }
  upto[1] += __shfl_sync(kFull, upto[0], 31);
  const int total = __shfl_sync(kFull, upto[1], 31) * segs;
  line.each = total / p.ranges;
  line.rest = total - line.each * p.ranges;
  const int u = line.start(range) - before;
  if (u < 0 || u >= total) return false;
  // The row of requests that holds u, then the request.
  const int row = __popc(__ballot_sync(kFull, upto[0] * segs <= u)) +
                  __popc(__ballot_sync(kFull, upto[1] * segs <= u));
  int from = row < 32 ? __shfl_sync(kFull, upto[0] - sum[0], row)
                      : __shfl_sync(kFull, upto[1] - sum[1], row - 32);
  if (rows > 1) units = units_at<KB, kAhead>(p, row * 32 + lane, bad);
  int x = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  const int n = min(__popc(__ballot_sync(kFull, (from + x) * segs <= u)), 31);
  at.b = min(row * 32 + n, p.batch - 1);
  at.units = max(__shfl_sync(kFull, units, n), 1);
  from += __shfl_sync(kFull, x, n) - at.units;
  at.seg = min(max((u - from * segs) / at.units, 0), segs - 1);
  at.off = max(u - from * segs - at.seg * at.units, 0);
  return true;
}

// Measures the line and gives the first unit of segment (at.b, at.seg), whose
// units it fills in.  For the join.
template <int KB>
__device__ __forceinline__ int segment_start(const DecodeParams &p, int segs, Place &at,
                                             Line &line) {
  int sum = 0, before = 0;
  bool bad = false;
  for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
    const int units = units_at<KB, true>(p, b, bad);
    sum += units;
    if (b < at.b) before += units;
  }
  const int total = __reduce_add_sync(kFull, sum) * segs;
  line.each = total / p.ranges;
  line.rest = total - line.each * p.ranges;
  at.units = units_of(p, span_of<KB>(p, length_of<true>(p, at.b)).blocks);
  at.off = 0;
  return __reduce_add_sync(kFull, before) * segs + at.seg * at.units;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a block in the ring is: a mask of its keys, and these.
enum : int {
  kPartBegins = 1 << 16,   // first block of a part
  kPartEnds = 1 << 17,
  kSegBegins = 1 << 18,    // first block of a segment
  kSegEnds = 1 << 19,
  kDone = 1 << 20,         // no block: the range is done
  kRowsFetched = 1 << 21   // the part's query rows are in the place of its turn
};

// Shared memory of one kernel of NW warps: a ring of S stages (K and V block
// each) per team, then per warp QS places for query rows that wait for their
// part and EXTRA bytes more.  In the end the sum of the whole CTA takes the place
// behind the rings.  Query rows are fetched ahead where that leaves three stages:
// under load a fetch takes 1 to 2 us, which a warp would spend waiting at each of its
// parts (1024 requests of 64 keys, 32 / 8 heads, D 128: 16 us more without).
template <typename T, int D, int RW, int TW, int KB, int EXTRA, int WARPS>
struct Shape {
  static constexpr int R = RW * TW;
  static constexpr int PAD = 4;
  static constexpr int kBlock = KB * D * int(sizeof(T));      // K or V block
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kPartial = R * (D + PAD) * 4;
  static constexpr int kQ = RW * D * int(sizeof(T));
  // The kernels' static arrays, in the steps of the ring's alignment.
  static constexpr int static_bytes(int nw, int s) {
    const int nt = nw / TW;
    return (nt * (R * 8 + 4) + nt * s * (TW > 1 ? 9 : 8) + (TW > 1 ? nt * 24 : 0) + 64 + 1023) /
           1024 * 1024;
  }
  // Most stages, up to 8, that fit.
  static constexpr int fit(int nw, int qs) {
    int s = 8;
    while (s > 0 &&
           nw / TW * s * kStage + nw * (qs * kQ + EXTRA) + static_bytes(nw, s) > 227 * 1024)
      --s;
    return s;
  }
  static constexpr int NW = fit(WARPS, EXTRA > 0) >= 2 ? WARPS : 4;
  static constexpr int NT = NW / TW;
  static constexpr int QS = fit(NW, 2) >= 3 ? 2 : (fit(NW, 1) >= 3 || EXTRA > 0) ? 1 : 0;
  static constexpr int S = fit(NW, QS);
  static constexpr int kWarpExtra = QS * kQ + EXTRA;
  static constexpr int kRing = S * kStage;
  static constexpr int kTail = NW * kWarpExtra > kPartial ? NW * kWarpExtra : kPartial;
  static constexpr int kSmem = NT * kRing + kTail;
  static_assert(S >= 2 && kRing >= kPartial && kSmem + static_bytes(NW, S) <= 227 * 1024,
                "decode stages");
};

// How a block of KB rows lies in shared memory: panels of PB bytes of every row,
// one behind the other, with the 16-byte chunks of a row swapped by its number as
// TMA's 128-byte (64-byte) swizzle does, so that eight rows' equal chunks fall
// into different banks.
template <int ROW_BYTES, int KB>
struct Tile {
  static constexpr int PB = ROW_BYTES % 128 == 0 ? 128 : 64;
  static constexpr int CPP = PB / 16;
  static __device__ __forceinline__ int at(int r, int ch) {
    const int panel = ch / CPP, c = ch % CPP;
    return panel * (KB * PB) + r * PB + ((c ^ (PB == 128 ? r & 7 : (r >> 1) & 3)) << 4);
  }
};

struct DecodeMaps {
  CUtensorMap k, v;
  int token_first;   // the maps' axes are dim, token, head, page, else dim, head, token, page
};

// One panel of KB tokens of one head, of K and of V.  All lanes execute it and one
// issues.
__device__ __forceinline__ void tma_load_panels_w(uint32_t dst_k, uint32_t dst_v,
                                                  const DecodeMaps &maps, uint32_t bar, int x,
                                                  int c1, int c2, int c3) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%2, {%5, %6, %7, %8}], [%4];\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%1], [%3, {%5, %6, %7, %8}], [%4];\n\t}" ::"r"(dst_k),
      "r"(dst_v), "l"(reinterpret_cast<uint64_t>(&maps.k)),
      "l"(reinterpret_cast<uint64_t>(&maps.v)), "r"(bar), "r"(x), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// All warps of a team.
template <int TW>
__device__ __forceinline__ void team_sync() {
  if constexpr (TW == 1) {
    __syncwarp();
  } else {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + int(threadIdx.x >> 5) / TW), "n"(32 * TW)
                 : "memory");
  }
}

// The loading side of a team: walks its range and keeps the ring filled.
// `look` finds the next block, `issue`, one block later, starts its copies.  All
// warps of the team walk alike, and meet at barriers on the strength of that; so one
// reads the lengths for all (`common`: two places for a length, in turn, and the range's
// beginning), and not even lengths that change during the call can part them.
// With pages of whole blocks (kTma) one lane starts
// TMA copies of whole panels, and the lanes hold the page ids of 32 blocks; else
// the lanes copy 16 bytes at a time, each warp its share, and hold the pages of
// their rows.  This runs once per block in a warp that has but one other to hide
// behind, so the usual step is kept short: some 40 instructions.
template <typename T, int D, typename Sh, int RW, int TW, int KB, bool kTma>
struct Loader {
  using Tl = Tile<D * int(sizeof(T)), KB>;
  static constexpr int VEC = 16 / int(sizeof(T));
  static constexpr int CPR = D / VEC;                   // 16-byte chunks per row
  static constexpr int kChunks = KB * CPR;              // ... and block
  static constexpr int kLoads = (kChunks + 32 * TW - 1) / (32 * TW);
  static constexpr int kAll = (1 << KB) - 1;
  static_assert(KB <= 16, "decode block");
  const DecodeParams &p;
  const DecodeMaps &maps;
  const int chunks, segs, lane, member;                 // member: warp of the team
  int left;                      // units left of the range
  int off, units, b, seg;        // units into the segment, and of it
  int blk, end;                  // next block of the part, and its end
  Span span;
  // The looked-up block: mask and flags, its request and segment, first row in the
  // request and in its page.
  int what, block_b, head, row, tok;
  int id;                        // block_b * segs + segment
  int page;                      // lane's page id ...
  int page_lane;                 // ... and, kTma, whose is the block's
  int err;
  int parts, parts_free;         // begun so far, and how many hold no query place any more
  int fifo_what, fifo_id;        // lane i: the block in stage i
  volatile int *const common;    // of teams of several warps
  int entered;                   // requests entered so far

  __device__ __forceinline__ Loader(const DecodeParams &p, const DecodeMaps &maps, int chunks,
                                    volatile int *common)
      : p(p), maps(maps), chunks(chunks), segs(p.n_kv * chunks), lane(threadIdx.x & 31),
        member((threadIdx.x >> 5) % TW), left(0), off(0), units(1), b(0), seg(0), blk(0), end(0),
        what(0), block_b(0), head(0), row(0), tok(0), id(0), page(-1), page_lane(0), err(0),
        parts(0), parts_free(0), fifo_what(kDone), fifo_id(0), common(common), entered(0) {
    const int team = (threadIdx.x >> 5) / TW;
    if (p.direct) {
      const int cta = blockIdx.x / p.direct, teams = p.direct * Sh::NT;
      b = cta / segs;
      seg = cta - b * segs;
      const int len = common_length();
      if ((len < 0 || len > p.max_pages * p.page_size) && p.error)
        atomicOr(p.error, FA_PAGED_BAD_LENGTH);
      // Its share as a range whose units are blocks.
      span = span_of<KB>(p, len);
      const int per = (span.blocks + teams - 1) / teams;
      off = min((int(blockIdx.x) * Sh::NT + team - cta * teams) * per, span.blocks);
      left = min(per, span.blocks - off);
      off += kSwitchBlocks;
      units = span.blocks + kSwitchBlocks;
      return;
    }
    const int range = blockIdx.x * Sh::NT + team;
    if (TW == 1 || member == 0) {
      Line line;
      Place at;
      if (find<KB, false>(p, segs, range, 0, line, at)) {
        left = line.each + (range < line.rest ? 1 : 0);
        b = at.b;
        seg = at.seg;
        off = at.off;
      }
    }
    if constexpr (TW > 1) {
      if (member == 0) {
        common[2] = left;
        common[3] = b;
        common[4] = seg;
        common[5] = off;
      }
      team_sync<TW>();
      left = common[2];
      b = common[3];
      seg = common[4];
      off = common[5];
    }
    if (left > 0) {
      enter();
      off = min(off, units - 1);
    }
  }

  // Request b's length, as one warp of the team reads it.  (A place is written again
  // two requests later, when all have met in between.)
  __device__ __forceinline__ int common_length() {
    if constexpr (TW == 1) {
      return length_of(p, b);
    } else {
      const int at = entered++ & 1;
      if (member == 0) common[at] = length_of(p, b);
      team_sync<TW>();
      return common[at];
    }
  }

  // Request b's span (its segments have the same).
  __device__ __forceinline__ void enter() {
    span = span_of<KB>(p, common_length());
    units = units_of(p, span.blocks);
  }

  __device__ __forceinline__ int page_index(int j) const {
    return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
  }
  // Lane i: the page of the block i behind the looked-up one.
  __device__ __forceinline__ void load_pages() {
    page_lane = 0;
    const int j = row + lane * KB;
    if (j < span.hi) page = p.table[block_b * p.table_stride + page_index(j)];
  }

  // The next part: the rest of the range inside the current segment.
  __device__ __forceinline__ bool open_part() {
    do {
      if (left <= 0) return false;
      if (off >= units) {          // on to the next segment
        off = 0;
        if (++seg == segs) {
          seg = 0;
          if (++b >= p.batch) {
            left = 0;
            return false;
          }
          enter();
        }
      }
      const int upto = min(off + left, units);
      blk = max((off << p.unit_shift) - kSwitchBlocks, 0);
      end = min((upto << p.unit_shift) - kSwitchBlocks, span.blocks);
      left -= upto - off;
      off = upto;
    } while (blk >= end);          // all of it is the segment's beginning
    block_b = b;
    head = chunks == 1 ? seg : seg / chunks;
    id = b * segs + seg;
    row = (span.blk0 + blk) * KB;
    if constexpr (kTma) {
      tok = row - page_index(row) * p.page_size;
      load_pages();
    }
    return true;
  }

  __device__ __forceinline__ void look() {
    what = 0;
    if (blk >= end) {
      if (!open_part()) {
        what = kDone;
        return;
      }
      what = kPartBegins | (blk == 0 ? kSegBegins : 0);
    } else {
      row += KB;
      if constexpr (kTma) {
        tok += KB;
        if (tok >= p.page_size) tok = 0;
        if (++page_lane == 32) load_pages();
      }
    }
    if (row >= span.lo && row + KB <= span.hi) {
      what |= kAll;
    } else {
      const int n_lo = max(span.lo - row, 0), n_hi = min(span.hi - row, KB);
      if (n_hi > n_lo) what |= (kAll >> (KB - n_hi)) & ~((1 << n_lo) - 1);
    }
    if (++blk >= end)
      what |= kPartEnds | (end == span.blocks ? kSegEnds : 0);
    if constexpr (!kTma) {
      if ((what >> (lane % KB)) & 1) {
        const int j = row + lane % KB, idx = page_index(j);
        tok = j - idx * p.page_size;
        page = p.table[block_b * p.table_stride + idx];
      }
    }
  }

  // `dst`: the stage, number `stage`; `bar`: its barrier; `q_places`: the warp's
  // places for query rows.
  __device__ __forceinline__ void issue(int stage, uint32_t dst, uint32_t bar,
                                        uint32_t q_places) {
    if (what & kDone) {
      if (lane == stage) fifo_what = kDone;
    } else {
      // The part's query rows, if the warp has a free place.
      const T *q = nullptr;
      uint32_t q_bytes = 0, q_to = 0;
      if (what & kPartBegins) {
        if (p.q_chunks && parts - parts_free < Sh::QS) {
          const int h0 = (chunks == 1 ? 0 : (id - block_b * segs) % chunks * (RW * TW)) +
                         member * RW;
          q = static_cast<const T *>(p.q) + block_b * p.q_stride +
              int64_t(head * p.group + h0) * D;
          q_bytes = uint32_t(min(max(p.group - h0, 0), RW) * D * int(sizeof(T)));
          q_to = q_places + (parts % (Sh::QS > 0 ? Sh::QS : 1)) * Sh::kQ;
          if (q_bytes) what |= kRowsFetched;
        }
        ++parts;
      }
      if constexpr (kTma) {
        const int my_page = __shfl_sync(kFull, page, page_lane);
        if (uint32_t(my_page) >= uint32_t(p.num_pages)) {
          if (what & kAll) err = FA_PAGED_BAD_PAGE;
          what &= ~kAll;
        }
        const bool copies = (TW == 1 || member == 0) && (what & kAll);
        sm103::mbar_arrive_expect_tx_w(bar, (copies ? Sh::kStage : 0) + q_bytes);
        if (copies) {
          const int c1 = maps.token_first ? tok : head, c2 = maps.token_first ? head : tok;
#pragma unroll
          for (int i = 0; i < CPR / Tl::CPP; ++i)
            tma_load_panels_w(dst + i * KB * Tl::PB, dst + Sh::kBlock + i * KB * Tl::PB, maps, bar,
                              i * Tl::CPP * VEC, c1, c2, my_page);
        }
        if (q_bytes) sm103::bulk_load_w(q_to, q, q_bytes, bar);
      } else {
        const bool fine = uint32_t(page) < uint32_t(p.num_pages);
        const int mask = what & kAll & __ballot_sync(kFull, fine);
        if (mask != (what & kAll)) err = FA_PAGED_BAD_PAGE;
        what = (what & ~kAll) | mask;
        const int64_t at =
            fine ? page * p.page_stride + tok * p.token_stride + head * p.head_stride : 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int c = (i * TW + member) * 32 + lane, r = c / CPR, ch = c % CPR;
          const int64_t o = __shfl_sync(kFull, at, r % KB);
          const bool take = (mask >> (r % KB)) & 1;
          if (kChunks % (32 * TW) == 0 || c < kChunks) {
            const int64_t from = (take ? o : 0) + ch * VEC;
            cp_async16(dst + Tl::at(r, ch), static_cast<const T *>(p.kc) + from, take);
            cp_async16(dst + Sh::kBlock + Tl::at(r, ch), static_cast<const T *>(p.vc) + from, take);
          }
        }
        for (int i = lane; i < int(q_bytes) / 16; i += 32)
          cp_async16(q_to + i * 16, q + i * VEC, true);
      }
      if (lane == stage) {
        fifo_what = what;
        fifo_id = id;
      }
    }
    if constexpr (!kTma) cp_async_commit();
  }
};

// Rows of a V block that do not count may hold anything (TMA brings whole
// blocks): they become zeros, which the weight 0 then leaves as they are.
template <int ROW_BYTES, int KB>
__device__ __forceinline__ void clear_rows(uint8_t *v, uint32_t mask) {
  for (int i = threadIdx.x & 31; i < KB * (ROW_BYTES / 16); i += 32) {
    const int r = i / (ROW_BYTES / 16), ch = i % (ROW_BYTES / 16);
    if (!((mask >> r) & 1))
      *reinterpret_cast<uint4 *>(v + Tile<ROW_BYTES, KB>::at(r, ch)) = make_uint4(0, 0, 0, 0);
  }
}

// Whether the phase with parity `parity` is complete.
__device__ __forceinline__ bool test_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for it, at most `limit` ns, or until *abort (if given) is set by another warp of
// the CTA whose wait ran out.  A try_wait may sleep for as long as the hardware likes,
// so short limits are kept by polling.  The wait proper is out of line: in line it cost
// the largest kernels registers (32 requests of 2000 to 8192 keys, 32 heads on one,
// D 192: 40.9 us in line, 38.4 so).
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, long long limit,
                                       const volatile int *abort) {
  const bool sleeps = limit >= 10000000;
  const uint64_t t0 = sm103::global_timer_ns();
  while (true) {
    if (sleeps ? sm103::mbar_try_wait(bar, parity) : test_phase(bar, parity)) return true;
    if (abort && *abort) return false;
    if (static_cast<long long>(sm103::global_timer_ns() - t0) > limit) return false;
  }
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, long long limit,
                                           const volatile int *abort) {
  return test_phase(bar, parity) || wait_slow(bar, parity, limit, abort);
}

// How a team gives up.  A warp whose wait for a stage runs out (p.wait_ns) goes on to the
// next step, where it leaves the loop before it refills that stage, whose copies may
// still be on the way.  The other warps of its team leave there too: in between all meet
// at the team's barrier, and the stage's flag, which they read behind it, is not
// written again before they have met once more.  (Until then only the stage of the
// step before is refilled, whose copies are in.)  Nothing more is issued; what was, from
// the stage that took too long on, is waited for here, again for a limited time, so
// that no copy is on its way to the shared memory of a CTA that is gone.  The call then
// ends with wrong results and FA_PAGED_TIMEOUT.  `stage` and `parity` are those of
// the stage behind it.
constexpr long long kDrainNs = 2000000000LL;
__device__ __noinline__ void drain(uint32_t full, int stages, int fifo_what, int stage,
                                   uint32_t parity) {
  if (--stage < 0) {
    stage = stages - 1;
    parity ^= 1;
  }
  for (int i = 0; i < stages; ++i) {
    if (__shfl_sync(kFull, fifo_what, stage) & kDone) break;   // nor any behind it
    wait_phase(full + stage * 8, parity, kDrainNs, nullptr);
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
}

// Floats of one workspace slot: o [rows][d], then the rows' maxima and sums.
__host__ __device__ constexpr int slot_floats(int rows, int d) { return rows * (d + 4); }

__device__ __forceinline__ float *slot_of(const DecodeParams &p, int range, int slot) {
  return p.part + (int64_t(range) * 2 + slot) * slot_floats(p.slot_rows, p.d);
}

__device__ __forceinline__ void write_stats(const DecodeParams &p, int b, int n, float mx,
                                            float sum) {
  if (!p.smax) return;
  const int64_t at = (int64_t(b) * p.n + n) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p.smax[at + i] = mx;
    p.ssum[at + i] = sum;
  }
}

// The parts of a direct call's CTA, one per team: o in the team's ring, which is
// free by then.
template <int NT, int R>
struct Partials {
  float m[NT][R], l[NT][R];
  int state[NT];                    // kHas | kSegBegins | kSegEnds of the part
};
constexpr int kHas = 1;

// Adds the parts of a direct call's CTA, which are those of its first teams.  A
// warp takes one row at a time.  The sum goes to y if it is the whole segment, else
// to `cta_part`.
template <typename T, int D, int R, typename Sh>
__device__ __forceinline__ void merge_cta(const DecodeParams &p, int chunks,
                                          const Partials<Sh::NT, R> &s, const uint8_t *rings,
                                          float *cta_part) {
  constexpr int NT = Sh::NT, PITCH = D + Sh::PAD;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int state = lane < NT ? s.state[lane] : 0;
  const int count = __popc(__ballot_sync(kFull, state & kHas));
  if (count == 0) return;
  const bool whole = __any_sync(kFull, state & kSegBegins) && __any_sync(kFull, state & kSegEnds);
  const int segs = p.n_kv * chunks, id = blockIdx.x / p.direct, b = id / segs, seg = id - b * segs;
  const int hk = chunks == 1 ? seg : seg / chunks, h0 = (seg - hk * chunks) * R;
  const int n0 = hk * p.group + h0, rows = min(R, p.group - h0);
#pragma unroll 1
  for (int r = warp; r < rows; r += Sh::NW) {
    const int mine = lane < count ? lane : 0;
    const float m = s.m[mine][r], l = s.l[mine][r];
    float mx = m;
#pragma unroll
    for (int o = 1; o < NT; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    const float f = sm103::ex2(m - (mx == -CUDART_INF_F ? 0.f : mx));
    float sum = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll 2
    for (int k = 0; k < count; ++k) {
      const float fk = __shfl_sync(kFull, f, k);
      sum += fk * __shfl_sync(kFull, l, k);
      const float *o = reinterpret_cast<const float *>(rings + k * Sh::kRing) + r * PITCH + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] += fk * o[32 * i];
    }
    if (whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T *y = static_cast<T *>(p.y) + b * p.y_stride + int64_t(n0 + r) * D + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[32 * i] = from_f<T>(acc[i] * inv);
      if (lane == 0) write_stats(p, b, n0 + r, mx * kLn2, sum);
    } else {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) cta_part[r * D + lane + 32 * i] = acc[i];
      if (lane == 0) {
        cta_part[R * D + r] = mx;
        cta_part[R * D + R + r] = sum;
      }
    }
  }
}

// The sums of a cluster's CTAs, each at `cta_part` of its shared memory, to y.
// A warp of the cluster takes one row.
template <typename T, int D, int R, int NW, int NT, int KB>
__device__ __forceinline__ void join_cluster(const DecodeParams &p, int chunks,
                                             const float *cta_part) {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int lane = threadIdx.x & 31, segs = p.n_kv * chunks;
  const int id = blockIdx.x / p.direct;
  const int b = id / segs, seg = id - b * segs;
  const int blocks = span_of<KB>(p, length_of(p, b)).blocks;
  const int per = (blocks + p.direct * NT - 1) / (p.direct * NT);
  const int parts = (blocks + per * NT - 1) / (per * NT);   // CTAs that have blocks
  int r = (blockIdx.x - id * p.direct) * NW + (threadIdx.x >> 5);
#pragma unroll 1
  for (; parts > 1 && r < R; r += p.direct * NW) {
    const int h = (chunks == 1 ? 0 : seg % chunks * R) + r;
    if (h >= p.group) break;
    const int n = (chunks == 1 ? seg : seg / chunks) * p.group + h;
    const uint32_t at = sm103::smem_u32(cta_part);
    const auto remote = [](uint32_t addr, int rank) {
      uint32_t a;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
      return a;
    };
    const auto load = [&](int rank, int i) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(x)
                   : "r"(remote(at + i * 4, rank))
                   : "memory");
      return x;
    };
    const int mine = lane < parts ? lane : 0;
    const float m = load(mine, R * D + r), l = load(mine, R * D + R + r);
    float mx = m;
#pragma unroll
    for (int o = 1; o < kMaxDirect; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    const float f = sm103::ex2(m - (mx == -CUDART_INF_F ? 0.f : mx));
    float sum = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float fk = __shfl_sync(kFull, f, k);
      sum += fk * __shfl_sync(kFull, l, k);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] += fk * load(k, r * D + lane + 32 * i);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    T *y = static_cast<T *>(p.y) + b * p.y_stride + int64_t(n) * D + lane;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) y[32 * i] = from_f<T>(acc[i] * inv);
    if (lane == 0) write_stats(p, b, n, mx * kLn2, sum);
  }
  // No CTA may leave while another reads its shared memory.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Tensor-core kernel, 16-bit types
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a b, or c = a b.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, bool first = false) {
  const float z0 = first ? 0.f : c[0], z1 = first ? 0.f : c[1], z2 = first ? 0.f : c[2],
              z3 = first ? 0.f : c[3];
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2),
          "f"(z3));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2),
          "f"(z3));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return std::is_same<T, __nv_bfloat16>::value ? sm103::pack_bf16(lo, hi)
                                               : sm103::pack_f16(lo, hi);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  const T *h = reinterpret_cast<const T *>(&x);
  return make_float2(to_f(h[0]), to_f(h[1]));
}

// Rows per team and the warps that share it.
template <int R>
struct TcTeam {
  static constexpr int RW = R == 8 ? 8 : 16, TW = R / RW;
};
// Warps of a CTA.  8 have registers for D up to 192.  With D 32 a block takes a warp
// little more than latencies, which 16 hide better (16 and 8, in us: 64 requests of 4000
// keys, 32 heads on 4, 39 and 47; 16 on one 15 and 20; 64 on one 39 and 48; one of 2048
// keys 7.4 and 7.1), but for 32 rows (32 on one: 32 and 29).  With D 64 they cost what
// they gain (32 on 4: 67 and 58).  With D 192 and 16 rows 8 warps have room for two
// stages each, of which one is on the way; 4 have four (4 and 8, in us: 32 requests of
// 5000 keys, 16 heads on one, 32 and 37; 500 of up to 200, 32 on two, 38 and 46; one of
// 2048 12.4 and 13.6; but 16 of 2048, 32 on two, 20.3 and 16.4).
constexpr int tc_warps(int d, int r) {
  return d == 32 && r != 32 ? 16 : d == 192 && r == 16 ? 4 : 8;
}
template <int D, int R>
using TcShape = Shape<__half, D, TcTeam<R>::RW, TcTeam<R>::TW, 16, 0, tc_warps(D, R)>;

// S = Q K^T and O = P V by m16n8k16 products: Q's rows are the group's query
// heads, padded to 16, and a team takes 16 keys at a time through its own ring of
// S stages (K and V), S - 1 of which are on the way: the stage read in one step is
// filled again in the next.  The maximum and the sum run along; O is corrected only
// in steps in which some row's maximum grows.
//
// P goes into the second product as the sum of two 16-bit numbers, so that
// its rounding (2^-17 for bf16, 2^-23 for fp16) stays below y's own.  With 8 rows the
// two halves share one product: rows 0-7 hold P rounded, rows 8-15 what is left
// of it, and the halves of the result are added at the end.  With 16 rows they
// are two products.  fp16 gets P times 2^15, which its range allows, and O is scaled
// back at a part's end: without that a weight below 2^-14 of the row's largest would
// lose digits, and one below 2^-25 all of them, which many keys can add up to much of y.
//
// Bound by memory for a few query heads per key head: each key is read once, for
// 4 R operations per element.  One CTA of 4 to 16 warps per SM, each with a ring of its
// own, because what keeps HBM busy is bytes on the way (150 to 200 KB per SM) and no
// warp has to meet another.  64 requests of 2048 keys, 32 / 8 heads,
// D 128, bf16: 90 us, 6.0 TB/s, 26% of the issue slots; a warp waits for its copies
// and for latencies (products, exponentials, shuffles) in equal parts.  At D 32 and 64 a
// block of 16 keys is so few bytes that what a warp does once per block bounds it (64
// requests of 4000 keys, 8 / 8 heads, D 32: 93 us for 39 us of bytes; 32 / 4, D 64: 57 for
// 39), and from about 16 rows the products' latency does (32 requests of 2000 to 8192 keys,
// 32 heads on one, D 192: 38 us, 108 TFLOP/s; 32 of 5000, 64 on one, D 128: 51 us for 12).
//
// mma.sync: with up to 16 query heads per key head the heads fill 8 or 16 of the 128 rows
// that tcgen05 multiplies at once.  With more heads, or with keys for rows, tcgen05
// would fit; such a kernel has not been built.  Not faster: a warp that only loads,
// K and V awaited apart, ranges taken from a counter.
template <typename T, int D, int R, bool kTma>
__global__ void __launch_bounds__(TcShape<D, R>::NW * 32, 1)
decode_tc_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ DecodeMaps maps) {
  using Sh = TcShape<D, R>;
  using Tl = Tile<D * 2, 16>;
  constexpr int RW = TcTeam<R>::RW, TW = TcTeam<R>::TW;
  constexpr int KB = 16, S = Sh::S, NW = Sh::NW, NT = Sh::NT;
  constexpr int NR = RW / 8;        // rows of a lane
  constexpr float kUp = std::is_same<T, __half>::value ? 32768.f : 1.f;   // P's factor
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Partials<NT, R> s_part;
  __shared__ uint64_t s_full[NT][S];
  __shared__ int s_abort;
  __shared__ volatile uint8_t s_gave_up[TW > 1 ? NT : 1][S];   // see drain
  __shared__ volatile int s_common[TW > 1 ? NT : 1][6];        // see Loader
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / TW;
  const int row0 = warp % TW * RW;  // first row of the team's that is the warp's
  uint8_t *my = smem + team * Sh::kRing;
  const uint32_t ring = sm103::smem_u32(my);
  const uint32_t q_places = sm103::smem_u32(smem) + NT * Sh::kRing + warp * Sh::kWarpExtra;
  const uint32_t full = sm103::smem_u32(&s_full[team][0]);
  const T *q = static_cast<const T *>(p.q);
  const int chunks = (p.group + R - 1) / R, segs = p.n_kv * chunks;
  if (lane == 0) s_part.state[team] = 0;
  if constexpr (kTma) {
    if (threadIdx.x == 0) {
      sm103::tma_prefetch_map(&maps.k);
      sm103::tma_prefetch_map(&maps.v);
      s_abort = 0;
      for (int i = 0; TW > 1 && i < NT * S; ++i) s_gave_up[i / S][i % S] = 0;
      for (int i = 0; i < NT * S; ++i) sm103::mbar_init(sm103::smem_u32(&s_full[0][0] + i), TW);
      sm103::mbar_fence_init();
    }
    __syncthreads();
  }

  // Launched while the kernel before on the stream may still run: nothing in
  // memory is read or written before this.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The join reads the lengths as soon as it runs, so it may not before this.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Loader<T, D, Sh, RW, TW, KB, kTma> load(p, maps, chunks, s_common[TW > 1 ? team : 0]);
  load.look();
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) {
    load.issue(i, ring + i * Sh::kStage, full + i * 8, q_places);
    load.look();
  }

  const int row = lane >> 2, col = (lane & 3) * 2;
  // ldmatrix addresses inside a block, K (n = key, k = dim) and V (transposed), of
  // chunk pairs: pair c of a panel is at the first one's address ^ 32 c, since
  // panels' rows begin at multiples of their length.
  constexpr int kPairs = Tl::CPP / 2;              // per panel
  const int k_at = Tl::at((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
  const int v_at = Tl::at((lane & 7) + (((lane >> 3) & 1) << 3), lane >> 4);
  int stage = 0, fill = S - 1, heads = 0, n0 = 0, id = 0, b = 0;
  uint32_t parity = 0;
  uint32_t qa[D / 16][2 * NR];
  float o[D / 8][4];
  float m[NR], l[NR];
  bool opens = false, gave_up = false;

#pragma unroll 1
  while (true) {
    if constexpr (!kTma) cp_async_wait<S - 2>();
    team_sync<TW>();                // the stage to fill has been read
    if constexpr (kTma && TW == 1) gave_up = __any_sync(kFull, gave_up);
    const int what = __shfl_sync(kFull, load.fifo_what, stage);
    if ((what & kDone) || (TW == 1 && gave_up)) break;
    if constexpr (kTma) {
      if (!wait_phase(full + stage * 8, parity, p.wait_ns, &s_abort)) {
        s_abort = 1;
        if constexpr (TW == 1)
          gave_up = true;
        else
          s_gave_up[team][stage] = 1;
      }
      if (TW > 1 && s_gave_up[team][fill]) break;
    }
    const uint32_t kb = ring + stage * Sh::kStage, vb = kb + Sh::kBlock;

    if (what & kPartBegins) {
      opens = what & kSegBegins;
      id = __shfl_sync(kFull, load.fifo_id, stage);
      b = id / segs;
      const int seg = id - b * segs, hk = chunks == 1 ? seg : seg / chunks;
      const int h0 = (chunks == 1 ? 0 : (seg - hk * chunks) * R) + row0;
      heads = min(RW, p.group - h0);           // may be negative
      n0 = hk * p.group + h0;
      if (what & kRowsFetched) {
        // Fragments by ldmatrix: rows behind the last head hold anything, and
        // nothing reads their results.
        const uint32_t qs = q_places + load.parts_free % (Sh::QS > 0 ? Sh::QS : 1) * Sh::kQ;
        const int q_row = NR == 1 ? (lane & 7) : (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += NR == 1 ? 2 : 1) {
          uint32_t x[4];
          const int ch = ks * 2 + (NR == 1 ? lane >> 3 : lane >> 4);
          ldsm4(x, qs + q_row * (D * 2) + ch * 16);
          if constexpr (NR == 1) {
            qa[ks][0] = x[0];
            qa[ks][1] = x[1];
            qa[ks + 1][0] = x[2];
            qa[ks + 1][1] = x[3];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[ks][i] = x[i];
          }
        }
        __syncwarp();               // the place is free
      } else {
        // Rows behind the last head repeat it.
        const T *qr = q + b * p.q_stride + int64_t(n0 - row0) * D;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) {
          // Fragment i of a step: rows row (and row + 8 for odd i with 16).
          const int r = min(row0 + row + (NR == 2 ? (i & 1) * 8 : 0),
                            max(heads + row0, 1) - 1);
          const uint16_t *h = reinterpret_cast<const uint16_t *>(
              qr + r * D + col + (NR == 2 ? i >> 1 : i) * 8);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            qa[ks][i] = uint32_t(h[ks * 16]) | uint32_t(h[ks * 16 + 1]) << 16;
        }
      }
      ++load.parts_free;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        m[i] = -CUDART_INF_F;
        l[i] = 0.f;
      }
    }
    load.issue(fill, ring + fill * Sh::kStage, full + fill * 8, q_places);
    load.look();
    fill = fill + 1 == S ? 0 : fill + 1;
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
    const int mask = what & 0xffff;
    if (kTma && mask != 0xffff) {
      // Each warp of the team clears them all, so none waits for another.
      clear_rows<D * 2, KB>(my + (vb - ring), mask);
      __syncwarp();
    }

    float sa[2][2][4];              // [chain][key half][fragment]
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t kf[4];
      ldsm4(kf, (kb + ks / kPairs * (KB * Tl::PB) + k_at) ^ (ks % kPairs * 32));
      uint32_t a[4];
      if constexpr (NR == 1) {
        a[0] = qa[ks][0];
        a[1] = 0;
        a[2] = qa[ks][1];
        a[3] = 0;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = qa[ks][i];
      }
      mma16816<T>(sa[ks & 1][0], a, kf[0], kf[1], ks < 2);
      mma16816<T>(sa[ks & 1][1], a, kf[2], kf[3], ks < 2);
    }
    float s[NR][4];                 // keys col, col + 1, col + 8, col + 9
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[i][e] = (sa[0][e >> 1][i * 2 + (e & 1)] + sa[1][e >> 1][i * 2 + (e & 1)]) * p.scale_log2;
    if (mask != 0xffff) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!((mask >> (col + (e & 1) + (e >> 1) * 8)) & 1)) {
#pragma unroll
          for (int i = 0; i < NR; ++i) s[i][e] = -CUDART_INF_F;
        }
    }
    float mn[NR];
    bool grows = false;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float t = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
      t = fmaxf(t, __shfl_xor_sync(kFull, t, 1));
      t = fmaxf(t, __shfl_xor_sync(kFull, t, 2));
      mn[i] = fmaxf(m[i], t);
      grows |= mn[i] > m[i];
    }
    if (__any_sync(kFull, grows)) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float f = m[i] == mn[i] ? 1.f : sm103::ex2(m[i] - mn[i]);
        m[i] = mn[i];
        l[i] *= f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          if constexpr (NR == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][e] *= f;
          } else {
            o[k][i * 2] *= f;
            o[k][i * 2 + 1] *= f;
          }
        }
      }
    }
    uint32_t hi[NR][2], lo[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float ref = m[i] == -CUDART_INF_F ? 0.f : m[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = sm103::ex2(s[i][e] - ref);
      l[i] += (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = s[i][2 * h] * kUp, p1 = s[i][2 * h + 1] * kUp;
        hi[i][h] = pack2<T>(p0, p1);
        const float2 back = unpack2<T>(hi[i][h]);
        lo[i][h] = pack2<T>(p0 - back.x, p1 - back.y);
      }
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      uint32_t vf[4];
      ldsm4_t(vf, (vb + dt / kPairs * (KB * Tl::PB) + v_at) ^ (dt % kPairs * 32));
      if constexpr (NR == 1) {
        const uint32_t a[4] = {hi[0][0], lo[0][0], hi[0][1], lo[0][1]};
        mma16816<T>(o[2 * dt], a, vf[0], vf[1]);
        mma16816<T>(o[2 * dt + 1], a, vf[2], vf[3]);
      } else {
        const uint32_t a[4] = {hi[0][0], hi[1][0], hi[0][1], hi[1][1]};
        const uint32_t c[4] = {lo[0][0], lo[1][0], lo[0][1], lo[1][1]};
        mma16816<T>(o[2 * dt], a, vf[0], vf[1]);
        mma16816<T>(o[2 * dt + 1], a, vf[2], vf[3]);
        mma16816<T>(o[2 * dt], c, vf[0], vf[1]);
        mma16816<T>(o[2 * dt + 1], c, vf[2], vf[3]);
      }
    }

    if (kTma && mask != 0xffff) sm103::fence_proxy_async_smem();   // before the next copy there

    if (what & kPartEnds) {
      const bool ends = what & kSegEnds;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        l[i] += __shfl_xor_sync(kFull, l[i], 1);
        l[i] += __shfl_xor_sync(kFull, l[i], 2);
      }
      if constexpr (kUp != 1.f) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][k] *= 1.f / kUp;
      }
      if (opens && ends) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = row + i * 8;
          if (r >= heads) continue;
          const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
          T *y = static_cast<T *>(p.y) + b * p.y_stride + int64_t(n0 + r) * D + col;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            const float x0 = (NR == 1 ? o[k][0] + o[k][2] : o[k][i * 2]) * inv;
            const float x1 = (NR == 1 ? o[k][1] + o[k][3] : o[k][i * 2 + 1]) * inv;
            if (p.y_pairs) {
              *reinterpret_cast<uint32_t *>(y + k * 8) = pack2<T>(x0, x1);
            } else {
              y[k * 8] = from_f<T>(x0);
              y[k * 8 + 1] = from_f<T>(x1);
            }
          }
          if ((lane & 3) == 0) write_stats(p, b, n0 + r, m[i] * kLn2, l[i]);
        }
      } else {
        // To the workspace, or, in a direct call, to shared memory: the ring, whose
        // last block this was.
        team_sync<TW>();
        const int pitch = p.direct ? D + Sh::PAD : D;
        float *slot = slot_of(p, blockIdx.x * NT + team, opens ? 1 : 0);
        float *dst = p.direct ? reinterpret_cast<float *>(my) : slot;
        float *dst_m = p.direct ? s_part.m[team] : slot + p.slot_rows * D;
        float *dst_l = p.direct ? s_part.l[team] : slot + p.slot_rows * (D + 1);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          if (row + i * 8 >= heads) continue;
          const int r = row0 + row + i * 8;
          if ((lane & 3) == 0) {
            dst_m[r] = m[i];
            dst_l[r] = l[i];
          }
#pragma unroll
          for (int k = 0; k < D / 8; ++k)
            *reinterpret_cast<float2 *>(dst + r * pitch + col + k * 8) =
                NR == 1 ? make_float2(o[k][0] + o[k][2], o[k][1] + o[k][3])
                       : make_float2(o[k][i * 2], o[k][i * 2 + 1]);
        }
        if (lane == 0)
          s_part.state[team] = kHas | (opens ? kSegBegins : 0) | (ends ? kSegEnds : 0);
      }
    }
  }
  if constexpr (kTma && TW > 1) gave_up = s_gave_up[team][fill];
  if (kTma && gave_up) {
    load.err |= FA_PAGED_TIMEOUT;
    drain(full, S, load.fifo_what, stage, parity);
  }
  if (p.direct) {
    __syncthreads();
    float *cta_part = reinterpret_cast<float *>(smem + NT * Sh::kRing);
    merge_cta<T, D, R, Sh>(p, chunks, s_part, smem, cta_part);
    if (p.direct > 1) join_cluster<T, D, R, NW, NT, KB>(p, chunks, cta_part);
  }
  if (load.err && p.error) atomicOr(p.error, load.err);
}

// ---------------------------------------------------------------------------
// fp32 kernel, on the CUDA cores
// ---------------------------------------------------------------------------
template <int D, int R>
using SimtShape = Shape<float, D, R, 1, 8, 8 * R * 4, 8>;

// Products in full fp32, which no tensor instruction offers.  A warp takes 8 keys at a
// time.  Scores: four lanes per key, each a quarter of the dims (every fourth chunk),
// so that a sum needs two shuffles and the banks do not collide.  Output: each lane
// D / 32 dims of all R heads, in registers; the keys' weights pass through shared
// memory.  Query rows are read from registers where a lane's quarter of them takes at
// most 128 (R D <= 512), else from shared memory for every block of keys.  Bound by
// memory with one or two heads per key head (16 requests of 2048 keys, 8 heads each
// with its own keys, D 128: 47 us, 5.7 TB/s), by shared memory and shuffles above that
// (32 heads on 8: 52 us, 62 with the rows in shared memory; 64 on 8, where they are:
// 96 us).
template <int D, int R, bool kTma>
__global__ void __launch_bounds__(SimtShape<D, R>::NW * 32, 1)
decode_simt_kernel(const __grid_constant__ DecodeParams p,
                   const __grid_constant__ DecodeMaps maps) {
  using Sh = SimtShape<D, R>;
  constexpr int KB = 8, S = Sh::S, NW = Sh::NW;
  using Tl = Tile<D * 4, KB>;
  constexpr int CPR = D / 4;
  constexpr int VW = D % 128 == 0 ? 4 : D % 64 == 0 ? 2 : 1;   // dims per access
  constexpr int NV = D / (32 * VW);                             // accesses per row
  constexpr bool kQRegs = R * D <= 512;   // query rows in registers
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Partials<NW, R> s_part;
  __shared__ uint64_t s_full[NW][S];
  __shared__ int s_abort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t *my = smem + warp * Sh::kRing;
  uint8_t *extra = smem + NW * Sh::kRing + warp * Sh::kWarpExtra;
  const uint32_t ring = sm103::smem_u32(my), q_places = sm103::smem_u32(extra);
  float *s_p = reinterpret_cast<float *>(extra + Sh::QS * Sh::kQ);   // weights [8][R]
  float *s_q = nullptr;                                               // the part's query rows
  const int chunks = (p.group + R - 1) / R, segs = p.n_kv * chunks;
  if (lane == 0) s_part.state[warp] = 0;

  const uint32_t full = sm103::smem_u32(&s_full[warp][0]);
  if constexpr (kTma) {
    if (threadIdx.x == 0) {
      sm103::tma_prefetch_map(&maps.k);
      sm103::tma_prefetch_map(&maps.v);
      s_abort = 0;
      for (int i = 0; i < NW * S; ++i) sm103::mbar_init(sm103::smem_u32(&s_full[0][0] + i), 1);
      sm103::mbar_fence_init();
    }
    __syncthreads();
  }

  asm volatile("griddepcontrol.wait;" ::: "memory");   // as above
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Loader<float, D, Sh, R, 1, KB, kTma> load(p, maps, chunks, nullptr);
  load.look();
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) {
    load.issue(i, ring + i * Sh::kStage, full + i * 8, q_places);
    load.look();
  }

  const int key = lane >> 2, quarter = lane & 3;
  int stage = 0, fill = S - 1, heads = 0, n0 = 0, id = 0, b = 0;
  uint32_t parity = 0;
  float o[R][NV * VW], m[R], l[R];
  float4 q_own[kQRegs ? R : 1][kQRegs ? CPR / 4 : 1];
  bool opens = false, gave_up = false;

#pragma unroll 1
  while (true) {
    if constexpr (!kTma) cp_async_wait<S - 2>();
    __syncwarp();                    // the stage to fill has been read
    if constexpr (kTma) gave_up = __any_sync(kFull, gave_up);
    const int what = __shfl_sync(kFull, load.fifo_what, stage);
    if ((what & kDone) || gave_up) break;
    if (what & kPartBegins) id = __shfl_sync(kFull, load.fifo_id, stage);
    if constexpr (kTma) {
      if (!wait_phase(full + stage * 8, parity, p.wait_ns, &s_abort)) gave_up = s_abort = true;
    }
    uint8_t *kb = my + stage * Sh::kStage, *vb = kb + Sh::kBlock;
    load.issue(fill, ring + fill * Sh::kStage, full + fill * 8, q_places);
    load.look();
    fill = fill + 1 == S ? 0 : fill + 1;
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
    const int mask = what & 0xff;
    if (kTma && mask != 0xff) clear_rows<D * 4, KB>(vb, mask);

    if (what & kPartBegins) {
      opens = what & kSegBegins;
      b = id / segs;
      const int seg = id - b * segs, hk = chunks == 1 ? seg : seg / chunks;
      const int h0 = chunks == 1 ? 0 : (seg - hk * chunks) * R;
      heads = min(R, p.group - h0);
      n0 = hk * p.group + h0;
      // A part keeps its place until it ends.
      s_q = reinterpret_cast<float *>(extra + load.parts_free % Sh::QS * Sh::kQ);
      if (!(what & kRowsFetched)) {
        const float *qr = static_cast<const float *>(p.q) + b * p.q_stride + int64_t(n0) * D;
        for (int i = lane; i < heads * D; i += 32) s_q[i] = qr[i];
        if (kTma) sm103::fence_proxy_async_smem();   // before a later copy to this place
        __syncwarp();
      }
      if constexpr (kQRegs) {
#pragma unroll
        for (int i = 0; i < CPR / 4; ++i) {
          const int c = (i * 4 + quarter) ^ ((key & 1) << 2);
#pragma unroll
          for (int r = 0; r < R; ++r)
            q_own[r][i] = *reinterpret_cast<const float4 *>(s_q + r * D + c * 4);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = -CUDART_INF_F;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < NV * VW; ++i) o[r][i] = 0.f;
      }
    }

    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 0.f;
#pragma unroll
    for (int i = 0; i < CPR / 4; ++i) {
      // Odd keys take the other half of a panel, for the banks' sake.
      const int c = (i * 4 + quarter) ^ ((key & 1) << 2);
      const float4 kv = *reinterpret_cast<const float4 *>(kb + Tl::at(key, c));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float4 qv;
        if constexpr (kQRegs)
          qv = q_own[r][i];
        else
          qv = *reinterpret_cast<const float4 *>(s_q + r * D + c * 4);
        s[r] = fmaf(kv.x, qv.x, s[r]);
        s[r] = fmaf(kv.y, qv.y, s[r]);
        s[r] = fmaf(kv.z, qv.z, s[r]);
        s[r] = fmaf(kv.w, qv.w, s[r]);
      }
    }
    const bool ok = (what >> key) & 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] += __shfl_xor_sync(kFull, s[r], 1);
      s[r] += __shfl_xor_sync(kFull, s[r], 2);
      s[r] = ok ? s[r] * p.scale_log2 : -CUDART_INF_F;
      float t = s[r];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, x));
      const float mn = fmaxf(m[r], t);
      if (mn > m[r]) {               // the same for the whole warp
        const float f = exp2f(m[r] - mn);
        m[r] = mn;
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < NV * VW; ++i) o[r][i] *= f;
      }
      s[r] = exp2f(s[r] - (m[r] == -CUDART_INF_F ? 0.f : m[r]));
      l[r] += s[r];                  // each key's weight in its four lanes
    }
    if (quarter == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) s_p[key * R + r] = s[r];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      float pk[R];
#pragma unroll
      for (int r = 0; r < R; ++r) pk[r] = s_p[k * R + r];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int d = (i * 32 + lane) * VW;
        const float *src = reinterpret_cast<const float *>(vb + Tl::at(k, d >> 2)) + (d & 3);
        float v[VW];
        if constexpr (VW == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(src);
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else if constexpr (VW == 2) {
          const float2 x = *reinterpret_cast<const float2 *>(src);
          v[0] = x.x; v[1] = x.y;
        } else {
          v[0] = *src;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < VW; ++e) o[r][i * VW + e] = fmaf(pk[r], v[e], o[r][i * VW + e]);
      }
    }

    if (kTma && mask != 0xff) sm103::fence_proxy_async_smem();   // before the next copy there

    if (what & kPartEnds) {
      ++load.parts_free;
      const bool ends = what & kSegEnds;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[r] += __shfl_xor_sync(kFull, l[r], x);
      }
      const bool whole = opens && ends;
      __syncwarp();                  // the ring has been read
      const int pitch = p.direct ? D + Sh::PAD : D;
      float *slot = slot_of(p, blockIdx.x * NW + warp, opens ? 1 : 0);
      float *dst = p.direct ? reinterpret_cast<float *>(my) : slot;
      float *dst_m = p.direct ? s_part.m[warp] : slot + p.slot_rows * D;
      float *dst_l = p.direct ? s_part.l[warp] : slot + p.slot_rows * (D + 1);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= heads) continue;
        const float inv = whole ? (l[r] == 0.f ? 0.f : 1.f / l[r]) : 1.f;
        float *to = whole ? static_cast<float *>(p.y) + b * p.y_stride + int64_t(n0 + r) * D
                          : dst + r * pitch;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VW; ++e) to[(i * 32 + lane) * VW + e] = o[r][i * VW + e] * inv;
        if (lane == 0) {
          if (whole) {
            write_stats(p, b, n0 + r, m[r] * kLn2, l[r]);
          } else {
            dst_m[r] = m[r];
            dst_l[r] = l[r];
          }
        }
      }
      if (lane == 0 && !whole)
        s_part.state[warp] = kHas | (opens ? kSegBegins : 0) | (ends ? kSegEnds : 0);
    }
  }
  if (kTma && gave_up) {
    load.err |= FA_PAGED_TIMEOUT;
    drain(full, S, load.fifo_what, stage, parity);
  }
  if (p.direct) {
    __syncthreads();
    float *cta_part = reinterpret_cast<float *>(smem + NW * Sh::kRing);
    merge_cta<float, D, R, Sh>(p, chunks, s_part, smem, cta_part);
    if (p.direct > 1) join_cluster<float, D, R, NW, NW, KB>(p, chunks, cta_part);
  }
  if (load.err && p.error) atomicOr(p.error, load.err);
}

// ---------------------------------------------------------------------------
// Adds the parts of the segments that were cut.  Which ranges share a segment
// follows from the lengths alone, so that is worked out before the main kernel is
// done.  Block x takes segment x, or, where there are more segments than ranges,
// the segment in which range x ends.  WPR warps take a query head's parts in turn,
// so that their loads overlap, and meet in shared memory, always in the same order.
// Bound by latency: a chain of two dependent loads (lengths, parts) and the launch,
// of which the first and the last hide behind the main kernel.  About 3 us of a call
// that is cut (16 requests of 512 keys: 11.7 us, of which 8.9 remain without the join
// and the search for ranges).
// ---------------------------------------------------------------------------
template <typename T, int D, int KB, int WPR>
__global__ void __launch_bounds__(WPR > 8 ? WPR * 32 : 256) join_kernel(
    const __grid_constant__ DecodeParams p, int by_segment) {
  constexpr int PL = D / 32;
  constexpr int kJoinWarps = WPR > 8 ? WPR : 8;
  constexpr int U = WPR > 8 ? 4 : 2;   // parts on the way at once, per warp
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float s_o[WPR > 1 ? kJoinWarps : 1][D];
  __shared__ int s_b, s_seg, s_first, s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = (p.group + p.rows - 1) / p.rows, segs = p.n_kv * chunks;
  // The lengths come past the L1 (length_of), so one warp reads them for all (eight:
  // 1024 requests of 64 keys 80 us, one: 69), but where they are few and the blocks many
  // each for itself (64 of 2048 keys, 32 heads on 8: 91.5 us, with one 94).
  int b = 0, seg = 0, i = 0, last = 0;
  const bool alone = WPR == 1 && by_segment;
  if (alone || warp == 0) {
    Line line;
    Place at{0, 0, 0, 1};
    int first_unit;                  // of the segment
    if (by_segment) {
      at.b = blockIdx.x / segs;
      at.seg = blockIdx.x - at.b * segs;
      first_unit = segment_start<KB>(p, segs, at, line);
    } else {
      find<KB, true>(p, segs, blockIdx.x + 1, 1, line, at);
      first_unit = line.start(blockIdx.x + 1) - 1 - at.off;
    }
    b = at.b;
    seg = at.seg;
    i = line.range_of(first_unit + (kSwitchBlocks >> p.unit_shift));
    last = min(line.range_of(first_unit + at.units - 1), p.ranges - 1);
    if (!alone && lane == 0) {
      s_b = b;
      s_seg = seg;
      s_first = i;
      s_last = last;
    }
  }
  if (!alone) {
    __syncthreads();
    b = s_b, seg = s_seg, i = s_first, last = s_last;
  }
  const int hk = chunks == 1 ? seg : seg / chunks, h0 = (seg - hk * chunks) * p.rows;
  const int rows = min(p.rows, p.group - h0);

  asm volatile("griddepcontrol.launch_dependents;");
  // Every block waits, also one with nothing to do: what follows on the stream
  // is behind the main kernel only through this one.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i >= last || (!by_segment && i != int(blockIdx.x))) return;
  const int parts = last - i + 1;
#pragma unroll 1
  for (int r = blockIdx.y * (kJoinWarps / WPR) + warp / WPR; r < rows;
       r += gridDim.y * (kJoinWarps / WPR)) {
    // Part 0 is in range i's slot 1, part k in range (i + k)'s slot 0.
    float mx = -CUDART_INF_F, sum = 0.f, acc[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) acc[k] = 0.f;
#pragma unroll 1
    for (int j0 = warp % WPR; j0 < parts; j0 += U * WPR) {
      float m2[U], l2[U], o2[U][PL];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = min(j0 + u * WPR, parts - 1);
        const float *src = slot_of(p, i + j, j == 0 ? 1 : 0);
        m2[u] = src[p.slot_rows * D + r];
        l2[u] = src[p.slot_rows * (D + 1) + r];
#pragma unroll
        for (int k = 0; k < PL; ++k) o2[u][k] = src[r * D + lane + 32 * k];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j0 + u * WPR >= parts) break;
        const float mn = fmaxf(mx, m2[u]), ref = mn == -CUDART_INF_F ? 0.f : mn;
        const float f = sm103::ex2(mx - ref), f2 = sm103::ex2(m2[u] - ref);
        mx = mn;
        sum = sum * f + l2[u] * f2;
#pragma unroll
        for (int k = 0; k < PL; ++k) acc[k] = acc[k] * f + o2[u][k] * f2;
      }
    }
    const int n = hk * p.group + h0 + r;
    T *y = static_cast<T *>(p.y) + b * p.y_stride + int64_t(n) * D;
    if constexpr (WPR == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int k = 0; k < PL; ++k) y[lane + 32 * k] = from_f<T>(acc[k] * inv);
      if (lane == 0) write_stats(p, b, n, mx * kLn2, sum);
    } else {
      // All warps are here: WPR is the whole block, and r its row.
      __syncthreads();
      if (lane == 0) {
        s_m[warp] = mx;
        s_l[warp] = sum;
      }
#pragma unroll
      for (int k = 0; k < PL; ++k) s_o[warp][lane + 32 * k] = acc[k];
      __syncthreads();
      const int d = threadIdx.x;
      if (d < D) {
        float top = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) top = fmaxf(top, s_m[k]);
        const float ref = top == -CUDART_INF_F ? 0.f : top;
        float total = 0.f, out = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) {
          const float f = sm103::ex2(s_m[k] - ref);
          total += f * s_l[k];
          out += f * s_o[k][d];
        }
        y[d] = from_f<T>(total == 0.f ? 0.f : out / total);
        if (d == 0) write_stats(p, b, n, top * kLn2, total);
      }
    }
  }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn decode_encode_fn() {
  static const EncodeFn fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeFn>(ptr);
  }();
  return fn;
}

// The cache as a 4-D tensor.  False: a block of KB keys may leave its page, or the
// strides are not those of nested axes, as TMA wants them.
template <typename T, int D, int KB>
bool make_page_maps(DecodeMaps &maps, const DecodeParams &p) {
  using Tl = Tile<D * int(sizeof(T)), KB>;
  const EncodeFn enc = decode_encode_fn();
  if (enc == nullptr || p.page_size % KB != 0) return false;
  const int64_t count[3] = {p.n_kv, p.page_size, p.num_pages};
  const int64_t stride[3] = {p.head_stride, p.token_stride, p.page_stride};
  cuuint64_t dims[4] = {D}, strides[3];
  cuuint32_t box[4] = {Tl::PB / sizeof(T), 1, 1, 1};
  const auto nested = [&](bool token_first) {
    const int order[3] = {token_first ? 1 : 0, token_first ? 0 : 1, 2};
    int64_t inner = 1, extent = D;   // stride and extent of the axis before, in elements
    for (int i = 0; i < 3; ++i) {
      const int a = order[i];
      const int64_t own = count[a] == 1 ? extent : stride[a];   // (an axis of one: any will do)
      if (own < extent || own % inner != 0 || own * int64_t(sizeof(T)) % 16 != 0 ||
          own * int64_t(sizeof(T)) >= (int64_t(1) << 40))
        return false;
      inner = own;
      extent = own * count[a];
      dims[i + 1] = cuuint64_t(count[a]);
      strides[i] = cuuint64_t(own) * sizeof(T);
      box[i + 1] = a == 1 ? KB : 1;
    }
    maps.token_first = token_first;
    return true;
  };
  if (!nested(false) && !nested(true)) return false;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type =
      std::is_same<T, float>::value    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
      : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto encode = [&](CUtensorMap *map, const void *base) {
    return enc(map, type, 4, const_cast<void *>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               Tl::PB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return encode(&maps.k, p.kc) && encode(&maps.v, p.vc);
}

// The main kernel and the join, which is launched as its dependent so that its
// launch overlaps the main kernel's run.
template <typename T, int D, typename Sh, int KB, typename Kernel>
cudaError_t launch_shape(DecodeParams p, Kernel with_tma, Kernel without, int sms,
                         cudaStream_t s) {
  constexpr int R = Sh::R, NW = Sh::NW, NT = Sh::NT;
  const int64_t segments = int64_t(p.batch) * p.n_kv * ((p.group + R - 1) / R);
  DecodeMaps maps;
  const bool tma = make_page_maps<T, D, KB>(maps, p);
  const Kernel kernel = tma ? with_tma : without;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  // Both kernels may be launched before the one before them is done, and wait for
  // it themselves.  A captured main kernel is not: what precedes it in a graph may
  // be no kernel.
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if ((e = cudaStreamIsCapturing(s, &capture)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.stream = s;
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.attrs = capture == cudaStreamCaptureStatusNone ? attrs : attrs + 1;
  cfg.numAttrs = capture == cudaStreamCaptureStatusNone ? 1 : 0;
  if (p.direct) {
    cfg.gridDim = dim3(unsigned(segments) * p.direct);
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = p.direct;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    ++cfg.numAttrs;
    return cudaLaunchKernelEx(&cfg, kernel, p, maps);
  }
  p.ranges = sms * NT;
  const int64_t blocks = (int64_t(p.max_pages) * p.page_size + KB - 1) / KB + 1 + kSwitchBlocks;
  p.unit_shift = 0;
  while (segments * ((blocks >> p.unit_shift) + 1) >= (int64_t(1) << 31)) ++p.unit_shift;
  cfg.gridDim = dim3(sms);
  if ((e = cudaLaunchKernelEx(&cfg, kernel, p, maps)) != cudaSuccess) return e;
  // 32 warps per query head where a segment has 16 parts and more and two such
  // blocks per SM suffice (152 parts take 2 us so, 10 us with 8 warps; 1024 heads of
  // 19 parts take 13 us less with 8); then 8 warps, and one where the GPU does not
  // hold blocks of those for all heads.
  const int by_segment = segments <= p.ranges;
  const int64_t heads = segments * p.slot_rows;
  const int warps = segments * 16 <= p.ranges && heads <= 2 * sms ? 32 : heads <= 8 * sms ? 8 : 1;
  cfg.gridDim = dim3(unsigned(by_segment ? segments : p.ranges),
                     unsigned(warps > 1 ? p.slot_rows : (p.slot_rows + 7) / 8));
  cfg.blockDim = dim3(warps == 32 ? 1024 : 256);
  cfg.dynamicSmemBytes = 0;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  return warps == 32  ? cudaLaunchKernelEx(&cfg, join_kernel<T, D, KB, 32>, p, by_segment)
         : warps == 8 ? cudaLaunchKernelEx(&cfg, join_kernel<T, D, KB, 8>, p, by_segment)
                      : cudaLaunchKernelEx(&cfg, join_kernel<T, D, KB, 1>, p, by_segment);
}

template <typename T, int D, int R>
cudaError_t launch_tc_rows(const DecodeParams &p, int sms, cudaStream_t s) {
  return launch_shape<T, D, TcShape<D, R>, 16>(p, decode_tc_kernel<T, D, R, true>,
                                               decode_tc_kernel<T, D, R, false>, sms, s);
}

template <typename T, int D>
cudaError_t launch_tc(const DecodeParams &p, int sms, cudaStream_t s) {
  switch (p.rows) {
    case 8: return launch_tc_rows<T, D, 8>(p, sms, s);
    case 16: return launch_tc_rows<T, D, 16>(p, sms, s);
    case 32: return launch_tc_rows<T, D, 32>(p, sms, s);
    default: return launch_tc_rows<T, D, 64>(p, sms, s);
  }
}

template <int D, int R>
cudaError_t launch_simt_rows(const DecodeParams &p, int sms, cudaStream_t s) {
  return launch_shape<float, D, SimtShape<D, R>, 8>(p, decode_simt_kernel<D, R, true>,
                                                    decode_simt_kernel<D, R, false>, sms, s);
}

template <int D>
cudaError_t launch_simt(const DecodeParams &p, int sms, cudaStream_t s) {
  switch (p.rows) {
    case 1: return launch_simt_rows<D, 1>(p, sms, s);
    case 2: return launch_simt_rows<D, 2>(p, sms, s);
    case 4: return launch_simt_rows<D, 4>(p, sms, s);
    default: return launch_simt_rows<D, 8>(p, sms, s);
  }
}

#define FAV_DECODE_BY_DIM(FN, ...)            \
  switch (p.d) {                              \
    case 32: return FN<__VA_ARGS__ 32>(p, sms, s);   \
    case 64: return FN<__VA_ARGS__ 64>(p, sms, s);   \
    case 96: return FN<__VA_ARGS__ 96>(p, sms, s);   \
    case 128: return FN<__VA_ARGS__ 128>(p, sms, s); \
    case 192: return FN<__VA_ARGS__ 192>(p, sms, s); \
  }                                           \
  return cudaErrorInvalidValue

}  // namespace
}  // namespace fav
