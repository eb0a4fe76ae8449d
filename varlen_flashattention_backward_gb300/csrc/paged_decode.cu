// Attention of one new token per request over the paged cache
// (fa_paged_decode): S_j = scale q . k_j, P = exp(S - max), y = P V / sum P.

#include <math_constants.h>

#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "sm103.cuh"

namespace fav {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kFull = 0xffffffffu;
// Beginning a segment costs a warp about as much as this many blocks of keys.
constexpr int kSwitchBlocks = 1;
// Most CTAs of a cluster that shares a segment, and blocks for each warp of it.
constexpr int kMaxDirect = 8;
constexpr int kDirectBlocks = 4;

// ---------------------------------------------------------------------------
// Division of the work
//
// A segment is one request, one key head and up to R of its query heads; its
// keys are cut into blocks of KB (at least one, which may hold no key).  The
// segments, each weighing its blocks plus kSwitchBlocks, form a line that is
// cut into ranges of equal weight, one per warp of the grid.  Weights count in
// units of 2^unit_shift blocks, which the host chooses so that 32 bits hold the
// line's length; the shift is 0 for any batch that fits a GPU's memory.
//
// A warp's share of a segment is a part.  A part that is a whole segment
// writes y from the warp's registers.  Of the others a warp has at most two,
// its first (slot A, where it does not begin its segment) and its last (slot B,
// where it does); they wait until the CTA's warps are done, when neighbouring
// parts of one segment are added.  What then still misses a neighbour, at most
// two sums per CTA, goes to the workspace: slot 0 where it does not begin its
// segment, slot 1 where it does.  join_kernel adds those, in order.
//
// Where there are few segments and none can be long (direct_ctas), a segment
// gets a cluster of CTAs instead: its blocks are dealt to their warps, and the
// CTAs' sums are added through distributed shared memory.  That saves finding
// the ranges, the workspace and the second kernel.
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

// Measures the line and finds unit `start(range)` on it.  Every warp that asks
// works it out for itself from all lengths, a lane taking a 32nd of them: that
// costs less than meeting other warps would.  False: nothing is there.
template <int KB>
__device__ __forceinline__ bool find(const DecodeParams &p, int segs, int range, int before,
                                     Line &line, Place &at) {
  const int lane = threadIdx.x & 31;
  const int per = (p.batch + 31) >> 5;
  const int b0 = lane * per;
  const int most = p.max_pages * p.page_size;
  int sum = 0, units = 0;
  bool bad = false;
#pragma unroll 4
  for (int i = 0; i < per; ++i) {
    if (b0 + i < p.batch) {
      const int len = __ldg(p.lens + b0 + i);
      bad |= len < 0 || len > most;
      units = units_of(p, span_of<KB>(p, len).blocks);
      sum += units;
    }
  }
  if (bad && range == 0 && p.error) atomicOr(p.error, FA_PAGED_BAD_LENGTH);
  sum *= segs;
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += y;
  }
  const int total = __shfl_sync(kFull, upto, 31);
  line.each = total / p.ranges;
  line.rest = total - line.each * p.ranges;
  const int u = line.start(range) - before;
  if (u < 0 || u >= total) return false;
  // The lane, then the request, inside which u falls.
  const int owner = __popc(__ballot_sync(kFull, upto <= u));
  int from = __shfl_sync(kFull, upto - sum, owner);
  at.b = owner * per;
  at.units = __shfl_sync(kFull, units, owner);
  if (per > 1) {
    for (int i = 0; i < per; i += 32) {
      const int b = owner * per + i + lane;
      const int w = i + lane < per && b < p.batch
                        ? units_of(p, span_of<KB>(p, __ldg(p.lens + b)).blocks)
                        : 0;
      int x = w * segs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      const int n = __popc(__ballot_sync(kFull, from + x <= u));
      if (n < 32) {
        at.b = owner * per + i + n;
        at.units = __shfl_sync(kFull, w, n);
        from += __shfl_sync(kFull, x, n) - at.units * segs;
        break;
      }
      from += __shfl_sync(kFull, x, 31);
    }
  }
  at.seg = (u - from) / at.units;
  at.off = u - from - at.seg * at.units;
  return true;
}

// Measures the line and gives the first unit of segment (at.b, at.seg), whose
// units it fills in.
template <int KB>
__device__ __forceinline__ int segment_start(const DecodeParams &p, int segs, Place &at,
                                             Line &line) {
  int sum = 0, before = 0;
  for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
    const int units = units_of(p, span_of<KB>(p, __ldg(p.lens + b)).blocks);
    sum += units;
    if (b < at.b) before += units;
  }
  const int total = __reduce_add_sync(kFull, sum) * segs;
  line.each = total / p.ranges;
  line.rest = total - line.each * p.ranges;
  at.units = units_of(p, span_of<KB>(p, __ldg(p.lens + at.b)).blocks);
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

// What a block in the ring is: x = mask of its keys | flags << 16, y = request,
// z = segment inside the request.
enum : int {
  kPartBegins = 1 << 16,   // first block of a part
  kPartEnds = 1 << 17,
  kSegBegins = 1 << 18,    // first block of a segment
  kSegEnds = 1 << 19,
  kRangeEnds = 1 << 20,    // last block of the warp's range
  kDone = 1 << 21          // no block: the range is done
};

// Shared memory of one kernel: NW rings of S stages (K and V block each), what
// the kernel adds per warp, and one partial result of the whole CTA.  Three stages of eight warps keep 128 KB on
// the way, which is what the memory needs; where they do not fit, four warps
// with more stages are taken if they do better (MINS: the stages that eight
// warps must have).
template <typename T, int D, int R, int KB, int EXTRA, int MINS>
struct Shape {
  static constexpr int PAD = 4;
  static constexpr int kBlock = KB * D * int(sizeof(T));      // K or V block of one warp
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kPartial = R * (D + PAD) * 4;
  static constexpr int kExtra = EXTRA;
  static constexpr int kBudget = 227 * 1024 - 4096 - kPartial;   // 4 KB of static arrays
  static constexpr int fit(int nw) { return (kBudget - nw * kExtra) / (nw * kStage); }
  static constexpr int NW = fit(8) >= MINS ? 8 : 4;
  static constexpr int S = fit(NW) > 8 ? 8 : fit(NW);
  static constexpr int kSmem = NW * (S * kStage + kExtra) + kPartial;
  static_assert(S >= 2 && S * kStage >= kPartial, "decode stages");
};

// The loading side of a warp: walks its range and keeps the ring filled.
// `look` finds the next block and starts the load of its page ids; `issue`,
// one block later, uses them to start the copies of its rows.
template <typename T, int D, int KB, int S, typename Swizzle>
struct Loader {
  static constexpr int VEC = 16 / int(sizeof(T));
  static constexpr int CPR = D / VEC;              // 16-byte chunks per row
  static constexpr int kLoads = KB * CPR / 32;     // chunks per lane, K or V
  static_assert(KB * CPR % 32 == 0 && KB <= 16, "decode block");
  const DecodeParams &p;
  const int chunks, segs, lane;
  int left;                      // units left of the range
  int off, units, b, seg;        // units into the segment, and of it
  int blk, end;                  // next block of the part, and its end
  bool begins;                   // blk begins its part
  Span span;
  int4 desc;
  int page, tok, head, err;
  bool inside;

  __device__ __forceinline__ Loader(const DecodeParams &p, int range, int chunks)
      : p(p), chunks(chunks), segs(p.n_kv * chunks), lane(threadIdx.x & 31), left(0), off(0),
        units(0), b(0), seg(0), blk(0), end(0), begins(false), page(-1), tok(0), head(0), err(0),
        inside(false) {
    if (p.direct) {
      const int id = blockIdx.x / p.direct, warps = p.direct * (blockDim.x >> 5);
      b = id / segs;
      seg = id - b * segs;
      head = chunks == 1 ? seg : seg / chunks;
      const int len = __ldg(p.lens + b);
      if ((len < 0 || len > p.max_pages * p.page_size) && p.error)
        atomicOr(p.error, FA_PAGED_BAD_LENGTH);
      span = span_of<KB>(p, len);
      const int per = (span.blocks + warps - 1) / warps;
      const int mine = range - id * warps;
      blk = min(mine * per, span.blocks);
      end = min(blk + per, span.blocks);
      begins = true;
      desc.y = b;
      desc.z = seg;
      return;
    }
    Line line;
    Place at;
    if (find<KB>(p, segs, range, 0, line, at)) {
      left = line.each + (range < line.rest ? 1 : 0);
      b = at.b;
      seg = at.seg;
      off = at.off;
      enter();
    }
  }

  // Request b's span (its segments have the same).
  __device__ __forceinline__ void enter() {
    span = span_of<KB>(p, __ldg(p.lens + b));
    units = units_of(p, span.blocks);
  }

  __device__ __forceinline__ void look() {
    while (blk >= end) {
      if (left <= 0) {
        desc.x = kDone;
        return;
      }
      // The next part: the rest of the range inside the current segment.
      const int upto = min(off + left, units);
      blk = max((off << p.unit_shift) - kSwitchBlocks, 0);
      end = min((upto << p.unit_shift) - kSwitchBlocks, span.blocks);
      begins = true;
      left -= upto - off;
      off = upto;
      if (blk >= end) continue;    // all of it is the segment's beginning
      desc.y = b;
      desc.z = seg;
      head = chunks == 1 ? seg : seg / chunks;
    }
    const int j = (span.blk0 + blk) * KB + (lane % KB);
    inside = j >= span.lo && j < span.hi;
    if (inside) {
      const int idx = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
      tok = j - idx * p.page_size;
      page = p.table[desc.y * p.table_stride + idx];
    }
    desc.x = (begins ? kPartBegins : 0) | (blk == 0 ? kSegBegins : 0);
    begins = false;
    if (++blk >= end) {
      desc.x |= kPartEnds | (end == span.blocks ? kSegEnds : 0) | (left == 0 ? kRangeEnds : 0);
      if (off == units) {          // on to the next segment
        off = 0;
        if (++seg == segs) {
          seg = 0;
          if (++b < p.batch && left > 0) enter();
        }
      }
    }
  }

  __device__ __forceinline__ void issue(uint32_t dst, int4 *at) {
    if (!(desc.x & kDone)) {
      int64_t o = -1;
      if (inside) {
        if (page >= 0 && page < p.num_pages)
          o = page * p.page_stride + tok * p.token_stride + head * p.head_stride;
        else
          err = FA_PAGED_BAD_PAGE;
      }
      const uint32_t mask = __ballot_sync(kFull, o >= 0) & ((1u << KB) - 1);
      if (lane == 0) *at = make_int4(desc.x | int(mask), desc.y, desc.z, 0);
      const T *kc = static_cast<const T *>(p.kc), *vc = static_cast<const T *>(p.vc);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int c = i * 32 + lane, r = c / CPR, ch = c % CPR;
        const int64_t row = __shfl_sync(kFull, o, r);
        const uint32_t to = dst + (r * CPR + (ch ^ Swizzle::at(r))) * 16;
        const int64_t from = (row < 0 ? 0 : row) + ch * VEC;
        cp_async16(to, kc + from, row >= 0);
        cp_async16(to + KB * CPR * 16, vc + from, row >= 0);
      }
    } else if (lane == 0) {
      *at = make_int4(kDone, 0, 0, 0);
    }
    cp_async_commit();
  }
};

// Floats of one workspace slot: o [rows][d], then the rows' maxima and sums.
__host__ __device__ constexpr int slot_floats(int rows, int d) { return rows * (d + 4); }

__device__ __forceinline__ float *slot_of(const DecodeParams &p, int cta, int slot, int rows) {
  return p.part + (int64_t(cta) * 2 + slot) * slot_floats(rows, p.d);
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

// The partial results of a CTA's warps: slot A of the part that does not begin
// its segment, slot B of the part that does and does not end it.
template <int NW, int R>
struct Partials {
  float m[2][NW][R], l[2][NW][R];
  const float *o[2][NW];            // [R][D + PAD]
  int id[2][NW];                    // segment (b * segs + seg), or -1
  int ends[2][NW];                  // whether the part ends it
};

// Where a warp puts the partial result of a part: its ring when the part is
// the last of its range (nothing is on the way behind it), else, so for a slot A
// that more parts follow, its place in the workspace.
template <int NW>
__device__ __forceinline__ float *partial_at(const DecodeParams &p, int rows, bool last,
                                             const uint8_t *ring) {
  if (last) return reinterpret_cast<float *>(const_cast<uint8_t *>(ring));
  return p.warp_part +
         (int64_t(blockIdx.x) * NW + (threadIdx.x >> 5)) * slot_floats(rows, p.d);
}

// Adds neighbouring partial results (see the top) once every warp is done.
// Run 0 begins with warp 0's slot A, run 1 + w with warp w's slot B; a run
// goes on with the slots A of the warps behind it.  A warp takes one row of
// one run at a time.
template <typename T, int D, int R, int NW, int PAD>
__device__ __forceinline__ void merge_partials(const DecodeParams &p, int chunks,
                                               const Partials<NW, R> &s, float *cta_part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(R, p.group);
  // Lane k < NW: the id in warp k's slot A, lane 16 + k: in its slot B.
  const int id_of = (lane & 15) < NW ? s.id[lane >> 4][lane & 15] : -1;
  const uint32_t held = __ballot_sync(kFull, id_of >= 0);
  // Runs begin at warp 0's slot A and at every slot B.
  uint32_t runs = held & 0xffff0001u;
  const int tasks = __popc(runs) * rows;
#pragma unroll 1
  for (int task = warp; task < tasks; task += NW) {
    const int run = task / rows, r = task - run * rows;
    uint32_t rest = runs;
    for (int i = 0; i < run; ++i) rest &= rest - 1;
    const int at = __ffs(rest) - 1, slot = at >> 4, w0 = at & 15;
    // Its members: w0, then the slots A behind it up to the first gap or the
    // first that ends the segment.
    int count = 1;
    bool ends = s.ends[slot][w0];
    while (!ends && w0 + count < NW) {
      ends = s.ends[0][w0 + count];
      ++count;
    }
    const int id = __shfl_sync(kFull, id_of, at);
    const int segs = p.n_kv * chunks;
    const int b = id / segs, seg = id - b * segs;
    const int h = (chunks == 1 ? 0 : seg % chunks * R) + r;
    if (h >= p.group) continue;
    const int n = (chunks == 1 ? seg : seg / chunks) * p.group + h;
    const int mine = lane < count ? lane : 0;
    const int my_slot = mine == 0 ? slot : 0;
    const float m = s.m[my_slot][w0 + mine][r], l = s.l[my_slot][w0 + mine][r];
    float mx = m;
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    const float f = sm103::ex2(m - (mx == -CUDART_INF_F ? 0.f : mx));
    float sum = 0.f;
    const bool whole = slot == 1 && ends;
    float *dst = p.direct ? cta_part : slot_of(p, blockIdx.x, slot, R);
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += 128) {
      const int d = d0 + lane * 4;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      sum = 0.f;
#pragma unroll 2
      for (int k = 0; k < count; ++k) {
        const float fk = __shfl_sync(kFull, f, k);
        sum += fk * __shfl_sync(kFull, l, k);
        if (d < D) {
          const float4 o = *reinterpret_cast<const float4 *>(
              s.o[k == 0 ? slot : 0][w0 + k] + r * (D + PAD) + d);
          acc.x += fk * o.x;
          acc.y += fk * o.y;
          acc.z += fk * o.z;
          acc.w += fk * o.w;
        }
      }
      if (d < D) {
        if (whole) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          T *y = static_cast<T *>(p.y) + b * p.y_stride + int64_t(n) * D + d;
          y[0] = from_f<T>(acc.x * inv);
          y[1] = from_f<T>(acc.y * inv);
          y[2] = from_f<T>(acc.z * inv);
          y[3] = from_f<T>(acc.w * inv);
        } else {
          *reinterpret_cast<float4 *>(dst + r * D + d) = acc;
        }
      }
    }
    if (lane == 0) {
      if (whole) {
        write_stats(p, b, n, mx * kLn2, sum);
      } else {
        dst[R * D + r] = mx;
        dst[R * D + R + r] = sum;
      }
    }
  }
}

// The sums of a cluster's CTAs, each at `cta_part` of its shared memory, to y.
// A warp of the cluster takes one row.
template <typename T, int D, int R, int NW, int KB>
__device__ __forceinline__ void join_cluster(const DecodeParams &p, int chunks,
                                             const float *cta_part) {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int lane = threadIdx.x & 31, segs = p.n_kv * chunks;
  const int id = blockIdx.x / p.direct;
  const int r = (blockIdx.x - id * p.direct) * NW + (threadIdx.x >> 5);
  const int b = id / segs, seg = id - b * segs;
  const int h = (chunks == 1 ? 0 : seg % chunks * R) + r;
  const int blocks = span_of<KB>(p, __ldg(p.lens + b)).blocks;
  const int per = (blocks + p.direct * NW - 1) / (p.direct * NW);
  const int parts = (blocks + per * NW - 1) / (per * NW);   // CTAs that have blocks
  if (parts > 1 && r < R && h < p.group) {
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
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Row r's chunk c of a block sits at chunk c ^ at(r) of the row, so that the
// eight rows of an 8x8 matrix fall into different banks (rows are an odd
// multiple of 64 bytes where CPR % 8 != 0).
template <int CPR>
struct TcSwizzle {
  static __device__ __forceinline__ int at(int r) {
    return CPR % 8 == 0 ? (r & 7) : ((r >> 1) & 3);
  }
};

template <int D, int R>
using TcShape = Shape<__half, D, R, 16, 0, 2>;

// S = Q K^T and O = P V by m16n8k16 products: Q's rows are the group's query
// heads, padded to 16, and a warp takes 16 keys at a time through its own ring
// of stages, filled by cp.async ahead of use.
//
// P goes into the second product as the sum of two 16-bit numbers, so that
// its rounding (2^-17 for bf16) stays below y's own.  With R = 8 the two
// halves share one product: rows 0-7 hold P rounded, rows 8-15 what is left
// of it, and the halves of the result are added at the end.  With R = 16 they
// are two products.
template <typename T, int D, int R>
__global__ void __launch_bounds__(TcShape<D, R>::NW * 32, 1)
decode_tc_kernel(const __grid_constant__ DecodeParams p) {
  using Sh = TcShape<D, R>;
  using Sw = TcSwizzle<D / 8>;
  constexpr int KB = 16, S = Sh::S, NW = Sh::NW;
  constexpr int CPR = D / 8;
  constexpr int NR = R / 8;         // rows of a lane
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Partials<NW, R> s_part;
  __shared__ int4 s_desc[NW][S];
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint8_t *my = smem + warp * S * Sh::kStage;
  const uint32_t ring = sm103::smem_u32(my);
  const T *q = static_cast<const T *>(p.q);
  const int chunks = (p.group + R - 1) / R, segs = p.n_kv * chunks;
  if (lane < 2) s_part.id[lane][warp] = -1;

  Loader<T, D, KB, S, Sw> load(p, blockIdx.x * NW + warp, chunks);
  load.look();
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) {
    load.issue(ring + i * Sh::kStage, &s_desc[warp][i]);
    load.look();
  }

  const int row = lane >> 2, col = (lane & 3) * 2;
  // ldmatrix addresses inside a block: K (n = key, k = dim) and V (transposed).
  const int k_row = (lane & 7) + ((lane >> 4) << 3), k_ch = (lane >> 3) & 1;
  const int v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_ch = lane >> 4;
  int stage = 0, fill = S - 1, heads = 0, n0 = 0;
  uint32_t qa[D / 16][2 * NR];
  float o[D / 8][4];
  float m[NR], l[NR];
  bool opens = false;

#pragma unroll 1
  while (true) {
    cp_async_wait<S - 2>();
    __syncwarp();
    const int4 desc = s_desc[warp][stage];
    if (desc.x & kDone) break;
    const uint32_t kb = ring + stage * Sh::kStage, vb = kb + Sh::kBlock;
    load.issue(ring + fill * Sh::kStage, &s_desc[warp][fill]);
    load.look();
    fill = fill + 1 == S ? 0 : fill + 1;
    stage = stage + 1 == S ? 0 : stage + 1;

    if (desc.x & kPartBegins) {
      const int hk = desc.z / chunks, h0 = (desc.z - hk * chunks) * R;
      heads = min(R, p.group - h0);
      n0 = hk * p.group + h0;
      opens = desc.x & kSegBegins;
      const T *qr = q + desc.y * p.q_stride + int64_t(n0) * D;
      // Fragment i of a step: rows row (and row + 8 for odd i with R = 16).  Rows
      // behind the last head repeat it; nothing reads their results.
#pragma unroll
      for (int i = 0; i < 2 * NR; ++i) {
        const int r = min(row + (NR == 2 ? (i & 1) * 8 : 0), heads - 1);
        const T *src = qr + r * D + col + (NR == 2 ? i >> 1 : i) * 8;
        if (p.q_pairs) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            qa[ks][i] = __ldg(reinterpret_cast<const uint32_t *>(src + ks * 16));
        } else {
          const uint16_t *h = reinterpret_cast<const uint16_t *>(src);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            qa[ks][i] = uint32_t(h[ks * 16]) | uint32_t(h[ks * 16 + 1]) << 16;
        }
      }
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

    float sa[2][2][4];              // [chain][key half][fragment]
#pragma unroll
    for (int i = 0; i < 16; ++i) (&sa[0][0][0])[i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t kf[4];
      ldsm4(kf, kb + (k_row * CPR + ((ks * 2 + k_ch) ^ Sw::at(k_row))) * 16);
      uint32_t a[4];
      if constexpr (R == 8) {
        a[0] = qa[ks][0];
        a[1] = 0;
        a[2] = qa[ks][1];
        a[3] = 0;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = qa[ks][i];
      }
      mma16816<T>(sa[ks & 1][0], a, kf[0], kf[1]);
      mma16816<T>(sa[ks & 1][1], a, kf[2], kf[3]);
    }
    float s[NR][4];                 // keys col, col + 1, col + 8, col + 9
    float mn[NR];
    bool grows = false;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float t = -CUDART_INF_F;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = col + (e & 1) + (e >> 1) * 8;
        const float x = (sa[0][e >> 1][i * 2 + (e & 1)] + sa[1][e >> 1][i * 2 + (e & 1)]) *
                        p.scale_log2;
        s[i][e] = (desc.x >> key) & 1 ? x : -CUDART_INF_F;
        t = fmaxf(t, s[i][e]);
      }
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
          if constexpr (R == 8) {
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
        hi[i][h] = pack2<T>(s[i][2 * h], s[i][2 * h + 1]);
        const float2 back = unpack2<T>(hi[i][h]);
        lo[i][h] = pack2<T>(s[i][2 * h] - back.x, s[i][2 * h + 1] - back.y);
      }
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      uint32_t vf[4];
      ldsm4_t(vf, vb + (v_row * CPR + ((dt * 2 + v_ch) ^ Sw::at(v_row))) * 16);
      if constexpr (R == 8) {
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

    if (desc.x & kPartEnds) {
      const bool ends = desc.x & kSegEnds;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        l[i] += __shfl_xor_sync(kFull, l[i], 1);
        l[i] += __shfl_xor_sync(kFull, l[i], 2);
      }
      const int id = desc.y * segs + desc.z;
      if (opens && ends) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = row + i * 8;
          if (r >= heads) continue;
          const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
          T *y = static_cast<T *>(p.y) + desc.y * p.y_stride + int64_t(n0 + r) * D + col;
#pragma unroll
          for (int k = 0; k < D / 8; ++k) {
            const float x0 = (R == 8 ? o[k][0] + o[k][2] : o[k][i * 2]) * inv;
            const float x1 = (R == 8 ? o[k][1] + o[k][3] : o[k][i * 2 + 1]) * inv;
            if (p.y_pairs) {
              *reinterpret_cast<uint32_t *>(y + k * 8) = pack2<T>(x0, x1);
            } else {
              y[k * 8] = from_f<T>(x0);
              y[k * 8 + 1] = from_f<T>(x1);
            }
          }
          if ((lane & 3) == 0) write_stats(p, desc.y, n0 + r, m[i] * kLn2, l[i]);
        }
      } else {
        __syncwarp();                // the ring has been read
        const int slot = opens ? 1 : 0;
        float *dst = partial_at<NW>(p, R, desc.x & kRangeEnds, my);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int r = row + i * 8;
          if ((lane & 3) == 0) {
            s_part.m[slot][warp][r] = m[i];
            s_part.l[slot][warp][r] = l[i];
          }
#pragma unroll
          for (int k = 0; k < D / 8; ++k)
            *reinterpret_cast<float2 *>(dst + r * (D + Sh::PAD) + col + k * 8) =
                R == 8 ? make_float2(o[k][0] + o[k][2], o[k][1] + o[k][3])
                       : make_float2(o[k][i * 2], o[k][i * 2 + 1]);
        }
        if (lane == 0) {
          s_part.id[slot][warp] = id;
          s_part.ends[slot][warp] = ends;
          s_part.o[slot][warp] = dst;
        }
      }
    }
  }
  __syncthreads();
  float *cta_part = reinterpret_cast<float *>(smem + NW * (S * Sh::kStage + Sh::kExtra));
  merge_partials<T, D, R, NW, Sh::PAD>(p, chunks, s_part, cta_part);
  if (p.direct > 1) join_cluster<T, D, R, NW, KB>(p, chunks, cta_part);
  if (load.err && p.error) atomicOr(p.error, load.err);
}

// ---------------------------------------------------------------------------
// fp32 kernel, on the CUDA cores
// ---------------------------------------------------------------------------
// Row r's chunk c at chunk c ^ at(r): the eight lanes of a 128-byte shared
// memory access read two rows' four neighbouring chunks.
struct SimtSwizzle {
  static __device__ __forceinline__ int at(int r) { return (r & 1) << 2; }
};

template <int D, int R>
using SimtShape = Shape<float, D, R, 8, (R * D + 8 * R) * 4, 2>;

// A warp takes 8 keys at a time.  Scores: four lanes per key, each a quarter
// of the dims (every fourth chunk).  Output: each lane D / 32 dims of all R heads.
template <int D, int R>
__global__ void __launch_bounds__(SimtShape<D, R>::NW * 32, 1)
decode_simt_kernel(const __grid_constant__ DecodeParams p) {
  using Sh = SimtShape<D, R>;
  constexpr int KB = 8, S = Sh::S, NW = Sh::NW;
  constexpr int CPR = D / 4;
  constexpr int VW = D % 128 == 0 ? 4 : D % 64 == 0 ? 2 : 1;   // dims per access
  constexpr int NV = D / (32 * VW);                             // accesses per row
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Partials<NW, R> s_part;
  __shared__ int4 s_desc[NW][S];
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *s_q = reinterpret_cast<float *>(smem + NW * S * Sh::kStage) + warp * (R * D + 8 * R);
  float *s_p = s_q + R * D;         // q [R][D], weights [8][R]
  const uint8_t *my = smem + warp * S * Sh::kStage;
  const uint32_t ring = sm103::smem_u32(my);
  const int chunks = (p.group + R - 1) / R, segs = p.n_kv * chunks;
  if (lane < 2) s_part.id[lane][warp] = -1;

  Loader<float, D, KB, S, SimtSwizzle> load(p, blockIdx.x * NW + warp, chunks);
  load.look();
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) {
    load.issue(ring + i * Sh::kStage, &s_desc[warp][i]);
    load.look();
  }

  const int key = lane >> 2, quarter = lane & 3;
  int stage = 0, fill = S - 1, heads = 0, n0 = 0;
  float o[R][NV * VW], m[R], l[R];
  bool opens = false;

#pragma unroll 1
  while (true) {
    cp_async_wait<S - 2>();
    __syncwarp();
    const int4 desc = s_desc[warp][stage];
    if (desc.x & kDone) break;
    const float *kb = reinterpret_cast<const float *>(my + stage * Sh::kStage);
    const float *vb = kb + KB * D;
    load.issue(ring + fill * Sh::kStage, &s_desc[warp][fill]);
    load.look();
    fill = fill + 1 == S ? 0 : fill + 1;
    stage = stage + 1 == S ? 0 : stage + 1;

    if (desc.x & kPartBegins) {
      const int hk = desc.z / chunks, h0 = (desc.z - hk * chunks) * R;
      heads = min(R, p.group - h0);
      n0 = hk * p.group + h0;
      opens = desc.x & kSegBegins;
      const float *qr = static_cast<const float *>(p.q) + desc.y * p.q_stride + int64_t(n0) * D;
      for (int i = lane; i < R * D; i += 32) s_q[i] = i < heads * D ? __ldg(qr + i) : 0.f;
      __syncwarp();
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
      const int c = i * 4 + quarter;
      const float4 kv =
          *reinterpret_cast<const float4 *>(kb + (key * CPR + (c ^ SimtSwizzle::at(key))) * 4);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 qv = *reinterpret_cast<const float4 *>(s_q + r * D + c * 4);
        s[r] = fmaf(kv.x, qv.x, s[r]);
        s[r] = fmaf(kv.y, qv.y, s[r]);
        s[r] = fmaf(kv.z, qv.z, s[r]);
        s[r] = fmaf(kv.w, qv.w, s[r]);
      }
    }
    const bool ok = (desc.x >> key) & 1;
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
        const float *src = vb + (k * CPR + ((d >> 2) ^ SimtSwizzle::at(k))) * 4 + (d & 3);
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

    if (desc.x & kPartEnds) {
      const bool ends = desc.x & kSegEnds;
      const int id = desc.y * segs + desc.z;
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[r] += __shfl_xor_sync(kFull, l[r], x);
      }
      const bool whole = opens && ends;
      const int slot = opens ? 1 : 0;
      float *dst = partial_at<NW>(p, R, desc.x & kRangeEnds, my);
      __syncwarp();                  // the ring has been read
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= heads) continue;
        const float inv = whole ? (l[r] == 0.f ? 0.f : 1.f / l[r]) : 1.f;
        float *to = whole ? static_cast<float *>(p.y) + desc.y * p.y_stride + int64_t(n0 + r) * D
                          : dst + r * (D + Sh::PAD);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VW; ++e) to[(i * 32 + lane) * VW + e] = o[r][i * VW + e] * inv;
        if (lane == 0) {
          if (whole) {
            write_stats(p, desc.y, n0 + r, m[r] * kLn2, l[r]);
          } else {
            s_part.m[slot][warp][r] = m[r];
            s_part.l[slot][warp][r] = l[r];
          }
        }
      }
      if (lane == 0 && !whole) {
        s_part.id[slot][warp] = id;
        s_part.ends[slot][warp] = ends;
        s_part.o[slot][warp] = dst;
      }
    }
  }
  __syncthreads();
  float *cta_part = reinterpret_cast<float *>(smem + NW * (S * Sh::kStage + Sh::kExtra));
  merge_partials<float, D, R, NW, Sh::PAD>(p, chunks, s_part, cta_part);
  if (p.direct > 1) join_cluster<float, D, R, NW, KB>(p, chunks, cta_part);
  if (load.err && p.error) atomicOr(p.error, load.err);
}

// ---------------------------------------------------------------------------
// Joins the sums of the segments that were cut between CTAs.  Block (x, r)
// takes query head r of segment x, or, where there are more segments than
// CTAs, of the segment in which CTA x's ranges end.  Which CTAs share it
// follows from the lengths alone, so all that is worked out before the main
// kernel is done.  The warps take the parts in turn, so that their loads
// overlap, and meet in shared memory, always in the same order.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <typename T, int D, int KB, int NW>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(
    const __grid_constant__ DecodeParams p, int rows, int by_segment) {
  constexpr int PL = D / 32;
  constexpr int U = 2;               // parts on the way at once, per warp
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float s_o[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
  const int chunks = (p.group + rows - 1) / rows, segs = p.n_kv * chunks;
  Line line;
  Place at;
  int first_unit;                    // of the segment
  if (by_segment) {
    at.b = blockIdx.x / segs;
    at.seg = blockIdx.x - at.b * segs;
    first_unit = segment_start<KB>(p, segs, at, line);
  } else {
    const int behind = (blockIdx.x + 1) * NW;
    find<KB>(p, segs, behind, 1, line, at);
    first_unit = line.start(behind) - 1 - at.off;
  }
  // The CTAs of its first and last block.
  const int i = line.range_of(first_unit + (kSwitchBlocks >> p.unit_shift)) / NW;
  const int last = line.range_of(first_unit + at.units - 1) / NW;
  const int h = (chunks == 1 ? 0 : at.seg % chunks * rows) + r;
  const int n = (chunks == 1 ? at.seg : at.seg / chunks) * p.group + h;

  // Every block waits, also one with nothing to do: what follows on the stream
  // is behind the main kernel only through this one.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (i == last || h >= p.group || (!by_segment && i != int(blockIdx.x))) return;
  // Part 0 is CTA i's slot 1, part k CTA (i + k)'s slot 0.
  const int parts = last - i + 1;
  float mx = -CUDART_INF_F, sum = 0.f, acc[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) acc[k] = 0.f;
#pragma unroll 1
  for (int j0 = warp; j0 < parts; j0 += U * kJoinWarps) {
    float m2[U], l2[U], o2[U][PL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * kJoinWarps, parts - 1);
      const float *src = slot_of(p, i + j, j == 0 ? 1 : 0, rows);
      m2[u] = src[rows * D + r];
      l2[u] = src[rows * D + rows + r];
#pragma unroll
      for (int k = 0; k < PL; ++k) o2[u][k] = src[r * D + lane + 32 * k];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j0 + u * kJoinWarps >= parts) break;
      const float mn = fmaxf(mx, m2[u]), ref = mn == -CUDART_INF_F ? 0.f : mn;
      const float f = sm103::ex2(mx - ref), f2 = sm103::ex2(m2[u] - ref);
      mx = mn;
      sum = sum * f + l2[u] * f2;
#pragma unroll
      for (int k = 0; k < PL; ++k) acc[k] = acc[k] * f + o2[u][k] * f2;
    }
  }
  if (lane == 0) {
    s_m[warp] = mx;
    s_l[warp] = sum;
  }
#pragma unroll
  for (int k = 0; k < PL; ++k) s_o[warp][lane + 32 * k] = acc[k];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
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
  static_cast<T *>(p.y)[at.b * p.y_stride + int64_t(n) * D + d] =
      from_f<T>(total == 0.f ? 0.f : out / total);
  if (d == 0) write_stats(p, at.b, n, top * kLn2, total);
}

// The main kernel and the join, which is launched as its dependent so that its
// launch overlaps the main kernel's run.
template <typename T, int D, int R, int KB, int NW, typename Kernel>
cudaError_t launch_both(DecodeParams p, Kernel kernel, int smem, int sms, cudaStream_t s) {
  const int64_t segments = int64_t(p.batch) * p.n_kv * ((p.group + R - 1) / R);
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (p.direct) {
    cfg.gridDim = dim3(unsigned(segments) * p.direct);
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.direct;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
  p.grid = sms;
  p.ranges = sms * NW;
  const int64_t blocks = (int64_t(p.max_pages) * p.page_size + KB - 1) / KB + 1 + kSwitchBlocks;
  p.unit_shift = 0;
  while (segments * ((blocks >> p.unit_shift) + 1) >= (int64_t(1) << 31)) ++p.unit_shift;
  kernel<<<p.grid, NW * 32, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int by_segment = segments <= p.grid;
  cfg.gridDim = dim3(unsigned(by_segment ? segments : p.grid), unsigned(p.group < R ? p.group : R));
  cfg.blockDim = dim3(kJoinWarps * 32);
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D, KB, NW>, p, R, by_segment);
}

template <int D, int R>
cudaError_t launch_simt(const DecodeParams &p, int sms, cudaStream_t s) {
  using Sh = SimtShape<D, R>;
  return launch_both<float, D, R, 8, Sh::NW>(p, decode_simt_kernel<D, R>, Sh::kSmem, sms, s);
}

template <typename T, int D, int R>
cudaError_t launch_tc(const DecodeParams &p, int sms, cudaStream_t s) {
  using Sh = TcShape<D, R>;
  return launch_both<T, D, R, 16, Sh::NW>(p, decode_tc_kernel<T, D, R>, Sh::kSmem, sms, s);
}

template <int D>
cudaError_t launch_d(const DecodeParams &p, fa_dtype dt, int rows, int sms, cudaStream_t s) {
  if (dt == FA_DTYPE_FP32) {
    switch (rows) {
      case 1: return launch_simt<D, 1>(p, sms, s);
      case 2: return launch_simt<D, 2>(p, sms, s);
      case 4: return launch_simt<D, 4>(p, sms, s);
      default: return launch_simt<D, 8>(p, sms, s);
    }
  }
  if (dt == FA_DTYPE_FP16)
    return rows == 8 ? launch_tc<__half, D, 8>(p, sms, s) : launch_tc<__half, D, 16>(p, sms, s);
  return rows == 8 ? launch_tc<__nv_bfloat16, D, 8>(p, sms, s)
                   : launch_tc<__nv_bfloat16, D, 16>(p, sms, s);
}

template <int D>
int warps_of_d(bool tc, int rows) {
  if (tc) return rows == 8 ? TcShape<D, 8>::NW : TcShape<D, 16>::NW;
  return rows == 1 ? SimtShape<D, 1>::NW : rows == 2 ? SimtShape<D, 2>::NW
         : rows == 4 ? SimtShape<D, 4>::NW : SimtShape<D, 8>::NW;
}

int warps_of(bool tc, int rows, int d) {
  switch (d) {
    case 32: return warps_of_d<32>(tc, rows);
    case 64: return warps_of_d<64>(tc, rows);
    case 96: return warps_of_d<96>(tc, rows);
    case 128: return warps_of_d<128>(tc, rows);
    default: return warps_of_d<192>(tc, rows);
  }
}

}  // namespace

// The shape of a call, from its scalars alone.
DecodePlan decode_plan(fa_dtype dt, int batch, int n_kv, int group, int d, int64_t max_keys,
                       int sms) {
  DecodePlan plan;
  // fp32: the heads whose outputs a lane's registers hold at once.  16-bit types:
  // the rows of one product, all 16 of which serve P rounded once a group has
  // more than 8 heads.
  const bool tc = dt != FA_DTYPE_FP32;
  plan.rows = tc ? (group <= 8 ? 8 : 16) : group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8;
  plan.warps = warps_of(tc, plan.rows, d);
  // The largest cluster per segment that still puts all of them on the GPU at
  // once, if its warps get at most kDirectBlocks blocks each.
  const int kb = tc ? 16 : 8;
  const int64_t blocks = (max_keys + kb - 1) / kb + 1;
  const int64_t segments = int64_t(batch) * n_kv * ((group + plan.rows - 1) / plan.rows);
  int ctas = 1;
  while (ctas < kMaxDirect && segments * ctas * 2 <= sms && ctas * plan.warps < blocks) ctas *= 2;
  plan.direct =
      segments * ctas <= sms && blocks <= int64_t(ctas) * plan.warps * kDirectBlocks ? ctas : 0;
  return plan;
}

size_t decode_part_floats(int rows, int d) { return size_t(slot_floats(rows, d)); }

cudaError_t launch_paged_decode(const DecodeParams &p, fa_dtype dt, int sms, cudaStream_t s) {
  const int rows = p.rows;
  switch (p.d) {
    case 32: return launch_d<32>(p, dt, rows, sms, s);
    case 64: return launch_d<64>(p, dt, rows, sms, s);
    case 96: return launch_d<96>(p, dt, rows, sms, s);
    case 128: return launch_d<128>(p, dt, rows, sms, s);
    case 192: return launch_d<192>(p, dt, rows, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fav
