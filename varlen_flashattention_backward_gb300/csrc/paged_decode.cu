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
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// A segment costs a CTA about this many blocks of keys beside its own.
constexpr int kSwitchBlocks = 2;

// ---------------------------------------------------------------------------
// Division of the work
//
// A segment is one request, one key head and up to R of its query heads; its
// keys are cut into blocks of KB.  The segments, each weighing its blocks plus
// kSwitchBlocks, form a line that is cut into `grid` ranges of equal weight,
// one per CTA.  A CTA's share of a segment is a part.  A part that is a whole
// segment writes y; of the others a CTA has at most two (its first and its
// last), which go to its two slots of the workspace: slot 0 for a part that
// does not begin its segment, slot 1 for one that begins it and does not end
// it.  join_kernel adds the parts of a segment in order.
// ---------------------------------------------------------------------------
struct Part {
  int b, seg;        // request; segment index inside the request
  int first, last;   // blocks [first, last), relative to the segment's first
  int blocks;        // of the whole segment
};

struct Span {
  int lo, hi;        // keys [lo, hi) that the query sees
  int blk0;          // first block (absolute)
  int blocks;
};

template <int KB>
__device__ __forceinline__ Span span_of(const DecodeParams &p, int b) {
  Span s;
  const int most = p.max_pages * p.page_size;
  int len = p.lens[b];
  len = len < 0 ? 0 : len > most ? most : len;
  s.hi = len;
  const int lo = len - 1 - p.pre;
  s.lo = lo < 0 ? 0 : lo > len ? len : lo;
  s.blk0 = s.lo / KB;
  s.blocks = s.hi > s.lo ? (s.hi + KB - 1) / KB - s.blk0 : 0;
  return s;
}

// Walks the parts of one CTA's range in order.
template <int KB>
struct Walk {
  int64_t left;      // weight left of the range
  int off;           // weight already passed inside the current segment
  int b, seg, segs;
  Span span;         // of request b
  Span part_span;    // of the part that next() gave

  __device__ __forceinline__ bool next(const DecodeParams &p, Part &part) {
    while (left > 0) {
      const int weight = span.blocks + kSwitchBlocks;
      const int end = int(min(off + left, int64_t(weight)));
      part.b = b;
      part.seg = seg;
      part.blocks = span.blocks;
      part.first = max(off - kSwitchBlocks, 0);
      part.last = max(end - kSwitchBlocks, 0);
      part_span = span;
      const bool opens = off == 0;
      left -= end - off;
      off = end;
      if (end == weight) {
        off = 0;
        if (++seg == segs) {
          seg = 0;
          if (++b < p.batch && left > 0) span = span_of<KB>(p, b);
        }
      }
      if (part.last > part.first || (part.blocks == 0 && opens)) return true;
    }
    return false;
  }
};

// Places `w` at the start of the CTA's range.  All threads of the CTA call it.
template <int KB>
__device__ void place(const DecodeParams &p, int segs, Walk<KB> &w) {
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_off;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = tid * per, b1 = min(b0 + per, p.batch);
  const int most = p.max_pages * p.page_size;
  int64_t sum = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    sum += int64_t(span_of<KB>(p, b).blocks + kSwitchBlocks) * segs;
    const int len = p.lens[b];
    bad |= len < 0 || len > most;
  }
  if (bad && blockIdx.x == 0 && p.error) atomicOr(p.error, FA_PAGED_BAD_LENGTH);
  int64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  int64_t before = x - sum, total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += s_sum[i];
    total += s_sum[i];
  }
  // Ranges differ by at most one block of weight.
  const int64_t each = total / p.grid, rest = total % p.grid;
  const int64_t i = blockIdx.x;
  const int64_t u0 = i * each + min(i, rest);
  w.left = each + (i < rest ? 1 : 0);
  if (w.left > 0 && u0 >= before && u0 < before + sum) {
    int64_t at = before;
    for (int b = b0; b < b1; ++b) {
      const int64_t mine = int64_t(span_of<KB>(p, b).blocks + kSwitchBlocks) * segs;
      if (u0 < at + mine) {
        s_b = b;
        s_off = u0 - at;
        break;
      }
      at += mine;
    }
  }
  __syncthreads();
  w.segs = segs;
  if (w.left > 0) {
    w.b = s_b;
    w.span = span_of<KB>(p, w.b);
    const int64_t weight = w.span.blocks + kSwitchBlocks;
    w.seg = int(s_off / weight);
    w.off = int(s_off - w.seg * weight);
  }
}

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

// What a CTA's parts left in the workspace, four words per CTA: the segment
// (b * segs + seg) whose part is in slot 0 (or -1), whether that part ends it,
// the segment in slot 1 (or -1).
struct Meta {
  int seg0 = -1, ends0 = 0, seg1 = -1;
  __device__ __forceinline__ void note(const Part &part, int segs) {
    const int id = part.b * segs + part.seg;
    if (part.first == 0) {
      seg1 = id;
    } else {
      seg0 = id;
      ends0 = part.last == part.blocks;
    }
  }
  __device__ __forceinline__ void store(const DecodeParams &p) const {
    *reinterpret_cast<int4 *>(p.meta + blockIdx.x * 4) = make_int4(seg0, ends0, seg1, 0);
  }
};

// The end of a part: the warps' maxima, sums and outputs in shared memory
// (o [warp][row][D + pad]) become y and the statistics, or a workspace slot.
// Four dims per thread.
template <typename T, int D, int R, int PAD>
__device__ __forceinline__ void finish_part(const DecodeParams &p, const Part &part, int n0,
                                            int heads, const float *s_o, const float *s_m,
                                            const float *s_l) {
  const bool whole = part.first == 0 && part.last == part.blocks;
  float *dst = slot_of(p, blockIdx.x, part.first == 0 ? 1 : 0, R);
  for (int i = threadIdx.x; i < heads * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
    float mx = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, s_m[k * R + r]);
    const float ref = mx == -CUDART_INF_F ? 0.f : mx;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float f = exp2f(s_m[k * R + r] - ref);
      const float4 o = *reinterpret_cast<const float4 *>(s_o + (k * R + r) * (D + PAD) + d);
      sum += f * s_l[k * R + r];
      acc.x += f * o.x;
      acc.y += f * o.y;
      acc.z += f * o.z;
      acc.w += f * o.w;
    }
    if (whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      T *y = static_cast<T *>(p.y) + part.b * p.y_stride + int64_t(n0 + r) * D + d;
      y[0] = from_f<T>(acc.x * inv);
      y[1] = from_f<T>(acc.y * inv);
      y[2] = from_f<T>(acc.z * inv);
      y[3] = from_f<T>(acc.w * inv);
      if (d == 0) write_stats(p, part.b, n0 + r, mx * kLn2, sum);
    } else {
      *reinterpret_cast<float4 *>(dst + r * D + d) = acc;
      if (d == 0) {
        dst[R * D + r] = mx;
        dst[R * D + R + r] = sum;
      }
    }
  }
}

// Page of key j of request b, or -1 (with `bad` set) where its id is none.
__device__ __forceinline__ int page_of(const DecodeParams &p, int j, int &in_page) {
  const int idx = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
  in_page = j - idx * p.page_size;
  return idx;
}

// ---------------------------------------------------------------------------
// Tensor-core kernel, 16-bit types
// ---------------------------------------------------------------------------
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

template <int D, int R>
struct TcShape {
  static constexpr int KB = 16;
  static constexpr int PAD = 4;
  static constexpr int kCtas = D <= 128 ? 2 : 1;            // per SM
  static constexpr int kStageBytes = KB * D * 2 * 2;        // one warp's K and V block
  static constexpr int kMergeBytes = kWarps * R * (D + PAD) * 4;
  static constexpr int kBudget = (kCtas == 2 ? 114 : 227) * 1024 - 2048;
  static constexpr int kFit = (kBudget - kMergeBytes) / (kWarps * kStageBytes);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kStages * kWarps * kStageBytes + kMergeBytes;
  static_assert(kStages >= 2, "decode stages");
};

// S = Q K^T and O = P V by m16n8k16 products: Q's rows are the group's query
// heads, padded to 16, and a warp takes 16 keys at a time through its own ring
// of stages, filled by cp.async ahead of use.  Warps meet only at the end of a
// part.
//
// P goes into the second product as the sum of two 16-bit numbers, so that
// its rounding (2^-17 for bf16) stays below y's own.  With R = 8 the two
// halves share one product: rows 0-7 hold P rounded, rows 8-15 what is left
// of it, and the halves of the result are added at the end.  With R = 16 they
// are two products.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, TcShape<D, R>::kCtas)
decode_tc_kernel(const __grid_constant__ DecodeParams p) {
  using Sh = TcShape<D, R>;
  constexpr int KB = Sh::KB, S = Sh::kStages;
  constexpr int CPR = D / 8;                       // 16-byte chunks per row
  constexpr int kLoads = KB * CPR / 32;            // chunks per lane, K or V
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float s_m[kWarps * R], s_l[kWarps * R];
  __shared__ uint32_t s_mask[kWarps][S];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *s_o = reinterpret_cast<float *>(smem + S * kWarps * Sh::kStageBytes);
  const uint32_t ring = sm103::smem_u32(smem) + warp * S * Sh::kStageBytes;
  const T *q = static_cast<const T *>(p.q);
  const T *kc = static_cast<const T *>(p.kc), *vc = static_cast<const T *>(p.vc);
  const int chunks = (p.group + R - 1) / R;

  Walk<KB> w;
  place<KB>(p, p.n_kv * chunks, w);

  // Row r's chunk c of a block sits at chunk c ^ swizzle(r) of the row, so that
  // the eight rows of an 8x8 matrix fall into different banks.
  auto swizzle = [](int r) { return CPR % 8 == 0 ? (r & 7) : ((r >> 1) & 3); };

  // --- The loading side: `look` finds the next block and loads its page ids
  // one block ahead of `issue`, which starts the copies.
  Walk<KB> pw = w;
  Part pp;
  pp.last = 0;
  int p_blk = 0;
  int nx_j = 0, nx_page = -1, nx_tok = 0, nx_head = 0;
  bool nx_any = true, nx_in = false;
  int err = 0;
  auto look = [&]() {
    while (nx_any && p_blk >= pp.last) {
      nx_any = pw.next(p, pp);
      p_blk = nx_any ? pp.first + warp : 0;
    }
    nx_in = false;
    if (!nx_any) return;
    const Span &sp = pw.part_span;
    nx_j = (sp.blk0 + p_blk) * KB + (lane & 15);
    nx_head = pp.seg / chunks;
    nx_in = nx_j >= sp.lo && nx_j < sp.hi;
    if (nx_in) nx_page = p.table[pp.b * p.table_stride + page_of(p, nx_j, nx_tok)];
    p_blk += kWarps;
  };
  auto issue = [&](int stage) {
    if (nx_any) {
      int64_t off = -1;
      if (nx_in) {
        if (nx_page >= 0 && nx_page < p.num_pages)
          off = nx_page * p.page_stride + nx_tok * p.token_stride + nx_head * p.head_stride;
        else
          err = FA_PAGED_BAD_PAGE;
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
      if (lane == 0) s_mask[warp][stage] = mask;
      const uint32_t dst = ring + stage * Sh::kStageBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int c = i * 32 + lane, r = c / CPR, ch = c % CPR;
        const int64_t o = __shfl_sync(0xffffffffu, off, r);
        const uint32_t to = dst + (r * CPR + (ch ^ swizzle(r))) * 16;
        const int64_t from = (o < 0 ? 0 : o) + ch * 8;
        cp_async16(to, kc + from, o >= 0);
        cp_async16(to + KB * D * 2, vc + from, o >= 0);
      }
    }
    cp_async_commit();
  };

  look();
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) {
    issue(i);
    look();
  }

  // --- The computing side.
  const int row = lane >> 2, col = (lane & 3) * 2;
  // ldmatrix addresses inside a block: K (n = key, k = dim) and V (transposed).
  const int k_row = (lane & 7) + ((lane >> 4) << 3), k_ch = (lane >> 3) & 1;
  const int v_row = (lane & 7) + (((lane >> 3) & 1) << 3), v_ch = lane >> 4;
  int stage = 0, fill = S - 1;
  Meta meta;
  Part part;
  while (w.next(p, part)) {
    const int hk = part.seg / chunks, h0 = (part.seg % chunks) * R;
    const int heads = min(R, p.group - h0), n0 = hk * p.group + h0;
    uint32_t qa[D / 16][R == 8 ? 2 : 4];
    {
      const T *qr = q + part.b * p.q_stride + int64_t(n0) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < (R == 8 ? 2 : 4); ++i) {
          const int r = R == 8 ? row : row + (i & 1) * 8;
          const int d = ks * 16 + col + (R == 8 ? i : i >> 1) * 8;
          uint32_t x = 0;
          if (r < heads) {
            T *h = reinterpret_cast<T *>(&x);
            h[0] = qr[r * D + d];
            h[1] = qr[r * D + d + 1];
          }
          qa[ks][i] = x;
        }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    constexpr int NR = R / 8;       // rows of a lane
    float m[NR], l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
    }

#pragma unroll 1
    for (int blk = part.first + warp; blk < part.last; blk += kWarps) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t kb = ring + stage * Sh::kStageBytes, vb = kb + KB * D * 2;
      const uint32_t mask = s_mask[warp][stage];
      issue(fill);
      look();
      fill = fill + 1 == S ? 0 : fill + 1;
      stage = stage + 1 == S ? 0 : stage + 1;

      float sa[2][2][4];            // [chain][key half][fragment]
#pragma unroll
      for (int i = 0; i < 16; ++i) (&sa[0][0][0])[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kf[4];
        ldsm4(kf, kb + (k_row * CPR + ((ks * 2 + k_ch) ^ swizzle(k_row))) * 16);
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
      float s[NR][4];               // keys col, col + 1, col + 8, col + 9
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
          s[i][e] = (mask >> key) & 1 ? x : -CUDART_INF_F;
          t = fmaxf(t, s[i][e]);
        }
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        mn[i] = fmaxf(m[i], t);
        grows |= mn[i] > m[i];
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          // m = -inf here means that o and l are 0 (or NaN) still.
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
        ldsm4_t(vf, vb + (v_row * CPR + ((dt * 2 + v_ch) ^ swizzle(v_row))) * 16);
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
    }

    __syncthreads();                // the last part's sums have been read
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) {
        s_m[warp * R + i * 8 + row] = m[i];
        s_l[warp * R + i * 8 + row] = l[i];
      }
      float *dst = s_o + (warp * R + i * 8 + row) * (D + Sh::PAD) + col;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const float2 x = R == 8 ? make_float2(o[k][0] + o[k][2], o[k][1] + o[k][3])
                                : make_float2(o[k][i * 2], o[k][i * 2 + 1]);
        *reinterpret_cast<float2 *>(dst + k * 8) = x;
      }
    }
    __syncthreads();
    finish_part<T, D, R, Sh::PAD>(p, part, n0, heads, s_o, s_m, s_l);
    if (part.first != 0 || part.last != part.blocks) meta.note(part, w.segs);
  }
  cp_async_wait<0>();
  if (tid == 0) meta.store(p);
  if (err && p.error) atomicOr(p.error, err);
}

// ---------------------------------------------------------------------------
// CUDA-core kernel.  One warp takes a block of KB keys at a time and holds all
// R heads' running maximum, sum and output; the warps of a CTA take blocks in
// turn and meet at the end of a part.
// ---------------------------------------------------------------------------
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads) decode_simt_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int KB = 8;
  constexpr int PL = D / 32;      // output dims per lane: lane, lane + 32, ...
  __shared__ float s_q[R][D];
  __shared__ __align__(16) float s_o[kWarps][R][D];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (p.group + R - 1) / R;
  Walk<KB> w;
  place<KB>(p, p.n_kv * chunks, w);
  const T *q = static_cast<const T *>(p.q), *kc = static_cast<const T *>(p.kc),
          *vc = static_cast<const T *>(p.vc);
  int err = 0;
  Meta meta;
  Part part;
  while (w.next(p, part)) {
    const Span sp = w.part_span;
    const int hk = part.seg / chunks, h0 = (part.seg % chunks) * R;
    const int heads = min(R, p.group - h0);
    const int n0 = hk * p.group + h0;
    __syncthreads();
    for (int i = tid; i < R * D; i += kThreads)
      s_q[i / D][i % D] =
          i / D < heads ? to_f(q[part.b * p.q_stride + int64_t(n0 + i / D) * D + i % D]) : 0.f;
    __syncthreads();
    float m[R], l[R], o[R][PL];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -CUDART_INF_F;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i) o[r][i] = 0.f;
    }
    for (int blk = part.first + warp; blk < part.last; blk += kWarps) {
      // Lane -> key lane / 4, dims (lane % 4) + 4 i.
      const int j = (sp.blk0 + blk) * KB + lane / 4;
      bool ok = j >= sp.lo && j < sp.hi;
      int64_t off = 0;
      if (ok) {
        int tok;
        const int page = p.table[part.b * p.table_stride + page_of(p, j, tok)];
        if (page >= 0 && page < p.num_pages) {
          off = page * p.page_stride + tok * p.token_stride + hk * p.head_stride;
        } else {
          ok = false;
          err = FA_PAGED_BAD_PAGE;
        }
      }
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
      if (ok) {
        for (int i = lane & 3; i < D; i += 4) {
          const float kv = to_f(kc[off + i]);
#pragma unroll
          for (int r = 0; r < R; ++r) s[r] = fmaf(s_q[r][i], kv, s[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
        s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
        s[r] = ok ? s[r] * p.scale_log2 : -CUDART_INF_F;
        float t = s[r];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, x));
        const float mn = fmaxf(m[r], t), ref = mn == -CUDART_INF_F ? 0.f : mn;
        const float a = exp2f(m[r] - ref);
        m[r] = mn;
        s[r] = exp2f(s[r] - ref);
        t = s[r];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
        l[r] = l[r] * a + t;
#pragma unroll
        for (int i = 0; i < PL; ++i) o[r][i] *= a;
      }
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const int64_t off_k = __shfl_sync(0xffffffffu, off, 4 * k);
        if (!__shfl_sync(0xffffffffu, int(ok), 4 * k)) continue;
        float pk[R];
#pragma unroll
        for (int r = 0; r < R; ++r) pk[r] = __shfl_sync(0xffffffffu, s[r], 4 * k);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          const float vv = to_f(vc[off_k + lane + 32 * i]);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][i] = fmaf(pk[r], vv, o[r][i]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (lane == 0) {
        s_m[warp][r] = m[r];
        s_l[warp][r] = l[r];
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) s_o[warp][r][lane + 32 * i] = o[r][i];
    }
    __syncthreads();
    finish_part<T, D, R, 0>(p, part, n0, heads, &s_o[0][0][0], &s_m[0][0], &s_l[0][0]);
    if (part.first != 0 || part.last != part.blocks) meta.note(part, w.segs);
  }
  if (tid == 0) meta.store(p);
  if (err && p.error) atomicOr(p.error, err);
}

// ---------------------------------------------------------------------------
// Joins the parts of the segments that were cut: block (i, r) takes query head
// r of the segment that CTA i began.  Its warps take the parts in turn, so
// that their loads overlap, and meet in shared memory, always in the same
// order.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(
    const __grid_constant__ DecodeParams p, int rows) {
  constexpr int PL = D / 32;
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  __shared__ float s_o[kJoinWarps][D];
  // Launched while the main kernel may still run: nothing of it is read before.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x, r = blockIdx.y;
  const int id = p.meta[i * 4 + 2];
  if (id < 0) return;
  const int chunks = (p.group + rows - 1) / rows;
  const int segs = p.n_kv * chunks;
  const int b = id / segs, seg = id % segs;
  const int h = (seg % chunks) * rows + r;
  if (h >= p.group) return;
  const int n = (seg / chunks) * p.group + h;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Part 0 is CTA i's slot 1, part k CTA (i + k)'s slot 0.
  int parts = 1;
  for (bool more = true; more; ) {
    const int j = i + parts + lane;
    const bool mine = j < p.grid && p.meta[j * 4] == id;
    const uint32_t got = __ballot_sync(0xffffffffu, mine);
    const int run = got == 0xffffffffu ? 32 : __ffs(~got) - 1;
    parts += run;
    more = run == 32;
  }
  float mx = -CUDART_INF_F, sum = 0.f, acc[PL];
#pragma unroll
  for (int k = 0; k < PL; ++k) acc[k] = 0.f;
#pragma unroll 2
  for (int j = warp; j < parts; j += kJoinWarps) {
    const float *src = slot_of(p, i + j, j == 0 ? 1 : 0, rows);
    const float m2 = src[rows * D + r], l2 = src[rows * D + rows + r];
    const float mn = fmaxf(mx, m2), ref = mn == -CUDART_INF_F ? 0.f : mn;
    const float f = exp2f(mx - ref), f2 = exp2f(m2 - ref);
    mx = mn;
    sum = sum * f + l2 * f2;
#pragma unroll
    for (int k = 0; k < PL; ++k) acc[k] = acc[k] * f + src[r * D + lane + 32 * k] * f2;
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
  float total = 0.f, o = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {
    const float f = exp2f(s_m[k] - ref);
    total += f * s_l[k];
    o += f * s_o[k][d];
  }
  static_cast<T *>(p.y)[b * p.y_stride + int64_t(n) * D + d] =
      from_f<T>(total == 0.f ? 0.f : o / total);
  if (d == 0) write_stats(p, b, n, top * kLn2, total);
}

// The join is launched as a dependent of the main kernel, so that its launch
// overlaps the main kernel's run.
template <typename T, int D>
cudaError_t launch_join(const DecodeParams &p, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.grid, rows);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D>, p, rows);
}

template <int D, int R>
cudaError_t launch_simt(DecodeParams p, int sms, cudaStream_t s) {
  p.grid = sms * kDecodeCtasPerSm;
  decode_simt_kernel<float, D, R><<<p.grid, kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<float, D>(p, R, s);
}

template <typename T, int D, int R>
cudaError_t launch_tc(DecodeParams p, int sms, cudaStream_t s) {
  using Sh = TcShape<D, R>;
  static_assert(Sh::kCtas <= kDecodeCtasPerSm, "workspace size");
  p.grid = sms * Sh::kCtas;
  const cudaError_t e = cudaFuncSetAttribute(
      decode_tc_kernel<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  decode_tc_kernel<T, D, R><<<p.grid, kThreads, Sh::kSmem, s>>>(p);
  const cudaError_t e2 = cudaGetLastError();
  return e2 != cudaSuccess ? e2 : launch_join<T, D>(p, R, s);
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

}  // namespace

// fp32: the heads that a lane's registers hold at once.  16-bit types: the
// rows of one product, all 16 of which serve P rounded once a group has more
// than 8 heads.
int decode_rows(fa_dtype dt, int group) {
  if (dt != FA_DTYPE_FP32) return group <= 8 ? 8 : 16;
  return group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8;
}

size_t decode_part_floats(int rows, int d) { return size_t(slot_floats(rows, d)); }

cudaError_t launch_paged_decode(const DecodeParams &p, fa_dtype dt, int sms, cudaStream_t s) {
  const int rows = decode_rows(dt, p.group);
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
