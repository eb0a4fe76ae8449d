// Attention of one new token per request over the paged cache
// (fa_paged_decode): S_j = scale q . k_j, P = exp(S - max), y = P V / sum P.

#include <math_constants.h>

#include "common.cuh"
#include "paged.h"

namespace fav {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
// A request costs a CTA about this many blocks of keys beside its own.
constexpr int kSwitchBlocks = 2;

// ---------------------------------------------------------------------------
// Division of the work
//
// A segment is one request, one key head and up to R of its query heads; its
// keys are cut into blocks.  The segments, each weighing its blocks plus
// kSwitchBlocks, form a line that is cut into `grid` ranges of equal weight,
// one per CTA.  A CTA's share of a segment is a part.  A part that is a whole
// segment writes y; of the others a CTA has at most two (its first and its
// last), which go to its two slots of the workspace: slot 0 for a part that
// does not begin its segment, slot 1 for one that begins it and does not end
// it.  join_kernel adds the parts of a segment in order.
// ---------------------------------------------------------------------------
struct Part {
  int b, seg;           // request; segment index inside the request
  int64_t first, last;  // blocks [first, last), relative to the request's first
  int64_t blocks;       // of the whole segment
};

struct Span {
  int lo, hi;       // keys [lo, hi) that the query sees
  int blk0;         // first block (absolute)
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
  int64_t left;    // weight left of the range
  int64_t off;     // weight already passed inside the current segment
  int b, seg, segs;
  Span span;

  __device__ __forceinline__ bool next(const DecodeParams &p, Part &part) {
    while (left > 0) {
      const int64_t weight = span.blocks + kSwitchBlocks;
      const int64_t end = min(off + left, weight);
      part.b = b;
      part.seg = seg;
      part.blocks = span.blocks;
      part.first = max(off - kSwitchBlocks, int64_t(0));
      part.last = max(end - kSwitchBlocks, int64_t(0));
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
    w.off = s_off - w.seg * weight;
  }
}

// Words of the workspace's meta block, four per CTA: the segment (b * segs +
// seg) whose part is in slot 0 (or -1), whether that part ends it, the segment
// in slot 1 (or -1).
__device__ __forceinline__ int64_t slot_at(const DecodeParams &p, int cta, int slot, int rows) {
  return (int64_t(cta) * 2 + slot) * rows * (p.d + 2);
}

template <typename T>
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

// ---------------------------------------------------------------------------
// CUDA-core kernel.  One warp takes a block of KB keys at a time and holds all
// R heads' running maximum, sum and output; the warps of a CTA take blocks in
// turn and meet at the end of a part.
// ---------------------------------------------------------------------------
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads) decode_simt_kernel(DecodeParams p) {
  constexpr int KB = 8;
  constexpr int PL = D / 32;      // output dims per lane: lane, lane + 32, ...
  __shared__ float s_q[R][D];
  __shared__ float s_o[kWarps][R][D];
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunks = (p.group + R - 1) / R;
  Walk<KB> w;
  place<KB>(p, p.n_kv * chunks, w);
  const T *q = static_cast<const T *>(p.q), *kc = static_cast<const T *>(p.kc),
          *vc = static_cast<const T *>(p.vc);
  int meta0 = -1, ends0 = 0, meta1 = -1, err = 0;
  Part part;
  while (w.next(p, part)) {
    const Span sp = span_of<KB>(p, part.b);
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
    for (int64_t blk = part.first + warp; blk < part.last; blk += kWarps) {
      // Lane -> key lane / 4, dims (lane % 4) + 4 i.
      const int j = int(sp.blk0 + blk) * KB + lane / 4;
      bool ok = j >= sp.lo && j < sp.hi;
      int64_t off = 0;
      if (ok) {
        const int page = p.table[part.b * p.table_stride + j / p.page_size];
        if (page >= 0 && page < p.num_pages) {
          off = page * p.page_stride + (j % p.page_size) * p.token_stride + hk * p.head_stride;
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
    const bool whole = part.first == 0 && part.last == part.blocks;
    const int slot = part.first == 0 ? 1 : 0;
    float *dst = p.part + slot_at(p, blockIdx.x, slot, R);
    for (int i = tid; i < heads * D; i += kThreads) {
      const int r = i / D, d = i % D;
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, s_m[k][r]);
      const float ref = mx == -CUDART_INF_F ? 0.f : mx;
      float sum = 0.f, acc = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float f = exp2f(s_m[k][r] - ref);
        sum += f * s_l[k][r];
        acc += f * s_o[k][r][d];
      }
      if (whole) {
        static_cast<T *>(p.y)[part.b * p.y_stride + int64_t(n0 + r) * D + d] =
            from_f<T>(sum == 0.f ? 0.f : acc / sum);
        if (d == 0) write_stats<T>(p, part.b, n0 + r, mx * kLn2, sum);
      } else {
        dst[i] = acc;
        if (d == 0) {
          dst[R * D + r] = mx;
          dst[R * D + R + r] = sum;
        }
      }
    }
    if (!whole) {
      const int id = part.b * w.segs + part.seg;
      if (slot == 0) {
        meta0 = id;
        ends0 = part.last == part.blocks;
      } else {
        meta1 = id;
      }
    }
  }
  if (tid == 0) {
    int32_t *meta = p.meta + blockIdx.x * 4;
    meta[0] = meta0;
    meta[1] = ends0;
    meta[2] = meta1;
  }
  if (err && p.error) atomicOr(p.error, err);
}

// ---------------------------------------------------------------------------
// Joins the parts of the segments that were cut: block (i, r) takes query head
// r of the segment that CTA i began.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(128) join_kernel(DecodeParams p, int rows) {
  const int i = blockIdx.x, r = blockIdx.y;
  const int id = p.meta[i * 4 + 2];
  if (id < 0) return;
  const int chunks = (p.group + rows - 1) / rows;
  const int segs = p.n_kv * chunks;
  const int b = id / segs, seg = id % segs;
  const int h = (seg % chunks) * rows + r;
  if (h >= p.group) return;
  const int n = (seg / chunks) * p.group + h;
  const int dim = p.d;
  for (int d = threadIdx.x; d < dim; d += blockDim.x) {
    const float *src = p.part + slot_at(p, i, 1, rows);
    float mx = src[rows * dim + r], sum = src[rows * dim + rows + r], acc = src[r * dim + d];
    for (int j = i + 1; j < p.grid && p.meta[j * 4] == id; ++j) {
      src = p.part + slot_at(p, j, 0, rows);
      const float m2 = src[rows * dim + r];
      const float mn = fmaxf(mx, m2), ref = mn == -CUDART_INF_F ? 0.f : mn;
      const float f = exp2f(mx - ref), f2 = exp2f(m2 - ref);
      mx = mn;
      sum = sum * f + src[rows * dim + rows + r] * f2;
      acc = acc * f + src[r * dim + d] * f2;
      if (p.meta[j * 4 + 1]) break;
    }
    static_cast<T *>(p.y)[b * p.y_stride + int64_t(n) * dim + d] =
        from_f<T>(sum == 0.f ? 0.f : acc / sum);
    if (d == 0) write_stats<T>(p, b, n, mx * kLn2, sum);
  }
}

template <typename T, int D, int R>
cudaError_t launch_r(DecodeParams p, cudaStream_t s) {
  decode_simt_kernel<T, D, R><<<p.grid, kThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  join_kernel<T><<<dim3(p.grid, R), 128, 0, s>>>(p, R);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const DecodeParams &p, int rows, cudaStream_t s) {
  switch (rows) {
    case 1: return launch_r<T, D, 1>(p, s);
    case 2: return launch_r<T, D, 2>(p, s);
    case 4: return launch_r<T, D, 4>(p, s);
    default: return launch_r<T, D, 8>(p, s);
  }
}

template <typename T>
cudaError_t launch_t(const DecodeParams &p, int rows, cudaStream_t s) {
  switch (p.d) {
    case 32: return launch_d<T, 32>(p, rows, s);
    case 64: return launch_d<T, 64>(p, rows, s);
    case 96: return launch_d<T, 96>(p, rows, s);
    case 128: return launch_d<T, 128>(p, rows, s);
    case 192: return launch_d<T, 192>(p, rows, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int decode_rows(fa_dtype, int group) {
  return group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8;
}

cudaError_t launch_paged_decode(const DecodeParams &p0, fa_dtype dt, int sms, cudaStream_t s) {
  DecodeParams p = p0;
  p.grid = sms * kDecodeCtasPerSm;
  const int rows = decode_rows(dt, p.group);
  if (dt == FA_DTYPE_FP32) return launch_t<float>(p, rows, s);
  if (dt == FA_DTYPE_FP16) return launch_t<__half>(p, rows, s);
  return launch_t<__nv_bfloat16>(p, rows, s);
}

}  // namespace fav
