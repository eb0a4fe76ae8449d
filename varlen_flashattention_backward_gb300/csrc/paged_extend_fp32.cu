// fa_paged_extend in fp32, on CUDA cores.
//
// A block is 64 packed query rows, a tile 32 keys.  128 threads, as 16 groups of 8:
// group g has the rows g, g + 16, g + 32, g + 48; of a tile's scores its lane x has the
// keys x, x + 8, x + 16, x + 24, and of the results the columns 4 x + 32 c.  K and V have
// one buffer each: the next K is on its way during the softmax and the products with
// V, the next V during the products with K.
//
// Bound by the shared memory that feeds the FMAs, 128 bytes a cycle: per four dims 32
// packed FMAs and 8 16-byte loads a thread in the first product, per four keys D / 2 and
// D / 8 + 4 in the second.  512 tokens behind 3500, 32 heads on 8, D 128: 765 us, 41
// TFLOP/s (single FMAs: 884; with half the warps and eight rows per thread, 12 loads for
// 64: 1024).  Three CTAs per multiprocessor up to head dim 64, two beyond: 263 and 291
// us at D 32, 422 and 443 at D 64; at D 128 three spill, 776.  Tables looked up a tile
// ahead gain nothing.

#include <type_traits>

#include "paged_extend.cuh"

namespace fav {
namespace {

constexpr int kBR = 64, kBN = 32, kThreads = 128;

template <int D>
struct Smem {
  float q[kBR][D + 4];
  float k[kBN][D + 4];
  float v[kBN][D + 4];
  float p[kBR][kBN + 4];
  int fine[2][kBN];      // the key's page is one of the cache's
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, D <= 64 ? 3 : 2) extend_fp32_kernel(const __grid_constant__ ExtendParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<D> &s = *reinterpret_cast<Smem<D> *>(raw);
  const int tid = threadIdx.x, x = tid & 7, g = tid >> 3;
  constexpr int C = D / 32;                 // column chunks of four per lane

  Walk<kBR, kBN> walk;
  {
    Line line;
    Place at;
    const bool any = measure<kBR, kBN, kThreads>(p, *reinterpret_cast<Measure *>(raw), line, at);
    walk.begin(p, line, at, any);
  }
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  Segment seg;
  // (Every thread walks for itself; the barriers below do not depend on what it reads
  // but for the number of segments and tiles, which one thread tells.)
  __shared__ Segment s_seg;
  __shared__ int s_more, s_flagged, s_odd;
  if (tid == 0) s_flagged = s_odd = 0;
  while (true) {
    if (tid == 0) {
      s_more = walk.next(p, seg);
      s_seg = seg;
    }
    __syncthreads();
    if (!s_more) break;
    seg = s_seg;
    const Request &r = seg.r;
    const int n0 = seg.h * p.group;
    const float flip = float(p.sign);
    // Query rows; zeros behind the last.
    for (int i = tid; i < kBR * (D / 4); i += kThreads) {
      const int row = i / (D / 4), c = i - row * (D / 4);
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < seg.k.rows) {
        const int packed = seg.k.row0 + row, t = packed / p.group;
        const float *src = static_cast<const float *>(p.q) + (r.start + t) * p.q_stride +
                           int64_t(n0 + packed - t * p.group) * D + c * 4;
        if (p.q_chunks) q = *reinterpret_cast<const float4 *>(src);
        else q = make_float4(src[0], src[1], src[2], src[3]);
      }
      q.x *= flip, q.y *= flip, q.z *= flip, q.w *= flip;
      *reinterpret_cast<float4 *>(&s.q[row][c * 4]) = q;
    }
    int lo[4], hi[4];
    float m[4], l[4], o[4][C * 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = g + 16 * i;
      lo[i] = hi[i] = 0;
      if (row < seg.k.rows) keys_of(p, r, (seg.k.row0 + row) / p.group, lo[i], hi[i]);
      m[i] = -CUDART_INF_F;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < C * 4; ++c) o[i][c] = 0.f;
    }

    // A thread copies a quarter of a key's row.
    const int key = tid >> 2, part = tid & 3;
    const auto load = [&](const void *cache, float (*dst)[D + 4], int t, int *fine) {
      const int j = (seg.k.tile0 + t) * kBN + key;
      const float *src = j < r.len ? cached<float>(p, cache, seg.b, seg.h, j) : nullptr;
      if (fine != nullptr && part == 0) {
        fine[key] = src != nullptr;
        if (j < r.len && src == nullptr) s_odd = 1;
      }
      const float *from = src != nullptr ? src : static_cast<const float *>(cache);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        cp_async16(sm103::smem_u32(&dst[key][(c * 4 + part) * 4]), from + (c * 4 + part) * 4, src != nullptr);
      cp_async_commit();
    };
    if (seg.t1 > seg.t0) {
      load(p.kc, s.k, seg.t0, s.fine[seg.t0 & 1]);
      load(p.vc, s.v, seg.t0, nullptr);
    }
    // R: how many of its four rows a thread has; drafts and the ends of chunks fill few.
    const auto tiles = [&](auto count) {
      constexpr int R = decltype(count)::value;
      for (int t = seg.t0; t < seg.t1; ++t) {
        const int k0 = (seg.k.tile0 + t) * kBN;
        cp_async_wait<1>();
        __syncthreads();
        float a[R][4], a2[R][4];      // sums over even and odd dims
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) a[i][c] = a2[i][c] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
          float4 q[R], k[4];
#pragma unroll
          for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4 *>(&s.q[g + 16 * i][d]);
#pragma unroll
          for (int c = 0; c < 4; ++c) k[c] = *reinterpret_cast<const float4 *>(&s.k[x + 8 * c][d]);
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              sm103::fma2(a[i][c], a2[i][c], q[i].x, q[i].y, k[c].x, k[c].y, a[i][c], a2[i][c]);
              sm103::fma2(a[i][c], a2[i][c], q[i].z, q[i].w, k[c].z, k[c].w, a[i][c], a2[i][c]);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) a[i][c] += a2[i][c];
        const int *fine = s.fine[t & 1];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float top = -CUDART_INF_F;
          bool seen[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = k0 + x + 8 * c;
            seen[c] = j >= lo[i] && j < hi[i] && fine[x + 8 * c];
            a[i][c] = seen[c] ? a[i][c] * p.scale_log2 : -CUDART_INF_F;
            top = fmaxf(top, a[i][c]);
          }
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
          const float mn = fmaxf(m[i], top), ref = mn == -CUDART_INF_F ? 0.f : mn;
          const float f = exp2f(m[i] - ref);
          m[i] = mn;
          l[i] *= f;
#pragma unroll
          for (int c = 0; c < C * 4; ++c) o[i][c] *= f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float w = exp2f(a[i][c] - ref);
            l[i] += w;                           // each lane its own keys
            s.p[g + 16 * i][x + 8 * c] = w;
          }
        }
        __syncthreads();                         // K has been read
        if (t + 1 < seg.t1) load(p.kc, s.k, t + 1, s.fine[(t + 1) & 1]);
        else cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
#pragma unroll 2
        for (int j = 0; j < kBN; j += 4) {
          float4 w[R];
#pragma unroll
          for (int i = 0; i < R; ++i) w[i] = *reinterpret_cast<const float4 *>(&s.p[g + 16 * i][j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const float4 v = *reinterpret_cast<const float4 *>(&s.v[j + e][x * 4 + 32 * c]);
#pragma unroll
              for (int i = 0; i < R; ++i) {
                const float we = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
                float *own = &o[i][4 * c];
                sm103::fma2(own[0], own[1], we, we, v.x, v.y, own[0], own[1]);
                sm103::fma2(own[2], own[3], we, we, v.z, v.w, own[2], own[3]);
              }
            }
          }
        }
        __syncthreads();                         // V and P have been read
        if (t + 1 < seg.t1) load(p.vc, s.v, t + 1, nullptr);
      }
    };
    if (seg.k.rows <= 16) tiles(std::integral_constant<int, 1>{});
    else if (seg.k.rows <= 32) tiles(std::integral_constant<int, 2>{});
    else tiles(std::integral_constant<int, 4>{});
    // Results.  A warp holds the rows 4 w .. 4 w + 3 and those 16, 32, 48 further on.
    cp_async_wait<0>();
    if (seg.t0 == 0 && tid < 2) p.flags[int64_t(seg.item) * 2 + tid] = 0;
    __syncthreads();
    float *slot = seg.slot >= 0 ? part_of<kBR>(p, blockIdx.x, seg.slot) : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = g + 16 * i;
#pragma unroll
      for (int sh = 1; sh < 8; sh <<= 1) l[i] += __shfl_xor_sync(kFull, l[i], sh);
      if (slot != nullptr) {
        if (row < seg.k.rows) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) slot[(x * 4 + 32 * c + e) * kBR + row] = o[i][4 * c + e];
          if (x == 0) {
            slot[D * kBR + row] = m[i];
            slot[(D + 1) * kBR + row] = l[i];
            slot[(D + 2) * kBR + row] = m[i];
          }
        }
        continue;
      }
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
      bool bad = false;
#pragma unroll
      for (int c = 0; c < C * 4; ++c) {
        bad |= !isfinite(o[i][c]);
        o[i][c] *= inv;
      }
      const uint32_t bads = __ballot_sync(kFull, bad);
      if (row >= seg.k.rows) continue;
      const int packed = seg.k.row0 + row, t = packed / p.group, n = n0 + packed - t * p.group;
      float *y = static_cast<float *>(p.y) + (r.start + t) * p.y_stride + int64_t(n) * D;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float *to = y + x * 4 + 32 * c;
        if (p.y_chunks) {
          *reinterpret_cast<float4 *>(to) = make_float4(o[i][4 * c], o[i][4 * c + 1], o[i][4 * c + 2], o[i][4 * c + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = o[i][4 * c + e];
        }
      }
      if (x == 0) {
        write_stats(p, int64_t(r.start + t) * p.n + n, m[i] * kLn2, l[i]);
        if ((bads >> (8 * (g & 3))) & 0xff) {
          s_flagged = 1;
          atomicOr(p.flags + int64_t(seg.item) * 2 + row / 32, 1u << (row & 31));
        }
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) {
    walk.rec.flagged = s_flagged;
    walk.rec.odd = s_odd;
    reinterpret_cast<Record *>(p.records)[blockIdx.x] = walk.rec;
  }
}

template <int D>
cudaError_t launch_dim(const ExtendParams &p, int ctas, cudaStream_t s) {
  const int smem = int(sizeof(Smem<D>) > sizeof(Measure) ? sizeof(Smem<D>) : sizeof(Measure));
  cudaError_t e = cudaFuncSetAttribute(extend_fp32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  extend_fp32_kernel<D><<<ctas, kThreads, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<float, D, kBR, kBN>(p, ctas, s);
}

}  // namespace

cudaError_t launch_paged_extend_fp32(const ExtendParams &p, int ctas, cudaStream_t s) {
  FAV_EXTEND_BY_DIM(launch_dim);
}

}  // namespace fav
