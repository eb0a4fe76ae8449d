// New key / value rows into the paged cache (fa_paged_write).

#include "paged.h"

namespace fav {
namespace {

constexpr int kThreads = 256;

template <typename V>
__device__ __forceinline__ V load_once(const V *p) {
  return *p;
}
template <>
__device__ __forceinline__ uint4 load_once<uint4>(const uint4 *p) {
  return __ldcs(p);
}

template <typename V>
__device__ __forceinline__ void store_once(V *p, V v) {
  *p = v;
}
template <>
__device__ __forceinline__ void store_once<uint4>(uint4 *p, uint4 v) {
  __stcs(p, v);
}

// A copy, bound by memory: a thread takes U pieces (of type V: 16 bytes where every row
// starts on a 16-byte boundary, else one element) of K and of V, kThreads apart, and
// has all its loads on the way before the first store.  Pieces are numbered token by token, so
// that a token's row is read, and where the layout allows written, in one sweep.
// Neither side is read again soon, so both are streamed past the caches.
// 39332 rows of 8 x 128 bf16: 49.7 us, 6.5 TB/s (one piece of each per thread 57,
// four 57, eight 83; without the streaming hints 51); with rows off those boundaries
// 290 us, bound by the number of pieces.
template <typename V, int U>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ WriteParams p,
                                                         int esize) {
  asm volatile("griddepcontrol.launch_dependents;");   // a decode may be launched behind it
  const int per = int(sizeof(V)) / esize;         // elements per piece
  const unsigned head_v = p.d / per;              // pieces per head
  const unsigned row_v = p.n_kv * head_v;         // ... and per token
  const int64_t first = int64_t(blockIdx.x) * (kThreads * U);
  // Token and piece of the block's first one; the others follow in 32 bits.
  const int64_t t0 = first / row_v;
  const unsigned r0 = unsigned(first - t0 * row_v) + threadIdx.x;
  V k[U], v[U];
  int64_t to[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned i = r0 + u * kThreads;
    const unsigned dt = i / row_v, r = i - dt * row_v;
    const int64_t t = t0 + dt;
    to[u] = -1;
    if (t >= p.tokens) continue;
    const int64_t slot = p.slots[t];
    if (slot < 0) continue;
    if (slot >= p.n_slots) {
      if (p.error && r == 0) atomicOr(p.error, FA_PAGED_BAD_SLOT);
      continue;
    }
    int64_t page, tok;
    if (p.page_shift >= 0) {
      page = slot >> p.page_shift;
      tok = slot & (p.page_size - 1);
    } else if (slot <= 0xffffffffll) {
      page = uint32_t(slot) / uint32_t(p.page_size);
      tok = slot - page * p.page_size;
    } else {
      page = slot / p.page_size;
      tok = slot - page * p.page_size;
    }
    const unsigned h = r / head_v, c = r - h * head_v;
    to[u] = (page * p.page_stride + tok * p.token_stride + h * p.head_stride) / per + c;
    k[u] = load_once(static_cast<const V *>(p.k) + (t * p.k_stride / per + r));
    v[u] = load_once(static_cast<const V *>(p.v) + (t * p.v_stride / per + r));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (to[u] < 0) continue;
    store_once(static_cast<V *>(p.kc) + to[u], k[u]);
    store_once(static_cast<V *>(p.vc) + to[u], v[u]);
  }
}

template <typename V, int U>
cudaError_t launch_u(const WriteParams &p, int esize, int64_t pieces, cudaStream_t s) {
  const int64_t blocks = (pieces + kThreads * U - 1) / (kThreads * U);
  write_kernel<V, U><<<unsigned(blocks), kThreads, 0, s>>>(p, esize);
  return cudaGetLastError();
}

template <typename V>
cudaError_t launch(const WriteParams &p, int esize, cudaStream_t s) {
  const int64_t pieces = int64_t(p.tokens) * p.n_kv * (p.d * esize / int(sizeof(V)));
  // Few rows: one piece per thread, to spread them over the SMs (the two cost the
  // same at 1024 rows of 8 x 128 bf16, two pieces 0.4 us less at 4096).
  if (pieces <= 152 * kThreads * 4) return launch_u<V, 1>(p, esize, pieces, s);
  return launch_u<V, 2>(p, esize, pieces, s);
}

}  // namespace

cudaError_t launch_paged_write(const WriteParams &p, fa_dtype dt, cudaStream_t s) {
  const int esize = dt == FA_DTYPE_FP32 ? 4 : 2;
  // Every row start a multiple of 16 bytes?
  const uint64_t mis = (reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v) |
                        uint64_t(p.k_stride * esize) | uint64_t(p.v_stride * esize)) & 15u;
  if (mis == 0) return launch<uint4>(p, esize, s);
  return esize == 4 ? launch<uint32_t>(p, esize, s) : launch<uint16_t>(p, esize, s);
}

}  // namespace fav
