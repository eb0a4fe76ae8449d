// New key / value rows into the paged cache (fa_paged_write).

#include "paged.h"

namespace fav {
namespace {

// One element of V per (token, head, position); V is the widest type that
// divides the rows' alignment.
template <typename V>
__global__ void __launch_bounds__(256) write_kernel(WriteParams p, int esize) {
  const int per = int(sizeof(V)) / esize;         // elements per V
  const int row_v = p.d / per;                    // V per head row
  const int64_t n = int64_t(p.tokens) * p.n_kv * row_v;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < n;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = i / (p.n_kv * row_v);
    const int r = int(i - t * (p.n_kv * row_v));
    const int h = r / row_v, c = r - h * row_v;
    const int64_t slot = p.slots[t];
    if (slot < 0) continue;
    if (slot >= p.n_slots) {
      if (p.error && r == 0) atomicOr(p.error, FA_PAGED_BAD_SLOT);
      continue;
    }
    const int64_t page = slot / p.page_size, tok = slot - page * p.page_size;
    const int64_t to =
        (page * p.page_stride + tok * p.token_stride + h * p.head_stride) / per + c;
    static_cast<V *>(p.kc)[to] = static_cast<const V *>(p.k)[t * p.k_stride / per + r];
    static_cast<V *>(p.vc)[to] = static_cast<const V *>(p.v)[t * p.v_stride / per + r];
  }
}

template <typename V>
cudaError_t launch(const WriteParams &p, int esize, cudaStream_t s) {
  const int64_t n = int64_t(p.tokens) * p.n_kv * (p.d * esize / int(sizeof(V)));
  int64_t blocks = (n + 255) / 256;
  if (blocks > 152 * 64) blocks = 152 * 64;
  write_kernel<V><<<int(blocks), 256, 0, s>>>(p, esize);
  return cudaGetLastError();
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
