// Host side of the paged-cache entry points: argument checks, the decode
// workspace and the launches.  Nothing here allocates or throws.

#include <cmath>

#include "internal.h"
#include "paged.h"

namespace fav {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxPageSize = 65536;
constexpr int64_t kMaxKeys = int64_t(1) << 30;
constexpr int64_t kMaxI32 = 2147483647;
// Extent of one axis (count * stride) in elements: offsets stay inside 64 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 58;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool known_dtype(fa_dtype dt) {
  return dt == FA_DTYPE_FP32 || dt == FA_DTYPE_FP16 || dt == FA_DTYPE_BF16;
}

// Multiprocessors of the current device; where there is none (a size call on
// a machine without a GPU) those of a whole GB300.
int sm_count() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) {
    cudaGetLastError();
    return 152;
  }
  return v;
}

fa_status check_table(int64_t batch, int64_t num_pages, int64_t page_size, int64_t max_pages,
                      int64_t table_stride) {
  if (batch < 1 || batch > kMaxBatch) return FA_ERR_INVALID;
  if (num_pages < 1 || num_pages > kMaxI32) return FA_ERR_INVALID;
  if (page_size < 1 || page_size > kMaxPageSize) return FA_ERR_INVALID;
  if (max_pages < 1 || max_pages > kMaxKeys || max_pages * page_size > kMaxKeys)
    return FA_ERR_INVALID;
  if (table_stride < max_pages || table_stride > kMaxExtent / batch) return FA_ERR_INVALID;
  return FA_OK;
}

fa_status check_heads(int64_t head_num, int64_t head_num_kv, int64_t head_dim, fa_dtype dtype) {
  if (!known_dtype(dtype)) return FA_ERR_INVALID;
  if (head_num < 1 || head_num > 256) return FA_ERR_INVALID;
  if (head_num_kv < 1 || head_num_kv > head_num || head_num % head_num_kv != 0)
    return FA_ERR_INVALID;
  if (head_dim < 1 || head_dim > 768) return FA_ERR_INVALID;
  if (head_dim != 32 && head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// Strides and bases of the cache.  The stride of an axis of one entry is
// never used: it becomes 0 and may be anything.
fa_status check_cache(const void *k_pages, const void *v_pages, int64_t num_pages,
                      int64_t page_size, int64_t n_kv, int64_t head_dim, int64_t &page_stride,
                      int64_t &token_stride, int64_t &head_stride, fa_dtype dtype) {
  const int64_t vec = dtype == FA_DTYPE_FP32 ? 4 : 8;   // elements in 16 bytes
  auto bad = [&](int64_t &stride, int64_t count) {
    if (count == 1) {
      stride = 0;
      return false;
    }
    return stride < head_dim || stride > kMaxExtent / count || stride % vec != 0;
  };
  if (bad(page_stride, num_pages) || bad(token_stride, page_size) || bad(head_stride, n_kv))
    return FA_ERR_INVALID;
  if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15u) != 0)
    return FA_ERR_INVALID;
  return FA_OK;
}

// Row stride of q, y, k or v: `count` rows of `row` elements.
bool bad_rows(int64_t &stride, int64_t count, int64_t row) {
  if (count <= 1) {
    stride = row;
    return false;
  }
  return stride < row || stride > kMaxExtent / count;
}

// q, y, k and v rows: aligned to their element type.
bool element_aligned(const void *ptr, fa_dtype dt) {
  return reinterpret_cast<uintptr_t>(ptr) % (dt == FA_DTYPE_FP32 ? 4 : 2) == 0;
}

// log2 of a power of 2, -1 for another number.
int log2_or_none(int64_t x) {
  if ((x & (x - 1)) != 0) return -1;
  int n = 0;
  while ((int64_t(1) << n) < x) ++n;
  return n;
}

// Bytes of a decode call's workspace: two partial results per range, none for a
// direct call.
size_t decode_bytes(const DecodePlan &plan, int sms, int group, int64_t head_dim) {
  if (plan.direct) return 0;
  const int rows = group < plan.rows ? group : plan.rows;
  return align_up(size_t(sms) * plan.teams * 2 * decode_part_floats(rows, int(head_dim)) *
                  sizeof(float));
}

// Keys that a query can see at most.
int64_t most_keys(int64_t max_pages, int64_t page_size, int64_t pre_tokens) {
  const int64_t keys = max_pages * page_size;
  return pre_tokens < 0 ? 0 : pre_tokens < keys ? pre_tokens + 1 : keys;
}

}  // namespace
}  // namespace fav

using namespace fav;

extern "C" {

fa_status fa_paged_plan(int32_t *block_table, int64_t max_pages, int64_t table_stride,
                        const int32_t *seq_lens, const int32_t *delta, int64_t batch,
                        int32_t *free_pages, const int64_t *free_state, int64_t num_pages,
                        int64_t page_size, int64_t *slots, int64_t max_tokens,
                        int64_t *cu_tokens, int32_t *seq_lens_out, int64_t *free_state_out,
                        int32_t *error, fa_stream_t stream) {
  if (!block_table || !seq_lens || !delta || !free_pages || !free_state || !cu_tokens ||
      !seq_lens_out || !free_state_out || (max_tokens > 0 && !slots))
    return FA_ERR_NULLPTR;
  const fa_status st = check_table(batch, num_pages, page_size, max_pages, table_stride);
  if (st != FA_OK) return st;
  if (max_tokens < 0 || max_tokens > kMaxI32) return FA_ERR_INVALID;
  PlanParams p{};
  p.table = block_table;
  p.table_stride = table_stride;
  p.lens = seq_lens;
  p.delta = delta;
  p.ring = free_pages;
  p.state = free_state;
  p.slots = slots;
  p.cu = cu_tokens;
  p.lens_out = seq_lens_out;
  p.state_out = free_state_out;
  p.error = error;
  p.max_tokens = max_tokens;
  p.batch = int(batch);
  p.max_pages = int(max_pages);
  p.num_pages = int(num_pages);
  p.page_size = int(page_size);
  p.page_shift = log2_or_none(page_size);
  return launch_paged_plan(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                     : FA_ERR_CUDA;
}

fa_status fa_paged_write(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                         const int64_t *slots, int64_t tokens, void *k_pages, void *v_pages,
                         int64_t num_pages, int64_t page_size, int64_t head_num_kv,
                         int64_t head_dim, int64_t page_stride, int64_t token_stride,
                         int64_t head_stride, fa_dtype dtype, int32_t *error,
                         fa_stream_t stream) {
  if (!k_pages || !v_pages || (tokens > 0 && (!k || !v || !slots))) return FA_ERR_NULLPTR;
  fa_status st = check_heads(head_num_kv, head_num_kv, head_dim, dtype);
  if (st != FA_OK) return st;
  st = check_table(1, num_pages, page_size, 1, 1);
  if (st != FA_OK) return st;
  st = check_cache(k_pages, v_pages, num_pages, page_size, head_num_kv, head_dim, page_stride,
                   token_stride, head_stride, dtype);
  if (st != FA_OK) return st;
  if (tokens < 0 || tokens > kMaxI32) return FA_ERR_INVALID;
  const int64_t row = head_num_kv * head_dim;
  if (bad_rows(k_stride, tokens, row) || bad_rows(v_stride, tokens, row)) return FA_ERR_INVALID;
  if (!element_aligned(k, dtype) || !element_aligned(v, dtype)) return FA_ERR_INVALID;
  if (tokens == 0) return FA_OK;
  WriteParams p{};
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.kc = k_pages;
  p.vc = v_pages;
  p.n_slots = num_pages * page_size;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.error = error;
  p.tokens = int(tokens);
  p.page_size = int(page_size);
  p.page_shift = log2_or_none(page_size);
  p.n_kv = int(head_num_kv);
  p.d = int(head_dim);
  return launch_paged_write(p, dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_paged_decode_workspace_size(int64_t batch, int64_t head_num, int64_t head_num_kv,
                                         int64_t head_dim, fa_dtype dtype, int64_t page_size,
                                         int64_t max_pages, int64_t pre_tokens,
                                         size_t *workspace_bytes) {
  if (!workspace_bytes) return FA_ERR_NULLPTR;
  fa_status st = check_table(batch, 1, page_size, max_pages, max_pages);
  if (st != FA_OK) return st;
  st = check_heads(head_num, head_num_kv, head_dim, dtype);
  if (st != FA_OK) return st;
  const int sms = sm_count();
  const DecodePlan plan = decode_plan(dtype, int(batch), int(head_num_kv),
                                      int(head_num / head_num_kv), int(head_dim),
                                      most_keys(max_pages, page_size, pre_tokens), sms);
  *workspace_bytes = decode_bytes(plan, sms, int(head_num / head_num_kv), head_dim);
  return FA_OK;
}

fa_status fa_paged_decode(const void *q, int64_t q_stride, const void *k_pages,
                          const void *v_pages, int64_t num_pages, int64_t page_size,
                          int64_t page_stride, int64_t token_stride, int64_t head_stride,
                          const int32_t *block_table, int64_t max_pages, int64_t table_stride,
                          const int32_t *seq_lens, int64_t batch, int64_t head_num,
                          int64_t head_num_kv, int64_t head_dim, fa_dtype dtype, double scale,
                          int64_t pre_tokens, void *y, int64_t y_stride, float *softmax_max,
                          float *softmax_sum, int32_t *error, void *workspace,
                          size_t workspace_bytes, fa_stream_t stream) {
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !y ||
      (!softmax_max != !softmax_sum))
    return FA_ERR_NULLPTR;
  fa_status st = check_heads(head_num, head_num_kv, head_dim, dtype);
  if (st != FA_OK) return st;
  st = check_table(batch, num_pages, page_size, max_pages, table_stride);
  if (st != FA_OK) return st;
  st = check_cache(k_pages, v_pages, num_pages, page_size, head_num_kv, head_dim, page_stride,
                   token_stride, head_stride, dtype);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale)) return FA_ERR_INVALID;
  const int64_t row = head_num * head_dim;
  if (bad_rows(q_stride, batch, row) || bad_rows(y_stride, batch, row)) return FA_ERR_INVALID;
  if (!element_aligned(q, dtype) || !element_aligned(y, dtype)) return FA_ERR_INVALID;
  const int sms = sm_count();
  const int group = int(head_num / head_num_kv);
  const DecodePlan plan =
      decode_plan(dtype, int(batch), int(head_num_kv), group, int(head_dim),
                  most_keys(max_pages, page_size, pre_tokens), sms);
  const size_t bytes = decode_bytes(plan, sms, group, head_dim);
  if (bytes > 0 && !workspace) return FA_ERR_NULLPTR;
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return FA_ERR_INVALID;
  if (workspace_bytes < bytes) return FA_ERR_WORKSPACE;

  DecodeParams p{};
  p.q = q;
  p.q_stride = q_stride;
  p.kc = k_pages;
  p.vc = v_pages;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.table = block_table;
  p.table_stride = table_stride;
  p.lens = seq_lens;
  p.y = y;
  p.y_stride = y_stride;
  p.smax = softmax_max;
  p.ssum = softmax_sum;
  p.error = error;
  p.part = static_cast<float *>(workspace);
  p.slot_rows = group < plan.rows ? group : plan.rows;
  p.num_pages = int(num_pages);
  p.page_size = int(page_size);
  p.page_shift = log2_or_none(page_size);
  p.max_pages = int(max_pages);
  p.batch = int(batch);
  p.n = int(head_num);
  p.n_kv = int(head_num_kv);
  p.d = int(head_dim);
  p.group = group;
  p.rows = plan.rows;
  p.direct = plan.direct;
  const auto pairs = [](const void *ptr, int64_t stride) {
    return reinterpret_cast<uintptr_t>(ptr) % 4 == 0 && stride % 2 == 0;
  };
  p.q_chunks = reinterpret_cast<uintptr_t>(q) % 16 == 0 &&
               q_stride % (dtype == FA_DTYPE_FP32 ? 4 : 8) == 0;
  p.y_pairs = pairs(y, y_stride);
  p.pre = int(pre_tokens < -1 ? -1 : pre_tokens > kMaxKeys ? kMaxKeys : pre_tokens);
  p.scale = float(scale);
  p.scale_log2 = float(scale * 1.4426950408889634);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == FA_DTYPE_FP32   ? launch_paged_decode_fp32(p, sms, cs)
                        : dtype == FA_DTYPE_FP16 ? launch_paged_decode_fp16(p, sms, cs)
                                                 : launch_paged_decode_bf16(p, sms, cs);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
