// Host side of the paged-cache entry points: argument checks, the decode
// workspace and the launches.  Nothing here allocates or throws.

#include <cfloat>
#include <cmath>

#include "internal.h"
#include "paged.h"

namespace fav {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxPageSize = 65536;
constexpr int64_t kMaxKeys = int64_t(1) << 30;
constexpr int64_t kMaxI32 = 2147483647;
constexpr int64_t kDefaultWaitNs = 2000000000;
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

// Whole numbers and statistics: aligned to their type (NULL is).
template <typename... Ptr>
bool misaligned(const Ptr *...ptr) {
  return (... || (reinterpret_cast<uintptr_t>(ptr) % sizeof(Ptr) != 0));
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

fa_status fa_paged_plan(const fa_paged_plan_args *args, fa_stream_t stream) {
  if (!args) return FA_ERR_NULLPTR;
  const auto &a = *args;
  if (!a.block_table || !a.seq_lens || !a.delta || !a.free_pages || !a.free_state ||
      !a.cu_tokens || !a.seq_lens_out || !a.free_state_out || (a.max_tokens > 0 && !a.slots))
    return FA_ERR_NULLPTR;
  const fa_status st =
      check_table(a.batch, a.num_pages, a.page_size, a.max_pages, a.table_stride);
  if (st != FA_OK) return st;
  if (a.max_tokens < 0 || a.max_tokens > kMaxI32) return FA_ERR_INVALID;
  if (misaligned(a.block_table, a.seq_lens, a.delta, a.free_pages, a.free_state, a.slots,
                 a.cu_tokens, a.seq_lens_out, a.free_state_out, a.error))
    return FA_ERR_INVALID;
  PlanParams p{};
  p.table = a.block_table;
  p.table_stride = a.table_stride;
  p.lens = a.seq_lens;
  p.delta = a.delta;
  p.ring = a.free_pages;
  p.state = a.free_state;
  p.slots = a.slots;
  p.cu = a.cu_tokens;
  p.lens_out = a.seq_lens_out;
  p.state_out = a.free_state_out;
  p.error = a.error;
  p.max_tokens = a.max_tokens;
  p.batch = int(a.batch);
  p.max_pages = int(a.max_pages);
  p.num_pages = int(a.num_pages);
  p.page_size = int(a.page_size);
  p.page_shift = log2_or_none(a.page_size);
  return launch_paged_plan(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                     : FA_ERR_CUDA;
}

fa_status fa_paged_write(const fa_paged_write_args *args, fa_stream_t stream) {
  if (!args) return FA_ERR_NULLPTR;
  const auto &a = *args;
  if (a.reserved != 0) return FA_ERR_INVALID;
  int64_t k_stride = a.k_stride;
  int64_t v_stride = a.v_stride;
  int64_t page_stride = a.page_stride;
  int64_t token_stride = a.token_stride;
  int64_t head_stride = a.head_stride;
  const fa_dtype dtype = static_cast<fa_dtype>(a.dtype);
  if (!a.k_pages || !a.v_pages || (a.tokens > 0 && (!a.k || !a.v || !a.slots)))
    return FA_ERR_NULLPTR;
  fa_status st = check_heads(a.head_num_kv, a.head_num_kv, a.head_dim, dtype);
  if (st != FA_OK) return st;
  st = check_table(1, a.num_pages, a.page_size, 1, 1);
  if (st != FA_OK) return st;
  st = check_cache(a.k_pages, a.v_pages, a.num_pages, a.page_size, a.head_num_kv, a.head_dim,
                   page_stride, token_stride, head_stride, dtype);
  if (st != FA_OK) return st;
  if (a.tokens < 0 || a.tokens > kMaxI32) return FA_ERR_INVALID;
  const int64_t row = a.head_num_kv * a.head_dim;
  if (bad_rows(k_stride, a.tokens, row) || bad_rows(v_stride, a.tokens, row))
    return FA_ERR_INVALID;
  if (!element_aligned(a.k, dtype) || !element_aligned(a.v, dtype) ||
      misaligned(a.slots, a.error))
    return FA_ERR_INVALID;
  if (a.tokens == 0) return FA_OK;
  WriteParams p{};
  p.k = a.k;
  p.v = a.v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = a.slots;
  p.kc = a.k_pages;
  p.vc = a.v_pages;
  p.n_slots = a.num_pages * a.page_size;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.error = a.error;
  p.tokens = int(a.tokens);
  p.page_size = int(a.page_size);
  p.page_shift = log2_or_none(a.page_size);
  p.n_kv = int(a.head_num_kv);
  p.d = int(a.head_dim);
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

fa_status fa_paged_decode(const fa_paged_decode_args *args, fa_stream_t stream) {
  return fa_paged_decode_ex(args, nullptr, stream);
}

fa_status fa_paged_decode_ex(const fa_paged_decode_args *args,
                             const fa_paged_decode_options *options, fa_stream_t stream) {
  if (!args) return FA_ERR_NULLPTR;
  const auto &a = *args;
  if (a.reserved != 0) return FA_ERR_INVALID;
  int64_t q_stride = a.q_stride;
  int64_t page_stride = a.page_stride;
  int64_t token_stride = a.token_stride;
  int64_t head_stride = a.head_stride;
  int64_t y_stride = a.y_stride;
  const fa_dtype dtype = static_cast<fa_dtype>(a.dtype);
  if (!a.q || !a.k_pages || !a.v_pages || !a.block_table || !a.seq_lens || !a.y ||
      (!a.softmax_max != !a.softmax_sum))
    return FA_ERR_NULLPTR;
  fa_status st = check_heads(a.head_num, a.head_num_kv, a.head_dim, dtype);
  if (st != FA_OK) return st;
  st = check_table(a.batch, a.num_pages, a.page_size, a.max_pages, a.table_stride);
  if (st != FA_OK) return st;
  st = check_cache(a.k_pages, a.v_pages, a.num_pages, a.page_size, a.head_num_kv, a.head_dim,
                   page_stride, token_stride, head_stride, dtype);
  if (st != FA_OK) return st;
  // The kernels hold it in 32 bits, where a larger one would make scores of 0 NaN.
  const double scale_log2 = a.scale * 1.4426950408889634;
  if (!(std::fabs(scale_log2) <= FLT_MAX)) return FA_ERR_INVALID;
  const int64_t row = a.head_num * a.head_dim;
  if (bad_rows(q_stride, a.batch, row) || bad_rows(y_stride, a.batch, row))
    return FA_ERR_INVALID;
  if (!element_aligned(a.q, dtype) || !element_aligned(a.y, dtype) ||
      misaligned(a.block_table, a.seq_lens, a.softmax_max, a.softmax_sum, a.error))
    return FA_ERR_INVALID;
  const int sms = sm_count();
  const int group = int(a.head_num / a.head_num_kv);
  const DecodePlan plan =
      decode_plan(dtype, int(a.batch), int(a.head_num_kv), group, int(a.head_dim),
                  most_keys(a.max_pages, a.page_size, a.pre_tokens), sms);
  const size_t bytes = decode_bytes(plan, sms, group, a.head_dim);
  if (bytes > 0 && !a.workspace) return FA_ERR_NULLPTR;
  if (reinterpret_cast<uintptr_t>(a.workspace) % 16 != 0) return FA_ERR_INVALID;
  if (a.workspace_bytes < bytes) return FA_ERR_WORKSPACE;

  DecodeParams p{};
  p.q = a.q;
  p.q_stride = q_stride;
  p.kc = a.k_pages;
  p.vc = a.v_pages;
  p.page_stride = page_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.table = a.block_table;
  p.table_stride = a.table_stride;
  p.lens = a.seq_lens;
  p.y = a.y;
  p.y_stride = y_stride;
  p.smax = a.softmax_max;
  p.ssum = a.softmax_sum;
  p.error = a.error;
  p.part = static_cast<float *>(a.workspace);
  p.slot_rows = group < plan.rows ? group : plan.rows;
  p.num_pages = int(a.num_pages);
  p.page_size = int(a.page_size);
  p.page_shift = log2_or_none(a.page_size);
  p.max_pages = int(a.max_pages);
  p.batch = int(a.batch);
  p.n = int(a.head_num);
  p.n_kv = int(a.head_num_kv);
  p.d = int(a.head_dim);
  p.group = group;
  p.rows = plan.rows;
  p.direct = plan.direct;
  const auto pairs = [](const void *ptr, int64_t stride) {
    return reinterpret_cast<uintptr_t>(ptr) % 4 == 0 && stride % 2 == 0;
  };
  p.q_chunks = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 &&
               q_stride % (dtype == FA_DTYPE_FP32 ? 4 : 8) == 0;
  p.y_pairs = pairs(a.y, y_stride);
  p.pre = int(a.pre_tokens < -1 ? -1 : a.pre_tokens > kMaxKeys ? kMaxKeys : a.pre_tokens);
  p.scale_log2 = float(scale_log2);
  p.wait_ns = options && options->wait_timeout_ns > 0 ? options->wait_timeout_ns : kDefaultWaitNs;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == FA_DTYPE_FP32   ? launch_paged_decode_fp32(p, sms, cs)
                        : dtype == FA_DTYPE_FP16 ? launch_paged_decode_fp16(p, sms, cs)
                                                 : launch_paged_decode_bf16(p, sms, cs);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
