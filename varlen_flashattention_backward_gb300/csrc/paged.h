// Declarations shared by the paged-cache entry points (paged_abi.cpp) and
// their kernels (paged_plan.cu, paged_write.cu, paged_decode.cuh,
// paged_pages.cu, paged_copy.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_varlen.h"

namespace fav {

struct PlanParams {
  int32_t *table;
  int64_t table_stride;
  const int32_t *lens, *delta;
  int32_t *ring;
  const int64_t *state;
  int64_t *slots, *cu;
  int32_t *lens_out;
  int64_t *state_out;
  int32_t *error;
  int64_t max_tokens;
  int batch, max_pages, num_pages, page_size, page_shift;   // page_shift: log2 or -1
  int phases;   // set at launch
};

struct WriteParams {
  const void *k, *v;
  int64_t k_stride, v_stride;
  const int64_t *slots;
  void *kc, *vc;
  int64_t n_slots;
  int64_t page_stride, token_stride, head_stride;
  int32_t *error;
  int tokens, page_size, page_shift, n_kv, d;
};

struct DecodeParams {
  const void *q;
  int64_t q_stride;
  const void *kc, *vc;
  int64_t page_stride, token_stride, head_stride;
  const int32_t *table;
  int64_t table_stride;
  const int32_t *lens;
  void *y;
  int64_t y_stride;
  float *smax, *ssum;
  int32_t *error;
  float *part;        // partial results: two slots per range (see paged_decode.cuh)
  int slot_rows;      // query heads in a slot
  int num_pages, page_size, page_shift;   // page_shift: log2(page_size), or -1
  int max_pages, batch, n, n_kv, d, group;
  int y_pairs;            // rows of y start on 4-byte boundaries
  int q_chunks;           // rows of q start on 16-byte boundaries
  int pre;            // pre_tokens clamped to [-1, 2^30]
  int rows, direct;   // DecodePlan
  int ranges;         // teams of the main kernel
  int unit_shift;     // log2 of the blocks in a unit of work
  float scale_log2;
  long long wait_ns;  // bound on every in-kernel wait
};

struct ForkParams {
  int32_t *table;
  int64_t table_stride;
  const int32_t *lens, *source;
  int32_t *shares, *ring;
  const int64_t *state;
  int32_t *copy_from, *copy_to;
  int32_t *lens_out;
  int64_t *state_out;
  int32_t *error;
  int64_t *work;   // see paged_pages.cu
  int batch, max_pages, num_pages, page_size;
  int phases, chunk;   // set at launch
};

struct CompactParams {
  const int32_t *table;
  int64_t table_stride;
  const int32_t *lens, *shares, *ring;
  const int64_t *state;
  int32_t *table_out;
  int64_t table_out_stride;
  int32_t *shares_out, *ring_out;
  int64_t *state_out;
  int32_t *copy_from, *copy_to;
  int32_t *error;
  int64_t *work;   // see paged_pages.cu
  int batch, max_pages, num_pages, page_size, new_pages, max_copies;
  int phases, chunk;   // set at launch
};

struct CopyParams {
  void *kc, *vc;
  const int32_t *from, *to;
  int32_t *error;
  int64_t page_stride, outer_stride, inner_stride;   // in 16-byte pieces
  int copies, num_pages;
  unsigned page_v, row_v, head_v;   // pieces of a page, of an outer entry, of an inner one
};

struct ExtendParams {
  const void *q;
  int64_t q_stride;
  const void *kc, *vc;
  int64_t page_stride, token_stride, head_stride;
  const int32_t *table;
  int64_t table_stride;
  const int32_t *lens;
  const int64_t *cu;
  void *y;
  int64_t y_stride;
  float *smax, *ssum;
  int32_t *error;
  // Workspace (see paged_extend.cuh).
  void *records;
  float *parts;
  uint32_t *flags;
  int num_pages, page_size, page_shift;   // page_shift: log2(page_size), or -1
  int max_pages, batch, tokens, n, n_kv, d, group;
  int pre, next;         // clamped to [-2^30, 2^30 - 1]
  int q_chunks, y_chunks, stat_chunks;   // rows of q, y, the statistics start on 16-byte boundaries
  int sign;              // of the scale; the query rows are multiplied by it
  int least_span;        // shortest span of a CTA
  float scale_log2;      // |scale| log2(e), above 0 (1 where the scale is 0)
  float bias;            // log2 of a factor that the sums of weights hold
  long long wait_ns;     // bound on every in-kernel wait
};

constexpr int kExtendRecord = 64;   // bytes of a CTA's record
constexpr int kExtendBiasFp16 = 7, kExtendBiasBf16 = -8;   // (see paged_extend_tc.cuh)

// How an extend call is run, and its workspace.
struct ExtendPlan {
  int rows;              // packed rows in a block
  int ctas;
  int64_t most_blocks;   // of one key head, that the rows can make
  size_t parts, flags, bytes;   // offsets (the records come first), and the end
};
ExtendPlan extend_plan(fa_dtype dt, int64_t batch, int64_t tokens, int n, int n_kv, int d, int sms);

// Bytes of the two workspaces.
size_t fork_work_bytes(int64_t batch, int64_t num_pages);
size_t compact_work_bytes(int64_t num_pages);

// How a decode call is run.
struct DecodePlan {
  int rows;     // query heads of one key head that a warp takes at a time
  int teams;    // per CTA
  int direct;   // CTAs per segment (see paged_decode.cuh), or 0: ranges and a join
};
DecodePlan decode_plan(fa_dtype dt, int batch, int n_kv, int group, int d, int64_t max_keys,
                       int sms);
// Floats of one partial result in the workspace.
size_t decode_part_floats(int rows, int d);

cudaError_t launch_paged_plan(const PlanParams &p, cudaStream_t s);
cudaError_t launch_paged_write(const WriteParams &p, fa_dtype dt, cudaStream_t s);
cudaError_t launch_paged_extend_bf16(const ExtendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_paged_extend_fp16(const ExtendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_paged_extend_fp32(const ExtendParams &p, int ctas, cudaStream_t s);
cudaError_t launch_paged_fork(const ForkParams &p, cudaStream_t s);
cudaError_t launch_paged_compact(const CompactParams &p, cudaStream_t s);
cudaError_t launch_paged_copy(const CopyParams &p, cudaStream_t s);
cudaError_t launch_paged_decode_bf16(const DecodeParams &p, int sms, cudaStream_t s);
cudaError_t launch_paged_decode_fp16(const DecodeParams &p, int sms, cudaStream_t s);
cudaError_t launch_paged_decode_fp32(const DecodeParams &p, int sms, cudaStream_t s);

}  // namespace fav
