// Declarations shared by the paged-cache entry points (paged_abi.cpp) and
// their kernels (paged_plan.cu, paged_write.cu, paged_decode.cuh).
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
cudaError_t launch_paged_decode_bf16(const DecodeParams &p, int sms, cudaStream_t s);
cudaError_t launch_paged_decode_fp16(const DecodeParams &p, int sms, cudaStream_t s);
cudaError_t launch_paged_decode_fp32(const DecodeParams &p, int sms, cudaStream_t s);

}  // namespace fav
