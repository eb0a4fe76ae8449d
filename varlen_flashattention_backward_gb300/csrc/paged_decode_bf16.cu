// fa_paged_decode, bf16.

#include "paged_decode.cuh"

namespace fav {

cudaError_t launch_paged_decode_bf16(const DecodeParams &p, int sms, cudaStream_t s) {
  FAV_DECODE_BY_DIM(launch_tc, __nv_bfloat16,);
}

}  // namespace fav
