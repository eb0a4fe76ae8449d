// fa_paged_decode, fp16.

#include "paged_decode.cuh"

namespace fav {

cudaError_t launch_paged_decode_fp16(const DecodeParams &p, int sms, cudaStream_t s) {
  FAV_DECODE_BY_DIM(launch_tc, __half,);
}

}  // namespace fav
