// gdna_attn_f16.cu -- the tensor-core attention kernels over fp16 caches.
#include "gdna_attn_tc.cuh"

namespace gdna {
template cudaError_t launch_attn_tc<GDNA_F16>(const AttnParams &, cudaStream_t);
template cudaError_t attn_wait_timeouts<GDNA_F16>(unsigned *);
}
