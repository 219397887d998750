// gdna_attn_bf16.cu -- the tensor-core attention kernels over bf16 caches.
#include "gdna_attn_tc.cuh"

namespace gdna {
template cudaError_t launch_attn_tc<GDNA_BF16>(const AttnParams &, cudaStream_t);
template cudaError_t attn_wait_timeouts<GDNA_BF16>(unsigned *);
}
