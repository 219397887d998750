// gdna_attn_e4m3.cu -- the tensor-core attention kernels over E4M3 caches.
#include "gdna_attn_tc.cuh"

namespace gdna {
template cudaError_t launch_attn_tc<GDNA_E4M3>(const AttnParams &, cudaStream_t);
template cudaError_t attn_wait_timeouts<GDNA_E4M3>(unsigned *);
}
