// gdnb_flash_128_bf16.cu -- attention of many query rows: the instances for head sizes up to 128, bf16 products.
#include "gdnb_flash.cuh"

namespace gdnb {
cudaError_t launch_flash_128_bf16(const FlashParams &p, cudaStream_t s) { return flash::launch_by_type<128, true>(p, s); }
cudaError_t flash_timeouts_128_bf16(unsigned *count) { return flash::wait_timeouts(count); }
}  // namespace gdnb
