// gdnb_flash_64_bf16.cu -- attention of many query rows: the instances for head sizes up to 64, bf16 products.
#include "gdnb_flash.cuh"

namespace gdnb {
cudaError_t launch_flash_64_bf16(const FlashParams &p, cudaStream_t s) { return flash::launch_by_type<64, true>(p, s); }
cudaError_t flash_timeouts_64_bf16(unsigned *count) { return flash::wait_timeouts(count); }
}  // namespace gdnb
