// gdnb_flash_128.cu -- attention of many query rows: the instances for head sizes up to 128.
#include "gdnb_flash.cuh"

namespace gdnb {
cudaError_t launch_flash_128(const FlashParams &p, cudaStream_t s) { return flash::launch_by_type<128>(p, s); }
cudaError_t flash_timeouts_128(unsigned *count) { return flash::wait_timeouts<128>(count); }
}  // namespace gdnb
