// gdnb_flash_64.cu -- attention of many query rows: the instances for head sizes up to 64.
#include "gdnb_flash.cuh"

namespace gdnb {
cudaError_t launch_flash_64(const FlashParams &p, cudaStream_t s) { return flash::launch_by_type<64>(p, s); }
cudaError_t flash_timeouts_64(unsigned *count) { return flash::wait_timeouts<64>(count); }
}  // namespace gdnb
