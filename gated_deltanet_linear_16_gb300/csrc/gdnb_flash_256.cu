// gdnb_flash_256.cu -- attention of many query rows: the instances for head sizes up to 256.
#include "gdnb_flash.cuh"

namespace gdnb {
cudaError_t launch_flash_256(const FlashParams &p, cudaStream_t s) { return flash::launch_by_type<256>(p, s); }
cudaError_t flash_timeouts_256(unsigned *count) { return flash::wait_timeouts<256>(count); }
}  // namespace gdnb
