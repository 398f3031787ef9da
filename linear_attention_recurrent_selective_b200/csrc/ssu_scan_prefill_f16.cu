// ssu_scan_prefill_f16.cu -- instances of the scan over prompts for x, dt, z, B and C in half precision.
#include "ssu_scan_prefill.cuh"

namespace ssu {

int launch_scan_prefill_f16(const ScanArgs &a, cudaStream_t s) { return launch_dt<SSU_F16>(a, s); }

}  // namespace ssu
