// ssu_scan_prefill_bf16.cu -- instances of the scan over prompts for x, dt, z, B and C in bfloat16.
#include "ssu_scan_prefill.cuh"

namespace ssu {

int launch_scan_prefill_bf16(const ScanArgs &a, cudaStream_t s) { return launch_dt<SSU_BF16>(a, s); }

}  // namespace ssu
