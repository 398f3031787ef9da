// ssu_scan_prefill_f32.cu -- instances of the scan over prompts for x, dt, z, B and C in fp32.
#include "ssu_scan_prefill.cuh"

namespace ssu {

int launch_scan_prefill_f32(const ScanArgs &a, cudaStream_t s) { return launch_dt<SSU_F32>(a, s); }

}  // namespace ssu
