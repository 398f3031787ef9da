// ssu_scan_prefill.cu -- the scan over prompts (ssu_scan_prefill.cuh): choice of the form, and
// its instances for inputs of any types.
#include "ssu_scan_prefill.cuh"

namespace ssu {
namespace {

// Whether a row of elements starts and steps on 16 bytes. With `first` (elements), so does
// every further block of that many.
bool rows16(const void *p, int dtype, int64_t ld, int64_t first = 0)
{
    const int e = esize(dtype);
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * e) % 16 == 0 && (first * e) % 16 == 0;
}

}  // namespace

int launch_scan_prefill(ScanArgs a, cudaStream_t s)
{
    if (!a.out)
        a.z = nullptr;
    // a CTA's channels start at a multiple of 8 within their group
    const int64_t per = a.G > 1 ? a.D / a.G : 0;
    const bool pairs = a.out && a.D % 2 == 0 && per % 2 == 0 &&
                       reinterpret_cast<uintptr_t>(a.out) % (2 * esize(a.x_dtype)) == 0;
    a.vec = (rows16(a.x, a.x_dtype, a.ldx, per) ? 1 : 0) |
            (rows16(a.dt, a.dt_dtype, a.lddt, per) ? 2 : 0) |
            (a.z && rows16(a.z, a.x_dtype, a.ldz, per) ? 4 : 0) | (pairs ? 8 : 0) |
            (rows16(a.B, a.bc_dtype, a.ldb, a.N) ? 16 : 0) |
            (a.out && rows16(a.C, a.bc_dtype, a.ldc, a.N) ? 32 : 0);
    // a type that all inputs share is compiled in: conversions and addresses by type at run
    // time cost as much as the scan's own arithmetic
    if (a.x_dtype == a.dt_dtype && a.x_dtype == a.bc_dtype) {
        if (a.x_dtype == SSU_BF16)
            return launch_scan_prefill_bf16(a, s);
        return a.x_dtype == SSU_F16 ? launch_scan_prefill_f16(a, s) : launch_scan_prefill_f32(a, s);
    }
    return launch_dt<-1>(a, s);
}

}  // namespace ssu
