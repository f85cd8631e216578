// gdn_prefill.hip -- launches of the chunked gated delta rule, bf16 inputs (gfx950); the kernel
// is gdn_walk.h's.
#include "gdn_walk.h"

namespace kda {
namespace {

template <int DK, int NCB>
__global__ __launch_bounds__((GCfg<DK, NCB>::THREADS)) void gdn_prefill_kernel(const PArgs a, const GdnTable tab) {
    gdn_walk<DK, NCB, false>(a, tab, blockIdx.x);
}

template <int DK, int NCB>
hipError_t launch(const GdnPrefillArgs& p, const GdnTable& tab, hipStream_t st) {
    typedef GCfg<DK, NCB> C;
    hipError_t e = hipFuncSetAttribute((const void*)gdn_prefill_kernel<DK, NCB>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                       C::LDS_BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdn_prefill_kernel<DK, NCB>), dim3((unsigned)walk_blocks(p)), dim3(C::THREADS), C::LDS_BYTES, st,
                       walk_args(p), tab);
    return hipGetLastError();
}

template <int DK>
hipError_t launch_nv(const GdnPrefillArgs& p, const GdnTable& tab, hipStream_t st) {
    switch (p.nv) {
        case 16: return launch<DK, 1>(p, tab, st);
        case 32: return launch<DK, 2>(p, tab, st);
        case 64: return launch<DK, 4>(p, tab, st);
        case 128: return launch<DK, 8>(p, tab, st);
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gdn_chunked(const GdnPrefillArgs& p, const GdnTable& tab, hipStream_t st) {
    return p.d.dk == 128 ? launch_nv<128>(p, tab, st) : launch_nv<64>(p, tab, st);
}

}  // namespace kda
