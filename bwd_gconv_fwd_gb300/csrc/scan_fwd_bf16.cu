// scan_fwd_bf16.cu -- instances of the selective scan's forward kernels for bf16 activations.
#include "scan_launch.cuh"

namespace gconv {

void scan_fwd_bf16(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    scan_fwd_start<__nv_bfloat16>(s, ends, a, st);
}

}  // namespace gconv
