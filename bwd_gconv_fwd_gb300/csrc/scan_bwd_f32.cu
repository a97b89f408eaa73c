// scan_bwd_f32.cu -- instances of the selective scan's gradient kernels for f32 activations.
#include "scan_launch.cuh"

namespace gconv {

void scan_bwd_f32(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    scan_bwd_start<float>(s, ends, a, st);
}

}  // namespace gconv
