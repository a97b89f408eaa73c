// scan_fwd_f32.cu -- instances of the selective scan's forward kernels for f32 activations.
#include "scan_launch.cuh"

namespace gconv {

void scan_fwd_f32(const ScanShape &s, bool ends, const ScanArgs &a, cudaStream_t st)
{
    scan_fwd_start<float>(s, ends, a, st);
}

}  // namespace gconv
