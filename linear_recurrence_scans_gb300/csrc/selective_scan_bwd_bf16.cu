// The selective scan's gradients for bf16 activations.
#include "selective_scan_bwd.cuh"

namespace mg {

mg_status ssm_bwd_bf16(const SsmArgs &p, bool wide, cudaStream_t s)
{
    return wide ? bwd_vec<bf16_t, 8>(p, s) : bwd_vec<bf16_t, 1>(p, s);
}

}  // namespace mg
