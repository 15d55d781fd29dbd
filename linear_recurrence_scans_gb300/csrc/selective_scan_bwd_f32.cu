// The selective scan's gradients for float32 activations.
#include "selective_scan_bwd.cuh"

namespace mg {

size_t ssm_bwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t)
{
    const Chunks ck = backward_chunks(B, T, D, N, G);
    return kControlBytes +
           sizeof(float) * (backward_tiles(D, N, G) * B * T * G * 2 * N + B * ck.n * D * (N + 2) + 4 +
                            B * (ck.n - 1) * (D * N + D));
}


mg_status ssm_bwd_f32(const SsmArgs &p, bool wide, cudaStream_t s)
{
    return wide ? bwd_vec<float, 4>(p, s) : bwd_vec<float, 1>(p, s);
}

}  // namespace mg
