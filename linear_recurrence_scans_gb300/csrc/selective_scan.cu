// Selective scan: the recurrence with N states a channel whose decay, input
// and output weights depend on the token,
//   h_r[d,n] = a_r h_{r-1}[d,n] + u_r B_r[n],  a_r = exp(delta_r A[d,n]),
//   u_r = delta_r x_r,  y_r[d] = sum_n C_r[n] h_r[d,n] + Dskip x_r,
// its gradients, and its form for single tokens.
//
// Four states of one channel are a thread's; L = ceil(N/4) lanes, rounded up
// to a power of two, share the channel, and sums over states are shuffles
// among them.  States past N have A = B = C = 0.
#include "ssm.cuh"

namespace mg {
namespace {

constexpr int kS = 4;         // states of a thread
constexpr int kSeg = 16;      // rows between two saved states
constexpr int kThreads = 128;

// delta from the raw step size, and d delta / d raw.
__device__ __forceinline__ float step_size(float raw, int softplus, float &slope)
{
    if (softplus) return softplus_f(raw, slope);
    slope = 1.f;
    return raw;
}

template <int L>
__device__ __forceinline__ float lane_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Four values of a row of B or C (zero past N).
template <typename T>
__device__ __forceinline__ void load_states(const T *p, int n0, int N, float (&o)[kS])
{
#pragma unroll
    for (int i = 0; i < kS; ++i) o[i] = n0 + i < N ? load1(p + n0 + i) : 0.f;
}

// A block's channels: a tile of one group.
struct Tile {
    int64_t tiles;    // tiles of a group
    int64_t width;    // channels of a group
};

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) ssm_fwd_kernel(SsmArgs p, Seqs q, Tile tl)
{
    constexpr int kCh = kThreads / L;
    const int64_t all_tiles = tl.tiles * p.G;
    const int64_t tile = blockIdx.x % all_tiles;
    const int s = int(blockIdx.x / all_tiles);
    if (blockIdx.x == 0) check_cu(q, error_word(p.ws), threadIdx.x, kThreads);
    const int g = int(tile / tl.tiles);
    const int64_t c = (tile % tl.tiles) * kCh + threadIdx.x / L;
    const bool live = c < tl.width;
    const int64_t d = g * tl.width + (live ? c : 0);
    const int sl = threadIdx.x % L, n0 = sl * kS;
    long long lo = q.begin(s), hi = q.begin(s + 1);
    lo = lo < 0 ? 0 : lo;
    hi = hi > q.rows ? q.rows : hi;
    float A2[kS], h[kS];
    load_states(p.A + d * p.N, n0, p.N, A2);
#pragma unroll
    for (int i = 0; i < kS; ++i) A2[i] *= kLog2eF;
    const int64_t state = (int64_t(s) * p.D + d) * p.N;
#pragma unroll
    for (int i = 0; i < kS; ++i) h[i] = 0.f;
    if (p.h0 != nullptr) load_states(p.h0 + state, n0, p.N, h);
    const float skip = p.Dskip != nullptr ? p.Dskip[d] : 0.f;
    const float bias = p.dt_bias != nullptr ? p.dt_bias[d] : 0.f;
    // dense batches save by their own rows, packed ones by packed rows
    const int64_t base = q.cu != nullptr ? 0 : lo, nseg = (p.T + kSeg - 1) / kSeg;
    const int64_t save0 = q.cu != nullptr ? 0 : int64_t(s) * nseg;
    for (int64_t r = lo; r < hi; ++r) {
        if (p.saved != nullptr && (r - base) % kSeg == 0 && live) {
            float *o = p.saved + ((save0 + (r - base) / kSeg) * p.D + d) * p.N;
#pragma unroll
            for (int i = 0; i < kS; ++i)
                if (n0 + i < p.N) o[n0 + i] = h[i];
        }
        const float x = load1(static_cast<const T *>(p.x) + r * p.ldx + d);
        float slope;
        const float delta = step_size(load1(static_cast<const T *>(p.raw) + r * p.ldraw + d) + bias,
                                      p.softplus, slope);
        const float u = delta * x;
        float Br[kS], Cr[kS], y = 0.f;
        load_states(static_cast<const T *>(p.Bm) + r * p.ldb + g * p.N, n0, p.N, Br);
        load_states(static_cast<const T *>(p.Cm) + r * p.ldc + g * p.N, n0, p.N, Cr);
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            h[i] = fmaf(ex2_sub(delta * A2[i]), h[i], u * Br[i]);
            y = fmaf(Cr[i], h[i], y);
        }
        y = lane_sum<L>(y);
        if (live && sl == 0) store1(static_cast<T *>(p.y) + r * p.D + d, fmaf(skip, x, y));
    }
    if (p.h_last != nullptr && live) {
#pragma unroll
        for (int i = 0; i < kS; ++i)
            if (n0 + i < p.N) p.h_last[state + n0 + i] = h[i];
    }
}

// Gradients of one sequence and tile, from its last saved segment to its
// first: the segment's states are computed again into shared memory, then the
// adjoint g walks back over them.  Parts of dB and dC (one for each tile of a
// group) and of dA, dDskip, ddt_bias (one for each sequence) are added by
// the kernels below.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) ssm_bwd_kernel(SsmArgs p, Seqs q, Tile tl, float *partB,
                                                           float *partA, float *partD)
{
    constexpr int kCh = kThreads / L;
    __shared__ float4 hist[kSeg][kThreads];      // a_r h_{r-1}
    __shared__ float red[2][4][L * kS];          // a row's dB and dC, by warp
    const int64_t all_tiles = tl.tiles * p.G;
    const int64_t tile = blockIdx.x % all_tiles;
    const int s = int(blockIdx.x / all_tiles);
    if (blockIdx.x == 0) check_cu(q, error_word(p.ws), threadIdx.x, kThreads);
    const int g = int(tile / tl.tiles);
    const int64_t c = (tile % tl.tiles) * kCh + threadIdx.x / L;
    const bool live = c < tl.width;
    const int64_t d = g * tl.width + (live ? c : 0);
    const int sl = threadIdx.x % L, n0 = sl * kS;
    long long lo = q.begin(s), hi = q.begin(s + 1);
    lo = lo < 0 ? 0 : lo;
    hi = hi > q.rows ? q.rows : hi;
    float A[kS], ag[kS] = {}, dA[kS] = {}, dD = 0.f, dbias = 0.f;
    load_states(p.A + d * p.N, n0, p.N, A);
    const int64_t state = (int64_t(s) * p.D + d) * p.N;
    if (p.dh_last != nullptr) load_states(p.dh_last + state, n0, p.N, ag);
    const float skip = p.Dskip != nullptr ? p.Dskip[d] : 0.f;
    const float bias = p.dt_bias != nullptr ? p.dt_bias[d] : 0.f;
    const int64_t base = q.cu != nullptr ? 0 : lo, nseg = (p.T + kSeg - 1) / kSeg;
    const int64_t save0 = q.cu != nullptr ? 0 : int64_t(s) * nseg;
    const T *x = static_cast<const T *>(p.x), *raw = static_cast<const T *>(p.raw);
    const T *dy = static_cast<const T *>(p.dy);
    const int64_t GN = int64_t(p.G) * p.N;
    for (int64_t k = hi > lo ? (hi - 1 - base) / kSeg : -1; k >= 0; --k) {
        const int64_t s0 = base + k * kSeg > lo ? base + k * kSeg : lo;
        const int64_t s1 = base + (k + 1) * kSeg < hi ? base + (k + 1) * kSeg : hi;
        if (s1 <= lo) break;
        float h[kS] = {};
        if (s0 == lo) {
            if (p.h0 != nullptr) load_states(p.h0 + state, n0, p.N, h);
        } else {
            load_states(p.saved_in + ((save0 + k) * p.D + d) * p.N, n0, p.N, h);
        }
        for (int64_t r = s0; r < s1; ++r) {
            float slope, Br[kS];
            const float delta = step_size(load1(raw + r * p.ldraw + d) + bias, p.softplus, slope);
            const float u = delta * load1(x + r * p.ldx + d);
            load_states(static_cast<const T *>(p.Bm) + r * p.ldb + g * p.N, n0, p.N, Br);
            float ah[kS];
#pragma unroll
            for (int i = 0; i < kS; ++i) {
                ah[i] = ex2_sub(delta * (A[i] * kLog2eF)) * h[i];
                h[i] = fmaf(u, Br[i], ah[i]);
            }
            hist[r - s0][threadIdx.x] = make_float4(ah[0], ah[1], ah[2], ah[3]);
        }
        for (int64_t r = s1 - 1; r >= s0; --r) {
            float slope, Br[kS], Cr[kS];
            const float delta = step_size(load1(raw + r * p.ldraw + d) + bias, p.softplus, slope);
            const float xv = load1(x + r * p.ldx + d), u = delta * xv;
            const float dyv = live ? load1(dy + r * p.lddy + d) : 0.f;
            load_states(static_cast<const T *>(p.Bm) + r * p.ldb + g * p.N, n0, p.N, Br);
            load_states(static_cast<const T *>(p.Cm) + r * p.ldc + g * p.N, n0, p.N, Cr);
            const float4 a4 = hist[r - s0][threadIdx.x];
            const float ah[kS] = {a4.x, a4.y, a4.z, a4.w};
            float s1v = 0.f, s2v = 0.f, dB[kS], dC[kS];
#pragma unroll
            for (int i = 0; i < kS; ++i) {
                const float gi = fmaf(Cr[i], dyv, ag[i]);
                dC[i] = live ? dyv * fmaf(u, Br[i], ah[i]) : 0.f;
                dB[i] = live ? gi * u : 0.f;
                s1v = fmaf(gi, Br[i], s1v);
                const float w = gi * ah[i];
                s2v = fmaf(w, A[i], s2v);
                dA[i] = fmaf(w, delta, dA[i]);
                ag[i] = ex2_sub(delta * (A[i] * kLog2eF)) * gi;
            }
            s1v = lane_sum<L>(s1v);
            s2v = lane_sum<L>(s2v);
            const float draw = fmaf(xv, s1v, s2v) * slope;
            if (live && sl == 0) {
                store1(static_cast<T *>(p.dx) + r * p.D + d, fmaf(delta, s1v, skip * dyv));
                store1(static_cast<T *>(p.draw) + r * p.D + d, draw);
                dbias += draw;
                dD = fmaf(dyv, xv, dD);
            }
#pragma unroll
            for (int i = 0; i < kS; ++i)
#pragma unroll
                for (int o = L; o < 32; o <<= 1) {
                    dB[i] += __shfl_xor_sync(~0u, dB[i], o);
                    dC[i] += __shfl_xor_sync(~0u, dC[i], o);
                }
            if ((threadIdx.x & 31) < L) {
#pragma unroll
                for (int i = 0; i < kS; ++i) {
                    red[0][threadIdx.x >> 5][n0 + i] = dB[i];
                    red[1][threadIdx.x >> 5][n0 + i] = dC[i];
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * L * kS; i += kThreads) {
                const int w = i / (L * kS), n = i % (L * kS);
                if (n < p.N)
                    partB[((tile % tl.tiles) * 2 + w) * q.rows * GN + r * GN + g * p.N + n] =
                        red[w][0][n] + red[w][1][n] + red[w][2][n] + red[w][3][n];
            }
            __syncthreads();
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < kS; ++i)
        if (n0 + i < p.N) {
            partA[state + n0 + i] = dA[i];
            if (p.dh0 != nullptr) p.dh0[state + n0 + i] = ag[i];
        }
    if (sl == 0) {
        partD[int64_t(s) * 2 * p.D + d] = dD;
        partD[int64_t(s) * 2 * p.D + p.D + d] = dbias;
    }
}

// dB and dC from the tiles' parts (tile-major, dB then dC), in order.
template <typename T>
__global__ void __launch_bounds__(256) sum_bc_kernel(const float *part, int64_t tiles, int64_t n,
                                                     T *dB, T *dC)
{
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float b = 0.f, c = 0.f;
    for (int64_t t = 0; t < tiles; ++t) {
        b += part[(2 * t) * n + i];
        c += part[(2 * t + 1) * n + i];
    }
    store1(dB + i, b);
    store1(dC + i, c);
}

// One token a row, the state updated in place.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(SsmStepArgs p)
{
    const int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = i < p.B * p.D;
    const int64_t b = live ? i / p.D : 0, d = live ? i - b * p.D : 0;
    const int sl = threadIdx.x % L, n0 = sl * kS;
    const int64_t slot = p.slots != nullptr ? __ldg(p.slots + b) : b;
    const bool on = live && slot >= 0 && slot < p.nslots;
    float y = 0.f, x = 0.f;
    if (on) {
        const int g = int(d / (p.D / p.G));
        x = load1(static_cast<const T *>(p.x) + b * p.ldx + d);
        float slope, A[kS], Br[kS], Cr[kS], h[kS];
        const float bias = p.dt_bias != nullptr ? p.dt_bias[d] : 0.f;
        const float delta = step_size(load1(static_cast<const T *>(p.raw) + b * p.ldraw + d) + bias,
                                      p.softplus, slope);
        load_states(p.A + d * p.N, n0, p.N, A);
        load_states(static_cast<const T *>(p.Bm) + b * p.ldb + g * p.N, n0, p.N, Br);
        load_states(static_cast<const T *>(p.Cm) + b * p.ldc + g * p.N, n0, p.N, Cr);
        float *st = p.state + (slot * p.D + d) * p.N;
        load_states(st, n0, p.N, h);
#pragma unroll
        for (int k = 0; k < kS; ++k) {
            h[k] = fmaf(ex2_sub(delta * (A[k] * kLog2eF)), h[k], delta * x * Br[k]);
            y = fmaf(Cr[k], h[k], y);
            if (n0 + k < p.N) st[n0 + k] = h[k];
        }
    }
    y = lane_sum<L>(y);
    if (live && sl == 0) {
        const float skip = on && p.Dskip != nullptr ? p.Dskip[d] : 0.f;
        store1(static_cast<T *>(p.y) + i, fmaf(skip, x, y));
    }
}

int lanes_for(int N)
{
    int L = 1;
    while (L * kS < N) L *= 2;
    return L;
}

Tile tile_for(int64_t D, int N, int G)
{
    Tile t;
    t.width = D / G;
    t.tiles = ceil_div(t.width, kThreads / lanes_for(N));
    return t;
}

template <typename T, int L>
mg_status fwd(const SsmArgs &p, cudaStream_t s)
{
    const Tile t = tile_for(p.D, p.N, p.G);
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    ssm_fwd_kernel<T, L><<<unsigned(t.tiles * p.G * p.nseq), kThreads, 0, s>>>(p, q, t);
    return launched("mg_selective_scan_fwd");
}

template <typename T, int L>
mg_status bwd(const SsmArgs &p, cudaStream_t s)
{
    const Tile t = tile_for(p.D, p.N, p.G);
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const int64_t n = q.rows * p.G * p.N, dn = p.D * p.N;
    float *partB = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    float *partA = partB + 2 * t.tiles * n;
    float *partD = partA + p.nseq * dn;
    ssm_bwd_kernel<T, L><<<unsigned(t.tiles * p.G * p.nseq), kThreads, 0, s>>>(p, q, t, partB, partA, partD);
    MG_TRY(launched("mg_selective_scan_bwd"));
    sum_bc_kernel<T><<<unsigned(ceil_div(n, 256)), 256, 0, s>>>(
        partB, t.tiles, n, static_cast<T *>(p.dBm), static_cast<T *>(p.dCm));
    MG_TRY(launched("mg_selective_scan_bwd"));
    MG_TRY(launch_sum_parts(partA, p.nseq, dn, dn, p.dA, s));
    if (p.dDskip != nullptr) MG_TRY(launch_sum_parts(partD, p.nseq, 2 * p.D, p.D, p.dDskip, s));
    if (p.ddt_bias != nullptr)
        MG_TRY(launch_sum_parts(partD + p.D, p.nseq, 2 * p.D, p.D, p.ddt_bias, s));
    return MG_OK;
}

template <typename T, int L>
mg_status step(const SsmStepArgs &p, cudaStream_t s)
{
    ssm_step_kernel<T, L><<<unsigned(ceil_div(p.B * p.D * L, kThreads)), kThreads, 0, s>>>(p);
    return launched("mg_selective_scan_step");
}

#define MG_SSM_L(F, T, p, s)             \
    switch (lanes_for((p).N)) {          \
    case 1: return F<T, 1>(p, s);        \
    case 2: return F<T, 2>(p, s);        \
    case 4: return F<T, 4>(p, s);        \
    case 8: return F<T, 8>(p, s);        \
    default: return F<T, 16>(p, s);      \
    }
#define MG_SSM(F, p, dt, s)                        \
    if (dt == MG_F32) { MG_SSM_L(F, float, p, s) } \
    MG_SSM_L(F, bf16_t, p, s)

}  // namespace

size_t ssm_fwd_ws_bytes(int64_t, int64_t, int64_t, int, int, int64_t) { return kControlBytes; }

size_t ssm_bwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t nseq)
{
    const Tile t = tile_for(D, N, G);
    return kControlBytes + sizeof(float) * (2 * t.tiles * B * T * G * N + nseq * (D * N + 2 * D));
}

size_t ssm_saved_bytes(int64_t B, int64_t T, int64_t D, int N)
{
    return size_t(B) * ceil_div(T, kSeg) * D * N * sizeof(float);
}
int ssm_saved_rows() { return kSeg; }

mg_status launch_ssm_fwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(fwd, p, dt, s) }
mg_status launch_ssm_bwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(bwd, p, dt, s) }
mg_status launch_ssm_step(const SsmStepArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(step, p, dt, s) }

}  // namespace mg
