// Group norm with an activation, channels last: each row's channels in G
// groups, each group normalised by itself, with a gate before or behind the
// norm (forward and gradients).
//
// A team of `tpg` neighbouring threads (a power of two) holds one row's
// group in registers: NV vectors of VEC channels a thread, read once.  The
// mean is taken first and the variance from the differences, both in
// registers, so there is no second pass over memory and no cancellation of
// E[p^2] against E[p]^2.  Memory bounds the kernels.
#include "ssm.cuh"

namespace mg {
namespace {

constexpr int kMaxTeam = 1024;

// Sum of v over each team; every thread of the team gets it.  buf: one float
// for each warp of the block.  All threads of the block call it.
__device__ __forceinline__ float team_sum(float v, int tpg, float *buf)
{
    const int in_warp = tpg < 32 ? tpg : 32;
    for (int o = in_warp / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (tpg <= 32) return v;
    const int warp = threadIdx.x >> 5, per = tpg >> 5, first = warp / per * per;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < per; ++i) v += buf[first + i];
    __syncthreads();
    return v;
}

__device__ __forceinline__ float act(float v, int silu) { return silu ? v * sigmoid_f(v) : v; }
// d act / dv
__device__ __forceinline__ float act_grad(float v, int silu)
{
    if (!silu) return 1.f;
    const float s = sigmoid_f(v);
    return s * fmaf(v, 1.f - s, 1.f);
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(NV == 16 ? kMaxTeam : 512)
norm_fwd_kernel(NormArgs p, int tpg, int64_t units)
{
    __shared__ float buf[32];
    const int teams = blockDim.x / tpg, lane = threadIdx.x & (tpg - 1);
    const int64_t u = int64_t(blockIdx.x) * teams + threadIdx.x / tpg;
    const bool live = u < units;
    const int64_t row = live ? u / p.G : 0, g = live ? u - row * p.G : 0, gs = p.D / p.G;
    const int64_t d0 = g * gs;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx + d0;
    const T *z = p.gate != MG_GATE_NONE ? static_cast<const T *>(p.z) + row * p.ldz + d0 : nullptr;
    Raw<T, VEC> xr[NV], zr[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t(i) * tpg + lane) * VEC;
        in[i] = live && c < gs;
        if (in[i]) {
            xr[i].load(x + c);
            if (z != nullptr) zr[i].load(z + c);
        }
    }
    const float inv = 1.f / float(gs);
    float f[NV][VEC], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                f[i][v] = p.gate == MG_GATE_FIRST ? xr[i][v] * act(zr[i][v], p.silu) : xr[i][v];
                sum += f[i][v];
            }
        }
    float mean = 0.f;
    if (!p.rms) mean = team_sum(sum, tpg, buf) * inv;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float e = f[i][v] - mean;
                sq = fmaf(e, e, sq);
            }
        }
    const float rstd = rsqrtf(fmaf(team_sum(sq, tpg, buf), inv, p.eps));
    if (!live) return;
    if (lane == 0 && p.stats != nullptr) {
        p.stats[2 * u] = mean;
        p.stats[2 * u + 1] = rstd;
    }
    T *y = static_cast<T *>(p.y) + row * p.D + d0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) {
            const int64_t c = (int64_t(i) * tpg + lane) * VEC;
            float w[VEC], b[VEC], o[VEC];
            load_vec<VEC>(p.w + d0 + c, w);
            if (p.bias != nullptr) load_vec<VEC>(p.bias + d0 + c, b);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                o[v] = (f[i][v] - mean) * rstd * w[v];
                if (p.bias != nullptr) o[v] += b[v];
                if (p.gate == MG_GATE_AFTER) o[v] *= act(zr[i][v], p.silu);
                if (p.gate == MG_GATE_NONE) o[v] = act(o[v], p.silu);
            }
            store_out<VEC>(y + c, o);
        }
}

// Gradients.  With n = (p - mean) rstd and dn = do w, over a group
//   dp = rstd (dn - mean(dn) - n mean(dn n))    (rms: without mean(dn))
// and the gate's chain rule around it.  A team keeps its group and walks over
// rows, so that a thread's channels stay the same and dw, dbias are summed in
// registers; the teams' sums are added in order by sum_parts_kernel.
template <typename T, int VEC, int NV, mg_gate GATE>
__global__ void __launch_bounds__(NV == 16 ? kMaxTeam : 512)
norm_bwd_kernel(NormArgs p, int tpg, int64_t row_teams, float *part)
{
    __shared__ float buf[32];
    const int teams = blockDim.x / tpg, lane = threadIdx.x & (tpg - 1);
    const int64_t t = int64_t(blockIdx.x) * teams + threadIdx.x / tpg;
    const int64_t g = t % p.G, slot = t / p.G, gs = p.D / p.G, d0 = g * gs;
    float dw[NV][VEC] = {}, db[NV][VEC] = {}, w[NV][VEC], b[NV][VEC];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t(i) * tpg + lane) * VEC;
        in[i] = slot < row_teams && c < gs;
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[i][v] = b[i][v] = 0.f;
        if (in[i]) {
            load_vec<VEC>(p.w + d0 + c, w[i]);
            if (GATE != MG_GATE_FIRST && p.bias != nullptr) load_vec<VEC>(p.bias + d0 + c, b[i]);
        }
    }
    const float inv = 1.f / float(gs);
    // the same count of rounds for every team: team_sum is for whole blocks
    const int64_t rounds = (p.M + row_teams - 1) / row_teams;
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t row = k * row_teams + slot;
        const bool live = slot < row_teams && row < p.M;
        const T *x = static_cast<const T *>(p.x) + row * p.ldx + d0;
        const T *z = static_cast<const T *>(p.z) + row * p.ldz + d0;
        const T *dy = static_cast<const T *>(p.dy) + row * p.lddy + d0;
        Raw<T, VEC> xr[NV], zr[NV], yr[NV];
        float mean = 0.f, rstd = 0.f;
        if (live) {
            mean = p.stats_in[2 * (row * p.G + g)];
            rstd = p.stats_in[2 * (row * p.G + g) + 1];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t(i) * tpg + lane) * VEC;
            if (live && in[i]) {
                xr[i].load(x + c);
                yr[i].load(dy + c);
                if (GATE != MG_GATE_NONE) zr[i].load(z + c);
            }
        }
        float n[NV][VEC], dn[NV][VEC], m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in[i]) {
                const int64_t c = (int64_t(i) * tpg + lane) * VEC;
                float dz[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float pv = GATE == MG_GATE_FIRST ? xr[i][v] * act(zr[i][v], p.silu) : xr[i][v];
                    n[i][v] = (pv - mean) * rstd;
                    float dov = yr[i][v];
                    if (GATE != MG_GATE_FIRST) {
                        const float o = fmaf(n[i][v], w[i][v], b[i][v]);
                        if (GATE == MG_GATE_AFTER) {
                            dz[v] = dov * o * act_grad(zr[i][v], p.silu);
                            dov *= act(zr[i][v], p.silu);
                        } else {
                            dov *= act_grad(o, p.silu);
                        }
                    }
                    dw[i][v] = fmaf(dov, n[i][v], dw[i][v]);
                    db[i][v] += dov;
                    dn[i][v] = dov * w[i][v];
                    m1 += dn[i][v];
                    m2 = fmaf(dn[i][v], n[i][v], m2);
                }
                if (GATE == MG_GATE_AFTER)
                    store_out<VEC>(static_cast<T *>(p.dz) + row * p.D + d0 + c, dz);
            }
        m1 = p.rms ? 0.f : team_sum(m1, tpg, buf) * inv;
        m2 = team_sum(m2, tpg, buf) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in[i]) {
                const int64_t c = (int64_t(i) * tpg + lane) * VEC;
                float dx[VEC], dz[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float dp = rstd * (dn[i][v] - m1 - n[i][v] * m2);
                    if (GATE == MG_GATE_FIRST) {
                        dx[v] = dp * act(zr[i][v], p.silu);
                        dz[v] = dp * xr[i][v] * act_grad(zr[i][v], p.silu);
                    } else {
                        dx[v] = dp;
                    }
                }
                store_out<VEC>(static_cast<T *>(p.dx) + row * p.D + d0 + c, dx);
                if (GATE == MG_GATE_FIRST)
                    store_out<VEC>(static_cast<T *>(p.dz) + row * p.D + d0 + c, dz);
            }
    }
    // part: row_teams rows of dw (D) and then of dbias (D)
    float *out = part + slot * 2 * p.D + d0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) {
            const int64_t c = (int64_t(i) * tpg + lane) * VEC;
            store_vec<VEC>(out + c, dw[i]);
            store_vec<VEC>(out + p.D + c, db[i]);
        }
}

// The team for groups of gs channels: the smallest power of two that covers
// it with NV vectors of vec channels a thread.
int team_for(int64_t gs, int vec, int nv)
{
    int t = 1;
    while (int64_t(t) * vec * nv < gs) t *= 2;
    return t;
}

constexpr int kNormBlock = 256;

// (vector width, vectors a thread) of a call.  Vectors are 16 bytes where
// the group's width and the rows allow, else one value.  More than one vector
// a thread is taken only where one would need a team of more than 512
// threads, beyond a group of 4096 bf16 channels: small teams keep more rows
// in flight.  8 x 512 float4 and 16 x 1024 single values hold the widest
// group, 16384 channels.
struct Shape {
    int vec, nv, tpg;
};
Shape shape_for(mg_dtype dt, int64_t gs, bool aligned)
{
    const int full = dt == MG_F32 ? 4 : 8;
    Shape c;
    c.vec = aligned && gs % full == 0 ? full : 1;
    for (int nv : {1, 2, 4, c.vec == 1 ? 16 : 8}) {
        c.nv = nv;
        c.tpg = team_for(gs, c.vec, nv);
        if (c.tpg <= 512 || (nv == 16 && c.tpg <= kMaxTeam)) return c;
    }
    c.tpg = 0;
    return c;
}

// Row teams of the backward: about 8 blocks of 256 threads for each SM, at
// most one for each row.
int64_t row_teams_for(int64_t M, int64_t G, int tpg)
{
    const int block = tpg > kNormBlock ? tpg : kNormBlock;
    const int64_t all = int64_t(152) * 8 * kNormBlock / block * (block / tpg);
    int64_t n = ceil_div(all, G);
    n = n < 1 ? 1 : n;
    return n < M ? n : M;
}

template <typename T, int VEC, int NV>
mg_status norm_fwd(const NormArgs &p, int tpg, cudaStream_t s)
{
    const int block = tpg > kNormBlock ? tpg : kNormBlock;
    const int64_t units = p.M * p.G;
    norm_fwd_kernel<T, VEC, NV><<<unsigned(ceil_div(units, block / tpg)), block, 0, s>>>(p, tpg, units);
    return launched("mg_group_norm_fwd");
}

template <typename T, int VEC, int NV>
mg_status norm_bwd(const NormArgs &p, int tpg, cudaStream_t s)
{
    const int block = tpg > kNormBlock ? tpg : kNormBlock;
    const int64_t rt = row_teams_for(p.M, p.G, tpg);
    const unsigned grid = unsigned(ceil_div(rt * p.G, block / tpg));
    float *part = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    switch (p.gate) {
    case MG_GATE_NONE:
        norm_bwd_kernel<T, VEC, NV, MG_GATE_NONE><<<grid, block, 0, s>>>(p, tpg, rt, part);
        break;
    case MG_GATE_AFTER:
        norm_bwd_kernel<T, VEC, NV, MG_GATE_AFTER><<<grid, block, 0, s>>>(p, tpg, rt, part);
        break;
    default:
        norm_bwd_kernel<T, VEC, NV, MG_GATE_FIRST><<<grid, block, 0, s>>>(p, tpg, rt, part);
    }
    MG_TRY(launched("mg_group_norm_bwd"));
    MG_TRY(launch_sum_parts(part, rt, 2 * p.D, p.D, p.dw, s));
    if (p.dbias != nullptr) return launch_sum_parts(part + p.D, rt, 2 * p.D, p.D, p.dbias, s);
    return MG_OK;
}

// Calls F<T, VEC, NV> for the call's shape.
#define MG_NORM_NV(F, T, VEC)                      \
    switch (c.nv) {                                \
    case 1: return F<T, VEC, 1>(p, c.tpg, s);      \
    case 2: return F<T, VEC, 2>(p, c.tpg, s);      \
    case 4: return F<T, VEC, 4>(p, c.tpg, s);      \
    }
#define MG_NORM(F)                                                                       \
    const int vec = dt == MG_F32 ? 4 : 8;                                                \
    const bool al = p.D % vec == 0 && p.ldx % vec == 0 &&                                \
                    (p.z == nullptr || p.ldz % vec == 0) &&                              \
                    (p.dy == nullptr || p.lddy % vec == 0);                              \
    const Shape c = shape_for(dt, p.D / p.G, al);                                        \
    if (c.tpg == 0)                                                                      \
        return fail(MG_ERR_UNSUPPORTED, "group of %lld channels too wide",               \
                    (long long)(p.D / p.G));                                             \
    if (dt == MG_F32) {                                                                  \
        if (c.vec == 4) {                                                                \
            MG_NORM_NV(F, float, 4)                                                      \
            return F<float, 4, 8>(p, c.tpg, s);                                          \
        }                                                                                \
        MG_NORM_NV(F, float, 1)                                                          \
        return F<float, 1, 16>(p, c.tpg, s);                                             \
    }                                                                                    \
    if (c.vec == 8) {                                                                    \
        MG_NORM_NV(F, bf16_t, 8)                                                         \
        return fail(MG_ERR_UNSUPPORTED, "group too wide");                               \
    }                                                                                    \
    MG_NORM_NV(F, bf16_t, 1)                                                             \
    return F<bf16_t, 1, 16>(p, c.tpg, s);

}  // namespace

size_t norm_ws_bytes(int64_t M, int64_t D, int64_t G)
{
    // the largest over the shapes that the call's type and strides may give
    size_t need = 0;
    for (mg_dtype dt : {MG_F32, MG_BF16})
        for (bool al : {false, true}) {
            const Shape c = shape_for(dt, D / G, al);
            if (c.tpg == 0) continue;
            const size_t n = size_t(row_teams_for(M, G, c.tpg)) * 2 * D * sizeof(float);
            need = n > need ? n : need;
        }
    return kControlBytes + need;
}

mg_status launch_norm_fwd(const NormArgs &p, mg_dtype dt, cudaStream_t s) { MG_NORM(norm_fwd) }
mg_status launch_norm_bwd(const NormArgs &p, mg_dtype dt, cudaStream_t s) { MG_NORM(norm_bwd) }

}  // namespace mg
