// Root-mean-square norm behind a residual's addition, with the output in the
// activations' type or in e4m3 with scales, and its gradients.
//
//   r = x + res (rounded once: what the layers behind see),  rstd = (mean r^2 + eps)^(-1/2)
//   y = r rstd w;  per block of channels scale = max|y| / 448, q = y / scale
//   dn = dy w, n = r rstd:  dx = rstd (dn - n mean(dn n)) + dr,  dw = sum over rows of dy n
//
// Memory bounds all of them: each input is read once and each output written
// once.  A team (a warp, or a whole block for wide rows) holds a row in
// registers, so that the sum of squares, the largest |y| and the outputs come
// from one read.  Sums are float32, first over a thread's values, then over the
// team in a fixed order.
#include "block.cuh"

namespace mg {
namespace {

constexpr int kSMs = 152;

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Add {
    static __device__ __forceinline__ float op(float a, float b) { return a + b; }
};
struct MaxNan {
    static __device__ __forceinline__ float op(float a, float b) { return max_nan(a, b); }
};

// v over the team, for every thread of it.  buf: a float for each warp, not the
// one of the call before.
template <bool WARP, typename R>
__device__ __forceinline__ float over_team(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = R::op(v, __shfl_xor_sync(~0u, v, o));
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = buf[0];
        for (int i = 1; i < int(blockDim.x >> 5); ++i) v = R::op(v, buf[i]);
    }
    return v;
}

// VEC values from p, in loads of LV (VEC, or 1 for rows of any alignment).
template <typename T, int VEC, int LV>
struct Held {
    Raw<T, LV> w[VEC / LV];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < VEC / LV; ++i) w[i].load(p + i * LV);
    }
    __device__ __forceinline__ float operator[](int i) const { return w[i / LV][i % LV]; }
};

__device__ __forceinline__ float rounded(float v, const float *) { return v; }
__device__ __forceinline__ float rounded(float v, const bf16_t *)
{
    return __bfloat162float(__float2bfloat16_rn(v));
}

__device__ __forceinline__ unsigned e4m3x2(float lo, float hi)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// What the forward writes in place of y: nothing else, or 8 bits with a scale
// for each block of channels or for the whole row.
enum Quant { kNone, kBlocks, kRow };

// One row for a team: threads t of `threads` hold vectors t, t + threads, ...
// of VEC channels, NV at most.
template <typename T, int VEC, int LV, int NV, bool WARP, Quant Q>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rms_fwd_kernel(const RmsArgs p)
{
    __shared__ float sums[32], most[32];
    const int64_t row = WARP ? int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.M) return;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
    const int vecs = int(p.D / VEC);
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.res != nullptr ? static_cast<const T *>(p.res) + row * p.ldres : nullptr;
    Held<T, VEC, LV> hx[NV], hr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
        if (j < vecs) hx[i].load(x + j * VEC);
    }
    if (res != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if (j < vecs) hr[i].load(res + j * VEC);
        }
    }
    float f[NV][VEC], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i][e] = 0.f;
        if (j >= vecs) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            f[i][e] = hx[i][e];
            if (res != nullptr) f[i][e] = rounded(f[i][e] + hr[i][e], x);
            ss = fmaf(f[i][e], f[i][e], ss);
        }
        if (p.r != nullptr) store_vec<VEC>(static_cast<T *>(p.r) + row * p.D + int64_t(j) * VEC, f[i]);
    }
    ss = over_team<WARP, Add>(ss, sums);
    const float rstd = rsqrtf(ss / float(p.D) + p.eps);
    if (p.rstd != nullptr && t == 0) p.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
        if (Q == kNone && j >= vecs) continue;
        float w[VEC] = {};
        if (j < vecs) load_vec<VEC>(p.w + j * VEC, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i][e] *= rstd * w[e];
        if constexpr (Q == kNone) store_vec<VEC>(static_cast<T *>(p.y) + row * p.D + int64_t(j) * VEC, f[i]);
        if constexpr (Q == kRow) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) top = max_nan(top, fabsf(f[i][e]));
        }
    }
    if constexpr (Q != kNone) {
        constexpr float kLeast = 1e-30f, kMost = 448.f;
        float scale = 0.f;
        if constexpr (Q == kRow) {
            scale = max_nan(over_team<WARP, MaxNan>(top, most), kLeast) / kMost;
            if (t == 0) p.scale[row] = scale;
        }
        const int lanes = int(p.block) / VEC;   // kBlocks: 4 to 32 lanes of one warp share a block
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if constexpr (Q == kBlocks) {
                top = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) top = max_nan(top, fabsf(f[i][e]));
                for (int o = lanes / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
                scale = max_nan(top, kLeast) / kMost;
                if (j < vecs && j % lanes == 0) p.scale[row * (p.D / p.block) + j / lanes] = scale;
            }
            if (j >= vecs) continue;
            // y times 1 / scale: off y / scale by 2^-23 at most, before a rounding of 2^-4
            const float inv = 1.f / scale;
            unsigned char *q = static_cast<unsigned char *>(p.q) + row * p.D + int64_t(j) * VEC;
            if constexpr (VEC == 8) {
                unsigned w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[h] = e4m3x2(f[i][4 * h] * inv, f[i][4 * h + 1] * inv) |
                           e4m3x2(f[i][4 * h + 2] * inv, f[i][4 * h + 3] * inv) << 16;
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
            } else if constexpr (VEC == 2) {
                *reinterpret_cast<unsigned short *>(q) = (unsigned short)e4m3x2(f[i][0] * inv, f[i][1] * inv);
            } else {
                *q = (unsigned char)e4m3x2(f[i][0] * inv, 0.f);
            }
        }
    }
}

// Gradients: teams walk over rows, the next row's values loaded before the
// barrier of the one at hand, and keep their channels' sums for dw; a block
// leaves one row of sums.
template <typename T, int VEC, int NV, bool WARP, int MOST>
__global__ void __launch_bounds__(MOST) rms_bwd_kernel(const RmsArgs p, float *part)
{
    __shared__ float sums[2][32];
    const int warps = blockDim.x >> 5;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
    const int vecs = int(p.D / VEC);
    const int64_t teams = WARP ? int64_t(gridDim.x) * warps : gridDim.x;
    int64_t row = WARP ? int64_t(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = 0.f;
        if (j < vecs) load_vec<VEC>(p.w + j * VEC, w[i]);
    }
    Raw<T, VEC> a[NV], b[NV], c[NV];
    float rstd = 0.f;
    auto fetch = [&](int64_t r) {
        if (r >= p.M) return;
        rstd = __ldg(p.rstd_in + r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if (j >= vecs) continue;
            a[i].load(static_cast<const T *>(p.dy) + r * p.lddy + j * VEC);
            b[i].load(static_cast<const T *>(p.x) + r * p.ldx + j * VEC);
            if (p.dr != nullptr) c[i].load(static_cast<const T *>(p.dr) + r * p.lddr + j * VEC);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) a[i].fill(0.f), b[i].fill(0.f), c[i].fill(0.f);
    fetch(row);
    int turn = 0;
    for (; row < p.M; row += teams, turn ^= 1) {
        Raw<T, VEC> dy[NV], x[NV], dr[NV];
        const float rs = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) dy[i] = a[i], x[i] = b[i], dr[i] = c[i];
        fetch(row + teams);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) dot = fmaf(dy[i][e] * w[i][e], x[i][e] * rs, dot);
        dot = over_team<WARP, Add>(dot, sums[turn]) / float(p.D);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if (j >= vecs) continue;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float n = x[i][e] * rs;
                dw[i][e] = fmaf(dy[i][e], n, dw[i][e]);
                o[e] = fmaf(rs, fmaf(-n, dot, dy[i][e] * w[i][e]), dr[i][e]);
            }
            store_vec<VEC>(static_cast<T *>(p.dx) + row * p.D + int64_t(j) * VEC, o);
        }
    }
    float *mine = part + int64_t(blockIdx.x) * p.D;
    if constexpr (!WARP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if (j < vecs) store_vec<VEC>(mine + int64_t(j) * VEC, dw[i]);
        }
    } else {
        extern __shared__ float all[];
        for (int turn_of = 0; turn_of < warps; ++turn_of) {
            if (int(threadIdx.x >> 5) == turn_of) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int j = i * threads + t;
                    if (j >= vecs) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        all[j * VEC + e] = turn_of == 0 ? dw[i][e] : all[j * VEC + e] + dw[i][e];
                }
            }
            __syncthreads();
        }
        for (int j = threadIdx.x; j < p.D; j += blockDim.x) mine[j] = all[j];
    }
}

// How a launch holds rows: vectors of vec channels, nv of them a thread, and
// a block of `threads` a row (0: a warp a row, 8 of them in a block).
struct Shape {
    int vec, nv, threads;
};

int vec_for(mg_dtype dt, int64_t D, std::initializer_list<int64_t> lds)
{
    int64_t all = D;
    for (int64_t ld : lds) all |= ld;
    if (all % 8 == 0) return 8;
    return dt == MG_BF16 && all % 2 == 0 ? 2 : 1;
}

// Up to 4 vectors a thread fit a warp's row; wider rows take a block of 2
// (vectors of 8), 4, 8 or 16 a thread, and as many threads as that leaves.
Shape shape_for(int vec, int64_t D)
{
    const int64_t n = D / vec;
    if (n <= 128) return {vec, n <= 32 ? 1 : n <= 64 ? 2 : 4, 0};
    const int nv = vec == 8 ? 2 : n <= 1024 ? 4 : n <= 4096 ? 8 : 16;
    return {vec, nv, int(align_up(size_t(ceil_div(n, nv)), 32))};
}

int64_t bwd_blocks(int64_t M, const Shape &c)
{
    const int64_t most = c.threads == 0 ? ceil_div(M, 8) : M;
    const int64_t resident = kSMs * (c.threads == 0 ? 3 : c.threads <= 128 ? 5 : c.threads <= 256 ? 3 : c.threads <= 512 ? 2 : 1);
    return most < resident ? most : resident;
}

template <typename T, int VEC, int LV, int NV, bool WARP, Quant Q>
mg_status fwd(const RmsArgs &p, const Shape &c, cudaStream_t s)
{
    const int64_t blocks = WARP ? ceil_div(p.M, 8) : p.M;
    MG_TRY(check_grids("mg_rms_norm", {blocks}));
    rms_fwd_kernel<T, VEC, LV, NV, WARP, Q><<<unsigned(blocks), WARP ? 256 : c.threads, 0, s>>>(p);
    return launched("mg_rms_norm");
}

template <typename T, int VEC, int NV, bool WARP, int MOST>
mg_status bwd_most(const RmsArgs &p, const Shape &c, cudaStream_t s)
{
    float *part = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    const int64_t blocks = bwd_blocks(p.M, c);
    rms_bwd_kernel<T, VEC, NV, WARP, MOST>
        <<<unsigned(blocks), WARP ? 256 : c.threads, WARP ? size_t(p.D) * 4 : 0, s>>>(p, part);
    MG_TRY(launched("mg_rms_norm_bwd"));
    return launch_sum_parts(part, blocks, {{p.dw, p.D}}, s);
}

// Registers for the threads that the block has.
template <typename T, int VEC, int NV, bool WARP>
mg_status bwd(const RmsArgs &p, const Shape &c, cudaStream_t s)
{
    if constexpr (!WARP) {
        if (c.threads > 512) return bwd_most<T, VEC, NV, WARP, 1024>(p, c, s);
        if (c.threads > 256) return bwd_most<T, VEC, NV, WARP, 512>(p, c, s);
    }
    return bwd_most<T, VEC, NV, WARP, 256>(p, c, s);
}

template <typename T, int VEC, int LV, Quant Q>
mg_status fwd_shape(const RmsArgs &p, cudaStream_t s)
{
    const Shape c = shape_for(VEC, p.D);
    if (c.threads == 0) {
        if (c.nv == 1) return fwd<T, VEC, LV, 1, true, Q>(p, c, s);
        if (c.nv == 2) return fwd<T, VEC, LV, 2, true, Q>(p, c, s);
        return fwd<T, VEC, LV, 4, true, Q>(p, c, s);
    }
    if constexpr (VEC == 8) {
        return fwd<T, VEC, LV, 2, false, Q>(p, c, s);
    } else {
        if (c.nv == 4) return fwd<T, VEC, LV, 4, false, Q>(p, c, s);
        if (c.nv == 8) return fwd<T, VEC, LV, 8, false, Q>(p, c, s);
        return fwd<T, VEC, LV, 16, false, Q>(p, c, s);
    }
}

template <typename T, int VEC>
mg_status bwd_shape(const RmsArgs &p, cudaStream_t s)
{
    const Shape c = shape_for(VEC, p.D);
    if (c.threads == 0) {
        if (c.nv == 1) return bwd<T, VEC, 1, true>(p, c, s);
        if (c.nv == 2) return bwd<T, VEC, 2, true>(p, c, s);
        return bwd<T, VEC, 4, true>(p, c, s);
    }
    if constexpr (VEC == 8) {
        return bwd<T, VEC, 2, false>(p, c, s);
    } else {
        if (c.nv == 4) return bwd<T, VEC, 4, false>(p, c, s);
        if (c.nv == 8) return bwd<T, VEC, 8, false>(p, c, s);
        return bwd<T, VEC, 16, false>(p, c, s);
    }
}

// Rows of whole vectors of 8 (of 2 in bf16), else single values; a scale for
// each block needs vectors of 8, which are then loaded value by value where
// the input's rows are not aligned.
template <typename T, Quant Q>
mg_status fwd_any(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    const int vec = vec_for(dt, p.D, {p.ldx, p.res != nullptr ? p.ldres : 0});
    if constexpr (Q == kBlocks) {
        if (vec != 8) return fwd_shape<T, 8, 1, Q>(p, s);
    }
    if (vec == 8) return fwd_shape<T, 8, 8, Q>(p, s);
    if constexpr (Q != kBlocks && sizeof(T) == 2) {
        if (vec == 2) return fwd_shape<T, 2, 2, Q>(p, s);
    }
    if constexpr (Q != kBlocks) return fwd_shape<T, 1, 1, Q>(p, s);
    return MG_OK;
}

template <typename T>
mg_status bwd_any(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    const int vec = vec_for(dt, p.D, {p.ldx, p.lddy, p.dr != nullptr ? p.lddr : 0});
    if (vec == 8) return bwd_shape<T, 8>(p, s);
    if constexpr (sizeof(T) == 2) {
        if (vec == 2) return bwd_shape<T, 2>(p, s);
    }
    return bwd_shape<T, 1>(p, s);
}

}  // namespace

size_t rms_ws_bytes(int64_t M, int64_t D)
{
    int64_t blocks = 0;   // the most over the vectors that types and strides may give
    for (int vec : {8, 2, 1}) {
        if (D % vec != 0) continue;
        const int64_t n = bwd_blocks(M, shape_for(vec, D));
        blocks = n > blocks ? n : blocks;
    }
    return kControlBytes + size_t(blocks) * D * sizeof(float);
}

mg_status launch_rms_fwd(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    return dt == MG_F32 ? fwd_any<float, kNone>(p, dt, s) : fwd_any<bf16_t, kNone>(p, dt, s);
}

mg_status launch_rms_quant(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    if (p.block == p.D || p.block == 0)
        return dt == MG_F32 ? fwd_any<float, kRow>(p, dt, s) : fwd_any<bf16_t, kRow>(p, dt, s);
    return dt == MG_F32 ? fwd_any<float, kBlocks>(p, dt, s) : fwd_any<bf16_t, kBlocks>(p, dt, s);
}

mg_status launch_rms_bwd(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    return dt == MG_F32 ? bwd_any<float>(p, dt, s) : bwd_any<bf16_t>(p, dt, s);
}

}  // namespace mg
