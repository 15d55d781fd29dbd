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
// team in a fixed order.  In bf16 with a residual: forward 32768 x 2048 80 us (6.7
// TB/s), with 8 bits and blocks of 128 at 32768 x 4096 164 us (5.8 TB/s, one vector
// of a row a thread instead of two 201), gradients of 32768 x 2048 89 us (6.0 TB/s).
#include <type_traits>

#include "block.cuh"
#include "flat_rows.h"
#include "umma.cuh"

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

// How rows lie.
enum Rows {
    kWhole,    // whole vectors of 8 on 16-byte boundaries
    kFlat,     // dense rows of any width: vectors on the boundaries of the flat array, of which a row's first and last hold fewer
    kLoose,    // whole vectors of 8, on no boundary: loaded value by value
    kSingle    // single values
};
template <Rows R>
constexpr int kVec = R == kSingle ? 1 : 8;
template <typename T>
constexpr int kWide = 16 / int(sizeof(T));   // values of 16 bytes

// The place of a row's first value between two such boundaries, for kFlat.
template <typename T, Rows R>
__device__ __forceinline__ int shift_of(int64_t row, int64_t D)
{
    return R == kFlat ? int((row * D) % kWide<T>) : 0;
}

// VEC values as loaded.
template <typename T, Rows R>
struct Held {
    static constexpr int LV = R == kSingle || R == kLoose ? 1 : kWide<T>;
    Raw<T, LV> w[kVec<R> / LV];
    // values i .. i + VEC - 1 of a row of D
    __device__ __forceinline__ void load(const T *row, int i, int D)
    {
#pragma unroll
        for (int c = 0; c < kVec<R> / LV; ++c) {
            const int at = i + c * LV;
            if (R != kFlat || (at >= 0 && at + LV <= D)) {
                w[c].load(row + at);
            } else {
                edge(w[c], row, at, D);
            }
        }
    }
    // The same of a row that lies in shared memory from its 16-byte boundary on,
    // `shift` values before it; `rest`: the row itself, for the piece that the copy
    // left out, from value `stop` on.
    __device__ __forceinline__ void take(const T *copy, int shift, int i, int D, const T *rest, int stop)
    {
        if constexpr (R != kSingle) {
#pragma unroll
            for (int c = 0; c < kVec<R> / LV; ++c) {
                const int at = i + c * LV;
                if (R != kFlat || (at >= 0 && at + LV <= D)) {
                    w[c].load(copy + at + shift);
                } else if (at >= stop) {
                    edge(w[c], rest, at, D);
                } else {
                    edge(w[c], copy + shift, at, D);
                }
            }
        }
    }
    __device__ __forceinline__ float operator[](int e) const { return w[e / LV][e % LV]; }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int c = 0; c < kVec<R> / LV; ++c) w[c].fill(0.f);
    }

  private:
    static __device__ __forceinline__ void edge(Raw<float, LV> &o, const float *row, int at, int D)
    {
#pragma unroll
        for (int e = 0; e < LV; ++e) o.w[e] = at + e >= 0 && at + e < D ? row[at + e] : 0.f;
    }
    static __device__ __forceinline__ void edge(Raw<bf16_t, LV> &o, const bf16_t *row, int at, int D)
    {
        if constexpr (LV > 1) {
#pragma unroll
            for (int e = 0; e < LV; e += 2) {
                const unsigned lo = at + e >= 0 && at + e < D ? row[at + e].bits : 0, hi = at + e + 1 >= 0 && at + e + 1 < D ? row[at + e + 1].bits : 0;
                o.w[e / 2] = lo | hi << 16;
            }
        }
    }
};

// Values i .. i + VEC - 1 of a row of D.
template <Rows R, typename T>
__device__ __forceinline__ void store_row(T *row, int i, int D, const float (&f)[kVec<R>])
{
    if constexpr (R == kSingle) {
        store1(row + i, f[0]);
    } else {
        constexpr int W = kWide<T>;
#pragma unroll
        for (int c = 0; c < 8 / W; ++c) {
            const int at = i + c * W;
            float v[W];
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = f[c * W + e];
            if (R != kFlat || (at >= 0 && at + W <= D)) {
                store_vec<W>(row + at, v);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (at + e >= 0 && at + e < D) store1(row + at + e, v[e]);
            }
        }
    }
}

// The weights that go with them, zeros beyond the row.  A flat row's are O values
// behind a boundary of 4, the same O for the whole row.
template <int O>
__device__ __forceinline__ void load_w_at(const float *p, int i, int D, float (&w)[8])
{
    float q[O == 0 ? 8 : 12];
#pragma unroll
    for (int c = 0; c < int(sizeof(q) / 16); ++c) {
        const int at = i - O + 4 * c;
        if (at >= 0 && at + 4 <= D) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(p + at));
            q[4 * c] = x.x, q[4 * c + 1] = x.y, q[4 * c + 2] = x.z, q[4 * c + 3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) q[4 * c + e] = at + e >= 0 && at + e < D ? __ldg(p + at + e) : 0.f;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = q[O + e];
}
template <Rows R>
__device__ __forceinline__ void load_w(const float *p, int i, int D, float (&w)[kVec<R>])
{
    if constexpr (R == kFlat) {
        switch (i & 3) {
        case 0: return load_w_at<0>(p, i, D, w);
        case 1: return load_w_at<1>(p, i, D, w);
        case 2: return load_w_at<2>(p, i, D, w);
        default: return load_w_at<3>(p, i, D, w);
        }
    } else {
        load_vec<kVec<R>>(p + i, w);
    }
}

// What the forward writes in place of y: nothing else, or 8 bits with a scale
// for each block of channels or for the whole row.
enum Quant { kNone, kBlocks, kRow };

// One row for a team: threads t of `threads` hold vectors t, t + threads, ...,
// NV at most.
template <typename T, Rows R, int NV, bool WARP, Quant Q>
__global__ void __launch_bounds__(WARP ? 256 : 1024, 1) rms_fwd_kernel(const RmsArgs p)
{
    constexpr int VEC = kVec<R>;
    __shared__ float sums[32], most[32];
    const int64_t row = WARP ? int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= p.M) return;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x, D = int(p.D);
    const int shift = shift_of<T, R>(row, p.D), vecs = (D + shift + VEC - 1) / VEC;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.res != nullptr ? static_cast<const T *>(p.res) + row * p.ldres : nullptr;
    Held<T, R> hx[NV], hr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
        if (j < vecs) hx[i].load(x, j * VEC - shift, D);
    }
    if (res != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if (j < vecs) hr[i].load(res, j * VEC - shift, D);
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
        if (p.r != nullptr) store_row<R>(static_cast<T *>(p.r) + row * p.D, j * VEC - shift, D, f[i]);
    }
    ss = over_team<WARP, Add>(ss, sums);
    const float rstd = rsqrtf(ss / float(D) + p.eps);
    if (p.rstd != nullptr && t == 0) p.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
        if (j >= vecs) continue;
        float w[VEC];
        load_w<R>(p.w, j * VEC - shift, D, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i][e] *= rstd * w[e];
        if constexpr (Q == kNone) store_row<R>(static_cast<T *>(p.y) + row * p.D, j * VEC - shift, D, f[i]);
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
                if (j < vecs && (t & (lanes - 1)) == 0) p.scale[row * (p.D / p.block) + j / lanes] = scale;
            }
            if (j >= vecs) continue;
            // y times 1 / scale: off y / scale by 2^-23 at most, before a rounding of 2^-4
            const float inv = __frcp_rn(scale);
            const int at = j * VEC - shift;
            unsigned char *q = static_cast<unsigned char *>(p.q) + row * p.D;
            if constexpr (VEC == 8) {
                unsigned w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w[h] = e4m3x2(f[i][4 * h] * inv, f[i][4 * h + 1] * inv) |
                           e4m3x2(f[i][4 * h + 2] * inv, f[i][4 * h + 3] * inv) << 16;
                if (R != kFlat) {
                    *reinterpret_cast<uint2 *>(q + at) = make_uint2(w[0], w[1]);
                } else {   // on 4-byte boundaries
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (at + 4 * h >= 0 && at + 4 * h + 4 <= D) {
                            *reinterpret_cast<unsigned *>(q + at + 4 * h) = w[h];
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (at + 4 * h + e >= 0 && at + 4 * h + e < D) q[at + 4 * h + e] = (unsigned char)(w[h] >> (8 * e));
                        }
                    }
                }
            } else {
                q[at] = (unsigned char)e4m3x2(f[i][0] * inv, 0.f);
            }
        }
    }
}

// Gradients: teams walk over rows and keep their channels' sums for dw; a block
// leaves one row of sums.  The next STAGES rows come by bulk copies into shared
// memory, so that a row's barrier does not hold up its successors: a flat row from
// the 16-byte boundary before it to the one behind it (flat_rows.h).  (A row ahead
// in registers: 125 us for 32768 x 2048 bf16 rows; 16-byte asynchronous copies by
// all threads: 116 us, and 160 for 16384 x 2048 float32 ones.)  The teams' number is a multiple
// of 8, so that a team's rows all begin at the same place between two boundaries.
// Single values are loaded as they are needed.
template <typename T, Rows R, int NV, bool WARP, int STAGES, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 ? 2 : 1) rms_bwd_kernel(const RmsArgs p, float *part, unsigned stage_bytes)
{
    constexpr int VEC = kVec<R>;
    constexpr bool kKeepW = MOST <= 512;   // registers for the weights
    using H = Held<T, R>;
    extern __shared__ __align__(16) char ring[];
    __shared__ float sums[2][32];
    __shared__ uint64_t full[WARP ? 8 : 1][STAGES];
    const int warps = blockDim.x >> 5, warp = WARP ? threadIdx.x >> 5 : 0;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x, D = int(p.D);
    const int64_t teams = WARP ? int64_t(gridDim.x) * warps : gridDim.x;
    int64_t row = WARP ? int64_t(blockIdx.x) * warps + warp : blockIdx.x;
    const int shift = shift_of<T, R>(row, p.D), vecs = (D + shift + VEC - 1) / VEC;
    const unsigned slot_bytes = stage_bytes / 3;
    const auto slot = [&](int stage, int k) { return reinterpret_cast<T *>(ring + (warp * STAGES + stage) * stage_bytes + k * slot_bytes); };
    const auto fetch = [&](int stage, int64_t r) {   // one thread of the team
        if (R == kSingle || r >= p.M) return;
        const int64_t pieces = flat_copy_end(r, p.D, p.M, kWide<T>) - flat_copy_begin(r, p.D, kWide<T>);
        const unsigned bytes = R == kFlat ? (pieces > 0 ? unsigned(pieces * sizeof(T)) : 0) : unsigned(D * sizeof(T));
        bar_expect(&full[warp][stage], bytes * (p.dr != nullptr ? 3 : 2));
        if (bytes == 0) return;
        copy_bytes(smem_addr(slot(stage, 0)), static_cast<const T *>(p.dy) + r * p.lddy - shift, bytes, &full[warp][stage]);
        copy_bytes(smem_addr(slot(stage, 1)), static_cast<const T *>(p.x) + r * p.ldx - shift, bytes, &full[warp][stage]);
        if (p.dr != nullptr) copy_bytes(smem_addr(slot(stage, 2)), static_cast<const T *>(p.dr) + r * p.lddr - shift, bytes, &full[warp][stage]);
    };
    if (R != kSingle && t == 0) {
        for (int s = 0; s < STAGES; ++s) bar_init(&full[warp][s]);
        fence_tiles();
        for (int s = 0; s < STAGES; ++s) fetch(s, row + s * teams);
    }
    float w[kKeepW ? NV : 1][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = i * threads + t;
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = w[kKeepW ? i : 0][e] = 0.f;
        if (kKeepW && j < vecs) load_w<R>(p.w, j * VEC - shift, D, w[i]);
    }
    __syncthreads();   // the barriers are set up
    float rstd = row < p.M ? __ldg(p.rstd_in + row) : 0.f;
    int turn = 0, stage = 0;
    unsigned phase = 0;
    for (; row < p.M; row += teams, turn ^= 1) {
        H dy[NV], x[NV], dr[NV];
        const float rs = rstd;
        if (row + teams < p.M) rstd = __ldg(p.rstd_in + row + teams);
        if constexpr (R != kSingle) {
            if (!bar_wait(&full[warp][stage], phase)) atomicOr(error_word(p.ws), kErrLookbackTimeout);
        }
        const T *gdy = static_cast<const T *>(p.dy) + row * p.lddy, *gx = static_cast<const T *>(p.x) + row * p.ldx;
        const T *gdr = p.dr != nullptr ? static_cast<const T *>(p.dr) + row * p.lddr : nullptr;
        const int stop = R == kFlat ? int(flat_copy_end(row, p.D, p.M, kWide<T>) - row * p.D) : D;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t, at = j * VEC - shift;
            dy[i].clear(), x[i].clear(), dr[i].clear();
            if (j >= vecs) continue;
            if constexpr (R == kSingle) {
                dy[i].load(gdy, at, D), x[i].load(gx, at, D);
                if (gdr != nullptr) dr[i].load(gdr, at, D);
            } else {
                dy[i].take(slot(stage, 0), shift, at, D, gdy, stop), x[i].take(slot(stage, 1), shift, at, D, gx, stop);
                if (gdr != nullptr) dr[i].take(slot(stage, 2), shift, at, D, gdr, stop);
            }
            if (!kKeepW) load_w<R>(p.w, at, D, w[0]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) dot = fmaf(dy[i][e] * w[kKeepW ? i : 0][e], x[i][e] * rs, dot);
        }
        dot = over_team<WARP, Add>(dot, sums[turn]) / float(D);
        if (WARP) __syncwarp();
        if (R != kSingle && t == 0) fetch(stage, row + STAGES * teams);   // the team has read the row
        if (++stage == STAGES) stage = 0, phase ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t;
            if (j >= vecs) continue;
            if (!kKeepW) load_w<R>(p.w, j * VEC - shift, D, w[0]);
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float n = x[i][e] * rs;
                dw[i][e] = fmaf(dy[i][e], n, dw[i][e]);
                o[e] = fmaf(rs, fmaf(-n, dot, dy[i][e] * w[kKeepW ? i : 0][e]), dr[i][e]);
            }
            store_row<R>(static_cast<T *>(p.dx) + row * p.D, j * VEC - shift, D, o);
        }
    }
    float *mine = part + int64_t(blockIdx.x) * p.D;
    if constexpr (!WARP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = i * threads + t, at = j * VEC - shift;
            if (j >= vecs) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (R != kFlat || (at + e >= 0 && at + e < D)) mine[at + e] = dw[i][e];
        }
    } else {
        __syncthreads();   // the ring is done with
        float *all = reinterpret_cast<float *>(ring);
        for (int j = threadIdx.x; j < D; j += blockDim.x) all[j] = 0.f;
        __syncthreads();
        for (int turn_of = 0; turn_of < warps; ++turn_of) {
            if (int(threadIdx.x >> 5) == turn_of) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int j = i * threads + t, at = j * VEC - shift;
                    if (j >= vecs) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (R != kFlat || (at + e >= 0 && at + e < D)) all[at + e] += dw[i][e];
                }
            }
            __syncthreads();
        }
        for (int j = threadIdx.x; j < D; j += blockDim.x) mine[j] = all[j];
    }
}

// dw from the blocks' rows of sums: 32 warps share a column, eight rows in flight
// each (with 8 warps and a row at a time it took half of the gradients of 16384 x
// 1002).
__global__ void __launch_bounds__(1024) rms_sum_kernel(const float *part, int64_t parts, int64_t D, float *dw)
{
    __shared__ float all[32][33];
    after_previous();
    const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.x;
    float v = 0.f;
    if (col < D) {
        for (int64_t r0 = threadIdx.y; r0 < parts; r0 += 32 * 8) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = r0 + 32 * u < parts ? part[(r0 + 32 * u) * D + col] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += x[u];
        }
    }
    all[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y > 0 || col >= D) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += all[i][threadIdx.x];
    dw[col] = v;
}

// How a launch holds rows: nv vectors a thread, and a block of `threads` a row
// (0: a warp a row, 8 of them in a block).
struct Shape {
    int nv, threads;
};

Rows rows_for(int64_t D, std::initializer_list<int64_t> lds)
{
    int64_t all = D;
    bool dense = true;
    for (int64_t ld : lds) all |= ld, dense = dense && ld == D;
    return all % 8 == 0 ? kWhole : dense ? kFlat : kSingle;
}

// A warp takes rows of up to 4 vectors a lane (2 in the gradients, which hold more
// for each), a block wider ones: 2 vectors a thread (single values: 4, 8 or 16).
// One vector a thread was slower: 8 bits of 32768 x 4096 bf16 rows 201 us against
// 167.  A flat row may have a vector more than it fills, which for the widest (from
// 16378 channels on) is one more than 1024 threads hold: 4 a thread.
Shape shape_for(Rows r, int64_t D, bool bwd)
{
    const int64_t n = r == kSingle ? D : r == kFlat ? (D + 14) / 8 : D / 8;
    if (n <= (bwd ? 64 : 128)) return {n <= 32 ? 1 : n <= 64 ? 2 : 4, 0};
    const int nv = r != kSingle ? (n <= 2048 ? 2 : 4) : n <= 1024 ? 4 : n <= 4096 ? 8 : 16;
    return {nv, int(align_up(size_t(ceil_div(n, nv)), 32))};
}

// The gradients' ring: bytes of a team's stage (three rows from boundary to
// boundary), stages, and blocks an SM, by shared memory and by 512 threads (128
// registers each).  So rows of up to 4096 channels have two blocks or more of up to
// 256 threads, wider ones one: bf16 16384 x 4096 93 us (5.8 TB/s), 32768 x 5120 234
// (5.7), 16384 x 8192 176 (6.1); flat rows of 4095 channels, with a 257th thread,
// have one block of 288 threads too: 174 us (3.1).  Above 8192 channels of float32
// 64 registers spill: 8192 x 8192 170 us (6.3), 4096 x 16384 246 (4.4).
struct Ring {
    unsigned stage;
    int stages;
    size_t bytes;
    int64_t per_sm;
};
Ring ring_for(Rows r, const Shape &c, int64_t D, size_t esize)
{
    const int threads = c.threads == 0 ? 256 : c.threads, teams = c.threads == 0 ? 8 : 1;
    Ring o{};
    o.stages = 1, o.per_sm = 512 / threads;
    if (r != kSingle) {
        o.stage = unsigned(3 * align_up(size_t(D) * esize + 32, 16));
        const size_t all = size_t(o.stage) * teams;
        o.stages = all * 3 <= 100 * 1024 ? 3 : all * 2 <= 200 * 1024 ? 2 : 1;
        const int64_t fit = int64_t(220 * 1024 / (all * o.stages));
        o.per_sm = fit < o.per_sm ? fit : o.per_sm;
    }
    o.bytes = size_t(o.stage) * teams * o.stages;
    if (c.threads == 0 && o.bytes < size_t(D) * 4) o.bytes = size_t(D) * 4;   // the sums of its warps
    if (o.per_sm < 1) o.per_sm = 1;
    return o;
}
int64_t bwd_blocks(int64_t M, const Shape &c, const Ring &r)
{
    const int64_t most = c.threads == 0 ? ceil_div(M, 8) : M;
    return most < kSMs * r.per_sm ? most : kSMs * r.per_sm;   // 152 is a multiple of 8
}

template <typename T, Rows R, int NV, bool WARP, Quant Q>
mg_status fwd(const RmsArgs &p, const Shape &c, cudaStream_t s)
{
    const int64_t blocks = WARP ? ceil_div(p.M, 8) : p.M;
    MG_TRY(check_grids("mg_rms_norm", {blocks}));
    rms_fwd_kernel<T, R, NV, WARP, Q><<<unsigned(blocks), WARP ? 256 : c.threads, 0, s>>>(p);
    return launched("mg_rms_norm");
}

template <typename T, Rows R, int NV, bool WARP, int STAGES, int MOST>
mg_status bwd_most(const RmsArgs &p, const Shape &c, const Ring &r, cudaStream_t s)
{
    float *part = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    const int64_t blocks = bwd_blocks(p.M, c, r);
    if (r.stages != STAGES) return fail(MG_ERR_UNSUPPORTED, "mg_rms_norm_bwd: a ring of %d stages", r.stages);
    MG_TRY((allow_shared<rms_bwd_kernel<T, R, NV, WARP, STAGES, MOST>>(r.bytes)));
    rms_bwd_kernel<T, R, NV, WARP, STAGES, MOST><<<unsigned(blocks), WARP ? 256 : c.threads, r.bytes, s>>>(p, part, r.stage);
    MG_TRY(launched("mg_rms_norm_bwd"));
    return launch_next("mg_rms_norm_bwd", rms_sum_kernel, ceil_div(p.D, 32), dim3(32, 32), 0, s, part, blocks, p.D, p.dw);
}

// Stages, and registers for the threads that the block has, of those that a type's
// rows come to (ring_for, shape_for).
template <typename T, Rows R, int NV, bool WARP>
mg_status bwd(const RmsArgs &p, const Shape &c, cudaStream_t s)
{
    constexpr bool kF32 = sizeof(T) == 4;
    const Ring r = ring_for(R, c, p.D, sizeof(T));
    if constexpr (R == kSingle) {
        if constexpr (NV == 16)
            if (c.threads > 512) return bwd_most<T, R, NV, WARP, 1, 1024>(p, c, r, s);
        return bwd_most<T, R, NV, WARP, 1, 512>(p, c, r, s);
    } else if constexpr (WARP) {
        if constexpr (kF32 && NV == 2)
            if (r.stages == 2) return bwd_most<T, R, NV, WARP, 2, 256>(p, c, r, s);
        return bwd_most<T, R, NV, WARP, 3, 256>(p, c, r, s);
    } else if constexpr (NV == 4) {
        return bwd_most<T, R, NV, WARP, kF32 ? 1 : 2, 1024>(p, c, r, s);
    } else {
        if constexpr (kF32)
            if (r.stages == 1) return bwd_most<T, R, NV, WARP, 1, 1024>(p, c, r, s);
        if (c.threads > 512) return bwd_most<T, R, NV, WARP, 2, 1024>(p, c, r, s);
        if (r.stages == 2) return bwd_most<T, R, NV, WARP, 2, 512>(p, c, r, s);
        if constexpr (!kF32)
            if (c.threads > 256) return bwd_most<T, R, NV, WARP, 3, 512>(p, c, r, s);
        return bwd_most<T, R, NV, WARP, 3, 256>(p, c, r, s);
    }
}

template <typename T, Rows R, Quant Q>
mg_status fwd_shape(const RmsArgs &p, cudaStream_t s)
{
    const Shape c = shape_for(R, p.D, false);
    if (c.threads == 0) {
        if (c.nv == 1) return fwd<T, R, 1, true, Q>(p, c, s);
        if (c.nv == 2) return fwd<T, R, 2, true, Q>(p, c, s);
        return fwd<T, R, 4, true, Q>(p, c, s);
    }
    if constexpr (R != kSingle) {
        if constexpr (R == kFlat)
            if (c.nv == 4) return fwd<T, R, 4, false, Q>(p, c, s);
        return fwd<T, R, 2, false, Q>(p, c, s);
    } else {
        if (c.nv == 4) return fwd<T, R, 4, false, Q>(p, c, s);
        if (c.nv == 8) return fwd<T, R, 8, false, Q>(p, c, s);
        return fwd<T, R, 16, false, Q>(p, c, s);
    }
}

template <typename T, Rows R>
mg_status bwd_shape(const RmsArgs &p, cudaStream_t s)
{
    const Shape c = shape_for(R, p.D, true);
    if (c.threads == 0) {
        if (c.nv == 1) return bwd<T, R, 1, true>(p, c, s);
        return bwd<T, R, 2, true>(p, c, s);
    }
    if constexpr (R != kSingle) {
        if constexpr (R == kFlat)
            if (c.nv == 4) return bwd<T, R, 4, false>(p, c, s);
        return bwd<T, R, 2, false>(p, c, s);
    } else {
        if (c.nv == 4) return bwd<T, R, 4, false>(p, c, s);
        if (c.nv == 8) return bwd<T, R, 8, false>(p, c, s);
        return bwd<T, R, 16, false>(p, c, s);
    }
}

// A scale for each block needs whole vectors of 8, which blocks of 32 and more
// are made of: loaded value by value where the input's rows are not aligned.
template <typename T, Quant Q>
mg_status fwd_any(const RmsArgs &p, cudaStream_t s)
{
    const Rows r = rows_for(p.D, {p.ldx, p.res != nullptr ? p.ldres : p.D});
    if constexpr (Q == kBlocks) {
        return r == kWhole ? fwd_shape<T, kWhole, Q>(p, s) : fwd_shape<T, kLoose, Q>(p, s);
    } else {
        if (r == kWhole) return fwd_shape<T, kWhole, Q>(p, s);
        if (r == kFlat) return fwd_shape<T, kFlat, Q>(p, s);
        return fwd_shape<T, kSingle, Q>(p, s);
    }
}

template <typename T>
mg_status bwd_any(const RmsArgs &p, cudaStream_t s)
{
    const Rows r = rows_for(p.D, {p.ldx, p.lddy, p.dr != nullptr ? p.lddr : p.D});
    if (r == kWhole) return bwd_shape<T, kWhole>(p, s);
    if (r == kFlat) return bwd_shape<T, kFlat>(p, s);
    return bwd_shape<T, kSingle>(p, s);
}

}  // namespace

size_t rms_ws_bytes(int64_t M, int64_t D)
{
    int64_t blocks = 0;   // the most over what types and strides may give
    for (Rows r : {kWhole, kFlat, kSingle})
        for (size_t esize : {2, 4}) {
            const Shape c = shape_for(r, D, true);
            const int64_t n = bwd_blocks(M, c, ring_for(r, c, D, esize));
            blocks = n > blocks ? n : blocks;
        }
    return kControlBytes + size_t(blocks) * D * sizeof(float);
}

mg_status launch_rms_fwd(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    return dt == MG_F32 ? fwd_any<float, kNone>(p, s) : fwd_any<bf16_t, kNone>(p, s);
}

mg_status launch_rms_quant(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    if (p.block == p.D || p.block == 0)
        return dt == MG_F32 ? fwd_any<float, kRow>(p, s) : fwd_any<bf16_t, kRow>(p, s);
    return dt == MG_F32 ? fwd_any<float, kBlocks>(p, s) : fwd_any<bf16_t, kBlocks>(p, s);
}

mg_status launch_rms_bwd(const RmsArgs &p, mg_dtype dt, cudaStream_t s)
{
    return dt == MG_F32 ? bwd_any<float>(p, s) : bwd_any<bf16_t>(p, s);
}

}  // namespace mg
