// Shared by the selective mixer's kernels (causal_conv.cu, selective_scan.cu,
// group_norm.cu): argument blocks, launchers, sequences and small device
// helpers.
#pragma once

#include <atomic>

#include "abi_checks.cuh"
#include "common.cuh"
#include "mg_ssm.h"

namespace mg {

// ------------------------------------------------------------ host side

struct ConvArgs {
    const void *x, *x0, *dy, *dx_last;
    int64_t ldx, lddy;
    const float *w, *bias;
    const int64_t *cu;
    int64_t nseq;
    int silu;
    void *y, *x_last, *dx, *dx0;
    float *dw, *dbias;
    int64_t B, T, D;
    int W;
    void *ws;
};
size_t conv_ws_bytes(int64_t B, int64_t T, int64_t D, int W);
mg_status launch_conv_fwd(const ConvArgs &p, mg_dtype dt, cudaStream_t s);
mg_status launch_conv_bwd(const ConvArgs &p, mg_dtype dt, cudaStream_t s);

struct ConvStepArgs {
    const void *x;
    int64_t ldx;
    const float *w, *bias;
    void *state;
    int64_t nslots;
    const int64_t *slots;
    int silu;
    void *y;
    int64_t B, D;
    int W;
};
mg_status launch_conv_step(const ConvStepArgs &p, mg_dtype dt, cudaStream_t s);

struct SsmArgs {
    const void *x, *raw, *Bm, *Cm, *dy;
    int64_t ldx, ldraw, ldb, ldc, lddy;
    const float *A, *Dskip, *dt_bias, *h0, *dh_last;
    int softplus;
    const int64_t *cu;
    int64_t nseq;
    void *y;
    float *h_last, *saved;
    const float *saved_in;
    void *dx, *draw, *dBm, *dCm;
    float *dA, *dDskip, *ddt_bias, *dh0;
    int64_t B, T, D;
    int N, G;
    void *ws;
};
constexpr int kSsmMaxN = 64;
size_t ssm_fwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t nseq);
size_t ssm_bwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t nseq);
size_t ssm_saved_bytes(int64_t B, int64_t T, int64_t D, int N);
int ssm_saved_rows();
mg_status launch_ssm_fwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s);
mg_status launch_ssm_bwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s);

struct SsmStepArgs {
    const void *x, *raw, *Bm, *Cm;
    int64_t ldx, ldraw, ldb, ldc;
    const float *A, *Dskip, *dt_bias;
    int softplus;
    float *state;
    int64_t nslots;
    const int64_t *slots;
    void *y;
    int64_t B, D;
    int N, G;
};
mg_status launch_ssm_step(const SsmStepArgs &p, mg_dtype dt, cudaStream_t s);

struct NormArgs {
    const void *x, *z, *dy;
    int64_t ldx, ldz, lddy;
    const float *w, *bias;
    float eps;
    int rms, silu;
    mg_gate gate;
    void *y, *dx, *dz;
    float *stats;
    const float *stats_in;
    float *dw, *dbias;
    int64_t M, D, G;
    void *ws;
};
size_t norm_ws_bytes(int64_t M, int64_t D, int64_t G);
mg_status launch_norm_fwd(const NormArgs &p, mg_dtype dt, cudaStream_t s);
mg_status launch_norm_bwd(const NormArgs &p, mg_dtype dt, cudaStream_t s);

// The last step of the sums over rows: each of `parts` rows of part holds the
// outputs' values one after another; out[i] = the sum of its column, in a fixed
// order, in one launch.  An output that is NULL is left out.
struct SumOut {
    float *out;
    int64_t n;
};
mg_status launch_sum_parts(const float *part, int64_t parts, std::initializer_list<SumOut> outs, cudaStream_t s);
inline int64_t sum_parts_blocks(int64_t columns) { return (columns + 31) / 32; }

// A call's block counts, all of them before its first launch: a grid holds
// 2^31 - 1 blocks.
inline mg_status check_grids(const char *what, std::initializer_list<int64_t> blocks)
{
    for (int64_t n : blocks)
        if (n > INT32_MAX)
            return fail(MG_ERR_UNSUPPORTED, "%s: %lld blocks in a launch, at most 2^31 - 1", what, (long long)n);
    return MG_OK;
}

inline mg_status launched(const char *what)
{
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MG_OK : fail(MG_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
}

// Launches a kernel that is set up while the kernel before it in the stream,
// one of the same call, comes to its end: until after_previous() it reads only
// the call's inputs.  1 x 2048 x 2048 channels of 16 states: forward (two
// kernels) 61 -> 58 us, gradients (four) 141 -> 133.  (Begun earlier, once the
// other's last blocks run, the second's blocks gather on the SMs that are
// free first: 74 us.)
template <typename... P, typename... A>
mg_status launch_next(const char *what, void (*kernel)(P...), int64_t grid, dim3 block, size_t smem, cudaStream_t s,
                      const A &...args)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(unsigned(grid));
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &early;
    c.numAttrs = 1;
    cudaLaunchKernelEx(&c, kernel, P(args)...);
    return launched(what);
}

// Dynamic shared memory beyond the default 48 KB (which count static shared
// memory too): allowed once for a kernel and device, up to what a block may
// have.  The set-up costs as much as a launch.
constexpr size_t kMostShared = 226 * 1024;
template <auto kKernel, size_t kMost = kMostShared>
mg_status allow_shared(size_t bytes)
{
    if (bytes <= 40 * 1024) return MG_OK;
    if (bytes > kMost) return fail(MG_ERR_UNSUPPORTED, "%zu bytes of shared memory", bytes);
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (e == cudaSuccess && (done.load() & bit) == 0) {
        e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost));
        if (e == cudaSuccess) done.fetch_or(bit);
    }
    return e == cudaSuccess ? MG_OK : fail(MG_ERR_LAUNCH, "shared memory: %s", cudaGetErrorString(e));
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------- device side

// Waits until the kernel before this one has ended and its writes are seen.
// Every kernel that launch_next starts has every block come here, so that the
// end of the last one means the end of all.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" : : : "memory"); }

// One value of an activation tensor.
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const bf16_t *p) { return bf16_bits_to_float(p->bits); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t *p, float v)
{
    p->bits = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// e^x for x <= 0.  The rounding of x log2 e costs a relative |x| 2^-24, no
// more than the rounding of the sum (raw + bias, a convolution) that x is.
__device__ __forceinline__ float exp_neg(float x) { return ex2_ftz(x * kLog2eF); }

// 1 / x to 1 ulp for x >= 1 (0 for infinity).
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log(1 + e) / e on [0, 1], the polynomial of degree 9 through a weighted
// least-squares fit at Chebyshev points (relative error 2.4e-8, with the
// evaluation's roundings 1.5e-7): times e it keeps relative accuracy for small
// e, where 1 + e would round e away.
__device__ constexpr float log1p_coef(int i)
{
    constexpr float c[10] = {1.f,           -0.499998897f, 0.333296657f,   -0.249511674f, 0.196610183f,
                             -0.152632743f, 0.105329506f,  -0.0562695265f, 0.0194876865f, -0.00316399941f};
    return c[i];
}

// log(1 + e), 0 <= e <= 1.
__device__ __forceinline__ float log1p_unit(float e)
{
    float c = log1p_coef(9);
#pragma unroll
    for (int i = 8; i >= 0; --i) c = fmaf(c, e, log1p_coef(i));
    return e * c;
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|).
__device__ __forceinline__ float softplus_f(float v)
{
    return fmaxf(v, 0.f) + log1p_unit(exp_neg(-fabsf(v)));
}

// ------------------------------------------------------- pairs of floats
// Two float32 in one 64-bit register pair: one instruction multiplies and
// adds both.
using pair_t = unsigned long long;

__device__ __forceinline__ pair_t pack2(float a, float b)
{
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(pair_t p, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c)
{
    pair_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b)
{
    pair_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ pair_t add2(pair_t a, pair_t b)
{
    pair_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// VEC neighbouring channels as pairs (or one float), and arithmetic on them.
template <int VEC>
struct Lanes {
    pair_t p[VEC / 2];
};
template <>
struct Lanes<1> {
    float p[1];
};
__device__ __forceinline__ pair_t op_fma(pair_t a, pair_t b, pair_t c) { return fma2(a, b, c); }
__device__ __forceinline__ pair_t op_mul(pair_t a, pair_t b) { return mul2(a, b); }
__device__ __forceinline__ pair_t op_add(pair_t a, pair_t b) { return add2(a, b); }
__device__ __forceinline__ float op_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float op_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float op_add(float a, float b) { return a + b; }
#define MG_LANES_EACH for (int i_ = 0; i_ < int(sizeof(Lanes<VEC>::p) / sizeof(Lanes<VEC>::p[0])); ++i_)
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vfma(const Lanes<VEC> &a, const Lanes<VEC> &b, const Lanes<VEC> &c)
{
    Lanes<VEC> r;
#pragma unroll
    MG_LANES_EACH r.p[i_] = op_fma(a.p[i_], b.p[i_], c.p[i_]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vmul(const Lanes<VEC> &a, const Lanes<VEC> &b)
{
    Lanes<VEC> r;
#pragma unroll
    MG_LANES_EACH r.p[i_] = op_mul(a.p[i_], b.p[i_]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vadd(const Lanes<VEC> &a, const Lanes<VEC> &b)
{
    Lanes<VEC> r;
#pragma unroll
    MG_LANES_EACH r.p[i_] = op_add(a.p[i_], b.p[i_]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vfrom(const float (&f)[VEC])
{
    Lanes<VEC> r;
    if constexpr (VEC == 1) {
        r.p[0] = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) r.p[i] = pack2(f[2 * i], f[2 * i + 1]);
    }
    return r;
}
template <int VEC>
__device__ __forceinline__ void vto(const Lanes<VEC> &a, float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        f[0] = a.p[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) unpack2(a.p[i], f[2 * i], f[2 * i + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vset(float c)
{
    float f[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = c;
    return vfrom<VEC>(f);
}
// sigmoid as 1 / (1 + 2^(-v log2 e)): for v far below 0 the power is infinite
// and the quotient 0.
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vsigmoid(const Lanes<VEC> &v)
{
    float f[VEC];
    vto<VEC>(vmul<VEC>(v, vset<VEC>(-kLog2eF)), f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = ex2_ftz(f[i]);
    vto<VEC>(vadd<VEC>(vfrom<VEC>(f), vset<VEC>(1.f)), f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = rcp_fast(f[i]);
    return vfrom<VEC>(f);
}

// The sequences of the flattened rows 0 .. B*T-1 of a batch: offsets from
// cu_seqlens, or B sequences of T rows.
struct Seqs {
    const long long *cu;
    long long T;       // rows of a dense sequence
    long long rows;    // all rows
    int nseq;
    __device__ __forceinline__ long long begin(int s) const
    {
        return cu != nullptr ? __ldg(cu + s) : (long long)s * T;
    }
    // The sequence that holds row r: the last s with begin(s) <= r.
    __device__ __forceinline__ int of(long long r) const
    {
        if (cu == nullptr) return int(r / T);
        int lo = 0, hi = nseq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(cu + mid) <= r) lo = mid; else hi = mid;
        }
        return lo;
    }
};

// Called by the threads of one block: sets the workspace's error bit if cu
// is not non-decreasing from 0 to rows.
__device__ __forceinline__ void check_cu(const Seqs &q, unsigned *err, int tid, int threads)
{
    if (q.cu == nullptr) return;
    bool bad = false;
    for (int s = tid; s < q.nseq; s += threads) {
        const long long a = __ldg(q.cu + s), b = __ldg(q.cu + s + 1);
        bad = bad || b < a || (s == 0 && a != 0) || (s + 1 == q.nseq && b != q.rows);
    }
    if (bad) atomicOr(err, kErrBadSeqlens);
}

inline Seqs make_seqs(const int64_t *cu, int64_t B, int64_t T, int64_t nseq)
{
    return Seqs{reinterpret_cast<const long long *>(cu), T, B * T, int(nseq)};
}

__device__ __forceinline__ unsigned *error_word(void *ws)
{
    return &static_cast<Control *>(ws)->error;
}

}  // namespace mg
