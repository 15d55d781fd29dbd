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

#ifndef MG_SSM_WHOLE
#define MG_SSM_WHOLE 256
#endif
#ifndef MG_SSM_BLOCKS
#define MG_SSM_BLOCKS 608
#endif

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

// The decay e^(delta A) = 2^(delta A log2 e) of two states.  ex2.approx comes
// out low by a relative 1.1e-8 on average for small exponents (measured), and
// a state that lives for 1 / (1 - a) rows would add that up; kDecayBias in
// the exponent, at no cost in the multiply-add, takes it out.  For larger
// exponents it is below their last bit, and the state is short-lived.
constexpr float kDecayBias = 1.6e-8f;

__device__ __forceinline__ pair_t decay2(pair_t delta, pair_t A2)
{
    float a, b;
    unpack2(fma2(delta, A2, pack2(kDecayBias, kDecayBias)), a, b);
    return pack2(ex2_ftz(a), ex2_ftz(b));
}

// ------------------------------------------------------------ chunk geometry

// Time is cut into chunks of `len` rows (a multiple of kSeg), `n` of them for
// a batch entry; block -> (tile, chunk, entry), tiles fastest.
struct Chunks {
    int64_t len;
    int64_t n;
};

constexpr int kTile = 16;   // rows of a staged tile

// How a thread block covers channels: a thread has S states of C channels,
// L lanes a channel.
template <int S_, int L_, int C_>
struct Cover {
    static constexpr int S = S_, L = L_, C = C_;
    static constexpr int NP = S * L;                       // states with padding
    static constexpr int kGroups = 32 / L;                 // channel groups of a warp
    static constexpr int kCh = kThreads / 32 * kGroups * C;  // channels of a block
};

// The (delta, u) pairs of a tile row lie as float4 of two channels; XORing
// the float4's index with bits of its octet spreads the staging writes (four
// consecutive float4 a thread) over all banks and leaves each octet's reads
// in one row of banks.
__device__ __forceinline__ int du_index(int ch) { return ((ch >> 1) ^ ((ch >> 4) & 3)) * 2 + (ch & 1); }

// Sum over the L lanes of a channel (lane bits 32/L .. 16) of G values each,
// G >= L: the lane of state group sl ends with values sl*G/L .. of v.
template <int G, int L>
__device__ __forceinline__ void spread_sum(float (&v)[G], int sl)
{
#pragma unroll
    for (int m = L / 2, w = G / 2; m > 0; m >>= 1, w >>= 1) {
        const bool up = (sl & m) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
            v[i] = keep + __shfl_xor_sync(~0u, give, m * (32 / L));
        }
    }
}

// A thread's S states of one channel.
template <int S>
__device__ __forceinline__ void load_group(const float *p, int n0, int N, float (&o)[S])
{
    if (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < S; i += 4) {
            const float4 v = n0 + i < N ? *reinterpret_cast<const float4 *>(p + n0 + i)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
            o[i] = v.x, o[i + 1] = v.y, o[i + 2] = v.z, o[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i) o[i] = n0 + i < N ? p[n0 + i] : 0.f;
    }
}
template <int S>
__device__ __forceinline__ void store_group(float *p, int n0, int N, const float (&o)[S])
{
    if (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < S; i += 4)
            if (n0 + i < N)
                *reinterpret_cast<float4 *>(p + n0 + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (n0 + i < N) p[n0 + i] = o[i];
    }
}
template <int S>
__device__ __forceinline__ void store_pairs(float *p, int n0, int N, const pair_t (&h)[S / 2])
{
    float o[S];
#pragma unroll
    for (int i = 0; i < S / 2; ++i) unpack2(h[i], o[2 * i], o[2 * i + 1]);
    store_group<S>(p, n0, N, o);
}

// ------------------------------------------------------------------ forward
//
// Two passes where time is cut: the first runs the recurrence of each chunk
// from 0 (from h0 at a sequence's start) and leaves its last state and its
// sum of delta; the second folds those of the chunks since its sequence's
// start into its own first state,
//   h <- exp(A sum_j delta) h + h_j,
// and runs the recurrence again with the outputs.  No block waits for
// another, and the order of every sum is fixed.
//
// A tile of kTile rows is staged at a time: the block's threads load x and
// raw for the next tile into registers while it works on this one, turn them
// into (delta, u) pairs in shared memory (softplus once for each row and
// channel), and the threads' recurrences read them from there, B and C next
// to them.  Rows past the chunk are staged as delta = u = 0, B = C = 0: the
// state passes through them.
//
// Per row and state: 4 float32 multiply-adds (2 instructions for a pair's
// 4) and one 2^x; 64 pairs and 32 2^x a clock and SM, so both pipes ask for
// the same time, and shared memory (2.1 or 3.9 clocks for a 16-byte load of a
// warp, by pattern) and the issue slots are close behind: a thread's S x C
// block of 8 x 2 states loads 5 x 16 bytes for its 16 states' row.
template <typename T, int VEC, typename CV, bool kFirst>
__global__ void __launch_bounds__(kThreads)
ssm_chunk_kernel(SsmArgs p, Seqs q, Tile tl, Chunks ck, float *agg_h, float *agg_s)
{
    constexpr int S = CV::S, L = CV::L, C = CV::C, NP = CV::NP, CH = CV::kCh, SP = S / 2;
    constexpr int kVecs = kTile * CH / VEC;                         // vectors of a tile
    constexpr int kPer = (kVecs + kThreads - 1) / kThreads;         // of a thread
    constexpr int kBc = (kTile * NP + kThreads - 1) / kThreads;     // values of B (or C) of a thread
    constexpr int G = L > 4 ? L : 4;                                // rows between two sums over lanes
    __shared__ __align__(16) float2 s_du[kTile][CH];
    __shared__ __align__(16) float s_b[kTile][NP], s_c[kFirst ? 1 : kTile][NP];
    __shared__ __align__(16) float s_y[kFirst ? 1 : kTile][CH];

    const int64_t all_tiles = tl.tiles * p.G;
    const int64_t tile = blockIdx.x % all_tiles, rest = blockIdx.x / all_tiles;
    const int64_t nch = kFirst ? ck.n - 1 : ck.n;                   // the last chunk has no successor
    const int64_t k = rest % nch, b = rest / nch;
    const int64_t rowb = b * p.T;
    const int64_t t0 = k * ck.len, t1 = t0 + ck.len < p.T ? t0 + ck.len : p.T;
    const int g = int(tile / tl.tiles);
    const int64_t c0 = (tile % tl.tiles) * CH, d0 = g * tl.width + c0;   // the tile's first channel
    const int64_t wide = tl.width - c0 < CH ? tl.width - c0 : CH;        // its channels
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sl = lane / CV::kGroups, n0 = sl * S;
    const int ch = (warp * CV::kGroups + lane % CV::kGroups) * C;        // the thread's first channel

    // The thread's channels.  Channels past the tile run on zeros.
    pair_t A2[C][SP], h[C][SP];
    float ssum[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float a[S];
        const bool live = ch + c < wide;
#pragma unroll
        for (int i = 0; i < S; ++i) a[i] = 0.f;
        if (live) load_group<S>(p.A + (d0 + ch + c) * p.N, n0, p.N, a);
#pragma unroll
        for (int i = 0; i < SP; ++i) {
            A2[c][i] = pack2(a[2 * i] * kLog2eF, a[2 * i + 1] * kLog2eF);
            h[c][i] = 0;
        }
        ssum[c] = 0.f;
    }
    auto start_state = [&](int s) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[S];
#pragma unroll
            for (int i = 0; i < S; ++i) v[i] = 0.f;
            if (p.h0 != nullptr && ch + c < wide)
                load_group<S>(p.h0 + (int64_t(s) * p.D + d0 + ch + c) * p.N, n0, p.N, v);
#pragma unroll
            for (int i = 0; i < SP; ++i) h[c][i] = pack2(v[2 * i], v[2 * i + 1]);
        }
    };
    int s = q.of(rowb + t0);
    long long next = q.begin(s + 1) - rowb;                         // where the sequence ends
    {
        const long long lo = q.begin(s) - rowb;
        if (lo >= t0) {
            start_state(s);
        } else if (!kFirst) {
            int64_t j = (lo < 0 ? 0 : lo) / ck.len;
            const int64_t base = b * (ck.n - 1);
            bool begin = true;
            for (; j < k; ++j) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (ch + c >= wide) continue;
                    const int64_t at = (base + j) * p.D + d0 + ch + c;
                    float v[S];
                    load_group<S>(agg_h + at * p.N, n0, p.N, v);
                    const float ds = agg_s[at];
#pragma unroll
                    for (int i = 0; i < SP; ++i) {
                        const pair_t hv = pack2(v[2 * i], v[2 * i + 1]);
                        h[c][i] = begin ? hv : fma2(decay2(pack2(ds, ds), A2[c][i]), h[c][i], hv);
                    }
                }
                begin = false;
            }
        }
    }

    // Staging: the thread's vectors of x and raw, and values of B and C.
    const T *xp = static_cast<const T *>(p.x) + rowb * p.ldx + d0;
    const T *rp = static_cast<const T *>(p.raw) + rowb * p.ldraw + d0;
    const T *bp = static_cast<const T *>(p.Bm) + rowb * p.ldb + int64_t(g) * p.N;
    const T *cp = static_cast<const T *>(p.Cm) + rowb * p.ldc + int64_t(g) * p.N;
    Raw<T, VEC> xr[kPer], rr[kPer];
    float br[kBc], cr[kFirst ? 1 : kBc];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = threadIdx.x + i * kThreads;
            const int64_t row = t + v / (CH / VEC);
            const int col = v % (CH / VEC) * VEC;
            xr[i].fill(0.f);
            rr[i].fill(0.f);
            if (v < kVecs && row < t1 && col < wide) {
                xr[i].load(xp + row * p.ldx + col);
                rr[i].load(rp + row * p.ldraw + col);
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = threadIdx.x + i * kThreads, n = e % NP;
            const int64_t row = t + e / NP;
            const bool in = e < kTile * NP && row < t1 && n < p.N;
            br[i] = in ? load1(bp + row * p.ldb + n) : 0.f;
            if (!kFirst) cr[i] = in ? load1(cp + row * p.ldc + n) : 0.f;
        }
    };

    // One row of the recurrence from the staged tile; y (without the sum over
    // lanes) comes back.
    auto step = [&](int tt, float (&y)[C]) {
        pair_t B[SP], Cw[SP];
#pragma unroll
        for (int i = 0; i < SP; i += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&s_b[tt][n0 + 2 * i]);
            B[i] = v.x, B[i + 1] = v.y;
            if (!kFirst) {
                const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&s_c[tt][n0 + 2 * i]);
                Cw[i] = w.x, Cw[i + 1] = w.y;
            }
        }
        float du[2 * C];
        if constexpr (C == 2) {
            const float4 v = *reinterpret_cast<const float4 *>(&s_du[tt][du_index(ch)]);
            du[0] = v.x, du[1] = v.y, du[2] = v.z, du[3] = v.w;
        } else {
            const float2 v = s_du[tt][du_index(ch)];
            du[0] = v.x, du[1] = v.y;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const pair_t dd = pack2(du[2 * c], du[2 * c]), uu = pack2(du[2 * c + 1], du[2 * c + 1]);
            pair_t acc = 0;
#pragma unroll
            for (int i = 0; i < SP; ++i) {
                h[c][i] = fma2(decay2(dd, A2[c][i]), h[c][i], mul2(uu, B[i]));
                if (!kFirst) acc = i == 0 ? mul2(Cw[i], h[c][i]) : fma2(Cw[i], h[c][i], acc);
            }
            if (kFirst) {
                ssum[c] += du[2 * c];
            } else {
                float a, e;
                unpack2(acc, a, e);
                y[c] = a + e;
            }
        }
    };

    fetch(t0);
    for (int64_t t = t0; t < t1; t += kTile) {
        // the tile's (delta, u), B and C
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = threadIdx.x + i * kThreads;
            const int row = v / (CH / VEC), col = v % (CH / VEC) * VEC;
            if (kVecs % kThreads == 0 || v < kVecs) {
                const bool in = t + row < t1 && col < wide;
                float2 o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float bias = in && p.dt_bias != nullptr ? __ldg(p.dt_bias + d0 + col + e) : 0.f;
                    const float r = rr[i][e] + bias;
                    const float delta = !in ? 0.f : p.softplus ? softplus_f(r) : r;
                    o[e] = make_float2(delta, delta * xr[i][e]);
                }
                if constexpr (VEC % 2 == 0) {
#pragma unroll
                    for (int e = 0; e < VEC; e += 2)
                        *reinterpret_cast<float4 *>(&s_du[row][du_index(col + e)]) =
                            make_float4(o[e].x, o[e].y, o[e + 1].x, o[e + 1].y);
                } else {
                    s_du[row][du_index(col)] = o[0];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = threadIdx.x + i * kThreads;
            if (kTile * NP % kThreads == 0 || e < kTile * NP) {
                s_b[e / NP][e % NP] = br[i];
                if (!kFirst) s_c[e / NP][e % NP] = cr[i];
            }
        }
        Raw<T, VEC> xk[kFirst ? 1 : kPer];
        if (!kFirst) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) xk[i] = xr[i];
        }
        __syncthreads();
        if (t + kTile < t1) fetch(t + kTile);
        if (!kFirst && p.saved != nullptr && t % kSeg == 0) {
            const int64_t at = b * ((p.T + kSeg - 1) / kSeg) + t / kSeg;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (ch + c < wide)
                    store_pairs<S>(p.saved + (at * p.D + d0 + ch + c) * p.N, n0, p.N, h[c]);
        }
        const int64_t end = t + kTile < t1 ? t + kTile : t1;
        auto last_state = [&]() {
            if (kFirst || p.h_last == nullptr) return;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (ch + c < wide)
                    store_pairs<S>(p.h_last + (int64_t(s) * p.D + d0 + ch + c) * p.N, n0, p.N, h[c]);
        };
        if (next >= end) {   // no sequence begins inside the tile
#pragma unroll 1
            for (int tt = 0; tt < kTile; tt += G) {
                float y[C][G];
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    float v[C];
                    step(tt + i, v);
#pragma unroll
                    for (int c = 0; c < C; ++c) y[c][i] = kFirst ? 0.f : v[c];
                }
                if (!kFirst) {
#pragma unroll
                    for (int c = 0; c < C; ++c) spread_sum<G, L>(y[c], sl);
#pragma unroll
                    for (int i = 0; i < G / L; ++i) {
                        float *o = &s_y[tt + sl * (G / L) + i][ch];
                        if constexpr (C == 2) *reinterpret_cast<float2 *>(o) = make_float2(y[0][i], y[1][i]);
                        else o[0] = y[0][i];
                    }
                }
            }
            if (next == end) last_state();
        } else {
#pragma unroll 1
            for (int tt = 0; tt < int(end - t); ++tt) {
                if (t + tt == next) {
                    ++s;
                    while (s + 1 < q.nseq && q.begin(s + 1) - rowb <= t + tt) ++s;   // empty ones
                    if (s >= q.nseq) s = q.nseq - 1;
                    next = q.begin(s + 1) - rowb;
                    start_state(s);
                }
                float y[C];
                step(tt, y);
                if (!kFirst) {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float v = y[c];
#pragma unroll
                        for (int m = CV::kGroups; m < 32; m <<= 1) v += __shfl_xor_sync(~0u, v, m);
                        if (sl == 0) s_y[tt][ch + c] = v;
                    }
                }
                if (t + tt + 1 == next) last_state();
            }
        }
        __syncthreads();
        if (!kFirst) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = threadIdx.x + i * kThreads;
                const int row = v / (CH / VEC), col = v % (CH / VEC) * VEC;
                if (v < kVecs && t + row < t1 && col < wide) {
                    float o[VEC];
                    load_vec<VEC>(&s_y[row][col], o);
                    if (p.Dskip != nullptr) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) o[e] = fmaf(__ldg(p.Dskip + d0 + col + e), xk[i][e], o[e]);
                    }
                    store_out<VEC>(static_cast<T *>(p.y) + (rowb + t + row) * p.D + d0 + col, o);
                }
            }
        }
    }
    if (kFirst) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (ch + c < wide) {
                const int64_t at = (b * (ck.n - 1) + k) * p.D + d0 + ch + c;
                store_pairs<S>(agg_h + at * p.N, n0, p.N, h[c]);
                if (sl == 0) agg_s[at] = ssum[c];
            }
    }
}

// Packed batches: checks cu_seqlens, and an empty sequence's last state is
// its first (its dh0 is dh_last): dst[s] = src[s], or 0.
__global__ void __launch_bounds__(256) empty_sequences_kernel(Seqs q, float *dst, const float *src,
                                                              int64_t n, unsigned *err)
{
    if (blockIdx.x == 0) check_cu(q, err, threadIdx.x, blockDim.x);
    if (dst == nullptr) return;
    for (int64_t s = blockIdx.x; s < q.nseq; s += gridDim.x)
        if (q.begin(int(s)) >= q.begin(int(s) + 1))
            for (int64_t i = threadIdx.x; i < n; i += blockDim.x) dst[s * n + i] = src != nullptr ? src[s * n + i] : 0.f;
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

// Where the forward cuts time, and how many channels a thread has.
struct Plan {
    int channels;    // C
    Chunks ck;
};

constexpr int64_t kMinChunk = 128;   // rows

// Lanes of a channel: 8 states a thread, 4 for N <= 8.
int forward_lanes(int N) { return N <= 16 ? 2 : N <= 32 ? 4 : 8; }

Plan forward_plan(int64_t B, int64_t T, int64_t D, int N, int G)
{
    const int L = forward_lanes(N);
    auto blocks = [&](int C) { return B * G * ceil_div(D / G, kThreads / L * C); };
    Plan f;
    f.channels = 2;
    f.ck.n = 1;
    if (blocks(2) < MG_SSM_WHOLE) {
        if (blocks(1) >= MG_SSM_WHOLE) {
            f.channels = 1;
        } else {
            f.ck.n = ceil_div(MG_SSM_BLOCKS, blocks(2));
        }
    }
    const int64_t most = ceil_div(T, kMinChunk);
    f.ck.n = f.ck.n < most ? f.ck.n : most;
    f.ck.len = ceil_div(ceil_div(T, f.ck.n), kSeg) * kSeg;
    f.ck.n = ceil_div(T, f.ck.len);
    return f;
}

template <typename T, int VEC, typename CV>
mg_status fwd_cover(const SsmArgs &p, const Plan &f, cudaStream_t s)
{
    const Tile t{ceil_div(p.D / p.G, CV::kCh), p.D / p.G};
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    float *agg_h = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    float *agg_s = agg_h + p.B * (f.ck.n - 1) * p.D * p.N;
    const int64_t tiles = t.tiles * p.G * p.B;
    if (p.cu != nullptr) {
        const int64_t n = p.D * p.N;
        empty_sequences_kernel<<<unsigned(p.nseq < 1024 ? p.nseq : 1024), 256, 0, s>>>(
            q, p.h_last, p.h0, n, &static_cast<Control *>(p.ws)->error);
        MG_TRY(launched("mg_selective_scan_fwd"));
    }
    if (f.ck.n > 1) {
        ssm_chunk_kernel<T, VEC, CV, true><<<unsigned(tiles * (f.ck.n - 1)), kThreads, 0, s>>>(
            p, q, t, f.ck, agg_h, agg_s);
        MG_TRY(launched("mg_selective_scan_fwd"));
    }
    ssm_chunk_kernel<T, VEC, CV, false><<<unsigned(tiles * f.ck.n), kThreads, 0, s>>>(p, q, t, f.ck, agg_h, agg_s);
    return launched("mg_selective_scan_fwd");
}

template <typename T, int VEC, int S, int L>
mg_status fwd_lanes(const SsmArgs &p, cudaStream_t s)
{
    const Plan f = forward_plan(p.B, p.T, p.D, p.N, p.G);
    if (f.channels == 2) return fwd_cover<T, VEC, Cover<S, L, 2>>(p, f, s);
    return fwd_cover<T, VEC, Cover<S, L, 1>>(p, f, s);
}

template <typename T, int VEC>
mg_status fwd_vec(const SsmArgs &p, cudaStream_t s)
{
    if (p.N <= 8) return fwd_lanes<T, VEC, 4, 2>(p, s);
    switch (forward_lanes(p.N)) {
    case 2: return fwd_lanes<T, VEC, 8, 2>(p, s);
    case 4: return fwd_lanes<T, VEC, 8, 4>(p, s);
    default: return fwd_lanes<T, VEC, 8, 8>(p, s);
    }
}

// 16-byte vectors of x and raw where the rows and the groups' channels allow.
bool wide_rows(const SsmArgs &p, int vec)
{
    return p.D / p.G % vec == 0 && p.ldx % vec == 0 && p.ldraw % vec == 0;
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

size_t ssm_fwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t)
{
    const Plan f = forward_plan(B, T, D, N, G);
    return kControlBytes + sizeof(float) * B * (f.ck.n - 1) * D * (N + 1);
}

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

mg_status launch_ssm_fwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s)
{
    if (dt == MG_F32) return wide_rows(p, 4) ? fwd_vec<float, 4>(p, s) : fwd_vec<float, 1>(p, s);
    return wide_rows(p, 8) ? fwd_vec<bf16_t, 8>(p, s) : fwd_vec<bf16_t, 1>(p, s);
}
mg_status launch_ssm_bwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(bwd, p, dt, s) }
mg_status launch_ssm_step(const SsmStepArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(step, p, dt, s) }

}  // namespace mg
