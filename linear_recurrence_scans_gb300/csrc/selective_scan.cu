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
#ifndef MG_SSM_BWD_BLOCKS
#define MG_SSM_BWD_BLOCKS 608
#endif
#ifndef MG_SSM_BLOCKS
#define MG_SSM_BLOCKS 608
#endif

constexpr int kS = 4;         // states of a thread
constexpr int kSeg = 16;      // rows between two saved states: a tile of the gradients
constexpr int kThreads = 128;
constexpr float kLn2 = 0.69314718f;

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
template <int S_, int L_, int C_, int THREADS_ = kThreads>
struct Cover {
    static constexpr int S = S_, L = L_, C = C_, THREADS = THREADS_;
    static constexpr int NP = S * L;                       // states with padding
    static constexpr int kGroups = 32 / L;                 // channel groups of a warp
    static constexpr int kCh = THREADS / 32 * kGroups * C;   // channels of a block
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
            if constexpr (!kFirst) {
                if (p.h_last == nullptr) return;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (ch + c < wide)
                        store_pairs<S>(p.h_last + (int64_t(s) * p.D + d0 + ch + c) * p.N, n0, p.N, h[c]);
            }
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

// ---------------------------------------------------------------- gradients
//
// With g_r the adjoint of h_r and q_r = a_r g_r what it hands to row r - 1:
//   g_r = C_r dy_r + q_{r+1},   w_r = g_r a_r h_{r-1},
//   dC_r += dy_r h_r, dB_r += u_r g_r        (sums over the group's channels)
//   s1 = sum_n g_r B_r, s2 = sum_n w_r A     (sums over the channel's states)
//   dx_r = delta_r s1 + Dskip dy_r,  draw_r = (x_r s1 + s2) slope_r,  dA += delta_r w_r
// Chunks go backwards: a first pass leaves each chunk's q at its first row,
// started from 0 (from dh_last at a sequence's end), and its sum of delta; the
// second folds its successors' up to its sequence's end and does the rest.
//
// A chunk's tiles of kTile rows are worked on from the last to the first.  The
// forward saved the state before each tile.  From it one sweep leaves the
// states before every kSub rows in shared memory; then, kSub rows at a time
// from the last, the states are computed once more with a_r and a_r h_{r-1}
// kept in registers for the walk back.  (Kept in shared memory for a whole
// tile instead, they would ask for more of its bandwidth than the second
// computation takes of the arithmetic.)
//
// Four states of four channels are a thread's: the sums over channels (8
// values of dB and dC over the warp's channel lanes) and over states (8
// values of s1 and s2) then take 13 shuffles a row, fewer than any other
// split of 16, and are halved at each step.  Pairs are of neighbouring
// channels.
constexpr int kSub = 4;

// v over LANES lanes (bits STRIDE .. of the lane index; `id` is the lane's
// place among them): while there are several values, each lane hands half of
// them over.  V >= LANES: lane id ends with values id V/LANES .. of the sum in
// v[0 .. V/LANES - 1]; else with value id V / LANES.
template <int V, int LANES, int STRIDE>
__device__ __forceinline__ void halve_sum(float (&v)[V], int id)
{
    int w = V / 2;
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1, w >>= 1) {
        if (w > 0) {
            const bool up = (id & m) != 0;
#pragma unroll
            for (int i = 0; i < w; ++i) {
                const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
                v[i] = keep + __shfl_xor_sync(~0u, give, m * STRIDE);
            }
        } else {
            v[0] += __shfl_xor_sync(~0u, v[0], m * STRIDE);
        }
    }
}

// The block's place in the gradient passes.
template <int CH>
struct Spot {
    int64_t tile, k, b, rowb, t0, t1, d0, wide;
    int g;
    __device__ __forceinline__ Spot(const SsmArgs &p, const Tile &tl, const Chunks &ck, bool first)
    {
        const int64_t all_tiles = tl.tiles * p.G;
        const int64_t at = blockIdx.x % all_tiles, rest = blockIdx.x / all_tiles;
        const int64_t nch = first ? ck.n - 1 : ck.n;      // the first chunk has nothing before it
        k = rest % nch + (first ? 1 : 0);
        b = rest / nch;
        rowb = b * p.T;
        t0 = k * ck.len;
        t1 = t0 + ck.len < p.T ? t0 + ck.len : p.T;
        g = int(at / tl.tiles);
        tile = at % tl.tiles;
        d0 = g * tl.width + tile * CH;
        wide = tl.width - tile * CH < CH ? tl.width - tile * CH : CH;
    }
};

// The sequences at a tile's rows, found only for tiles that hold a first or
// last row of one: the sequence that row starts / ends there, or -1.
__device__ __forceinline__ void edge_rows(const Seqs &q, int64_t rowb, int64_t ta, int rows,
                                          int (&first)[kTile], int (&last)[kTile])
{
    const int i = threadIdx.x;
    if (i >= kTile) return;
    int f = -1, e = -1;
    if (i < rows) {
        const long long r = rowb + ta + i;
        const int s = q.of(r);
        if (q.begin(s) == r) f = s;
        if (q.begin(s + 1) == r + 1) e = s;
    }
    first[i] = f;
    last[i] = e;
}

// A thread's 4 x 4 states of float arrays (.., D, N), as channel pairs.
template <int S>
__device__ __forceinline__ void load_block(const float *base, int64_t d, int ch, int64_t wide, int n0,
                                           int N, pair_t (&o)[S][2])
{
    float v[4][S];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int i = 0; i < S; ++i) v[c][i] = 0.f;
        if (base != nullptr && ch + c < wide) load_group<S>(base + (d + c) * N, n0, N, v[c]);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
        o[i][0] = pack2(v[0][i], v[1][i]);
        o[i][1] = pack2(v[2][i], v[3][i]);
    }
}
template <int S>
__device__ __forceinline__ void store_block(float *base, int64_t d, int ch, int64_t wide, int n0, int N,
                                            const pair_t (&o)[S][2])
{
    float v[4][S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        unpack2(o[i][0], v[0][i], v[1][i]);
        unpack2(o[i][1], v[2][i], v[3][i]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (ch + c < wide) store_group<S>(base + (d + c) * N, n0, N, v[c]);
}

__device__ __forceinline__ pair_t dup2(float a) { return pack2(a, a); }

// First pass: q at the first row of chunks 1 .. n-1.
template <typename T, int VEC, typename CV>
__global__ void __launch_bounds__(CV::THREADS)
ssm_adjoint_chunk_kernel(SsmArgs p, Seqs q, Tile tl, Chunks ck, float *agg_q, float *agg_s)
{
    constexpr int S = CV::S, NP = CV::NP, CH = CV::kCh;
    constexpr int kVecs = kTile * CH / VEC, kPer = (kVecs + CV::THREADS - 1) / CV::THREADS;
    constexpr int kBc = (kTile * NP + CV::THREADS - 1) / CV::THREADS;
    __shared__ __align__(16) float s_d[kTile][CH], s_dy[kTile][CH], s_c[kTile][NP];
    __shared__ int s_last[kTile], s_first[kTile];
    const Spot<CH> w(p, tl, ck, true);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sl = lane / CV::kGroups, n0 = sl * S;
    const int ch = (warp * CV::kGroups + lane % CV::kGroups) * 4;
    pair_t A2[S][2], ag[S][2];
    load_block<S>(p.A, w.d0 + ch, ch, w.wide, n0, p.N, A2);
    float ssum[4] = {};
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            A2[i][c] = mul2(A2[i][c], dup2(kLog2eF));
            ag[i][c] = 0;
        }
    const T *rp = static_cast<const T *>(p.raw) + w.rowb * p.ldraw + w.d0;
    const T *yp = static_cast<const T *>(p.dy) + w.rowb * p.lddy + w.d0;
    const T *cp = static_cast<const T *>(p.Cm) + w.rowb * p.ldc + int64_t(w.g) * p.N;
    Raw<T, VEC> rr[kPer], yr[kPer];
    float cr[kBc];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = threadIdx.x + i * CV::THREADS;
            const int64_t row = t + v / (CH / VEC);
            const int col = v % (CH / VEC) * VEC;
            rr[i].fill(0.f);
            yr[i].fill(0.f);
            if (v < kVecs && row < w.t1 && col < w.wide) {
                rr[i].load(rp + row * p.ldraw + col);
                yr[i].load(yp + row * p.lddy + col);
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = threadIdx.x + i * CV::THREADS, n = e % NP;
            const int64_t row = t + e / NP;
            cr[i] = e < kTile * NP && row < w.t1 && n < p.N ? load1(cp + row * p.ldc + n) : 0.f;
        }
    };
    int64_t t = w.t0 + (w.t1 - 1 - w.t0) / kTile * kTile;
    int s = q.of(w.rowb + w.t1 - 1);
    long long lo = q.begin(s) - w.rowb, hi = q.begin(s + 1) - w.rowb;
    fetch(t);
    for (; t >= w.t0; t -= kTile) {
        const int64_t end = t + kTile < w.t1 ? t + kTile : w.t1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = threadIdx.x + i * CV::THREADS;
            const int row = v / (CH / VEC), col = v % (CH / VEC) * VEC;
            if (kVecs % CV::THREADS == 0 || v < kVecs) {
                const bool in = t + row < w.t1 && col < w.wide;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float bias = in && p.dt_bias != nullptr ? __ldg(p.dt_bias + w.d0 + col + e) : 0.f;
                    const float r = rr[i][e] + bias;
                    s_d[row][col + e] = !in ? 0.f : p.softplus ? softplus_f(r) : r;
                    s_dy[row][col + e] = yr[i][e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = threadIdx.x + i * CV::THREADS;
            if (kTile * NP % CV::THREADS == 0 || e < kTile * NP) s_c[e / NP][e % NP] = cr[i];
        }
        const bool edges = lo >= t || hi == end;
        if (edges) edge_rows(q, w.rowb, t, int(end - t), s_first, s_last);
        __syncthreads();
        if (t > w.t0) fetch(t - kTile);
#pragma unroll 4
        for (int tt = kTile - 1; tt >= 0; --tt) {
            if (edges && s_last[tt] >= 0) {
                load_block<S>(p.dh_last != nullptr ? p.dh_last + int64_t(s_last[tt]) * p.D * p.N : nullptr,
                              w.d0 + ch, ch, w.wide, n0, p.N, ag);
            }
            const float4 d4 = *reinterpret_cast<const float4 *>(&s_d[tt][ch]);
            const ulonglong2 y2 = *reinterpret_cast<const ulonglong2 *>(&s_dy[tt][ch]);
            const float4 c4 = *reinterpret_cast<const float4 *>(&s_c[tt][n0]);
            const pair_t dl[2] = {pack2(d4.x, d4.y), pack2(d4.z, d4.w)}, dy[2] = {y2.x, y2.y};
            const float cv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    ag[i][c] = mul2(decay2(dl[c], A2[i][c]), fma2(dup2(cv[i]), dy[c], ag[i][c]));
            ssum[0] += d4.x, ssum[1] += d4.y, ssum[2] += d4.z, ssum[3] += d4.w;
        }
        if (lo >= t && t > w.t0) {
            s = q.of(w.rowb + t - 1);
            lo = q.begin(s) - w.rowb;
        }
        hi = q.begin(s + 1) - w.rowb;
        __syncthreads();
    }
    const int64_t at = (w.b * (ck.n - 1) + w.k - 1) * p.D;
    store_block<S>(agg_q + at * p.N, w.d0 + ch, ch, w.wide, n0, p.N, ag);
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (sl == 0 && ch + c < w.wide) agg_s[at + w.d0 + ch + c] = ssum[c];
}

// Shared memory of the second pass.
template <typename T, int VEC, typename CV>
struct BwdShared {
    static constexpr int CH = CV::kCh, NP = CV::NP;
    static constexpr int kVecs = kTile * CH / VEC;
    float d[kTile][CH], x[kTile][CH], dy[kTile][CH], slope[kTile][CH];
    float s12[kTile][2 * CH];                      // (s1, s2) of each channel
    float b[kTile][NP], c[kTile][NP];
    float red[kTile][CV::THREADS / 32][2 * NP];       // each warp's dB, then dC
    float4 ck[kTile / kSub][4][CV::THREADS];          // states before each kSub rows, by thread
    float acc[2 * VEC][CV::THREADS];                  // each thread's dDskip and ddt_bias
    uint4 raw[VEC == 1 ? 1 : 3][VEC == 1 ? 1 : kVecs];   // the next tile's x, raw, dy as loaded
    int first[kTile], last[kTile];
};

template <typename T, int VEC, typename CV>
__global__ void __launch_bounds__(CV::THREADS, 2)
ssm_bwd_kernel(SsmArgs p, Seqs q, Tile tl, Chunks ck, const float *agg_q, const float *agg_s,
               float *partB, float *partA, float *partD)
{
    constexpr int S = CV::S, L = CV::L, NP = CV::NP, CH = CV::kCh;
    constexpr int kVecs = kTile * CH / VEC, kPer = (kVecs + CV::THREADS - 1) / CV::THREADS;
    constexpr int kBc = (kTile * NP + CV::THREADS - 1) / CV::THREADS;
    static_assert(S == 4, "four states a thread");
    extern __shared__ __align__(16) unsigned char shared_bytes[];
    BwdShared<T, VEC, CV> &sm = *reinterpret_cast<BwdShared<T, VEC, CV> *>(shared_bytes);
    const Spot<CH> w(p, tl, ck, false);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sl = lane / CV::kGroups, cg = lane % CV::kGroups, n0 = sl * S;
    const int ch = (warp * CV::kGroups + cg) * 4;
    const bool vec_n = p.N % 4 == 0;

    pair_t A2[S][2], ag[S][2], dA[S][2];
    load_block<S>(p.A, w.d0 + ch, ch, w.wide, n0, p.N, A2);
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            A2[i][c] = mul2(A2[i][c], dup2(kLog2eF));
            ag[i][c] = dA[i][c] = 0;
        }
#pragma unroll
    for (int e = 0; e < 2 * VEC; ++e) sm.acc[e][tid] = 0.f;

    int s = q.of(w.rowb + w.t1 - 1);
    long long lo = q.begin(s) - w.rowb, hi = q.begin(s + 1) - w.rowb;
    if (hi > w.t1) {   // the chunk's last sequence goes on: fold its later chunks
        int64_t j = ((hi < p.T ? hi : p.T) - 1) / ck.len;
        bool begin = true;
        for (; j > w.k; --j) {
            const int64_t at = (w.b * (ck.n - 1) + j - 1) * p.D;
            pair_t v[S][2];
            load_block<S>(agg_q + at * p.N, w.d0 + ch, ch, w.wide, n0, p.N, v);
            float ds[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) ds[c] = ch + c < w.wide ? agg_s[at + w.d0 + ch + c] : 0.f;
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    ag[i][c] = begin ? v[i][c]
                                     : fma2(decay2(pack2(ds[2 * c], ds[2 * c + 1]), A2[i][c]), ag[i][c], v[i][c]);
            begin = false;
        }
    }

    const T *xp = static_cast<const T *>(p.x) + w.rowb * p.ldx + w.d0;
    const T *rp = static_cast<const T *>(p.raw) + w.rowb * p.ldraw + w.d0;
    const T *yp = static_cast<const T *>(p.dy) + w.rowb * p.lddy + w.d0;
    const T *bp = static_cast<const T *>(p.Bm) + w.rowb * p.ldb + int64_t(w.g) * p.N;
    const T *cp = static_cast<const T *>(p.Cm) + w.rowb * p.ldc + int64_t(w.g) * p.N;
    const int64_t nseg = (p.T + kSeg - 1) / kSeg;
    float br[kBc], cr[kBc];
    // Starts the copies of a tile's x, raw and dy (each thread its vectors),
    // and loads its B and C.
    auto fetch = [&](int64_t t) {
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = tid + i * CV::THREADS;
                const int64_t row = t + v / (CH / VEC);
                const int col = v % (CH / VEC) * VEC;
                if (v < kVecs && row < w.t1 && col < w.wide) {
                    cp_async16(&sm.raw[0][v], xp + row * p.ldx + col);
                    cp_async16(&sm.raw[1][v], rp + row * p.ldraw + col);
                    cp_async16(&sm.raw[2][v], yp + row * p.lddy + col);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = tid + i * CV::THREADS, n = e % NP;
            const int64_t row = t + e / NP;
            const bool in = e < kTile * NP && row < w.t1 && n < p.N;
            br[i] = in ? load1(bp + row * p.ldb + n) : 0.f;
            cr[i] = in ? load1(cp + row * p.ldc + n) : 0.f;
        }
    };
    // The saved states before a tile, into the thread's first checkpoint.
    auto fetch_state = [&](int64_t t) {
        const float *o = p.saved_in + ((w.b * nseg + t / kSeg) * p.D + w.d0 + ch) * p.N;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float4 *to = &sm.ck[0][c][tid];
            if (ch + c >= w.wide || n0 >= p.N) {
                *to = make_float4(0.f, 0.f, 0.f, 0.f);
            } else if (vec_n) {
                cp_async16(to, o + c * p.N + n0);
            } else {
                float v[S];
                load_group<S>(o + c * p.N, n0, p.N, v);
                *to = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    };
    pair_t h[S][2];
    auto get_state = [&](int i) {
        const float4 a = sm.ck[i][0][tid], b = sm.ck[i][1][tid], c = sm.ck[i][2][tid], d = sm.ck[i][3][tid];
        h[0][0] = pack2(a.x, b.x), h[0][1] = pack2(c.x, d.x);
        h[1][0] = pack2(a.y, b.y), h[1][1] = pack2(c.y, d.y);
        h[2][0] = pack2(a.z, b.z), h[2][1] = pack2(c.z, d.z);
        h[3][0] = pack2(a.w, b.w), h[3][1] = pack2(c.w, d.w);
    };
    // (kept as channel pairs: [state pair][..] would do as well; a float4 a channel)
    auto put_state = [&](int i) {
        float a[4], b[4], c[4], d[4];
#pragma unroll
        for (int n = 0; n < S; ++n) {
            unpack2(h[n][0], a[n], b[n]);
            unpack2(h[n][1], c[n], d[n]);
        }
        sm.ck[i][0][tid] = make_float4(a[0], a[1], a[2], a[3]);
        sm.ck[i][1][tid] = make_float4(b[0], b[1], b[2], b[3]);
        sm.ck[i][2][tid] = make_float4(c[0], c[1], c[2], c[3]);
        sm.ck[i][3][tid] = make_float4(d[0], d[1], d[2], d[3]);
    };

    int64_t t = w.t0 + (w.t1 - 1 - w.t0) / kTile * kTile;
    fetch(t);
    fetch_state(t);
    cp_async_commit();
    for (; t >= w.t0; t -= kTile) {
        const int64_t end = t + kTile < w.t1 ? t + kTile : w.t1;
        cp_async_wait<0>();
        // the thread's vectors as float32: delta, x, dy and the slope of delta
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = tid + i * CV::THREADS;
            const int row = v / (CH / VEC), col = v % (CH / VEC) * VEC;
            if (kVecs % CV::THREADS == 0 || v < kVecs) {
                const bool in = t + row < w.t1 && col < w.wide;
                float xv[VEC], rv[VEC], yv[VEC], sv[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[e] = rv[e] = yv[e] = sv[e] = 0.f;
                if (in) {
                    if constexpr (VEC > 1) {
                        load_vec<VEC>(reinterpret_cast<const T *>(&sm.raw[0][v]), xv);
                        load_vec<VEC>(reinterpret_cast<const T *>(&sm.raw[1][v]), rv);
                        load_vec<VEC>(reinterpret_cast<const T *>(&sm.raw[2][v]), yv);
                    } else {
                        xv[0] = load1(xp + (t + row) * p.ldx + col);
                        rv[0] = load1(rp + (t + row) * p.ldraw + col);
                        yv[0] = load1(yp + (t + row) * p.lddy + col);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        if (p.dt_bias != nullptr) rv[e] += __ldg(p.dt_bias + w.d0 + col + e);
                        sv[e] = 1.f;
                        if (p.softplus) rv[e] = softplus_f(rv[e], sv[e]);
                    }
                }
                store_vec<VEC>(&sm.d[row][col], rv);
                store_vec<VEC>(&sm.x[row][col], xv);
                store_vec<VEC>(&sm.dy[row][col], yv);
                store_vec<VEC>(&sm.slope[row][col], sv);
            }
        }
#pragma unroll
        for (int i = 0; i < kBc; ++i) {
            const int e = tid + i * CV::THREADS;
            if (kTile * NP % CV::THREADS == 0 || e < kTile * NP) {
                sm.b[e / NP][e % NP] = br[i];
                sm.c[e / NP][e % NP] = cr[i];
            }
        }
        const bool edges = lo >= t || hi == end;
        if (edges) edge_rows(q, w.rowb, t, int(end - t), sm.first, sm.last);
        __syncthreads();
        if (t > w.t0) fetch(t - kTile);
        cp_async_commit();

        auto enter = [&](int tt) {   // a sequence's first row starts from its h0
            const int f = sm.first[tt];
            if (f >= 0)
                load_block<S>(p.h0 != nullptr ? p.h0 + int64_t(f) * p.D * p.N : nullptr, w.d0 + ch, ch,
                              w.wide, n0, p.N, h);
        };
        get_state(0);
#pragma unroll 1
        for (int sb = 1; sb < kTile / kSub; ++sb) {
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const int tt = (sb - 1) * kSub + i;
                if (edges) enter(tt);
                const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(&sm.d[tt][ch]);
                const ulonglong2 x2 = *reinterpret_cast<const ulonglong2 *>(&sm.x[tt][ch]);
                const float4 b4 = *reinterpret_cast<const float4 *>(&sm.b[tt][n0]);
                const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
                const pair_t dl[2] = {d2.x, d2.y}, u[2] = {mul2(d2.x, x2.x), mul2(d2.y, x2.y)};
#pragma unroll
                for (int n = 0; n < S; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        h[n][c] = fma2(decay2(dl[c], A2[n][c]), h[n][c], mul2(u[c], dup2(bv[n])));
            }
            put_state(sb);
        }
#pragma unroll 1
        for (int sb = kTile / kSub - 1; sb >= 0; --sb) {
            if (sb < kTile / kSub - 1) get_state(sb);
            if (sb == 0 && t > w.t0) {
                fetch_state(t - kTile);
                cp_async_commit();
            }
            pair_t a[kSub][S][2], ah[kSub][S][2];
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const int tt = sb * kSub + i;
                if (edges) enter(tt);
                const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(&sm.d[tt][ch]);
                const ulonglong2 x2 = *reinterpret_cast<const ulonglong2 *>(&sm.x[tt][ch]);
                const float4 b4 = *reinterpret_cast<const float4 *>(&sm.b[tt][n0]);
                const float bv[4] = {b4.x, b4.y, b4.z, b4.w};
                const pair_t dl[2] = {d2.x, d2.y}, u[2] = {mul2(d2.x, x2.x), mul2(d2.y, x2.y)};
#pragma unroll
                for (int n = 0; n < S; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        a[i][n][c] = decay2(dl[c], A2[n][c]);
                        ah[i][n][c] = mul2(a[i][n][c], h[n][c]);
                        h[n][c] = fma2(u[c], dup2(bv[n]), ah[i][n][c]);
                    }
            }
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
                const int tt = sb * kSub + i;
                if (edges && sm.last[tt] >= 0)
                    load_block<S>(p.dh_last != nullptr ? p.dh_last + int64_t(sm.last[tt]) * p.D * p.N : nullptr,
                                  w.d0 + ch, ch, w.wide, n0, p.N, ag);
                const ulonglong2 d2 = *reinterpret_cast<const ulonglong2 *>(&sm.d[tt][ch]);
                const ulonglong2 x2 = *reinterpret_cast<const ulonglong2 *>(&sm.x[tt][ch]);
                const ulonglong2 y2 = *reinterpret_cast<const ulonglong2 *>(&sm.dy[tt][ch]);
                const float4 b4 = *reinterpret_cast<const float4 *>(&sm.b[tt][n0]);
                const float4 c4 = *reinterpret_cast<const float4 *>(&sm.c[tt][n0]);
                const float bv[4] = {b4.x, b4.y, b4.z, b4.w}, cv[4] = {c4.x, c4.y, c4.z, c4.w};
                const pair_t dl[2] = {d2.x, d2.y}, dy[2] = {y2.x, y2.y};
                const pair_t u[2] = {mul2(d2.x, x2.x), mul2(d2.y, x2.y)};
                pair_t s1[2], s2[2];
                float bc[2 * S];
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    const pair_t bn = dup2(bv[n]), cn = dup2(cv[n]);
                    pair_t db = 0, dc = 0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const pair_t g = fma2(cn, dy[c], ag[n][c]);
                        const pair_t hh = fma2(u[c], bn, ah[i][n][c]);
                        dc = c == 0 ? mul2(dy[c], hh) : fma2(dy[c], hh, dc);
                        db = c == 0 ? mul2(u[c], g) : fma2(u[c], g, db);
                        s1[c] = n == 0 ? mul2(g, bn) : fma2(g, bn, s1[c]);
                        const pair_t wv = mul2(g, ah[i][n][c]);
                        s2[c] = n == 0 ? mul2(wv, A2[n][c]) : fma2(wv, A2[n][c], s2[c]);
                        dA[n][c] = fma2(wv, dl[c], dA[n][c]);
                        ag[n][c] = mul2(a[i][n][c], g);
                    }
                    float lo2, hi2;
                    unpack2(db, lo2, hi2);
                    bc[n] = lo2 + hi2;
                    unpack2(dc, lo2, hi2);
                    bc[S + n] = lo2 + hi2;
                }
                if (edges && p.dh0 != nullptr && sm.first[tt] >= 0)
                    store_block<S>(p.dh0 + int64_t(sm.first[tt]) * p.D * p.N, w.d0 + ch, ch, w.wide, n0, p.N, ag);
                // dB, dC over the warp's channel lanes
                constexpr int kG = CV::kGroups, kOut = 2 * S / kG > 0 ? 2 * S / kG : 1;
                halve_sum<2 * S, kG, 1>(bc, cg);
                if (kG <= 2 * S || cg % (kG / (2 * S) > 0 ? kG / (2 * S) : 1) == 0) {
                    const int v0 = kG <= 2 * S ? cg * kOut : cg / (kG / (2 * S) > 0 ? kG / (2 * S) : 1);
#pragma unroll
                    for (int o = 0; o < kOut; ++o)
                        sm.red[tt][warp][(v0 + o) / S * NP + n0 + (v0 + o) % S] = bc[o];
                }
                // s1, s2 over the channel's state lanes
                float sv[8];
                unpack2(s1[0], sv[0], sv[2]);
                unpack2(s1[1], sv[4], sv[6]);
                unpack2(s2[0], sv[1], sv[3]);
                unpack2(s2[1], sv[5], sv[7]);
                constexpr int kOs = 8 / L > 0 ? 8 / L : 1;
                halve_sum<8, L, kG>(sv, sl);
                if (L <= 8 || sl % (L / 8 > 0 ? L / 8 : 1) == 0) {
                    const int v0 = L <= 8 ? sl * kOs : sl / (L / 8 > 0 ? L / 8 : 1);
#pragma unroll
                    for (int o = 0; o < kOs; ++o) sm.s12[tt][2 * ch + v0 + o] = sv[o];
                }
            }
        }
        if (lo >= t && t > w.t0) {
            s = q.of(w.rowb + t - 1);
            lo = q.begin(s) - w.rowb;
        }
        hi = q.begin(s + 1) - w.rowb;
        __syncthreads();
        // outputs of the tile
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int v = tid + i * CV::THREADS;
            const int row = v / (CH / VEC), col = v % (CH / VEC) * VEC;
            if (v < kVecs && t + row < w.t1 && col < w.wide) {
                float dx[VEC], dr[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float s1 = sm.s12[row][2 * (col + e)], s2 = sm.s12[row][2 * (col + e) + 1] * kLn2;
                    const float dyv = sm.dy[row][col + e], xv = sm.x[row][col + e];
                    const float skip = p.Dskip != nullptr ? __ldg(p.Dskip + w.d0 + col + e) : 0.f;
                    dx[e] = fmaf(sm.d[row][col + e], s1, skip * dyv);
                    dr[e] = fmaf(xv, s1, s2) * sm.slope[row][col + e];
                    sm.acc[e][tid] = fmaf(dyv, xv, sm.acc[e][tid]);
                    sm.acc[VEC + e][tid] += dr[e];
                }
                const int64_t o = (w.rowb + t + row) * p.D + w.d0 + col;
                store_out<VEC>(static_cast<T *>(p.dx) + o, dx);
                store_out<VEC>(static_cast<T *>(p.draw) + o, dr);
            }
        }
        auto bc_sum = [&](int row, int v) {
            float a = sm.red[row][0][v];
#pragma unroll
            for (int k = 1; k < CV::THREADS / 32; ++k) a += sm.red[row][k][v];
            return a;
        };
        for (int i = tid; i < kTile * 2 * NP; i += CV::THREADS) {
            const int row = i / (2 * NP), v = i % (2 * NP), n = v % NP;
            if (n < p.N && t + row < w.t1)
                partB[((w.tile * q.rows + w.rowb + t + row) * p.G + w.g) * 2 * p.N + v / NP * p.N + n] =
                    bc_sum(row, v);
        }
    }
    const int64_t part = w.b * ck.n + w.k;
    store_block<S>(partA + part * p.D * p.N, w.d0 + ch, ch, w.wide, n0, p.N, dA);
    // dDskip and ddt_bias: the threads of a column, in order
    __syncthreads();
    if (tid < CH / VEC && tid * VEC < w.wide) {
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) {
            float v = 0.f;
            for (int i = tid; i < CV::THREADS; i += CH / VEC) v += sm.acc[e][i];
            partD[(part * 2 + e / VEC) * p.D + w.d0 + tid * VEC + e % VEC] = v;
        }
    }
}

// dB and dC from the tiles' parts, in order: part (tile, row, group, dB or
// dC, N).
template <typename T>
__global__ void __launch_bounds__(256) sum_bc_kernel(const float *part, int64_t tiles, int64_t rows_g,
                                                     int N, T *dB, T *dC)
{
    const int64_t n = rows_g * 2 * N, i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float a = 0.f;
    for (int64_t t = 0; t < tiles; ++t) a += part[t * n + i];
    const int64_t rg = i / (2 * N);
    const int v = int(i - rg * 2 * N);
    T *o = v < N ? dB : dC;
    store1(o + rg * N + (v < N ? v : v - N), a);
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

// The gradients' chunks: four channels a thread, two blocks for each SM.
int backward_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
// Threads of a block: shared memory holds the tiles of 128 channels.
constexpr int backward_threads(int L) { return L == 1 ? 32 : L == 2 ? 64 : kThreads; }
int64_t backward_tiles(int64_t D, int N, int G)
{
    const int L = backward_lanes(N);
    return ceil_div(D / G, backward_threads(L) / L * 4);
}

Chunks backward_chunks(int64_t B, int64_t T, int64_t D, int N, int G)
{
    const int64_t blocks = B * G * backward_tiles(D, N, G);
    Chunks ck;
    ck.n = ceil_div(MG_SSM_BWD_BLOCKS, blocks);
    const int64_t most = ceil_div(T, kMinChunk);
    ck.n = ck.n < most ? ck.n : most;
    ck.len = ceil_div(ceil_div(T, ck.n), kSeg) * kSeg;
    ck.n = ceil_div(T, ck.len);
    return ck;
}

template <typename T, int VEC, int L>
mg_status bwd(const SsmArgs &p, cudaStream_t s)
{
    using CV = Cover<4, L, 4, backward_threads(L)>;
    const Tile t{backward_tiles(p.D, p.N, p.G), p.D / p.G};
    const Chunks ck = backward_chunks(p.B, p.T, p.D, p.N, p.G);
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const int64_t rows_g = q.rows * p.G, dn = p.D * p.N, parts = p.B * ck.n;
    float *partB = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    float *partA = partB + t.tiles * rows_g * 2 * p.N;
    float *partD = partA + parts * dn;
    float *agg_q = partD + parts * 2 * p.D;
    float *agg_s = agg_q + p.B * (ck.n - 1) * dn;
    const int64_t tiles = t.tiles * p.G * p.B;
    if (p.cu != nullptr) {
        empty_sequences_kernel<<<unsigned(p.nseq < 1024 ? p.nseq : 1024), 256, 0, s>>>(
            q, p.dh0, p.dh_last, dn, &static_cast<Control *>(p.ws)->error);
        MG_TRY(launched("mg_selective_scan_bwd"));
    }
    if (ck.n > 1) {
        ssm_adjoint_chunk_kernel<T, VEC, CV><<<unsigned(tiles * (ck.n - 1)), CV::THREADS, 0, s>>>(
            p, q, t, ck, agg_q, agg_s);
        MG_TRY(launched("mg_selective_scan_bwd"));
    }
    constexpr size_t smem = sizeof(BwdShared<T, VEC, CV>);
    static_assert(smem <= 227 * 1024, "shared memory of a block");
    const cudaError_t e = cudaFuncSetAttribute(ssm_bwd_kernel<T, VEC, CV>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return fail(MG_ERR_LAUNCH, "mg_selective_scan_bwd: %s", cudaGetErrorString(e));
    ssm_bwd_kernel<T, VEC, CV><<<unsigned(tiles * ck.n), CV::THREADS, smem, s>>>(p, q, t, ck, agg_q, agg_s, partB,
                                                                             partA, partD);
    MG_TRY(launched("mg_selective_scan_bwd"));
    sum_bc_kernel<T><<<unsigned(ceil_div(rows_g * 2 * p.N, 256)), 256, 0, s>>>(
        partB, t.tiles, rows_g, p.N, static_cast<T *>(p.dBm), static_cast<T *>(p.dCm));
    MG_TRY(launched("mg_selective_scan_bwd"));
    MG_TRY(launch_sum_parts(partA, parts, dn, dn, p.dA, s));
    if (p.dDskip != nullptr) MG_TRY(launch_sum_parts(partD, parts, 2 * p.D, p.D, p.dDskip, s));
    if (p.ddt_bias != nullptr)
        MG_TRY(launch_sum_parts(partD + p.D, parts, 2 * p.D, p.D, p.ddt_bias, s));
    return MG_OK;
}

template <typename T, int VEC>
mg_status bwd_vec(const SsmArgs &p, cudaStream_t s)
{
    switch (backward_lanes(p.N)) {
    case 1: return bwd<T, VEC, 1>(p, s);
    case 2: return bwd<T, VEC, 2>(p, s);
    case 4: return bwd<T, VEC, 4>(p, s);
    case 8: return bwd<T, VEC, 8>(p, s);
    default: return bwd<T, VEC, 16>(p, s);
    }
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

size_t ssm_bwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t)
{
    const Chunks ck = backward_chunks(B, T, D, N, G);
    return kControlBytes +
           sizeof(float) * (backward_tiles(D, N, G) * B * T * G * 2 * N + B * ck.n * (D * N + 2 * D) +
                            B * (ck.n - 1) * (D * N + D));
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
mg_status launch_ssm_bwd(const SsmArgs &p, mg_dtype dt, cudaStream_t s)
{
    const int vec = dt == MG_F32 ? 4 : 8;
    const bool wide = wide_rows(p, vec) && p.lddy % vec == 0;
    if (dt == MG_F32) return wide ? bwd_vec<float, 4>(p, s) : bwd_vec<float, 1>(p, s);
    return wide ? bwd_vec<bf16_t, 8>(p, s) : bwd_vec<bf16_t, 1>(p, s);
}
mg_status launch_ssm_step(const SsmStepArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(step, p, dt, s) }

}  // namespace mg
