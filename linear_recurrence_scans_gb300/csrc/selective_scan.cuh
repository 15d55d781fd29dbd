// Shared by the selective scan's kernels: pairs of floats, the decay, how
// threads cover channels and states, and how time is cut into chunks.
#pragma once

#include "ssm.cuh"

namespace mg {

constexpr int kSeg = 16;      // rows between two saved states: a tile of the gradients
constexpr int kTile = kSeg;
constexpr int kThreads = 128;
constexpr float kLn2 = 0.69314718f;

// A block's channels: a tile of one group.
struct Tile {
    int64_t tiles;    // tiles of a group
    int64_t width;    // channels of a group
};

// softplus of two values, from e = e^-|v| (as softplus_f).
__device__ __forceinline__ pair_t softplus2(pair_t v, float &e0, float &e1)
{
    float v0, v1;
    unpack2(v, v0, v1);
    e0 = exp_neg(-fabsf(v0));
    e1 = exp_neg(-fabsf(v1));
    const pair_t e = pack2(e0, e1);
    pair_t c = pack2(log1p_coef(9), log1p_coef(9));
#pragma unroll
    for (int i = 8; i >= 0; --i) c = fma2(c, e, pack2(log1p_coef(i), log1p_coef(i)));
    return fma2(e, c, pack2(fmaxf(v0, 0.f), fmaxf(v1, 0.f)));
}
__device__ __forceinline__ pair_t softplus2(pair_t v)
{
    float e0, e1;
    return softplus2(v, e0, e1);
}
// The same, and sigmoid of both.
__device__ __forceinline__ pair_t softplus2(pair_t v, pair_t &sig)
{
    float e0, e1, v0, v1;
    const pair_t d = softplus2(v, e0, e1);
    unpack2(v, v0, v1);
    const float r0 = rcp_fast(1.f + e0), r1 = rcp_fast(1.f + e1);
    sig = pack2(v0 >= 0.f ? r0 : e0 * r0, v1 >= 0.f ? r1 : e1 * r1);
    return d;
}

// The decay e^(delta A) = 2^(delta A log2 e) of two states.  ex2.approx comes
// out low by a relative 1.1e-8 on average for small exponents (measured), and
// a state that lives for 1 / (1 - a) rows would add that up; kDecayBias in
// the exponent, at no cost in the multiply-add, takes it out.  For larger
// exponents it is below their last bit, and the state is short-lived.
//
// The exponents are single multiply-adds on purpose: the SM reads registers
// for two operands of an instruction a clock, a multiply-add of three
// different registers runs at 2/3 rate (measured, pairs and singles alike),
// and a constant third operand is part of a single's instruction (26 against
// 29 clocks for the core of a warp's row).
constexpr float kDecayBias = 1.6e-8f;

__device__ __forceinline__ pair_t decay2(float d0, float d1, pair_t A2)
{
    float a, b;
    unpack2(A2, a, b);
    return pack2(ex2_ftz(fmaf(d0, a, kDecayBias)), ex2_ftz(fmaf(d1, b, kDecayBias)));
}
__device__ __forceinline__ pair_t decay2(pair_t d, pair_t A2)
{
    float d0, d1;
    unpack2(d, d0, d1);
    return decay2(d0, d1, A2);
}

// ------------------------------------------------------------ chunk geometry

// Time is cut into chunks of `len` rows (a multiple of kSeg), `n` of them for
// a batch entry; block -> (tile, chunk, entry), tiles fastest.
struct Chunks {
    int64_t len;
    int64_t n;
};

// How a warp covers channels: a thread has S states of C channels, L lanes a
// channel.
template <int S_, int L_, int C_, int THREADS_ = kThreads>
struct Cover {
    static constexpr int S = S_, L = L_, C = C_, THREADS = THREADS_;
    static constexpr int NP = S * L;                         // states with padding
    static constexpr int kGroups = 32 / L;                   // channel groups of a warp
    static constexpr int kWarpCh = kGroups * C;              // channels of a warp
    static constexpr int kCh = THREADS / 32 * kWarpCh;       // channels of a block
};

// Place of a row's (delta, u) of channel ch, as float2: they lie as float4 of
// two channels, and XORing the float4's index with its octet and the row
// spreads the staging writes (four consecutive float4 a lane, several rows an
// octet of lanes) over the banks; a row's reads stay within their octets.
template <int WCH>
__device__ __forceinline__ int du_index(int row, int ch)
{
    const int f = ch >> 1;
    const int x = WCH >= 32 ? ((f >> 3) & 1) | ((row & 1) << 1) : row & (WCH / 2 - 1) & 3;
    return (f ^ x) * 2 + (ch & 1);
}

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

// ------------------------------------------------- rows of any alignment
// A row segment of WCH channels that 16-byte copies do not fit arrives as
// 4-byte words from the one that holds its first value; with 2-byte values
// that value may be a word's upper half (the shift).
template <typename T, int WCH>
struct Words {
    static constexpr int kWords = sizeof(T) == 4 ? WCH : WCH / 2 + 1;
    static constexpr int kPitch = kWords * 4 / int(sizeof(T));   // values
};

// `bytes` (0, 2 or 4) of a 4-byte word, the rest zero.
__device__ __forceinline__ void cp_async4(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" : : "r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}

// (Loaded value by value where they are used instead, rows of 1001 bf16
// channels took 386 us where they now take 142, and their gradients 568 for
// 288: 2 x 4096 rows of 16 states.)
//
// Starts the copies of the words of ROWS row segments: row r's first channel
// is value first + r * ld of base, its channels `wide`, and rows from `rows`
// on are zero.  A word past the last channel's value is not read beyond it.
template <typename T, int WCH, int ROWS>
__device__ __forceinline__ void fetch_words(T (*dst)[Words<T, WCH>::kPitch], const T *base, int64_t first, int64_t ld,
                                            int rows, int wide, int lane)
{
    constexpr int kWords = Words<T, WCH>::kWords, kPer = (ROWS * kWords + 31) / 32;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int v = lane + i * 32, row = v / kWords, w = v % kWords;
        if (ROWS * kWords % 32 == 0 || v < ROWS * kWords) {
            const int64_t at = first + row * ld;
            const int shift = sizeof(T) == 4 ? 0 : int(at & 1), per = 4 / int(sizeof(T));
            const int c = w * per - shift;   // the word's first value, as a channel
            const int bytes = row >= rows || c >= wide ? 0 : c + per <= wide ? 4 : int(sizeof(T));
            cp_async4(reinterpret_cast<unsigned *>(dst[row]) + w, bytes > 0 ? base + at + c : base, bytes);
        }
    }
}

// How rows of B and C are read: value by value, by 4 bytes, by 16 bytes.
enum BcMode { kBcValues, kBcWords, kBcVectors };
template <typename T>
inline int bc_mode(int N, int64_t ldb, int64_t ldc)
{
    const int per16 = 16 / int(sizeof(T)), per4 = 4 / int(sizeof(T));
    if (N % per16 == 0 && ldb % per16 == 0 && ldc % per16 == 0) return kBcVectors;
    return N % per4 == 0 && ldb % per4 == 0 && ldc % per4 == 0 ? kBcWords : kBcValues;
}

// 16 bytes, or 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(void *dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" : : "r"(smem_addr(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}

// ---------------------------------------------------------- host side

constexpr int64_t kSms = 152;

// The time that an SM's blocks take for a row, by how many there are; more
// than the last go in turns.
struct RowTime {
    double ns[4];
    int most;   // blocks that an SM holds
    double first;   // the first pass's time as a part of the second's
    double of(int64_t blocks) const
    {
        const int64_t m = ceil_div(blocks, kSms), rest = m % most;
        return double(m / most) * ns[most] + ns[rest];
    }
};

constexpr int64_t kMinChunk = 32;   // rows
constexpr double kFoldNs = 500;      // a launch and a step of the fold over chunks

// Cuts T rows into chunks for `blocks` blocks a chunk, so that the two passes
// together take least: more chunks fill the SMs, and pay a first pass over
// all but the last of them.
inline Chunks cut_time(int64_t blocks, int64_t T, const RowTime &r)
{
    Chunks best{ceil_div(T, kSeg) * kSeg, 1};
    double least = double(T) * r.of(blocks);
    const int64_t most = ceil_div(T, kMinChunk);
    for (int64_t n = 2; n <= most && blocks * (n - 1) <= 4 * r.most * kSms; ++n) {
        Chunks ck;
        ck.len = ceil_div(ceil_div(T, n), kSeg) * kSeg;
        ck.n = ceil_div(T, ck.len);
        if (ck.n != n) continue;
        const double t = double(ck.len) * (r.of(blocks * n) + r.first * r.of(blocks * (n - 1))) + kFoldNs * double(n);
        if (t < least) {
            least = t;
            best = ck;
        }
    }
    return best;
}

// Packed batches: checks cu_seqlens, and gives empty sequences the state that
// they were given: dst[s] = src[s], or 0 (selective_scan.cu).
mg_status launch_empty_sequences(const Seqs &q, float *dst, const float *src, int64_t n, void *ws, cudaStream_t s);

// 16-byte vectors of x and raw where the rows and the groups' channels allow.
inline bool wide_rows(const SsmArgs &p, int vec)
{
    return p.D / p.G % vec == 0 && p.ldx % vec == 0 && p.ldraw % vec == 0;
}

// The gradients' first pass: q at the first row of chunks 1 .. ck.n-1, and
// each one's sum of delta, and its block count (selective_scan.cu).
int64_t adjoint_blocks(const SsmArgs &p, const Chunks &ck);
mg_status launch_ssm_adjoint(const SsmArgs &p, mg_dtype dt, bool wide, const Chunks &ck, float *agg_q,
                             float *agg_s, cudaStream_t s);

// The gradients by activation type (selective_scan_bwd_*.cu).
mg_status ssm_bwd_f32(const SsmArgs &p, bool wide, cudaStream_t s);
mg_status ssm_bwd_bf16(const SsmArgs &p, bool wide, cudaStream_t s);

}  // namespace mg
