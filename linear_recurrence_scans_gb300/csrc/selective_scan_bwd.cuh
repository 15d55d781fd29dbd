// The selective scan's gradients (see selective_scan.cu for the recurrence):
// kernels and launchers, instantiated by activation type in
// selective_scan_bwd_*.cu.
#pragma once

#include <type_traits>

#include "selective_scan.cuh"

namespace mg {

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
// Four states of four channels are a thread's (of two, up to 8 states): the
// sums over channels (8 values of dB and dC over the warp's channel lanes) and
// over states (s1 and s2 of its channels) then take 13 shuffles a row, fewer
// than any other split of 16 states, and are halved at each step.  Pairs are of
// neighbouring channels.  The lane that a channel's s1 and s2 end at writes its
// dx and draw and sums its dDskip and ddt_bias.  Each warp stages its own
// channels, the block its B and C (staged by every warp for itself they took
// shared memory for a second block: 2 x 4096 x 1024 channels of 64 states 1246
// -> 838 us); the block's warps meet once a tile to add their dB and dC.
//
// 4 x 4096 x 2048 channels of 16 states take 775 us, 0.69e12 states a second:
// 120 for the first pass, 616 here and 18 for the sums of the parts.
// Instructions bound it: 23 a state (10 of them the formulas', each state's
// exponential taken twice), at half the issue slots with two warps a
// scheduler, which is what the registers of kSub rows leave.  (B and C kept
// twice over as ready pairs: 847 us; u staged next to x: no change.)
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

// The block's place.
template <int CH>
struct Spot {
    int64_t tile, k, b, rowb, t0, t1, d0, wide;
    int g;
    __device__ __forceinline__ Spot(const SsmArgs &p, const Tile &tl, const Chunks &ck)
    {
        const int64_t all_tiles = tl.tiles * p.G;
        const int64_t at = blockIdx.x % all_tiles, rest = blockIdx.x / all_tiles;
        k = rest % ck.n;
        b = rest / ck.n;
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
// last row of one: the sequence that row starts / ends there, or -1.  Rows past
// the batch's end start from 0 (kNoRow): an infinite last state times their
// adjoints of 0 would make dA NaN.
constexpr int kNoRow = -2;
__device__ __forceinline__ void edge_rows(const Seqs &q, int64_t rowb, int64_t ta, int rows,
                                          int (&first)[kTile], int (&last)[kTile])
{
    const int i = threadIdx.x;
    if (i >= kTile) return;
    int f = i < rows ? -1 : kNoRow, e = -1;
    if (i < rows) {
        const long long r = rowb + ta + i;
        const int s = q.of(r);
        if (q.begin(s) == r) f = s;
        if (q.begin(s + 1) == r + 1) e = s;
    }
    first[i] = f;
    last[i] = e;
}

// A thread's states of 2 CP channels of float arrays (.., D, N), as channel
// pairs.
template <int S, int CP>
__device__ __forceinline__ void load_block(const float *base, int64_t d, int ch, int64_t wide, int n0,
                                           int N, pair_t (&o)[S][CP])
{
    float v[2 * CP][S];
#pragma unroll
    for (int c = 0; c < 2 * CP; ++c) {
#pragma unroll
        for (int i = 0; i < S; ++i) v[c][i] = 0.f;
        if (base != nullptr && ch + c < wide) load_group<S>(base + (d + c) * N, n0, N, v[c]);
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int c = 0; c < CP; ++c) o[i][c] = pack2(v[2 * c][i], v[2 * c + 1][i]);
}
template <int S, int CP>
__device__ __forceinline__ void store_block(float *base, int64_t d, int ch, int64_t wide, int n0, int N,
                                            const pair_t (&o)[S][CP])
{
    float v[2 * CP][S];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int c = 0; c < CP; ++c) unpack2(o[i][c], v[2 * c][i], v[2 * c + 1][i]);
#pragma unroll
    for (int c = 0; c < 2 * CP; ++c)
        if (ch + c < wide) store_group<S>(base + (d + c) * N, n0, N, v[c]);
}
// A row's values of a thread's channels in shared memory.
template <int CP>
__device__ __forceinline__ void load_pairs(const float *from, pair_t (&o)[CP])
{
    if constexpr (CP == 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(from);
        o[0] = v.x, o[1] = v.y;
    } else {
        o[0] = *reinterpret_cast<const pair_t *>(from);
    }
}

__device__ __forceinline__ pair_t dup2(float a) { return pack2(a, a); }

// s1 and s2 of V channels over LANES lanes (bits STRIDE ..): lane id ends
// with the sums of channels id V/LANES .. (or id / (LANES/V)) in a[0], b[0], ..
template <int LANES, int STRIDE, int V>
__device__ __forceinline__ void halve_channels(float (&a)[V], float (&b)[V], int id)
{
    int w = V / 2;
#pragma unroll
    for (int m = LANES / 2; m > 0; m >>= 1, w >>= 1) {
        if (w > 0) {
            const bool up = (id & m) != 0;
#pragma unroll
            for (int i = 0; i < w; ++i) {
                const float ka = up ? a[i + w] : a[i], ga = up ? a[i] : a[i + w];
                const float kb = up ? b[i + w] : b[i], gb = up ? b[i] : b[i + w];
                a[i] = ka + __shfl_xor_sync(~0u, ga, m * STRIDE);
                b[i] = kb + __shfl_xor_sync(~0u, gb, m * STRIDE);
            }
        } else {
            a[0] += __shfl_xor_sync(~0u, a[0], m * STRIDE);
            b[0] += __shfl_xor_sync(~0u, b[0], m * STRIDE);
        }
    }
}

// Shared memory of the second pass: a warp's, and the block's.
template <typename T, int VEC, typename CV>
struct BwdWarp {
    static constexpr int WCH = CV::kWarpCh, NP = CV::NP;
    float d[kTile][WCH], x[kTile][WCH], dy[kTile][WCH], slope[kTile][WCH];
    float4 ck[kTile / kSub][CV::C][32];                // states before each kSub rows, by lane
    float bias[WCH];
    T raw[3][kTile][VEC > 1 ? WCH : Words<T, WCH>::kPitch];   // the next tile's x, raw, dy as loaded
};
template <typename T, int VEC, typename CV>
struct alignas(16) BwdShared {
    BwdWarp<T, VEC, CV> warp[CV::THREADS / 32];
    float bc[kTile][2][CV::NP];                       // the tile's B and C
    alignas(16) T rawbc[kTile][2][CV::NP];            // the next tile's as loaded
    float red[kTile][CV::THREADS / 32][2 * CV::NP];   // each warp's dB, then dC
    int first[kTile], last[kTile];
};

// Blocks that share an SM.
template <typename CV>
constexpr int backward_blocks() { return (CV::C == 2 ? 3 : 2) * (kThreads / CV::THREADS); }

template <typename T, int VEC, typename CV>
__global__ void __launch_bounds__(CV::THREADS, backward_blocks<CV>())
ssm_bwd_kernel(SsmArgs p, Seqs q, Tile tl, Chunks ck, const float *agg_q, const float *agg_s,
               float *partB, float *partA, int mode)
{
    constexpr int S = CV::S, L = CV::L, C = CV::C, CP = C / 2, NP = CV::NP, CH = CV::kCh, WCH = CV::kWarpCh, kWarps = CV::THREADS / 32;
    constexpr int kCols = WCH / VEC, kVecs = kTile * kCols, kPer = (kVecs + 31) / 32;
    constexpr int kCv = NP < 16 / int(sizeof(T)) ? NP : 16 / int(sizeof(T));   // values of a vector of B or C
    constexpr int kBcCols = NP / kCv, kBcVecs = kTile * 2 * kBcCols, kBcPer = (kBcVecs + CV::THREADS - 1) / CV::THREADS;
    constexpr int kG = CV::kGroups;
    static_assert(S == 4 && (C == 2 || C == 4), "four states of two or four channels a thread");
    extern __shared__ __align__(16) unsigned char shared_bytes[];
    BwdShared<T, VEC, CV> &block = *reinterpret_cast<BwdShared<T, VEC, CV> *>(shared_bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    BwdWarp<T, VEC, CV> &sm = block.warp[warp];
    const Spot<CH> w(p, tl, ck);
    const int sl = lane / kG, cg = lane % kG, n0 = sl * S;
    const int ch = cg * C;                                       // of the warp's channels
    const int64_t dw = w.d0 + warp * WCH;                        // the warp's first channel
    const int wide = int(w.wide - warp * WCH < WCH ? w.wide - warp * WCH : WCH);   // its channels (may be <= 0)
    const bool vec_n = p.N % 4 == 0;

    pair_t A2[S][CP], ag[S][CP], dA[S][CP];
    load_block<S, CP>(p.A, dw + ch, ch, wide, n0, p.N, A2);
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            // (a padded state's A is -1: with 0 an infinite delta would make its decay NaN, and with it s1)
            A2[i][c] = n0 + i < p.N ? mul2(A2[i][c], dup2(kLog2eF)) : dup2(-1.f);
            ag[i][c] = dA[i][c] = 0;
        }
    for (int i = lane; i < WCH; i += 32)
        sm.bias[i] = p.dt_bias != nullptr && i < wide ? p.dt_bias[dw + i] : 0.f;
    // the channels whose outputs are this lane's (lanes that share one: the first writes)
    constexpr int kOut = L <= C ? C / L : 1, kSame = L > C ? L / C : 1;
    const int oc = ch + (L <= C ? sl * kOut : sl / kSame);
    const bool writes = sl % kSame == 0;
    float skip[kOut], sum_d[kOut], sum_b[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
        skip[o] = p.Dskip != nullptr && oc + o < wide ? p.Dskip[dw + oc + o] : 0.f;
        sum_d[o] = sum_b[o] = 0.f;
    }

    int s = q.of(w.rowb + w.t1 - 1);
    long long lo = q.begin(s) - w.rowb, hi = q.begin(s + 1) - w.rowb;
    const T *x0p = static_cast<const T *>(p.x), *r0p = static_cast<const T *>(p.raw), *y0p = static_cast<const T *>(p.dy);
    const int64_t xf = w.rowb * p.ldx + dw, rf = w.rowb * p.ldraw + dw, yf = w.rowb * p.lddy + dw;
    const T *xp = x0p + xf, *rp = r0p + rf, *yp = y0p + yf;
    const T *bp = static_cast<const T *>(p.Bm) + w.rowb * p.ldb + int64_t(w.g) * p.N;
    const T *cp = static_cast<const T *>(p.Cm) + w.rowb * p.ldc + int64_t(w.g) * p.N;
    const int64_t nseg = (p.T + kSeg - 1) / kSeg;
    // Starts the copies of a tile's x, raw, dy, B and C: each lane its vectors.
    auto fetch = [&](int64_t t) {
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = lane + i * 32, row = v / kCols, col = v % kCols * VEC;
                if (v < kVecs && col < wide && t + row < w.t1) {
                    cp_async16(&sm.raw[0][row][col], xp + (t + row) * p.ldx + col);
                    cp_async16(&sm.raw[1][row][col], rp + (t + row) * p.ldraw + col);
                    cp_async16(&sm.raw[2][row][col], yp + (t + row) * p.lddy + col);
                }
            }
        } else {
            const int rows = wide > 0 ? int(w.t1 - t < kTile ? w.t1 - t : kTile) : 0;
            fetch_words<T, WCH, kTile>(sm.raw[0], x0p, xf + t * p.ldx, p.ldx, rows, wide, lane);
            fetch_words<T, WCH, kTile>(sm.raw[1], r0p, rf + t * p.ldraw, p.ldraw, rows, wide, lane);
            fetch_words<T, WCH, kTile>(sm.raw[2], y0p, yf + t * p.lddy, p.lddy, rows, wide, lane);
        }
        if (mode == kBcValues) return;
#pragma unroll
        for (int i = 0; i < kBcPer; ++i) {
            const int v = tid + i * CV::THREADS, n = v % kBcCols * kCv, which = v / kBcCols % 2, row = v / kBcCols / 2;
            if (v >= kBcVecs) continue;
            const bool in = t + row < w.t1;
            const T *src = which == 0 ? bp + (t + row) * p.ldb + n : cp + (t + row) * p.ldc + n;
            T *to = &block.rawbc[row][which][n];
            if (kCv * sizeof(T) == 16 && mode == kBcVectors) {
                cp_async16_or_zero(to, in && n < p.N ? static_cast<const void *>(src) : p.Bm, in && n < p.N);
            } else {
                constexpr int kPer4 = 4 / int(sizeof(T));
#pragma unroll
                for (int e = 0; e < kCv; e += kPer4) {
                    const bool ok = in && n + e < p.N;
                    cp_async4(to + e, ok ? static_cast<const void *>(src + e) : p.Bm, ok ? 4 : 0);
                }
            }
        }
    };
    // The saved states before a tile, into the lane's first checkpoint.
    auto fetch_state = [&](int64_t t) {
        const float *o = p.saved_in + ((w.b * nseg + t / kSeg) * p.D + dw + ch) * p.N;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float4 *to = &sm.ck[0][c][lane];
            if (ch + c >= wide || n0 >= p.N) {
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
    pair_t h[S][CP];
    auto get_state = [&](int i) {
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            const float4 a = sm.ck[i][2 * c][lane], b = sm.ck[i][2 * c + 1][lane];
            h[0][c] = pack2(a.x, b.x), h[1][c] = pack2(a.y, b.y);
            h[2][c] = pack2(a.z, b.z), h[3][c] = pack2(a.w, b.w);
        }
    };
    auto put_state = [&](int i) {
#pragma unroll
        for (int c = 0; c < CP; ++c) {
            float4 a, b;
            unpack2(h[0][c], a.x, b.x), unpack2(h[1][c], a.y, b.y);
            unpack2(h[2][c], a.z, b.z), unpack2(h[3][c], a.w, b.w);
            sm.ck[i][2 * c][lane] = a;
            sm.ck[i][2 * c + 1][lane] = b;
        }
    };

    // A staged row's values for the thread: delta and u = delta x of its
    // channel pairs, and B of its states.
    auto row_in = [&](int tt, pair_t (&dl)[CP], pair_t (&u)[CP], float (&bv)[4]) {
        pair_t x[CP];
        load_pairs<CP>(&sm.d[tt][ch], dl);
        load_pairs<CP>(&sm.x[tt][ch], x);
        const float4 b4 = *reinterpret_cast<const float4 *>(&block.bc[tt][0][n0]);
#pragma unroll
        for (int c = 0; c < CP; ++c) u[c] = mul2(dl[c], x[c]);
        bv[0] = b4.x, bv[1] = b4.y, bv[2] = b4.z, bv[3] = b4.w;
    };

    // One tile; kEdges: it holds a sequence's first or last row.
    auto tile = [&](int64_t t, auto edges) {
        constexpr bool kEdges = decltype(edges)::value;
        auto enter = [&](int tt) {   // a sequence's first row starts from its h0
            if constexpr (kEdges) {
                const int f = block.first[tt];
                if (f != -1)
                    load_block<S, CP>(f >= 0 && p.h0 != nullptr ? p.h0 + int64_t(f) * p.D * p.N : nullptr, dw + ch, ch,
                                      wide, n0, p.N, h);
            }
        };
        const int rows = int(w.t1 - t);
        int64_t out = (w.rowb + t + kTile - 1) * p.D + dw + oc;   // of the row at hand, from the last
        get_state(0);
#pragma unroll 1
        for (int sb = 1; sb < kTile / kSub; ++sb) {
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const int tt = (sb - 1) * kSub + i;
                enter(tt);
                pair_t dl[CP], u[CP];
                float bv[4];
                row_in(tt, dl, u, bv);
#pragma unroll
                for (int n = 0; n < S; ++n)
#pragma unroll
                    for (int c = 0; c < CP; ++c)
                        h[n][c] = fma2(decay2(dl[c], A2[n][c]), h[n][c], mul2(u[c], dup2(bv[n])));
            }
            put_state(sb);
        }
#pragma unroll 1
        for (int sb = kTile / kSub - 1; sb >= 0; --sb) {
            if (sb < kTile / kSub - 1) get_state(sb);
            if (sb == 0) {
                if (t > w.t0) fetch_state(t - kTile);
                cp_async_commit();
            }
            pair_t a[kSub][S][CP], ah[kSub][S][CP];
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const int tt = sb * kSub + i;
                enter(tt);
                pair_t dl[CP], u[CP];
                float bv[4];
                row_in(tt, dl, u, bv);
#pragma unroll
                for (int n = 0; n < S; ++n)
#pragma unroll
                    for (int c = 0; c < CP; ++c) {
                        a[i][n][c] = decay2(dl[c], A2[n][c]);
                        ah[i][n][c] = mul2(a[i][n][c], h[n][c]);
                        h[n][c] = fma2(u[c], dup2(bv[n]), ah[i][n][c]);
                    }
            }
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
                const int tt = sb * kSub + i;
                if constexpr (kEdges) {
                    if (block.last[tt] >= 0)
                        load_block<S, CP>(p.dh_last != nullptr ? p.dh_last + int64_t(block.last[tt]) * p.D * p.N : nullptr,
                                      dw + ch, ch, wide, n0, p.N, ag);
                }
                pair_t dl[CP], u[CP];
                float bv[4];
                row_in(tt, dl, u, bv);
                pair_t dy[CP], s1[CP], s2[CP];
                load_pairs<CP>(&sm.dy[tt][ch], dy);
                const float4 c4 = *reinterpret_cast<const float4 *>(&block.bc[tt][1][n0]);
                const float cv[4] = {c4.x, c4.y, c4.z, c4.w};
                float bc[2 * S];
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    const pair_t bn = dup2(bv[n]), cn = dup2(cv[n]);
                    pair_t db = 0, dc = 0;
#pragma unroll
                    for (int c = 0; c < CP; ++c) {
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
                if constexpr (kEdges) {
                    if (p.dh0 != nullptr && block.first[tt] >= 0)
                        store_block<S, CP>(p.dh0 + int64_t(block.first[tt]) * p.D * p.N, dw + ch, ch, wide, n0, p.N, ag);
                }
                // dB, dC over the warp's channel lanes
                constexpr int kBcOut = 2 * S / kG > 0 ? 2 * S / kG : 1, kShare = kG / (2 * S) > 0 ? kG / (2 * S) : 1;
                halve_sum<2 * S, kG, 1>(bc, cg);
                if (cg % kShare == 0) {
                    const int v0 = cg / kShare * kBcOut;
#pragma unroll
                    for (int o = 0; o < kBcOut; ++o)
                        block.red[tt][warp][(v0 + o) / S * NP + n0 + (v0 + o) % S] = bc[o];
                }
                // s1, s2 over the channel's state lanes, and the outputs
                float s1v[C], s2v[C];
#pragma unroll
                for (int c = 0; c < CP; ++c) {
                    unpack2(s1[c], s1v[2 * c], s1v[2 * c + 1]);
                    unpack2(s2[c], s2v[2 * c], s2v[2 * c + 1]);
                }
                halve_channels<L, kG>(s1v, s2v, sl);
#pragma unroll
                for (int o = 0; o < kOut; ++o) {
                    const float xv = sm.x[tt][oc + o], dyv = sm.dy[tt][oc + o];
                    const float dx = fmaf(sm.d[tt][oc + o], s1v[o], skip[o] * dyv);
                    const float dr = fmaf(xv, s1v[o], s2v[o] * kLn2) * sm.slope[tt][oc + o];
                    sum_d[o] = fmaf(dyv, xv, sum_d[o]);
                    sum_b[o] += dr;
                    if (writes && tt < rows && oc + o < wide) {
                        store1(static_cast<T *>(p.dx) + out + o, dx);
                        store1(static_cast<T *>(p.draw) + out + o, dr);
                    }
                }
                out -= p.D;
            }
        }
    };

    int64_t t = w.t0 + (w.t1 - 1 - w.t0) / kTile * kTile;
    fetch(t);
    fetch_state(t);
    cp_async_commit();
    after_previous();   // the chunks' states
    if (hi > w.t1) {   // the chunk's last sequence goes on: fold its later chunks
        int64_t j = ((hi < p.T ? hi : p.T) - 1) / ck.len;
        bool begin = true;
        for (; j > w.k; --j) {
            const int64_t at = (w.b * (ck.n - 1) + j - 1) * p.D;
            pair_t v[S][CP];
            load_block<S, CP>(agg_q + at * p.N, dw + ch, ch, wide, n0, p.N, v);
            float ds[C];
#pragma unroll
            for (int c = 0; c < C; ++c) ds[c] = ch + c < wide ? agg_s[at + dw + ch + c] : 0.f;
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int c = 0; c < CP; ++c)
                    ag[i][c] = begin ? v[i][c]
                                     : fma2(decay2(ds[2 * c], ds[2 * c + 1], A2[i][c]), ag[i][c], v[i][c]);
            begin = false;
        }
    }
    for (; t >= w.t0; t -= kTile) {
        const int64_t end = t + kTile < w.t1 ? t + kTile : w.t1;
        cp_async_wait<0>();
        __syncwarp();
        // the lane's vectors as float32: delta, x, dy and the slope of delta
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = lane + i * 32, row = v / kCols, col = v % kCols * VEC;
                if (v < kVecs) {
                    float xv[VEC], rv[VEC], yv[VEC], sv[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) xv[e] = rv[e] = yv[e] = sv[e] = 0.f;
                    if (col < wide && t + row < w.t1) {
                        float bias[VEC];
                        load_vec<VEC>(&sm.bias[col], bias);
                        load_vec<VEC>(&sm.raw[0][row][col], xv);
                        load_vec<VEC>(&sm.raw[1][row][col], rv);
                        load_vec<VEC>(&sm.raw[2][row][col], yv);
#pragma unroll
                        for (int e = 0; e < VEC; e += 2) {
                            pair_t sg;
                            const pair_t r = add2(pack2(rv[e], rv[e + 1]), pack2(bias[e], bias[e + 1]));
                            const pair_t sp = softplus2(r, sg);
                            unpack2(p.softplus ? sp : r, rv[e], rv[e + 1]);
                            unpack2(p.softplus ? sg : dup2(1.f), sv[e], sv[e + 1]);
                        }
                    }
                    store_vec<VEC>(&sm.d[row][col], rv);
                    store_vec<VEC>(&sm.x[row][col], xv);
                    store_vec<VEC>(&sm.dy[row][col], yv);
                    store_vec<VEC>(&sm.slope[row][col], sv);
                }
            }
        } else {   // single values, two at a time
            static_assert(VEC > 1 || (kVecs % 64 == 0 && kPer % 2 == 0), "pairs");
#pragma unroll 2
            for (int i = 0; i < kPer; i += 2) {
                float xv[2], rv[2], yv[2], sv[2], bias[2];
                bool in[2];
                int row[2], col[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int v = lane + (i + e) * 32;
                    row[e] = v / kCols, col[e] = v % kCols;
                    in[e] = col[e] < wide && t + row[e] < w.t1;
                    auto shift = [&](int64_t first, int64_t ld) {   // of the row's words
                        return sizeof(T) == 4 ? 0 : (int(first) ^ ((int(t) + row[e]) & int(ld))) & 1;
                    };
                    xv[e] = load1(&sm.raw[0][row[e]][col[e] + shift(xf, p.ldx)]);
                    rv[e] = load1(&sm.raw[1][row[e]][col[e] + shift(rf, p.ldraw)]);
                    yv[e] = load1(&sm.raw[2][row[e]][col[e] + shift(yf, p.lddy)]);
                    bias[e] = sm.bias[col[e]];
                }
                pair_t sg;
                const pair_t r = add2(pack2(rv[0], rv[1]), pack2(bias[0], bias[1])), sp = softplus2(r, sg);
                unpack2(p.softplus ? sp : r, rv[0], rv[1]);
                unpack2(p.softplus ? sg : dup2(1.f), sv[0], sv[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sm.d[row[e]][col[e]] = in[e] ? rv[e] : 0.f;
                    sm.x[row[e]][col[e]] = in[e] ? xv[e] : 0.f;
                    sm.dy[row[e]][col[e]] = in[e] ? yv[e] : 0.f;
                    sm.slope[row[e]][col[e]] = in[e] ? sv[e] : 0.f;
                }
            }
        }
        // the thread's vectors of B and C, which it copied itself
        if (mode != kBcValues) {
#pragma unroll
            for (int i = 0; i < kBcPer; ++i) {
                const int v = tid + i * CV::THREADS;
                if (v < kBcVecs) {
                    float o[kCv];
                    load_vec<kCv>(&block.rawbc[v / kBcCols / 2][v / kBcCols % 2][v % kBcCols * kCv], o);
                    store_vec<kCv>(&block.bc[v / kBcCols / 2][v / kBcCols % 2][v % kBcCols * kCv], o);
                }
            }
        } else {
            for (int e = tid; e < kTile * 2 * NP; e += CV::THREADS) {
                const int n = e % NP, which = e / NP % 2, row = e / NP / 2;
                const bool in = t + row < w.t1 && n < p.N;
                block.bc[row][which][n] =
                    !in ? 0.f : load1(which == 0 ? bp + (t + row) * p.ldb + n : cp + (t + row) * p.ldc + n);
            }
        }
        const bool edges = lo >= t || hi == end;
        if (edges) edge_rows(q, w.rowb, t, int(end - t), block.first, block.last);
        __syncthreads();   // edges; and the block's dB and dC of the tile before are read
        if (t > w.t0) fetch(t - kTile);
        cp_async_commit();
        if (edges) tile(t, std::true_type());
        else tile(t, std::false_type());
        if (lo >= t && t > w.t0) {
            s = q.of(w.rowb + t - 1);
            lo = q.begin(s) - w.rowb;
        }
        hi = q.begin(s + 1) - w.rowb;
        __syncthreads();
        for (int i = tid; i < kTile * 2 * NP; i += CV::THREADS) {
            const int row = i / (2 * NP), v = i % (2 * NP), n = v % NP;
            if (n < p.N && t + row < w.t1) {
                float a = block.red[row][0][v];
#pragma unroll
                for (int k = 1; k < kWarps; ++k) a += block.red[row][k][v];
                partB[((w.tile * q.rows + w.rowb + t + row) * p.G + w.g) * 2 * p.N + v / NP * p.N + n] = a;
            }
        }
    }
    // a part is dA, then dDskip and ddt_bias
    float *part = partA + (w.b * ck.n + w.k) * p.D * (p.N + 2);
    if (p.N % 4 == 0 && p.D % 2 == 0) {
        store_block<S, CP>(part, dw + ch, ch, wide, n0, p.N, dA);
    } else {   // parts that are not 16-byte aligned
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float a, b;
                unpack2(dA[i][c / 2], a, b);
                if (ch + c < wide && n0 + i < p.N) part[(dw + ch + c) * p.N + n0 + i] = c % 2 ? b : a;
            }
    }
#pragma unroll
    for (int o = 0; o < kOut; ++o)
        if (writes && oc + o < wide) {
            part[p.D * p.N + dw + oc + o] = sum_d[o];
            part[p.D * (p.N + 1) + dw + oc + o] = sum_b[o];
        }
}

// dB and dC from the tiles' parts, in order: part (tile, row, group, dB or
// dC, N).
template <typename T>
__global__ void __launch_bounds__(256) sum_bc_kernel(const float *part, int64_t tiles, int64_t rows_g,
                                                     int N, T *dB, T *dC)
{
    const int64_t n = rows_g * 2 * N, i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    after_previous();
    if (i >= n) return;
    float a = 0.f;
    for (int64_t t = 0; t < tiles; ++t) a += part[t * n + i];
    const int64_t rg = i / (2 * N);
    const int v = int(i - rg * 2 * N);
    T *o = v < N ? dB : dC;
    store1(o + rg * N + (v < N ? v : v - N), a);
}

// The gradients' threads: states of four channels, or, up to 8 states, of two,
// whose registers let three blocks share an SM instead of two (2 x 4096 x 1024
// channels of 8 states: 235 -> 162 us; of 16 it would be 821 -> 857, the sums
// over lanes being of fewer values).  A block holds 128 channels, 64 from 17
// states on and 32 from 33 on.
inline int backward_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
constexpr int backward_channels(int L) { return L <= 2 ? 2 : 4; }
constexpr int backward_threads(int L) { return L == 1 ? 64 : kThreads; }
inline int64_t backward_tiles(int64_t D, int N, int G)
{
    const int L = backward_lanes(N);
    return ceil_div(D / G, backward_threads(L) / L * backward_channels(L));
}

inline Chunks backward_chunks(int64_t B, int64_t T, int64_t D, int N, int G)
{
    // measured: 1024 rows of 152, 304 and 456 blocks
    static constexpr RowTime two{{0, 405, 495, 625}, 3, 0.2}, four{{0, 520, 705, 0}, 2, 0.2};
    return cut_time(B * G * backward_tiles(D, N, G), T, backward_channels(backward_lanes(N)) == 2 ? two : four);
}

template <typename T, int VEC, int L>
mg_status bwd(const SsmArgs &p, cudaStream_t s)
{
    using CV = Cover<4, L, backward_channels(L), backward_threads(L)>;
    const Tile t{backward_tiles(p.D, p.N, p.G), p.D / p.G};
    const Chunks ck = backward_chunks(p.B, p.T, p.D, p.N, p.G);
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const int64_t rows_g = q.rows * p.G, dn = p.D * p.N, parts = p.B * ck.n;
    float *partB = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    float *partA = partB + t.tiles * rows_g * 2 * p.N;
    float *agg_q = partA + ceil_div(parts * p.D * (p.N + 2), 4) * 4;
    float *agg_s = agg_q + p.B * (ck.n - 1) * dn;
    const int64_t tiles = t.tiles * p.G * p.B;
    const int mode = bc_mode<T>(p.N, p.ldb, p.ldc);
    const int64_t bc_blocks = ceil_div(rows_g * 2 * p.N, 256);
    MG_TRY(check_grids("mg_selective_scan_bwd", {tiles * ck.n, adjoint_blocks(p, ck), bc_blocks,
                                                 sum_parts_blocks(p.D * (p.N + 2))}));
    if (p.cu != nullptr) {
        MG_TRY(launch_empty_sequences(q, p.dh0, p.dh_last, dn, p.ws, s));
    }
    if (ck.n > 1) {
        constexpr mg_dtype dt = sizeof(T) == 4 ? MG_F32 : MG_BF16;
        MG_TRY(launch_ssm_adjoint(p, dt, VEC > 1, ck, agg_q, agg_s, s));
    }
    constexpr size_t smem = sizeof(BwdShared<T, VEC, CV>);
    static_assert(smem <= kMostShared, "shared memory of a block");
    MG_TRY(allow_shared<ssm_bwd_kernel<T, VEC, CV>>(smem));
    constexpr const char *what = "mg_selective_scan_bwd";
    auto kernel = ssm_bwd_kernel<T, VEC, CV>;
    if (ck.n > 1 || p.cu != nullptr) {   // not the call's first
        MG_TRY(launch_next(what, kernel, tiles * ck.n, CV::THREADS, smem, s, p, q, t, ck, agg_q, agg_s, partB, partA, mode));
    } else {
        kernel<<<unsigned(tiles), CV::THREADS, smem, s>>>(p, q, t, ck, agg_q, agg_s, partB, partA, mode);
        MG_TRY(launched(what));
    }
    MG_TRY(launch_next(what, sum_bc_kernel<T>, bc_blocks, 256, 0, s, partB, t.tiles, rows_g, p.N,
                       static_cast<T *>(p.dBm), static_cast<T *>(p.dCm)));
    return launch_sum_parts(partA, parts, {{p.dA, dn}, {p.dDskip, p.D}, {p.ddt_bias, p.D}}, s);
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

}  // namespace mg
