// Selective scan, forward and for single tokens: the recurrence with N states
// a channel whose decay, input and output weights depend on the token,
//   h_r[d,n] = a_r h_{r-1}[d,n] + u_r B_r[n],  a_r = exp(delta_r A[d,n]),
//   u_r = delta_r x_r,  y_r[d] = sum_n C_r[n] h_r[d,n] + Dskip x_r.
//
// L lanes share a channel's states, and sums over states are shuffles among
// them.  States past N have A = B = C = 0.
#include "selective_scan.cuh"

namespace mg {
namespace {

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
// The gradients' first pass is the same walk backwards in time, with
// q <- a_r (q + C_r dy_r) in the recurrence's place (ChunkPass kAdjoint).
//
// Each warp works by itself, on its own channels and its own copy of B and C:
// no barrier lines up the warps of an SM.  Stages of kRows rows pass through
// shared memory.  The rows' x, raw, B and C arrive by asynchronous copies,
// kRing stages ahead; while the warp runs the recurrence over one stage, the
// next one's (delta, u) pairs (softplus once for each row and channel) are
// computed in the same instruction stream, so that their latency hides behind
// the recurrence's even with a single warp on a scheduler, and written to the
// other of two buffers.  Rows past the chunk are staged as delta = u = 0,
// B = C = 0: the state passes through them.
//
// Per row and state: 4 float32 multiply-adds and one 2^x.  64 pairs of
// multiply-adds and 32 2^x a clock and SM would need the same time; a
// multiply-add of three registers runs at 2/3 of that, so the core of a
// warp's row of 512 states takes 26 clocks of its SM where 16 would be the
// pipes' own.  A thread's block of 8 x 2 states loads 5 x 16 bytes from
// shared memory for its 16 states' row (2.1 or 3.9 clocks for a warp's load,
// by pattern), which is below that.
//
// 4 x 4096 x 2048 bf16 channels of 16 states take 287 us with a cold L2, 1.9e12
// states a second: 121 for the states at the chunks' ends, the rest for the
// outputs (178 where states are saved for the gradients).  The bytes would need
// 30 us.  Of a warp's row of 512 states the formulas are 48 instructions in the
// first pass and 56 in the second; executed are 89 and 124: staging, addresses,
// conversions and the sum over lanes, in both passes.  Three warps a scheduler
// (the registers of 16 states a thread) issue in 65 and 62% of the slots.
constexpr int kRows = 8;    // rows of a stage
constexpr int kRing = 4;    // stages in flight or in use

// What a launch of ssm_chunk_kernel does.
enum ChunkPass { kOutputs, kStates, kAdjoint };

template <typename T, int VEC, int WCH, int NP, bool kFirst>
struct alignas(16) FwdShared {   // of a warp
    static constexpr int kBc = kFirst ? 1 : 2;
    float2 du[2][kRows][WCH];
    float bc[2][kRows][kBc][NP];
    float y[kFirst ? 1 : kRows][kFirst ? 4 : WCH];
    float bias[WCH], skip[WCH];
    // as loaded: x, raw, and B (and C)
    T raw[kRing][2][kRows][VEC > 1 ? WCH : Words<T, WCH>::kPitch];
    alignas(16) T rawbc[kRing][kRows][kBc][NP];
};

template <typename T, int VEC, typename CV, ChunkPass kPass>
__global__ void __launch_bounds__(kThreads, 3)
ssm_chunk_kernel(SsmArgs p, Seqs q, Tile tl, Chunks ck, float *agg_h, float *agg_s, int mode)
{
    constexpr bool kFirst = kPass != kOutputs, kBack = kPass == kAdjoint;
    constexpr int S = CV::S, L = CV::L, C = CV::C, NP = CV::NP, SP = S / 2, WCH = CV::kWarpCh;
    constexpr int kBc = kFirst ? 1 : 2;
    // A lane's part of staging: kPer pieces of VEC channels, kStep rows apart.
    constexpr int kCols = WCH / VEC, kStep = 32 / kCols;
    constexpr int kPer = kStep < kRows ? kRows / kStep : 1;
    constexpr int kCv = 16 / int(sizeof(T));                        // values of a vector of B or C
    constexpr int kBcCols = NP / kCv, kBcVecs = kRows * kBc * kBcCols, kBcPer = (kBcVecs + 31) / 32;
    constexpr int kBcW = kRows * kBc * NP * int(sizeof(T)) / 4, kRowW = NP * int(sizeof(T)) / 4;
    static_assert(C == 2 && WCH % VEC == 0 && kCols <= 32 && (VEC > 1 || kPer % 2 == 0), "staging");
    using Shared = FwdShared<T, VEC, WCH, NP, kFirst>;
    extern __shared__ __align__(16) unsigned char shared_bytes[];
    if (kFirst) after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Shared &sm = reinterpret_cast<Shared *>(shared_bytes)[warp];

    const int64_t all_tiles = tl.tiles * p.G;
    const int64_t tile = blockIdx.x % all_tiles, rest = blockIdx.x / all_tiles;
    const int64_t nch = kFirst ? ck.n - 1 : ck.n;      // the last (backwards: first) chunk has no successor
    const int64_t k = rest % nch + (kBack ? 1 : 0), b = rest / nch;
    const int64_t rowb = b * p.T;
    const int64_t t0 = k * ck.len, t1 = t0 + ck.len < p.T ? t0 + ck.len : p.T;
    const int g = int(tile / tl.tiles);
    const int64_t c0 = (tile % tl.tiles) * CV::kCh + warp * WCH, d0 = g * tl.width + c0;   // the warp's first channel
    if (c0 >= tl.width) return;
    const int wide = int(tl.width - c0 < WCH ? tl.width - c0 : WCH);                       // its channels
    const int sl = lane / CV::kGroups, n0 = sl * S;
    const int ch = lane % CV::kGroups * C;             // the thread's first channel

    // Staging: the lane's vectors of x and raw (one column, kStep rows apart),
    // and of B and C.
    const int row0 = lane / kCols, col = lane % kCols * VEC;
    const bool col_in = col < wide && row0 < kRows;
    // Backwards, rows count from the chunk's last one down: dy stands for x, C
    // for B, and the strides are negative.
    const int64_t ldx = kBack ? -p.lddy : p.ldx, ldr = kBack ? -p.ldraw : p.ldraw;
    const int64_t ldb = kBack ? -p.ldc : p.ldb, ldc = p.ldc;
    const int64_t rf = rowb + (kBack ? t1 - 1 : t0);   // the chunk's first row in that order
    const T *x0p = static_cast<const T *>(kBack ? p.dy : p.x), *r0p = static_cast<const T *>(p.raw);
    const int64_t xf = rf * (kBack ? p.lddy : p.ldx) + d0, rawf = rf * p.ldraw + d0;   // its first values
    const T *xp = x0p + xf + row0 * ldx + col, *rp = r0p + rawf + row0 * ldr + col;
    const int64_t xs = kStep * ldx, rs = kStep * ldr;
    const T *bp = static_cast<const T *>(kBack ? p.Cm : p.Bm) + rf * (kBack ? p.ldc : p.ldb) + int64_t(g) * p.N;
    const T *cp = static_cast<const T *>(p.Cm) + rf * p.ldc + int64_t(g) * p.N;
    const int rows = int(t1 - t0);
    // Starts the copies of the rows from `at` on into ring slot `slot`.
    auto fetch = [&](int at, int slot) {
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int row = at + row0 + i * kStep;
                const bool in = col_in && row < rows;
                if (row0 < kRows) {
                    cp_async16_or_zero(&sm.raw[slot][0][row0 + i * kStep][col], in ? xp + at * ldx + i * xs : p.x, in);
                    cp_async16_or_zero(&sm.raw[slot][1][row0 + i * kStep][col], in ? rp + at * ldr + i * rs : p.raw, in);
                }
            }
        } else {
            fetch_words<T, WCH, kRows>(sm.raw[slot][0], x0p, xf + at * ldx, ldx, rows - at, wide, lane);
            fetch_words<T, WCH, kRows>(sm.raw[slot][1], r0p, rawf + at * ldr, ldr, rows - at, wide, lane);
        }
        if (mode == kBcVectors) {
#pragma unroll
            for (int i = 0; i < kBcPer; ++i) {
                const int v = lane + i * 32, n = v % kBcCols * kCv, which = v / kBcCols % kBc, row = v / kBcCols / kBc;
                const bool in = at + row < rows && n < p.N;
                const void *src = !in          ? p.Bm
                                  : which == 0 ? static_cast<const void *>(bp + (at + row) * ldb + n)
                                               : static_cast<const void *>(cp + (at + row) * ldc + n);
                if (kBcVecs % 32 == 0 || v < kBcVecs) cp_async16_or_zero(&sm.rawbc[slot][row][which][n], src, in);
            }
        } else if (mode == kBcWords) {
#pragma unroll 4
            for (int v = lane; v < kBcW; v += 32) {
                const int n = v % kRowW * (4 / int(sizeof(T))), which = v / kRowW % kBc, row = v / kRowW / kBc;
                const bool in = at + row < rows && n < p.N;
                const T *src = which == 0 ? bp + (at + row) * ldb + n : cp + (at + row) * ldc + n;
                cp_async4(&sm.rawbc[slot][row][which][n], in ? static_cast<const void *>(src) : p.Bm, in ? 4 : 0);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch(i * kRows, i);

    // The thread's channels.  Channels past the group run on zeros.
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
    for (int i = lane; i < WCH; i += 32) {
        sm.bias[i] = p.dt_bias != nullptr && i < wide ? p.dt_bias[d0 + i] : 0.f;
        sm.skip[i] = !kFirst && p.Dskip != nullptr && i < wide ? p.Dskip[d0 + i] : 0.f;
    }
    __syncwarp();
    const float *edge = kBack ? p.dh_last : p.h0;      // the state that a sequence starts from
    auto start_state = [&](int s) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[S];
#pragma unroll
            for (int i = 0; i < S; ++i) v[i] = 0.f;
            if (edge != nullptr && ch + c < wide)
                load_group<S>(edge + (int64_t(s) * p.D + d0 + ch + c) * p.N, n0, p.N, v);
#pragma unroll
            for (int i = 0; i < SP; ++i) h[c][i] = pack2(v[2 * i], v[2 * i + 1]);
        }
    };
    int s = q.of(rf);
    // where the sequence ends, in rows from the chunk's first
    auto ends = [&]() { return kBack ? rowb + t1 - q.begin(s) : q.begin(s + 1) - (rowb + t0); };
    long long next = ends();
    if (!kFirst) after_previous();   // the chunks' states
    {
        const long long lo = q.begin(s) - rowb;
        if (kBack ? q.begin(s + 1) - rowb <= t1 : lo >= t0) {
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
                        h[c][i] = begin ? hv : fma2(decay2(ds, ds, A2[c][i]), h[c][i], hv);
                    }
                }
                begin = false;
            }
        }
    }

    // The next stage's staged values, from what the copies brought: computed
    // (convert) and written to buffer `to` (put) apart from each other.
    constexpr int kPairs = kPer * VEC / 2;   // of channels, or (VEC = 1) of a channel's rows
    pair_t dl[kPairs], uu[kPairs];
    float bcv[kBcPer][kCv];
    // parity of the rows' first values, for the words' shifts
    const int xpar = int(xf & 1), xstep = int(ldx & 1), rpar = int(rawf & 1), rstep = int(ldr & 1);
    auto word_value = [&](const T *row_words, int shift) { return load1(row_words + shift + col); };
    auto convert = [&](int at, int slot) {
        if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const bool in = col_in && at + row0 + i * kStep < rows;
                float xv[VEC], rv[VEC], bias[VEC];
                load_vec<VEC>(&sm.raw[slot][0][(row0 + i * kStep) % kRows][col], xv);
                load_vec<VEC>(&sm.raw[slot][1][(row0 + i * kStep) % kRows][col], rv);
                load_vec<VEC>(&sm.bias[col], bias);
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const pair_t r = add2(pack2(rv[e], rv[e + 1]), pack2(bias[e], bias[e + 1]));
                    const pair_t sp = softplus2(r), xx = pack2(xv[e], xv[e + 1]);
                    const pair_t d = !in ? 0 : p.softplus ? sp : r;
                    dl[(i * VEC + e) / 2] = d;
                    uu[(i * VEC + e) / 2] = kBack ? xx : mul2(d, xx);
                }
            }
        } else {
            const float bias = sm.bias[col];
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                const int a = row0 + i * kStep, b = a + kStep;
                const bool in0 = col_in && at + a < rows, in1 = col_in && at + b < rows;
                const int sx = sizeof(T) == 4 ? 0 : 1, ra = at + a, rb = at + b;
                const float r0 = word_value(sm.raw[slot][1][a % kRows], sx & (rpar ^ (ra & rstep)));
                const float r1 = word_value(sm.raw[slot][1][b % kRows], sx & (rpar ^ (rb & rstep)));
                const float x0 = word_value(sm.raw[slot][0][a % kRows], sx & (xpar ^ (ra & xstep)));
                const float x1 = word_value(sm.raw[slot][0][b % kRows], sx & (xpar ^ (rb & xstep)));
                const pair_t r = add2(pack2(r0, r1), pack2(bias, bias)), sp = softplus2(r);
                float d0v, d1v;
                unpack2(p.softplus ? sp : r, d0v, d1v);
                const pair_t d = pack2(in0 ? d0v : 0.f, in1 ? d1v : 0.f);
                // (a channel past the group reads a neighbour's or stale values)
                const pair_t xx = pack2(in0 ? x0 : 0.f, in1 ? x1 : 0.f);
                dl[i / 2] = d;
                uu[i / 2] = kBack ? xx : mul2(d, xx);
            }
        }
        if (mode != kBcValues) {
#pragma unroll
            for (int i = 0; i < kBcPer; ++i) {
                const int v = lane + i * 32;
                if (kBcVecs % 32 == 0 || v < kBcVecs)
                    load_vec<kCv>(&sm.rawbc[slot][v / kBcCols / kBc][v / kBcCols % kBc][v % kBcCols * kCv], bcv[i]);
            }
        }
    };
    auto put = [&](int at, int to) {
        if (row0 < kRows) {
            if constexpr (VEC > 1) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int row = row0 + i * kStep;
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) {
                        float4 o;
                        unpack2(dl[(i * VEC + e) / 2], o.x, o.z);
                        unpack2(uu[(i * VEC + e) / 2], o.y, o.w);
                        *reinterpret_cast<float4 *>(&sm.du[to][row][du_index<WCH>(row, col + e)]) = o;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPer; i += 2) {
                    const int a = row0 + i * kStep, b = a + kStep;
                    float2 oa, ob;
                    unpack2(dl[i / 2], oa.x, ob.x);
                    unpack2(uu[i / 2], oa.y, ob.y);
                    sm.du[to][a][du_index<WCH>(a, col)] = oa;
                    sm.du[to][b][du_index<WCH>(b, col)] = ob;
                }
            }
        }
        if (mode != kBcValues) {
#pragma unroll
            for (int i = 0; i < kBcPer; ++i) {
                const int v = lane + i * 32;
                if (kBcVecs % 32 == 0 || v < kBcVecs)
                    store_vec<kCv>(&sm.bc[to][v / kBcCols / kBc][v / kBcCols % kBc][v % kBcCols * kCv], bcv[i]);
            }
        } else {
            for (int e = lane; e < kRows * kBc * NP; e += 32) {
                const int n = e % NP, which = e / NP % kBc, row = e / NP / kBc;
                const bool in = at + row < rows && n < p.N;
                sm.bc[to][row][which][n] =
                    !in ? 0.f : load1(which == 0 ? bp + (at + row) * ldb + n : cp + (at + row) * ldc + n);
            }
        }
    };

    // One row of the recurrence from the staged tile; y (without the sum over
    // lanes) comes back.
    auto step = [&](int buf, int tt, float (&y)[C]) {
        pair_t B[SP], Cw[SP];
#pragma unroll
        for (int i = 0; i < SP; i += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&sm.bc[buf][tt][0][n0 + 2 * i]);
            B[i] = v.x, B[i + 1] = v.y;
            if (!kFirst) {
                const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sm.bc[buf][tt][kBc - 1][n0 + 2 * i]);
                Cw[i] = w.x, Cw[i + 1] = w.y;
            }
        }
        const float4 du4 = *reinterpret_cast<const float4 *>(&sm.du[buf][tt][du_index<WCH>(tt, ch)]);
        const float du[4] = {du4.x, du4.y, du4.z, du4.w};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const pair_t u2 = pack2(du[2 * c + 1], du[2 * c + 1]);
            pair_t acc = 0;
#pragma unroll
            for (int i = 0; i < SP; ++i) {
                const pair_t a = decay2(du[2 * c], du[2 * c], A2[c][i]);
                h[c][i] = kBack ? mul2(a, fma2(u2, B[i], h[c][i])) : fma2(a, h[c][i], mul2(u2, B[i]));
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

    T *yp = static_cast<T *>(p.y) + (rowb + t0 + row0) * p.D + d0 + col;
    cp_async_wait<kRing - 1>();
    __syncwarp();   // words are other lanes' copies
    convert(0, 0);
    put(0, 0);
    __syncwarp();
    int slot = 0, buf = 0;
#pragma unroll 1
    for (int at = 0; at < rows; at += kRows) {
        if (!kFirst && p.saved != nullptr && (t0 + at) % kSeg == 0) {
            const int64_t o = b * ((p.T + kSeg - 1) / kSeg) + (t0 + at) / kSeg;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (ch + c < wide)
                    store_pairs<S>(p.saved + (o * p.D + d0 + ch + c) * p.N, n0, p.N, h[c]);
        }
        const int end = at + kRows < rows ? at + kRows : rows;
        auto last_state = [&]() {
            if constexpr (!kFirst) {
                if (p.h_last == nullptr) return;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (ch + c < wide)
                        store_pairs<S>(p.h_last + (int64_t(s) * p.D + d0 + ch + c) * p.N, n0, p.N, h[c]);
            }
        };
        cp_async_wait<kRing - 2>();
        __syncwarp();
        const int ns = slot + 1 < kRing ? slot + 1 : 0;
        if (next >= end) {   // no sequence begins inside the stage
            convert(at + kRows, ns);
            float y[C][kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float v[C];
                step(buf, i, v);
#pragma unroll
                for (int c = 0; c < C; ++c) y[c][i] = kFirst ? 0.f : v[c];
            }
            if constexpr (!kFirst) {
#pragma unroll
                for (int c = 0; c < C; ++c) spread_sum<kRows, L>(y[c], sl);
#pragma unroll
                for (int i = 0; i < kRows / L; ++i)
                    *reinterpret_cast<float2 *>(&sm.y[sl * (kRows / L) + i][ch]) = make_float2(y[0][i], y[1][i]);
            }
            if (next == end) last_state();
        } else {
#pragma unroll 1
            for (int tt = 0; tt < end - at; ++tt) {
                if (at + tt == next) {   // the next sequence that has rows
                    s = q.of(kBack ? rf - (at + tt) : rf + at + tt);
                    next = ends();
                    start_state(s);
                }
                float y[C];
                step(buf, tt, y);
                if constexpr (!kFirst) {
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float v = y[c];
#pragma unroll
                        for (int m = CV::kGroups; m < 32; m <<= 1) v += __shfl_xor_sync(~0u, v, m);
                        if (sl == 0) sm.y[tt][ch + c] = v;
                    }
                }
                if (at + tt + 1 == next) last_state();
            }
            convert(at + kRows, ns);
        }
        put(at + kRows, buf ^ 1);
        __syncwarp();
        if constexpr (!kFirst) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int row = row0 + i * kStep;
                if (col_in && at + row < rows) {
                    float o[VEC], x[VEC], skip[VEC];
                    load_vec<VEC>(&sm.y[row % kRows][col], o);
                    load_vec<VEC>(&sm.skip[col], skip);
                    if constexpr (VEC > 1) load_vec<VEC>(&sm.raw[slot][0][row % kRows][col], x);
                    else x[0] = word_value(sm.raw[slot][0][row % kRows],
                                           (sizeof(T) == 4 ? 0 : 1) & (xpar ^ ((at + row) & xstep)));
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = fmaf(skip[e], x[e], o[e]);
                    store_out<VEC>(yp + (at + i * kStep) * p.D, o);
                }
            }
        }
        if (VEC == 1) __syncwarp();   // the slot's x is read
        fetch(at + kRing * kRows, slot);
        __syncwarp();
        slot = ns;
        buf ^= 1;
    }
    cp_async_wait<0>();
    if (kFirst) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (ch + c < wide) {
                const int64_t at = (b * (ck.n - 1) + (kBack ? k - 1 : k)) * p.D + d0 + ch + c;
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

// ------------------------------------------------------------ single tokens
//
// A thread keeps four states' A of one channel for kTokens rows of the batch,
// L lanes a channel; everything is loaded before the first of it is used.  The
// states read and written bound it: 256 x 4096 channels of 16 states take 34
// us, 4.1 TB/s (one row a thread 41 us; four need registers that cost as many
// warps).
constexpr int kS = 4;        // states of a thread
constexpr int kTokens = 2;   // rows of a thread

int lanes_for(int N)
{
    int L = 1;
    while (L * kS < N) L *= 2;
    return L;
}

// The first n of kS values from p on, the rest zero.
__device__ __forceinline__ void load_some(const float *p, int n, Raw<float, kS> &o)
{
#pragma unroll
    for (int i = 0; i < kS; ++i)
        if (i < n) o.w[i] = p[i];
}
__device__ __forceinline__ void load_some(const bf16_t *p, int n, Raw<bf16_t, kS> &o)
{
#pragma unroll
    for (int i = 0; i < kS; ++i)
        if (i < n) o.w[i / 2] |= unsigned(p[i].bits) << (i % 2 * 16);
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 8) ssm_step_kernel(SsmStepArgs p, unsigned chan_blocks, int bc_wide)
{
    const int d = (blockIdx.x % chan_blocks * kThreads + threadIdx.x) / L, D = int(p.D);
    const bool live = d < D;
    const int sl = threadIdx.x % L, n0 = sl * kS;
    const int dd = live ? d : 0, g = dd / (D / p.G);
    const int64_t b0 = int64_t(blockIdx.x / chan_blocks) * kTokens;
    const int rows = int(p.B - b0 < kTokens ? p.B - b0 : kTokens);
    // everything is loaded before the first of it is used
    float h[kTokens][kS], x[kTokens], raw[kTokens];
    Raw<T, kS> B[kTokens], C[kTokens];
    float *st[kTokens];
    bool on[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int64_t b = b0 + (k < rows ? k : 0);
        const int64_t slot = k >= rows ? -1 : p.slots != nullptr ? __ldg(p.slots + b) : b;
        on[k] = live && slot >= 0 && slot < p.nslots;
        st[k] = p.state + ((on[k] ? slot : 0) * p.D + dd) * p.N;
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int64_t b = b0 + (k < rows ? k : 0);
        const T *bp = static_cast<const T *>(p.Bm) + b * p.ldb + int64_t(g) * p.N + n0;
        const T *cp = static_cast<const T *>(p.Cm) + b * p.ldc + int64_t(g) * p.N + n0;
#pragma unroll
        for (int i = 0; i < kS; ++i) h[k][i] = 0.f;
        if (on[k]) load_group<kS>(st[k], n0, p.N, h[k]);
        x[k] = load1(static_cast<const T *>(p.x) + b * p.ldx + dd);
        raw[k] = load1(static_cast<const T *>(p.raw) + b * p.ldraw + dd);
        B[k].fill(0.f);
        C[k].fill(0.f);
        if (n0 < p.N) {
            if (bc_wide) {
                B[k].load(bp);
                C[k].load(cp);
            } else {
                load_some(bp, p.N - n0, B[k]);
                load_some(cp, p.N - n0, C[k]);
            }
        }
    }
    float A2[kS];
    load_group<kS>(p.A + int64_t(dd) * p.N, n0, p.N, A2);
    const float bias = p.dt_bias != nullptr ? p.dt_bias[dd] : 0.f, skip = p.Dskip != nullptr ? p.Dskip[dd] : 0.f;
#pragma unroll
    for (int i = 0; i < kS; ++i) A2[i] *= kLog2eF;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const float v = raw[k] + bias, delta = p.softplus ? softplus_f(v) : v, u = delta * x[k];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            h[k][i] = fmaf(ex2_ftz(fmaf(delta, A2[i], kDecayBias)), h[k][i], u * B[k][i]);
            y = fmaf(C[k][i], h[k][i], y);
        }
        if (on[k]) store_group<kS>(st[k], n0, p.N, h[k]);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(~0u, y, o);
        if (live && sl == 0 && k < rows)
            store1(static_cast<T *>(p.y) + (b0 + k) * p.D + d, on[k] ? fmaf(skip, x[k], y) : 0.f);
    }
}

// Lanes of a channel: 8 states a thread, 4 for N <= 8.
int forward_lanes(int N) { return N <= 16 ? 2 : N <= 32 ? 4 : 8; }

int64_t forward_tiles(int64_t D, int N, int G)
{
    return ceil_div(D / G, kThreads / forward_lanes(N) * 2);
}
Chunks forward_chunks(int64_t B, int64_t T, int64_t D, int N, int G)
{
    // measured at 152 m blocks of 2048 rows: 273, 386, 537 us
    static constexpr RowTime r{{0, 133, 188, 262}, 3, 0.65};
    return cut_time(B * G * forward_tiles(D, N, G), T, r);
}

template <typename T, int VEC, typename CV>
mg_status fwd_cover(const SsmArgs &p, cudaStream_t s)
{
    const Tile t{forward_tiles(p.D, p.N, p.G), p.D / p.G};
    const Chunks ck = forward_chunks(p.B, p.T, p.D, p.N, p.G);
    const int mode = bc_mode<T>(p.N, p.ldb, p.ldc);
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    float *agg_h = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    float *agg_s = agg_h + p.B * (ck.n - 1) * p.D * p.N;
    const int64_t tiles = t.tiles * p.G * p.B;
    MG_TRY(check_grids("mg_selective_scan_fwd", {tiles * ck.n}));
    if (p.cu != nullptr) {
        const int64_t n = p.D * p.N;
        MG_TRY(launch_empty_sequences(q, p.h_last, p.h0, n, p.ws, s));
    }
    constexpr size_t sm1 = kThreads / 32 * sizeof(FwdShared<T, VEC, CV::kWarpCh, CV::NP, true>);
    constexpr size_t sm2 = kThreads / 32 * sizeof(FwdShared<T, VEC, CV::kWarpCh, CV::NP, false>);
    MG_TRY(allow_shared<ssm_chunk_kernel<T, VEC, CV, kStates>>(sm1));
    MG_TRY(allow_shared<ssm_chunk_kernel<T, VEC, CV, kOutputs>>(sm2));
    bool first = p.cu == nullptr;   // of the call's kernels
    auto ours = [&](auto kernel, int64_t grid, size_t smem) {
        constexpr const char *what = "mg_selective_scan_fwd";
        if (!first) return launch_next(what, kernel, grid, kThreads, smem, s, p, q, t, ck, agg_h, agg_s, mode);
        kernel<<<unsigned(grid), kThreads, smem, s>>>(p, q, t, ck, agg_h, agg_s, mode);
        return launched(what);
    };
    if (ck.n > 1) {
        MG_TRY(ours(ssm_chunk_kernel<T, VEC, CV, kStates>, tiles * (ck.n - 1), sm1));
        first = false;
    }
    return ours(ssm_chunk_kernel<T, VEC, CV, kOutputs>, tiles * ck.n, sm2);
}

template <typename T, int VEC, typename CV>
mg_status adjoint_cover(const SsmArgs &p, const Chunks &ck, float *agg_q, float *agg_s, cudaStream_t s)
{
    const Tile t{forward_tiles(p.D, p.N, p.G), p.D / p.G};
    const int mode = bc_mode<T>(p.N, p.ldc, p.ldc);
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    constexpr size_t sm = kThreads / 32 * sizeof(FwdShared<T, VEC, CV::kWarpCh, CV::NP, true>);
    MG_TRY(allow_shared<ssm_chunk_kernel<T, VEC, CV, kAdjoint>>(sm));
    const int64_t grid = adjoint_blocks(p, ck);
    auto kernel = ssm_chunk_kernel<T, VEC, CV, kAdjoint>;
    if (p.cu != nullptr)
        return launch_next("mg_selective_scan_bwd", kernel, grid, kThreads, sm, s, p, q, t, ck, agg_q, agg_s, mode);
    kernel<<<unsigned(grid), kThreads, sm, s>>>(p, q, t, ck, agg_q, agg_s, mode);
    return launched("mg_selective_scan_bwd");
}

// F<CV>(...) for the states of the call.
#define MG_COVER(F, T, VEC, ...)                                                     \
    if (p.N <= 8) return F<T, VEC, Cover<4, 2, 2>>(__VA_ARGS__);                     \
    switch (forward_lanes(p.N)) {                                                    \
    case 2: return F<T, VEC, Cover<8, 2, 2>>(__VA_ARGS__);                           \
    case 4: return F<T, VEC, Cover<8, 4, 2>>(__VA_ARGS__);                           \
    default: return F<T, VEC, Cover<8, 8, 2>>(__VA_ARGS__);                          \
    }
template <typename T, int VEC>
mg_status fwd_vec(const SsmArgs &p, cudaStream_t s)
{
    MG_COVER(fwd_cover, T, VEC, p, s)
}
template <typename T, int VEC>
mg_status adjoint_vec(const SsmArgs &p, const Chunks &ck, float *agg_q, float *agg_s, cudaStream_t s)
{
    MG_COVER(adjoint_cover, T, VEC, p, ck, agg_q, agg_s, s)
}

template <typename T, int L>
mg_status step(const SsmStepArgs &p, cudaStream_t s)
{
    const int64_t chan_blocks = ceil_div(p.D * L, kThreads), blocks = ceil_div(p.B, kTokens) * chan_blocks;
    MG_TRY(check_grids("mg_selective_scan_step", {blocks}));
    if (p.D > (int64_t(1) << 31) / L - kThreads)
        return fail(MG_ERR_UNSUPPORTED, "mg_selective_scan_step: B = %lld, D = %lld", (long long)p.B, (long long)p.D);
    // rows of B and C as vectors of four
    const int bc_wide = p.N % 4 == 0 && p.ldb % 4 == 0 && p.ldc % 4 == 0;
    ssm_step_kernel<T, L><<<unsigned(blocks), kThreads, 0, s>>>(p, unsigned(chan_blocks), bc_wide);
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

mg_status launch_empty_sequences(const Seqs &q, float *dst, const float *src, int64_t n, void *ws, cudaStream_t s)
{
    empty_sequences_kernel<<<unsigned(q.nseq < 1024 ? q.nseq : 1024), 256, 0, s>>>(
        q, dst, src, n, &static_cast<Control *>(ws)->error);
    return launched("selective scan: empty sequences");
}

int64_t adjoint_blocks(const SsmArgs &p, const Chunks &ck)
{
    return forward_tiles(p.D, p.N, p.G) * p.G * p.B * (ck.n - 1);
}
mg_status launch_ssm_adjoint(const SsmArgs &p, mg_dtype dt, bool wide, const Chunks &ck, float *agg_q,
                             float *agg_s, cudaStream_t s)
{
    if (dt == MG_F32)
        return wide ? adjoint_vec<float, 4>(p, ck, agg_q, agg_s, s) : adjoint_vec<float, 1>(p, ck, agg_q, agg_s, s);
    return wide ? adjoint_vec<bf16_t, 8>(p, ck, agg_q, agg_s, s) : adjoint_vec<bf16_t, 1>(p, ck, agg_q, agg_s, s);
}

size_t ssm_fwd_ws_bytes(int64_t B, int64_t T, int64_t D, int N, int G, int64_t)
{
    const Chunks ck = forward_chunks(B, T, D, N, G);
    return kControlBytes + sizeof(float) * B * (ck.n - 1) * D * (N + 1);
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
    return dt == MG_F32 ? ssm_bwd_f32(p, wide, s) : ssm_bwd_bf16(p, wide, s);
}
mg_status launch_ssm_step(const SsmStepArgs &p, mg_dtype dt, cudaStream_t s) { MG_SSM(step, p, dt, s) }

}  // namespace mg
