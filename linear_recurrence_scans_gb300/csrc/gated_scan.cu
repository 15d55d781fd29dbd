// Gated recurrence with a matrix state per head: what its passes share, the
// float32 kernels, and single tokens.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
//
// In a chunk of L rows with G_i the sum of its gates up to row i, S the state
// before the chunk, D the adjoint of the state behind it, A_ij = e^{G_i - G_j}
// (j <= i, else 0) and dO' = scale dO:
//
//   O  = scale [(Q K^T . A) V + e^{G_i} Q S],    S' = e^{G_L} S + (e^{G_L - G_j} K)^T V
//   dQ = (dO' V^T . A) K + e^{G_i} dO' S^T,      dK = (dO' V^T . A)^T Q + e^{G_L - G_j} V D^T
//   dV = (Q K^T . A)^T dO' + e^{G_L - G_j} K D,  D' = e^{G_L} D + (e^{G_i} Q)^T dO'
//   dg_t = sum_{i >= t > j} W_ij + sum_{i >= t} q_i . (e^{G_i} S dO'_i)
//          + sum_{j < t} k_j . (e^{G_L - G_j} D v_j) + e^{G_L} <S, D>,   W = (Q K^T)(dO' V^T) . A
//
// so a call is: what each chunk adds to the state (all chunks at once), a pass
// over the chunks, and the outputs (all chunks at once); backwards the same
// for the adjoints.  dg is summed inside its chunk: a running sum over the whole
// sequence of q . dq - k . dk gives the same, but its rounding errors grow
// with the length.  The sums G are taken and kept as two floats, so
// that a row that forgets everything costs the differences behind it nothing.
//
// The float32 kernels multiply with FFMA (the tensor cores' 10 or 7 bits would
// take three to nine products for float32's) in chunks of 64 rows, by blocks of
// 256 threads that hold a 64 x 64 product in 4 x 4 values each.  At 5003 rows in
// one packed batch x 6 heads x 80 x 48 a call takes 75 us (2.8 us of bytes):
// 510 blocks of each kernel are less than two rounds, and a block's chain of
// loads, products and barriers is what it takes; 25 us for what chunks add, 40
// for the outputs.  3x509x6x24x40 with gradients: 77 us for seven launches.
#include "gated_scan.cuh"

namespace mg {
namespace {

// ------------------------------------------------------------ chunk table

// A block a cut.  Nothing of a cu that breaks the rules is used: its tables
// name no chunks.
__global__ void __launch_bounds__(1024) chunk_table_kernel(const Chunks c0, const Chunks c1, void *ws)
{
    __shared__ int sums[32];
    const Chunks &c = blockIdx.x == 0 ? c0 : c1;
    int *first = const_cast<int *>(c.first);
    check_cu(c.q, error_word(ws), threadIdx.x, blockDim.x);
    bool bad = false;
    for (int s = threadIdx.x; s < c.q.nseq; s += 1024) {
        const long long a = __ldg(c.q.cu + s), b = __ldg(c.q.cu + s + 1);
        bad = bad || b < a || (s == 0 && a != 0) || (s + 1 == c.q.nseq && b != c.q.rows);
    }
    bad = __syncthreads_or(bad);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int base = 0;
    if (threadIdx.x == 0) first[0] = 0;
    for (int s0 = 0; s0 < c.q.nseq; s0 += 1024) {
        const int s = s0 + threadIdx.x;
        int v = s < c.q.nseq && !bad ? int((__ldg(c.q.cu + s + 1) - __ldg(c.q.cu + s) + c.L - 1) / c.L) : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int before = base;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before += sums[w];
            base += sums[w];
        }
        if (s < c.q.nseq) first[s + 1] = before + v;
        __syncthreads();
    }
}

// ------------------------------------------------------- pass over chunks

// A thread keeps VEC of a state's values and walks over the chunks, kAhead of
// them loaded before they are needed.
template <int VEC, bool BACK>
__global__ void __launch_bounds__(256) over_chunks_kernel(const Chunks c, float *states, const float *totals,
                                                          const float *from, float *to, int H, int64_t NP,
                                                          int blocks_per)
{
    after_previous();
    constexpr int kAhead = 8;
    const int64_t sh = blockIdx.x / blocks_per;   // sequence and head
    const int seq = int(sh / H), h = int(sh % H);
    const int64_t at = (int64_t(blockIdx.x % blocks_per) * 256 + threadIdx.x) * VEC;
    if (at >= NP) return;
    const int64_t lo = c.begin(seq), hi = c.end(seq);
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.f;
    if (from != nullptr) load_vec<VEC>(from + sh * NP + at, s);
    // + 0: a caller's signalling NaN must not get into the workspace as it is
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] += 0.f;
    for (int64_t i0 = 0; i0 < hi - lo; i0 += kAhead) {
        float add[kAhead][VEC], decay[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t i = i0 + u;
            if (i >= hi - lo) continue;
            const int64_t ch = (BACK ? hi - 1 - i : lo + i) * H + h;
            load_vec<VEC>(states + ch * NP + at, add[u]);
            decay[u] = totals[ch];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t i = i0 + u;
            if (i >= hi - lo) continue;
            const int64_t ch = (BACK ? hi - 1 - i : lo + i) * H + h;
            store_vec<VEC>(states + ch * NP + at, s);
            const float d = expf(decay[u]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = fmaf(d, s[e], add[u][e]);
        }
    }
    if (to != nullptr) store_vec<VEC>(to + sh * NP + at, s);
}

// ---------------------------------------------------------- float32 kernels
// Chunks of 64 rows in shared memory, 16 x 16 threads.  The arithmetic is float32 multiply-adds: bf16 tensor products of float32 values
// would need six products of three-way splits, and tf32 ones three.

constexpr int kL = 64, kThreads = 256;
constexpr int kStaged = 4096;                  // values of a state in shared memory at a time, for the outputs
constexpr size_t kRoom = kMostShared - 4096;   // beside a kernel's own gates and sums

// Products of operands in shared memory.  A thread's rows are ty + 16 i; its
// columns tx + 16 j, or for kQuads neighbouring ones, 4 (2) at a time, so that one
// load brings them.  Operands whose rows run along the summed index are read 4
// of its steps at a time: their row strides are 4 above a multiple of 32 values,
// which spreads the 16 rows of a load over all banks.  (With single values
// loaded, 8 loads for 16 multiply-adds, the loads bound the kernels.)
enum Columns { kStrided, kQuads };
template <Columns C, int NJ>
__device__ __forceinline__ int column(int j)
{
    const int tx = threadIdx.x & 15;
    return C == kStrided ? tx + 16 * j : NJ == 2 ? 2 * tx + j : 4 * tx + (j & 3) + 64 * (j >> 2);
}

// acc[i][j] += sum_k A(row i, k) B(k, column j).  AT: A lies as [k][row], else as
// [row][k]; BT: B lies as [column][k] (columns kStrided), else as [k][column].
// Not AT: K is rounded up to a multiple of 4, with zeros behind.
template <int MI, int NJ, bool AT, bool BT, Columns C, int LA, int LB>
__device__ __forceinline__ void mm(float (&acc)[MI][NJ], const float *A, const float *B, int K)
{
    static_assert(!BT || (!AT && C == kStrided), "both along k");
    const int ty = threadIdx.x >> 4;
    constexpr int S = AT ? 1 : 4;
#pragma unroll(AT ? 4 : 2)
    for (int k = 0; k < K; k += S) {
        float x[MI][S], y[S][NJ];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if constexpr (AT) x[i][0] = A[k * LA + ty + 16 * i];
            else load_vec<4>(A + (ty + 16 * i) * LA + k, x[i]);
        }
        if constexpr (BT) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                float v[4];
                load_vec<4>(B + column<C, NJ>(j) * LB + k, v);
#pragma unroll
                for (int u = 0; u < 4; ++u) y[u][j] = v[u];
            }
        } else {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                constexpr int W = C == kStrided ? 1 : NJ == 2 ? 2 : 4;
#pragma unroll
                for (int j = 0; j < NJ; j += W) {
                    float v[W];
                    load_vec<W>(B + (k + u) * LB + column<C, NJ>(j), v);
#pragma unroll
                    for (int e = 0; e < W; ++e) y[u][j + e] = v[e];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = fmaf(x[i][u], y[u][j], acc[i][j]);
    }
}

template <int MI, int NJ>
__device__ __forceinline__ void clear(float (&acc)[MI][NJ])
{
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
}

// `rows` x `cols` values, times `by`, as ROWS x CB with row stride LD; zeros
// beside and below.
template <int ROWS, int CB, int LD>
__device__ __forceinline__ void load_tile(float *to, const float *from, int64_t ld, int rows, int cols, float by = 1.f)
{
#pragma unroll 8
    for (int i = threadIdx.x; i < ROWS * CB; i += kThreads) {
        const int r = i / CB, c = i % CB;
        to[r * LD + c] = r < rows && c < cols ? __ldg(from + r * ld + c) * by : 0.f;
    }
}

// Warp 0: a chunk's gate sums as two floats (rows behind the chunk have gate
// 0).
struct Gates {
    float hi[kL], lo[kL];
};
__device__ __forceinline__ void load_gates(Gates &s, const float *g, int64_t ldg, int len)
{
    if (threadIdx.x >= 32) return;
    const int i = 2 * threadIdx.x;
    const float a = i < len ? gate_of(__ldg(g + i * ldg)) : 0.f, b = i + 1 < len ? gate_of(__ldg(g + (i + 1) * ldg)) : 0.f;
    float h = a, l = 0.f;
    add_two(h, l, b, 0.f);
    for (int o = 1; o < 32; o <<= 1) {
        const float uh = __shfl_up_sync(~0u, h, o), ul = __shfl_up_sync(~0u, l, o);
        if (int(threadIdx.x) >= o) add_two(h, l, uh, ul);
    }
    s.hi[i + 1] = h, s.lo[i + 1] = l;
    float bh = __shfl_up_sync(~0u, h, 1), bl = __shfl_up_sync(~0u, l, 1);   // before the lane's own two
    if (threadIdx.x == 0) bh = bl = 0.f;
    add_two(bh, bl, a, 0.f);
    s.hi[i] = bh, s.lo[i] = bl;
}
__device__ __forceinline__ float span(const Gates &s, int i, int j)   // e^{G_i - G_j}
{
    return expf((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j]));
}
__device__ __forceinline__ float span(const Gates &s, int i) { return expf(s.hi[i]) * (1.f + s.lo[i]); }

// What a chunk adds to the state (to its adjoint with BACK), and its total gate.
template <int NB, int PB, bool BACK>
__global__ void __launch_bounds__(kThreads) gated_add_kernel(const GatedCall p)
{
    after_previous();
    extern __shared__ float sm[];
    __shared__ Gates gates;
    const GatedArgs &a = p.a;
    const int c = int(blockIdx.x / unsigned(a.H)), h = int(blockIdx.x % unsigned(a.H)), grp = h / (a.H / a.G);
    const Chunks::One ch = p.c.get(c);
    if (ch.len == 0) return;
    float *K = sm, *V = sm + kL * NB;
    load_gates(gates, a.g + ch.row * a.ldg + h, a.ldg, ch.len);
    load_tile<kL, NB, NB>(K, static_cast<const float *>(BACK ? a.q : a.k) + ch.row * (BACK ? a.ldq : a.ldk) + grp * a.N,
                          BACK ? a.ldq : a.ldk, ch.len, a.N, BACK ? a.scale : 1.f);
    load_tile<kL, PB, PB>(V, static_cast<const float *>(BACK ? a.dout : a.v) + ch.row * (BACK ? a.lddo : a.ldv) + h * a.P,
                          BACK ? a.lddo : a.ldv, ch.len, a.P);
    __syncthreads();
    __shared__ float by[kL];
    if (threadIdx.x < kL) by[threadIdx.x] = BACK ? span(gates, threadIdx.x) : span(gates, kL - 1, threadIdx.x);
    __syncthreads();
    for (int i = threadIdx.x; i < kL * PB; i += kThreads) V[i] *= by[i / PB];
    __syncthreads();
    float acc[NB / 16][PB / 16];
    clear(acc);
    mm<NB / 16, PB / 16, true, false, kQuads, NB, PB>(acc, K, V, ch.len);
    float *out = (BACK ? p.adjoints : p.states) + (int64_t(c) * a.H + h) * a.N * a.P;
    const int ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < NB / 16; ++i)
#pragma unroll
        for (int j = 0; j < PB / 16; ++j) {
            const int n = ty + 16 * i, q = column<kQuads, PB / 16>(j);
            if (n < a.N && q < a.P) out[n * a.P + q] = acc[i][j];
        }
    if (threadIdx.x == 0) p.totals[int64_t(c) * a.H + h] = gates.hi[kL - 1];
}

// o of a chunk and head.
template <int NB, int PB>
__global__ void __launch_bounds__(kThreads) gated_out_kernel(const GatedCall p)
{
    after_previous();
    extern __shared__ float sm[];
    __shared__ Gates gates;
    constexpr int LN = NB + 4, LP = kL + 4, KN = LN > LP ? LN : LP, SR = kStaged / PB < NB ? kStaged / PB : NB;
    const GatedArgs &a = p.a;
    const int c = int(blockIdx.x / unsigned(a.H)), h = int(blockIdx.x % unsigned(a.H)), grp = h / (a.H / a.G);
    const Chunks::One ch = p.c.get(c);
    if (ch.len == 0) return;
    float *Q = sm, *K = Q + kL * LN, *V = K + kL * KN, *St = V + kL * PB, *W = K;   // weights take K's place
    load_gates(gates, a.g + ch.row * a.ldg + h, a.ldg, ch.len);
    load_tile<kL, NB, LN>(Q, static_cast<const float *>(a.q) + ch.row * a.ldq + grp * a.N, a.ldq, ch.len, a.N, a.scale);
    load_tile<kL, NB, LN>(K, static_cast<const float *>(a.k) + ch.row * a.ldk + grp * a.N, a.ldk, ch.len, a.N);
    load_tile<kL, PB, PB>(V, static_cast<const float *>(a.v) + ch.row * a.ldv + h * a.P, a.ldv, ch.len, a.P);
    __syncthreads();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float w[4][4];
    clear(w);
    mm<4, 4, false, true, kStrided, LN, LN>(w, Q, K, a.N);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = ty + 16 * i, q = tx + 16 * j;
            W[r * LP + q] = q <= r ? w[i][j] * span(gates, r, q) : 0.f;
        }
    // Q S, the state SR rows at a time
    float acc[4][PB / 16];
    clear(acc);
    const float *S = p.states + (int64_t(c) * a.H + h) * a.N * a.P;
    for (int n0 = 0; n0 < a.N; n0 += SR) {
        const int rows = a.N - n0 < SR ? a.N - n0 : SR;
        if (n0 > 0) __syncthreads();
        load_tile<SR, PB, PB>(St, S + n0 * a.P, a.P, rows, a.P);
        __syncthreads();
        mm<4, PB / 16, false, false, kQuads, LN, PB>(acc, Q + n0, St, rows);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float up = span(gates, ty + 16 * i);
#pragma unroll
        for (int j = 0; j < PB / 16; ++j) acc[i][j] *= up;
    }
    mm<4, PB / 16, false, false, kQuads, LP, PB>(acc, W, V, ch.len);
    float *o = static_cast<float *>(a.o) + (ch.row * a.H + h) * a.P;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < PB / 16; ++j) {
            const int r = ty + 16 * i, q = column<kQuads, PB / 16>(j);
            if (r < ch.len && q < a.P) o[int64_t(r) * a.H * a.P + q] = acc[i][j];
        }
}

// Sums over the 16 lanes that share a row.
__device__ __forceinline__ float over_row(float v)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// dv and dg of a chunk's heads, and dq and dk summed over them: a group's heads,
// or a part of them whose sums then go to `partial`.
template <int NB, int PB>
__global__ void __launch_bounds__(kThreads) gated_grad_kernel(const GatedCall p)
{
    after_previous();
    extern __shared__ float sm[];
    __shared__ Gates gates;
    __shared__ float col[8][kL], sum_row[kL], sum_key[kL], through[8];
    constexpr int LN = NB + 4, LV = PB + 4, LP = kL + 4, HN = NB < 64 ? NB : 64, NJ = NB / 16, HJ = HN / 16, PJ = PB / 16;
    const GatedArgs &a = p.a;
    const int split = int(blockIdx.x % p.splits), grp = int(blockIdx.x / p.splits % a.G);
    const int c = int(blockIdx.x / unsigned(p.splits) / unsigned(a.G));
    const Chunks::One ch = p.c.get(c);
    if (ch.len == 0) return;
    float *Q = sm, *K = Q + kL * LN, *V = K + kL * LN, *dO = V + kL * LV, *W = dO + kL * LV, *dW = W + kL * LP, *St = dW + kL * LP;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    load_tile<kL, NB, LN>(Q, static_cast<const float *>(a.q) + ch.row * a.ldq + grp * a.N, a.ldq, ch.len, a.N);
    load_tile<kL, NB, LN>(K, static_cast<const float *>(a.k) + ch.row * a.ldk + grp * a.N, a.ldk, ch.len, a.N);
    const int per_group = a.H / a.G, h0 = split * p.heads, h1 = h0 + p.heads < per_group ? h0 + p.heads : per_group;
    float dq[4][NJ], dk[4][NJ];
    clear(dq), clear(dk);
    for (int hh = h0; hh < h1; ++hh) {
        const int h = grp * per_group + hh;
        __syncthreads();
        load_gates(gates, a.g + ch.row * a.ldg + h, a.ldg, ch.len);
        load_tile<kL, PB, LV>(V, static_cast<const float *>(a.v) + ch.row * a.ldv + h * a.P, a.ldv, ch.len, a.P);
        load_tile<kL, PB, LV>(dO, static_cast<const float *>(a.dout) + ch.row * a.lddo + h * a.P, a.lddo, ch.len, a.P, a.scale);
        __syncthreads();
        {
            float s[4][4], d[4][4], cols[4] = {};
            clear(s), clear(d);
            mm<4, 4, false, true, kStrided, LN, LN>(s, Q, K, a.N);
            mm<4, 4, false, true, kStrided, LV, LV>(d, dO, V, a.P);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i;
                float row = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = tx + 16 * j;
                    const float by = q <= r ? span(gates, r, q) : 0.f;
                    const float w = q <= r ? s[i][j] * by : 0.f, dw = q <= r ? d[i][j] * by : 0.f;
                    const float both = q < r ? s[i][j] * dw : 0.f;
                    W[r * LP + q] = w, dW[r * LP + q] = dw;
                    row += both, cols[j] += both;
                }
                row = over_row(row);
                if (tx == 0) sum_row[r] = row;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cols[j] += __shfl_xor_sync(~0u, cols[j], 16);
                if (lane < 16) col[warp][tx + 16 * j] = cols[j];
            }
        }
        __syncthreads();
        mm<4, NJ, false, false, kStrided, LP, LN>(dq, dW, K, kL);
        mm<4, NJ, true, false, kStrided, LP, LN>(dk, dW, Q, kL);
        float dv[4][PJ], in_d[4][PJ];
        clear(dv), clear(in_d);
        mm<4, PJ, true, false, kQuads, LP, LV>(dv, W, dO, kL);
        float of_q[4] = {}, of_k[4] = {}, dot = 0.f;
        const float *S = p.states + (int64_t(c) * a.H + h) * a.N * a.P, *D = p.adjoints + (int64_t(c) * a.H + h) * a.N * a.P;
#pragma unroll
        for (int n0 = 0; n0 < NB; n0 += HN) {
            const int rows = a.N - n0 < HN ? a.N - n0 : HN;   // below 1: none
            // the adjoint behind the chunk
            __syncthreads();
            load_tile<HN, PB, LV>(St, D + n0 * a.P, a.P, rows, a.P);
            __syncthreads();
            float t[4][HJ];
            clear(t);
            mm<4, HJ, false, true, kStrided, LV, LV>(t, V, St, a.P);
            mm<4, PJ, false, false, kQuads, LN, LV>(in_d, K + n0, St, rows);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float tail = span(gates, kL - 1, ty + 16 * i);
#pragma unroll
                for (int j = 0; j < HJ; ++j) {
                    const float x = t[i][j] * tail;
                    dk[i][n0 / 16 + j] += x;
                    of_k[i] = fmaf(x, K[(ty + 16 * i) * LN + n0 + tx + 16 * j], of_k[i]);
                }
            }
            // <S, D>, and the state before the chunk
            for (int i = tid; i < rows * a.P; i += kThreads) dot = fmaf(__ldg(S + n0 * a.P + i), St[i / a.P * LV + i % a.P], dot);
            __syncthreads();
            load_tile<HN, PB, LV>(St, S + n0 * a.P, a.P, rows, a.P);
            __syncthreads();
            clear(t);
            mm<4, HJ, false, true, kStrided, LV, LV>(t, dO, St, a.P);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float up = span(gates, ty + 16 * i);
#pragma unroll
                for (int j = 0; j < HJ; ++j) {
                    const float x = t[i][j] * up;
                    dq[i][n0 / 16 + j] += x;
                    of_q[i] = fmaf(x, Q[(ty + 16 * i) * LN + n0 + tx + 16 * j], of_q[i]);
                }
            }
        }
        float *out = static_cast<float *>(a.dv) + (ch.row * a.H + h) * a.P;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 16 * i;
            const float tail = span(gates, kL - 1, r);
#pragma unroll
            for (int j = 0; j < PJ; ++j) {
                const int q = column<kQuads, PJ>(j);
                if (r < ch.len && q < a.P) out[int64_t(r) * a.H * a.P + q] = fmaf(tail, in_d[i][j], dv[i][j]);
            }
            const float x = over_row(of_q[i]), y = over_row(of_k[i]);
            if (tx == 0) sum_row[r] += x, sum_key[r] = y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
        if (lane == 0) through[warp] = dot;
        __syncthreads();
        if (warp == 0) {   // dg: two rows a lane
            float x[2], z[2];
            for (int u = 0; u < 2; ++u) {
                const int r = 2 * lane + u;
                x[u] = sum_row[r], z[u] = sum_key[r];
                for (int w = 0; w < 8; ++w) x[u] -= col[w][r];
            }
            float after = x[0] + x[1], before = z[0] + z[1], whole = 0.f;
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_down_sync(~0u, after, o), v = __shfl_up_sync(~0u, before, o);
                if (lane + o < 32) after += u;
                if (lane >= o) before += v;
            }
            before -= z[1];
            for (int w = 0; w < 8; ++w) whole += through[w];
            whole *= expf(gates.hi[kL - 1]);
            float *dg = a.dg + ch.row * a.H + h;
            if (2 * lane < ch.len) dg[int64_t(2 * lane) * a.H] = after + (before - z[0]) + whole;
            if (2 * lane + 1 < ch.len) dg[int64_t(2 * lane + 1) * a.H] = (after - x[0]) + before + whole;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int r = ty + 16 * i, n = tx + 16 * j;
            if (r >= ch.len || n >= a.N) continue;
            const int64_t at = (ch.row + r) * a.G * a.N + grp * a.N + n;
            if (p.splits == 1) {
                static_cast<float *>(a.dq)[at] = dq[i][j];
                static_cast<float *>(a.dk)[at] = dk[i][j];
            } else {
                float *part = p.partial + (int64_t(split) * 2 * a.B * a.T * a.G * a.N) + at;
                part[0] = dq[i][j], part[a.B * a.T * a.G * a.N] = dk[i][j];
            }
        }
}

// dq and dk from their parts.
__global__ void __launch_bounds__(256) gated_join_kernel(const float *part, int splits, int64_t n, float *dq, float *dk)
{
    after_previous();
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < 2 * n; i += int64_t(gridDim.x) * 256) {
        float v = 0.f;
        for (int s = 0; s < splits; ++s) v += part[s * 2 * n + i];
        *(i < n ? dq + i : dk + (i - n)) = v;
    }
}

// ------------------------------------------------------------------ tokens

// Bytes bound it: the state is read and written once (256 x 32 heads of 128 x 64:
// 82 us, 6.6 TB/s).  One row of 16 heads of 128 x 128 takes 6.7 us: the latency of a
// launch, and of a thread's four rounds of loads and stores, one behind the other,
// on 16 of the SMs.
// A block takes a row's head: a state of N x P, walked by rows of P values, VEC
// a thread; the threads beside each other in P share an n, and the others' sums
// are joined at the end.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedStepArgs p)
{
    __shared__ float acc[256 * VEC];
    __shared__ float qs[kGatedMax], ks[kGatedMax];
    const int64_t row = blockIdx.x / p.H;
    const int h = int(blockIdx.x % p.H), grp = h / (p.H / p.G);
    const int per = (p.P + VEC - 1) / VEC, rows = 256 / per;   // threads along P, rows of the state at a time
    const int x = threadIdx.x % per, y = threadIdx.x / per;
    const int64_t slot = p.slots != nullptr ? p.slots[row] : row;
    T *o = static_cast<T *>(p.o) + (row * p.H + h) * p.P;
    if (slot < 0 || slot >= p.nslots) {
        for (int i = threadIdx.x; i < p.P; i += 256) store1(o + i, 0.f);
        return;
    }
    const T *q = static_cast<const T *>(p.q) + row * p.ldq + grp * p.N, *k = static_cast<const T *>(p.k) + row * p.ldk + grp * p.N;
    for (int i = threadIdx.x; i < p.N; i += 256) qs[i] = load1(q + i), ks[i] = load1(k + i);
    float v[VEC], s[VEC];
    if (y < rows)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = load1(static_cast<const T *>(p.v) + row * p.ldv + h * p.P + x * VEC + e), s[e] = 0.f;
    const float d = expf(gate_of(p.g[row * p.ldg + h]));
    float *S = p.state + ((slot * p.H + h) * p.N) * p.P + x * VEC;
    __syncthreads();
    if (y < rows)
        for (int n0 = y; n0 < p.N; n0 += 4 * rows) {
            float old[4][VEC];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (n0 + u * rows < p.N) load_vec<VEC>(S + int64_t(n0 + u * rows) * p.P, old[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int n = n0 + u * rows;
                if (n >= p.N) continue;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    old[u][e] = fmaf(d, old[u][e], ks[n] * v[e]);
                    s[e] = fmaf(qs[n], old[u][e], s[e]);
                }
                store_vec<VEC>(S + int64_t(n) * p.P, old[u]);
            }
        }
    if (y < rows) store_vec<VEC>(acc + (y * per + x) * VEC, s);
    __syncthreads();
    for (int i = threadIdx.x; i < p.P; i += 256) {
        float sum = 0.f;
        for (int r = 0; r < rows; ++r) sum += acc[r * per * VEC + i];
        store1(o + i, p.scale * sum);
    }
}

// ------------------------------------------------------------------- host

// How many blocks take a group's heads, so that about `kWant` run in all; what
// more than one takes is summed afterwards.
int splits_for(int64_t chunks, int H, int G)
{
    constexpr int64_t kWant = 2 * 152;
    const int per = H / G;
    int64_t n = ceil_div(kWant, chunks * G > 0 ? chunks * G : 1);
    n = n > per ? per : n;
    const int heads = int(ceil_div(per, n));
    return int(ceil_div(per, heads));
}

// The call's first kernel, or the second where a chunk table comes before it.
template <int NB, int PB, bool BACK>
mg_status add_chunks(const GatedCall &p, int64_t blocks, size_t smem, cudaStream_t s)
{
    if (p.a.cu != nullptr) return launch_next("mg_gated_scan", gated_add_kernel<NB, PB, BACK>, blocks, dim3(kThreads), smem, s, p);
    gated_add_kernel<NB, PB, BACK><<<unsigned(blocks), kThreads, smem, s>>>(p);
    return launched("mg_gated_scan");
}

template <int NB, int PB>
mg_status fwd_sized(const GatedCall &p, cudaStream_t s)
{
    const GatedArgs &a = p.a;
    const int64_t blocks = int64_t(p.c.most) * a.H;
    constexpr int LN = NB + 4, KN = LN > kL + 4 ? LN : kL + 4;
    constexpr size_t add = size_t(kL) * (NB + PB) * 4, out = (size_t(kL) * (LN + KN + PB) + kStaged) * 4;
    MG_TRY((allow_shared<gated_add_kernel<NB, PB, false>, kRoom>(add)));
    MG_TRY((allow_shared<gated_out_kernel<NB, PB>, kRoom>(out)));
    MG_TRY((add_chunks<NB, PB, false>(p, blocks, add, s)));
    MG_TRY(launch_over_chunks(p.c, p.states, p.totals, a.S0, a.S_last, a.H, int64_t(a.N) * a.P, false, s));
    return launch_next("mg_gated_scan_fwd", gated_out_kernel<NB, PB>, blocks, dim3(kThreads), out, s, p);
}

template <int NB, int PB>
mg_status bwd_sized(const GatedCall &p, cudaStream_t s)
{
    const GatedArgs &a = p.a;
    const int64_t blocks = int64_t(p.c.most) * a.H, grads = int64_t(p.c.most) * a.G * p.splits;
    constexpr size_t add = size_t(kL) * (NB + PB) * 4;
    constexpr size_t grad = size_t(kL) * (2 * (NB + 4) + 2 * (PB + 4) + 2 * (kL + 4)) * 4 + size_t(NB < 64 ? NB : 64) * (PB + 4) * 4;
    MG_TRY((allow_shared<gated_add_kernel<NB, PB, true>, kRoom>(add)));
    MG_TRY((allow_shared<gated_grad_kernel<NB, PB>, kRoom>(grad)));
    MG_TRY((add_chunks<NB, PB, true>(p, blocks, add, s)));
    MG_TRY(launch_over_chunks(p.c, p.adjoints, p.totals, a.dS_last, a.dS0, a.H, int64_t(a.N) * a.P, true, s));
    MG_TRY(launch_next("mg_gated_scan_bwd", gated_grad_kernel<NB, PB>, grads, dim3(kThreads), grad, s, p));
    if (p.splits == 1) return MG_OK;
    const int64_t n = a.B * a.T * a.G * a.N, want = ceil_div(2 * n, 256);
    return launch_next("mg_gated_scan_bwd", gated_join_kernel, want < 8192 ? want : 8192, dim3(256), 0, s, p.partial, p.splits, n,
                       static_cast<float *>(a.dq), static_cast<float *>(a.dk));
}

// F<NB, PB> for the sizes that hold N and P.
#define MG_GATED_P(F, NB)                           \
    if (p.a.P <= 32) return F<NB, 32>(p, s);        \
    if (p.a.P <= 64) return F<NB, 64>(p, s);        \
    return F<NB, 128>(p, s);
#define MG_GATED(F)                                 \
    if (p.a.N <= 32) { MG_GATED_P(F, 32) }          \
    if (p.a.N <= 64) { MG_GATED_P(F, 64) }          \
    MG_GATED_P(F, 128)
mg_status fwd_any(const GatedCall &p, cudaStream_t s) { MG_GATED(fwd_sized) }
mg_status bwd_any(const GatedCall &p, cudaStream_t s) { MG_GATED(bwd_sized) }

// The call's chunks, checked against what a grid and the chunk table's 32-bit
// counts hold.
mg_status make_call(const GatedArgs &a, bool bwd, GatedCall &p)
{
    const bool packed = a.cu != nullptr;
    const GatedWs w = gated_ws(a.B, a.T, a.H, a.N, a.P, a.nseq, packed, kL, bwd || a.saved == nullptr);
    char *ws = static_cast<char *>(a.ws);
    p.a = a;
    p.c.q = make_seqs(a.cu, a.B, a.T, a.nseq);
    p.c.first = reinterpret_cast<const int *>(ws + w.first);
    p.c.per = int(ceil_div(a.T, kL)), p.c.L = kL, p.c.most = int(w.chunks);
    p.totals = reinterpret_cast<float *>(ws + w.totals);
    float *states = reinterpret_cast<float *>(ws + w.states);
    p.states = bwd ? const_cast<float *>(a.saved_in) : a.saved != nullptr ? a.saved : states;
    p.adjoints = bwd ? states : nullptr;
    p.partial = reinterpret_cast<float *>(ws + w.more);
    p.splits = splits_for(w.chunks, a.H, a.G);
    p.heads = int(ceil_div(a.H / a.G, p.splits));
    return check_grids(bwd ? "mg_gated_scan_bwd" : "mg_gated_scan_fwd",
                       {w.chunks * a.H, w.chunks * a.G * p.splits, a.nseq * a.H * ceil_div(int64_t(a.N) * a.P, 256)});
}

}  // namespace

mg_status launch_chunk_tables(const Chunks &c, const Chunks &d, void *ws, cudaStream_t s)
{
    chunk_table_kernel<<<c.first == d.first ? 1 : 2, 1024, 0, s>>>(c, d, ws);
    return launched("chunk tables");
}

mg_status launch_over_chunks(const Chunks &c, float *states, const float *totals, const float *from, float *to, int H,
                             int64_t NP, bool backward, cudaStream_t s)
{
    const int vec = NP % 4 == 0 ? 4 : 1;
    const int per = int(ceil_div(NP, 256 * vec));
    auto *kernel = vec == 4 ? (backward ? over_chunks_kernel<4, true> : over_chunks_kernel<4, false>)
                            : (backward ? over_chunks_kernel<1, true> : over_chunks_kernel<1, false>);
    return launch_next("pass over chunks", kernel, int64_t(c.q.nseq) * H * per, dim3(256), 0, s, c, states, totals, from, to, H, NP, per);
}

size_t gated_saved_bytes(int64_t B, int64_t T, int64_t H, int64_t N, int64_t P, int64_t nseq, bool packed, mg_dtype dt)
{
    if (dt == MG_BF16) return gated_tc_saved_bytes(B, T, int(H), int(N), int(P), nseq, packed);
    return size_t(chunks_most(B, T, nseq, packed, kL)) * H * N * P * 4;
}

size_t gated_ws_bytes(int64_t B, int64_t T, int64_t H, int64_t G, int64_t N, int64_t P, int64_t nseq, bool packed,
                      mg_dtype dt, bool bwd)
{
    if (dt == MG_BF16) return gated_tc_ws_bytes(B, T, int(H), int(G), int(N), int(P), nseq, packed, bwd);
    const GatedWs w = gated_ws(B, T, H, N, P, nseq, packed, kL, true);
    const int splits = bwd ? splits_for(w.chunks, int(H), int(G)) : 1;
    return w.more + (splits > 1 ? size_t(splits) * 2 * B * T * G * N * 4 : 0);
}

mg_status launch_gated_fwd(const GatedArgs &a, mg_dtype dt, cudaStream_t s)
{
    if (dt == MG_BF16) return launch_gated_tc_fwd(a, s);
    GatedCall p{};
    MG_TRY(make_call(a, false, p));
    if (a.cu != nullptr) MG_TRY(launch_chunk_tables(p.c, p.c, a.ws, s));
    return fwd_any(p, s);
}

mg_status launch_gated_bwd(const GatedArgs &a, mg_dtype dt, cudaStream_t s)
{
    if (dt == MG_BF16) return launch_gated_tc_bwd(a, s);
    GatedCall p{};
    MG_TRY(make_call(a, true, p));
    if (a.cu != nullptr) MG_TRY(launch_chunk_tables(p.c, p.c, a.ws, s));
    return bwd_any(p, s);
}

mg_status launch_gated_step(const GatedStepArgs &p, mg_dtype dt, cudaStream_t s)
{
    const int64_t blocks = p.B * p.H;
    MG_TRY(check_grids("mg_gated_scan_step", {blocks}));
    const bool vec = p.P % 4 == 0;
    if (dt == MG_F32) {
        if (vec) gated_step_kernel<float, 4><<<unsigned(blocks), 256, 0, s>>>(p);
        else gated_step_kernel<float, 1><<<unsigned(blocks), 256, 0, s>>>(p);
    } else {
        if (vec) gated_step_kernel<bf16_t, 4><<<unsigned(blocks), 256, 0, s>>>(p);
        else gated_step_kernel<bf16_t, 1><<<unsigned(blocks), 256, 0, s>>>(p);
    }
    return launched("mg_gated_scan_step");
}

}  // namespace mg
