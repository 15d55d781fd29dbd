// Short causal depthwise convolution, channels last, with an optional SiLU:
//   v_r = bias + sum_{k<W} w_k x_{r-W+1+k},  y_r = silu(v_r)
// and its gradients.
//
// The rows of a batch lie back to back (row r of B*T, or of the packed
// batch); a thread owns VEC neighbouring channels and walks a run of rows
// with the last W-1 inputs in registers, so each input is read once but for
// the W-1 rows before its run.  At a sequence's first row the window is
// loaded from the sequence's x0 (a select, so nothing of the sequence before
// reaches it).  The kernels move 2 W + 4 flops a value: memory bounds them.
#include "ssm.cuh"

namespace mg {
namespace {

constexpr int kUnroll = 4;   // rows loaded before the first of them is used

// A thread's place: its channels and its run of rows.
struct Place {
    int64_t d, r0, r1;
    bool live;
};

__device__ __forceinline__ Place place(int64_t chan_blocks, int vec, int64_t D, int64_t rows,
                                       int64_t run)
{
    const int64_t cb = blockIdx.x % chan_blocks, rb = blockIdx.x / chan_blocks;
    Place w;
    w.d = (cb * blockDim.x + threadIdx.x) * vec;
    w.r0 = (rb * blockDim.y + threadIdx.y) * run;
    w.r1 = w.r0 + run < rows ? w.r0 + run : rows;
    w.live = w.d < D && w.r0 < rows;
    return w;
}

// The sequence a run is in.  lo and hi are its bounds, lo kept within
// [0, row] whatever cu holds.
struct Walk {
    int s;
    long long lo, hi;
    __device__ __forceinline__ void start(const Seqs &q, long long r)
    {
        s = q.of(r);
        lo = q.begin(s);
        hi = q.begin(s + 1);
        lo = lo < 0 ? 0 : (lo > r ? r : lo);
    }
};

// A sequence's edge state (W-1 rows), x0 or dx_last: row j, or zero.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_edge(const T *edge, int s, int j, int64_t D, int64_t d,
                                          float (&o)[VEC])
{
    if (edge != nullptr) {
        load_vec<VEC>(edge + (int64_t(s) * (W - 1) + j) * D + d, o);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = 0.f;
    }
}

// An empty sequence hands its edge state on: dst[s] = src[s] (or zero).
template <typename T, int VEC, int W>
__device__ __forceinline__ void copy_edge(T *dst, const T *src, int s, int64_t D, int64_t d)
{
    if (dst == nullptr) return;
    for (int j = 0; j < W - 1; ++j) {
        float o[VEC];
        load_edge<T, VEC, W>(src, s, j, D, d, o);
        store_vec<VEC>(dst + (int64_t(s) * (W - 1) + j) * D + d, o);
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs p, Seqs q, int64_t chan_blocks,
                                                       int64_t run)
{
    if (blockIdx.x == 0)
        check_cu(q, error_word(p.ws), threadIdx.y * blockDim.x + threadIdx.x,
                 blockDim.x * blockDim.y);
    const Place at = place(chan_blocks, VEC, p.D, q.rows, run);
    if (!at.live) return;
    const int64_t D = p.D, d = at.d;
    const T *x = static_cast<const T *>(p.x), *x0 = static_cast<const T *>(p.x0);
    T *y = static_cast<T *>(p.y), *x_last = static_cast<T *>(p.x_last);
    float w[W][VEC], bias[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        bias[v] = p.bias != nullptr ? __ldg(p.bias + d + v) : 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][v] = __ldg(p.w + (d + v) * W + k);
    }
    Walk k;
    k.start(q, at.r0);
    if (k.lo == at.r0)   // empty sequences that lie at this row
        for (int e = k.s - 1; e >= 0 && q.begin(e) == at.r0; --e) copy_edge<T, VEC, W>(x_last, x0, e, D, d);
    float win[W][VEC];   // inputs r-W+1 .. r
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t r = at.r0 - (W - 1) + j;
        if (r >= k.lo) load_vec<VEC>(x + r * p.ldx + d, win[j + 1]);
        else load_edge<T, VEC, W>(x0, k.s, int(r - k.lo + W - 1), D, d, win[j + 1]);
    }
    for (int64_t rb = at.r0; rb < at.r1; rb += kUnroll) {
        Raw<T, VEC> in[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (rb + i < at.r1) in[i].load(x + (rb + i) * p.ldx + d);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t r = rb + i;
            if (r >= at.r1) break;
            if (r == k.hi) {   // a new sequence (empty ones on the way)
                ++k.s;
                while (k.s + 1 < q.nseq && q.begin(k.s + 1) <= r) {
                    copy_edge<T, VEC, W>(x_last, x0, k.s, D, d);
                    ++k.s;
                }
                if (k.s >= q.nseq) k.s = q.nseq - 1;
                k.hi = q.begin(k.s + 1);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) load_edge<T, VEC, W>(x0, k.s, j, D, d, win[j + 1]);
            }
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) win[j][v] = win[j + 1][v];
                win[W - 1][v] = in[i][v];
                float a = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) a = fmaf(w[j][v], win[j][v], a);
                o[v] = p.silu ? a * sigmoid_f(a) : a;
            }
            store_vec<VEC>(y + r * D + d, o);
            if (r + 1 == k.hi && x_last != nullptr) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    store_vec<VEC>(x_last + (int64_t(k.s) * (W - 1) + j) * D + d, win[j + 1]);
            }
        }
    }
    if (at.r1 == q.rows)   // empty sequences at the end
        for (int e = k.s + 1; e < q.nseq; ++e) copy_edge<T, VEC, W>(x_last, x0, e, D, d);
}

// Gradients.  The walk carries, next to the window, the sums that the rows
// r-W+2 .. r of dx have so far: row r sends w_k dv_r to row r-W+1+k, and the
// oldest of them is then complete.  A run goes W-1 rows past its end for its
// last rows' sums.  dw and dbias are summed over the run in registers, over
// the block in shared memory and over the blocks by sum_parts_kernel.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(256) conv_bwd_kernel(ConvArgs p, Seqs q, int64_t chan_blocks,
                                                       int64_t run, float *part)
{
    extern __shared__ float sums[];   // [blockDim.y][blockDim.x][VEC * (W + 1)]
    constexpr int NS = VEC * (W + 1);
    if (blockIdx.x == 0)
        check_cu(q, error_word(p.ws), threadIdx.y * blockDim.x + threadIdx.x,
                 blockDim.x * blockDim.y);
    const Place at = place(chan_blocks, VEC, p.D, q.rows, run);
    const int64_t D = p.D, d = at.d, rows = q.rows;
    float dw[W][VEC] = {}, db[VEC] = {};
    if (at.live) {
        const T *x = static_cast<const T *>(p.x), *x0 = static_cast<const T *>(p.x0);
        const T *dy = static_cast<const T *>(p.dy), *dx_last = static_cast<const T *>(p.dx_last);
        T *dx = static_cast<T *>(p.dx), *dx0 = static_cast<T *>(p.dx0);
        float w[W][VEC], bias[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            bias[v] = p.bias != nullptr ? __ldg(p.bias + d + v) : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][v] = __ldg(p.w + (d + v) * W + k);
        }
        Walk k;
        k.start(q, at.r0);
        if (k.lo == at.r0)
            for (int e = k.s - 1; e >= 0 && q.begin(e) == at.r0; --e)
                copy_edge<T, VEC, W>(dx0, dx_last, e, D, d);
        float win[W][VEC], acc[W][VEC] = {};
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t r = at.r0 - (W - 1) + j;
            if (r >= k.lo) load_vec<VEC>(x + r * p.ldx + d, win[j + 1]);
            else load_edge<T, VEC, W>(x0, k.s, int(r - k.lo + W - 1), D, d, win[j + 1]);
        }
        // dx of row r, or of a row before the sequence, is complete.
        auto emit = [&](int64_t r, const float (&v)[VEC]) {
            if (r >= k.lo) {
                if (r >= at.r0 && r < at.r1) store_vec<VEC>(dx + r * D + d, v);
            } else if (dx0 != nullptr && k.lo >= at.r0 && k.lo < at.r1 && r >= k.lo - (W - 1)) {
                store_vec<VEC>(dx0 + (int64_t(k.s) * (W - 1) + (r - k.lo + W - 1)) * D + d, v);
            }
        };
        const int64_t stop = at.r1 + W - 1 < rows ? at.r1 + W - 1 : rows;
        bool done = false;
        for (int64_t rb = at.r0; rb < stop && !done; rb += kUnroll) {
            Raw<T, VEC> in[kUnroll], gy[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i)
                if (rb + i < stop) {
                    in[i].load(x + (rb + i) * p.ldx + d);
                    gy[i].load(dy + (rb + i) * p.lddy + d);
                }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t r = rb + i;
                if (r >= stop || done) break;
                if (r == k.hi) {
                    ++k.s;
                    while (k.s + 1 < q.nseq && q.begin(k.s + 1) <= r) {
                        copy_edge<T, VEC, W>(dx0, dx_last, k.s, D, d);
                        ++k.s;
                    }
                    if (k.s >= q.nseq) k.s = q.nseq - 1;
                    k.lo = r;
                    k.hi = q.begin(k.s + 1);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        load_edge<T, VEC, W>(x0, k.s, j, D, d, win[j + 1]);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) acc[j + 1][v] = 0.f;
                    }
                }
                const bool own = r < at.r1;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) {
                        win[j][v] = win[j + 1][v];
                        acc[j][v] = acc[j + 1][v];
                    }
                    win[W - 1][v] = in[i][v];
                    acc[W - 1][v] = 0.f;
                    float dv = gy[i][v];
                    if (p.silu) {
                        float a = bias[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) a = fmaf(w[j][v], win[j][v], a);
                        const float sg = sigmoid_f(a);
                        dv *= sg * fmaf(a, 1.f - sg, 1.f);
                    }
                    if (own) db[v] += dv;
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        acc[j][v] = fmaf(w[j][v], dv, acc[j][v]);
                        if (own) dw[j][v] = fmaf(dv, win[j][v], dw[j][v]);
                    }
                }
                emit(r - (W - 1), acc[0]);
                if (r + 1 == k.hi) {   // the sequence ends: the rest is complete too
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        float o[VEC];
                        load_edge<T, VEC, W>(dx_last, k.s, j, D, d, o);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) o[v] += acc[j + 1][v];
                        emit(r - (W - 2) + j, o);
                    }
                    done = r + 1 >= at.r1;
                }
            }
        }
        if (at.r1 == rows)
            for (int e = k.s + 1; e < q.nseq; ++e) copy_edge<T, VEC, W>(dx0, dx_last, e, D, d);
    }
    // the block's sums over its runs, in order
    float *mine = sums + (threadIdx.y * blockDim.x + threadIdx.x) * NS;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) mine[v * W + k] = dw[k][v];
        mine[VEC * W + v] = db[v];
    }
    __syncthreads();
    if (threadIdx.y == 0 && d < D) {
        const int64_t rb = blockIdx.x / chan_blocks;
        float *out = part + rb * D * (W + 1);
        for (int i = 0; i < NS; ++i) {
            float a = 0.f;
            for (int yy = 0; yy < blockDim.y; ++yy) a += sums[(yy * blockDim.x + threadIdx.x) * NS + i];
            if (i < VEC * W) out[d * W + i] = a;
            else out[D * W + d + (i - VEC * W)] = a;
        }
    }
}

// One token: the state's rows move up by one and x enters as the last.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvStepArgs p)
{
    const int64_t per = (p.D + VEC - 1) / VEC;
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= p.B * per) return;
    const int64_t b = i / per, d = (i - b * per) * VEC, D = p.D;
    const int64_t slot = p.slots != nullptr ? __ldg(p.slots + b) : b;
    T *y = static_cast<T *>(p.y) + b * D + d;
    float o[VEC];
    if (slot < 0 || slot >= p.nslots) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = 0.f;
        store_vec<VEC>(y, o);
        return;
    }
    T *st = static_cast<T *>(p.state) + slot * (W - 1) * D + d;
    float win[W][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_vec<VEC>(st + j * D, win[j]);
    load_vec<VEC>(static_cast<const T *>(p.x) + b * p.ldx + d, win[W - 1]);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float a = p.bias != nullptr ? __ldg(p.bias + d + v) : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) a = fmaf(__ldg(p.w + (d + v) * W + j), win[j][v], a);
        o[v] = p.silu ? a * sigmoid_f(a) : a;
    }
    store_vec<VEC>(y, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_vec<VEC>(st + j * D, win[j + 1]);
}

// out[i] = sum_j part[j * stride + i]: 8 threads take every 8th part of a
// column, and their sums are added in order.
__global__ void __launch_bounds__(256) sum_parts_kernel(const float *part, int64_t parts,
                                                        int64_t stride, int64_t n, float *out)
{
    __shared__ float s[8][33];
    const int64_t i = int64_t(blockIdx.x) * 32 + threadIdx.x;
    float a = 0.f;
    if (i < n)
        for (int64_t j = threadIdx.y; j < parts; j += 8) a += part[j * stride + i];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && i < n) {
        float t = 0.f;
        for (int k = 0; k < 8; ++k) t += s[k][threadIdx.x];
        out[i] = t;
    }
}

// How a launch cuts rows and channels.
struct Cut {
    dim3 block;
    int64_t chan_blocks, run, row_blocks;
};

// Lanes run over channels (a multiple of a warp, at most 128), the rest of
// 256 threads over runs; runs of `least` rows or more, long enough for about
// `blocks` blocks in all.
Cut cut(int64_t rows, int64_t D, int vec, int64_t least, int64_t blocks)
{
    Cut c;
    const int64_t lanes = ceil_div(D, vec);
    const int bx = lanes <= 32 ? 32 : lanes <= 64 ? 64 : 128, by = 256 / bx;
    c.block = dim3(bx, by);
    c.chan_blocks = ceil_div(lanes, bx);
    const int64_t want = ceil_div(blocks, c.chan_blocks) * by;
    c.run = ceil_div(rows, want);
    c.run = c.run < least ? least : c.run;
    c.row_blocks = ceil_div(ceil_div(rows, c.run), by);
    return c;
}

constexpr int64_t kBwdBlocks = 608;   // 4 blocks for each of 152 SMs

Cut cut_bwd(int64_t rows, int64_t D, int vec) { return cut(rows, D, vec, 16, kBwdBlocks); }

bool rows_aligned(int64_t D, int64_t ld1, int64_t ld2, int vec)
{
    return D % vec == 0 && ld1 % vec == 0 && ld2 % vec == 0;
}

template <typename T, int VEC, int W>
mg_status conv_fwd(const ConvArgs &p, cudaStream_t s)
{
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const Cut c = cut(q.rows, p.D, VEC, 16, 4096);
    conv_fwd_kernel<T, VEC, W><<<unsigned(c.chan_blocks * c.row_blocks), c.block, 0, s>>>(
        p, q, c.chan_blocks, c.run);
    return launched("mg_causal_conv_fwd");
}

template <typename T, int VEC, int W>
mg_status conv_bwd(const ConvArgs &p, cudaStream_t s)
{
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const Cut c = cut_bwd(q.rows, p.D, VEC);
    float *part = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    const size_t smem = 256 * size_t(VEC * (W + 1)) * sizeof(float);
    conv_bwd_kernel<T, VEC, W><<<unsigned(c.chan_blocks * c.row_blocks), c.block, smem, s>>>(
        p, q, c.chan_blocks, c.run, part);
    MG_TRY(launched("mg_causal_conv_bwd"));
    const int64_t n = p.D * (W + 1);
    MG_TRY(launch_sum_parts(part, c.row_blocks, n, p.D * W, p.dw, s));
    if (p.dbias != nullptr)
        return launch_sum_parts(part + p.D * W, c.row_blocks, n, p.D, p.dbias, s);
    return MG_OK;
}

template <typename T, int VEC, int W>
mg_status conv_step(const ConvStepArgs &p, cudaStream_t s)
{
    const int64_t threads = p.B * ceil_div(p.D, VEC);
    conv_step_kernel<T, VEC, W><<<unsigned(ceil_div(threads, 128)), 128, 0, s>>>(p);
    return launched("mg_causal_conv_step");
}

// Calls F<T, VEC, W> for the call's type, alignment and width.
#define MG_CONV_W(F, T, VEC, p, s)                \
    switch ((p).W) {                              \
    case 1: return F<T, VEC, 1>(p, s);            \
    case 2: return F<T, VEC, 2>(p, s);            \
    case 3: return F<T, VEC, 3>(p, s);            \
    case 4: return F<T, VEC, 4>(p, s);            \
    case 5: return F<T, VEC, 5>(p, s);            \
    case 6: return F<T, VEC, 6>(p, s);            \
    case 7: return F<T, VEC, 7>(p, s);            \
    case 8: return F<T, VEC, 8>(p, s);            \
    }                                             \
    return fail(MG_ERR_UNSUPPORTED, "W = %d outside [1, 8]", (p).W)

}  // namespace

size_t conv_ws_bytes(int64_t B, int64_t T, int64_t D, int W)
{
    // the parts of either vector width
    size_t need = 0;
    for (int vec : {1, 4}) {
        const Cut c = cut_bwd(B * T, D, vec);
        const size_t n = size_t(c.row_blocks) * D * (W + 1) * sizeof(float);
        need = n > need ? n : need;
    }
    return kControlBytes + need;
}

mg_status launch_conv_fwd(const ConvArgs &p, mg_dtype dt, cudaStream_t s)
{
    const bool wide = rows_aligned(p.D, p.ldx, p.ldx, 4);
    if (dt == MG_F32) {
        if (wide) { MG_CONV_W(conv_fwd, float, 4, p, s); }
        MG_CONV_W(conv_fwd, float, 1, p, s);
    }
    if (wide) { MG_CONV_W(conv_fwd, bf16_t, 4, p, s); }
    MG_CONV_W(conv_fwd, bf16_t, 1, p, s);
}

mg_status launch_conv_bwd(const ConvArgs &p, mg_dtype dt, cudaStream_t s)
{
    const bool wide = rows_aligned(p.D, p.ldx, p.lddy, 4);
    if (dt == MG_F32) {
        if (wide) { MG_CONV_W(conv_bwd, float, 4, p, s); }
        MG_CONV_W(conv_bwd, float, 1, p, s);
    }
    if (wide) { MG_CONV_W(conv_bwd, bf16_t, 4, p, s); }
    MG_CONV_W(conv_bwd, bf16_t, 1, p, s);
}

mg_status launch_conv_step(const ConvStepArgs &p, mg_dtype dt, cudaStream_t s)
{
    const bool wide = rows_aligned(p.D, p.ldx, p.ldx, 4);
    if (dt == MG_F32) {
        if (wide) { MG_CONV_W(conv_step, float, 4, p, s); }
        MG_CONV_W(conv_step, float, 1, p, s);
    }
    if (wide) { MG_CONV_W(conv_step, bf16_t, 4, p, s); }
    MG_CONV_W(conv_step, bf16_t, 1, p, s);
}

mg_status launch_sum_parts(const float *part, int64_t parts, int64_t stride, int64_t n, float *out,
                           cudaStream_t s)
{
    sum_parts_kernel<<<unsigned(ceil_div(n, 32)), dim3(32, 8), 0, s>>>(part, parts, stride, n, out);
    return launched("sum over parts");
}

}  // namespace mg
