// Short causal depthwise convolution, channels last, with an optional SiLU:
//   v_r = bias + sum_{k<W} w_k x_{r-W+1+k},  y_r = silu(v_r)
// and its gradients.
//
// The rows of a batch lie back to back (row r of B*T, or of the packed
// batch); a thread owns VEC neighbouring channels and walks a run of rows
// with the last W-1 inputs in registers, so each input is read once but for
// the W-1 rows before its run.  At a sequence's first row the window is
// loaded from the sequence's x0 (a select, so nothing of the sequence before
// reaches it).  A value takes 2 W + 4 flops: memory bounds the forward.  32768
// x 4096 bf16 channels, W = 4, take 97 us forward with a cold L2, 5.5 TB/s, and
// 164 us for the gradients, 4.9 TB/s; float32 reaches 5.7 and 5.1 TB/s at half
// the width.  The gradients fill neither DRAM (55% at 2048 channels) nor the
// issue slots (51%): their 128 registers leave 14 warps an SM, which wait for
// their own results.
#include "ssm.cuh"

namespace mg {
namespace {

// Rows of a group, and groups of a thread's ring.
constexpr int kUnroll = 4;
constexpr int kGroups = 3;
constexpr int kBlock = 128;
// Blocks that an SM holds: the registers allow 6 of the forward's and 4 of the
// gradients'; one more or fewer of either was slower.
constexpr int kFwdPerSm = 6, kBwdPerSm = 4;

// VEC neighbouring channels of a row.
template <typename T, int VEC>
__device__ __forceinline__ void store_lanes(T *to, const Lanes<VEC> &v)
{
    float o[VEC];
    vto<VEC>(v, o);
    store_vec<VEC>(to, o);
}
template <typename T, int VEC>
__device__ __forceinline__ Lanes<VEC> load_lanes(const T *from)
{
    float o[VEC];
    load_vec<VEC>(from, o);
    return vfrom<VEC>(o);
}

// A thread's own ring of rows in shared memory, filled by asynchronous copies
// kGroups - 1 groups ahead of the one at hand: what is in flight takes no
// registers, and no other thread reads it, so nothing but the thread's own
// copies is waited for.  A single bf16 comes as the 4-byte word that it is a
// half of, with the value before it, or alone (8 x 4096 x 1001 channels: 54
// us and 91 for the gradients, where loads at the use took 64 and 120).
template <typename T, int VEC>
struct Ring {
    static constexpr bool kHalf = sizeof(T) * VEC == 2;
    static constexpr int kBytes = kHalf ? 4 : int(sizeof(T)) * VEC;
    static constexpr size_t bytes(int threads) { return size_t(kGroups) * kUnroll * threads * kBytes; }
    unsigned char *mine;   // the thread's slot of ring row 0
    const T *next;         // the next row to be copied
    int64_t ld;
    bool upper, turns;     // kHalf: a group's first row is an upper half; its rows take turns
    __device__ __forceinline__ Ring(unsigned char *base, const T *first, int64_t stride) : next(first), ld(stride)
    {
        mine = base + (threadIdx.y * blockDim.x + threadIdx.x) * kBytes;
        upper = reinterpret_cast<uintptr_t>(first) % 4 != 0;
        turns = stride % 2 != 0;
    }
    __device__ __forceinline__ unsigned char *at(int row) const { return mine + row * kBlock * kBytes; }
    static_assert(kUnroll % 2 == 0, "a group begins like the first one");
    __device__ __forceinline__ bool half(int i) const { return upper != (turns && i % 2 != 0); }
    // Starts the copies of the rows i0 .. of a run of n into ring group g.
    __device__ __forceinline__ void fetch(int g, int i0, int n)
    {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (i0 + i < n) {
                const unsigned to = smem_addr(at(g * kUnroll + i));
                if constexpr (kHalf)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" : : "r"(to),
                                 "l"(half(i) ? next - 1 : next), "r"(half(i) ? 4 : 2) : "memory");
                else if constexpr (kBytes == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(to), "l"(next) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" : : "r"(to), "l"(next), "n"(kBytes)
                                 : "memory");
            }
            next += ld;
        }
    }
    // Row i of ring group g, the group at hand.
    __device__ __forceinline__ Lanes<VEC> get(int g, int i) const
    {
        if constexpr (kHalf) {
            const unsigned w = *reinterpret_cast<const unsigned *>(at(g * kUnroll + i));
            Lanes<VEC> v;
            v.p[0] = __uint_as_float(half(i) ? w & 0xffff0000u : w << 16);
            return v;
        } else {
            return load_lanes<T, VEC>(reinterpret_cast<const T *>(at(g * kUnroll + i)));
        }
    }
};

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

// The sequence that a run is in, its bounds counted from the run's first row
// (a run has fewer than kFar rows; lo <= 0 whatever cu holds).
constexpr int kFar = 1 << 30;
struct Walk {
    int s, lo, hi;
    __device__ __forceinline__ void bounds(const Seqs &q, long long r0)
    {
        const long long a = q.begin(s) - r0, b = q.begin(s + 1) - r0;
        lo = int(a < -kFar ? -kFar : a > kFar ? kFar : a);
        hi = int(b < -kFar ? -kFar : b > kFar ? kFar : b);
    }
    __device__ __forceinline__ void start(const Seqs &q, long long r0)
    {
        s = q.of(r0);
        bounds(q, r0);
        if (lo > 0 || lo < -r0) lo = 0;
    }
};

// A sequence's edge state (W-1 rows), x0 or dx_last: row j, or zero.
template <typename T, int VEC, int W>
__device__ __forceinline__ Lanes<VEC> load_edge(const T *edge, int s, int j, int64_t D, int64_t d)
{
    if (edge == nullptr) return vset<VEC>(0.f);
    float o[VEC];
    load_vec<VEC>(edge + (int64_t(s) * (W - 1) + j) * D + d, o);
    return vfrom<VEC>(o);
}
// An empty sequence hands its edge state on: dst[s] = src[s] (or zero).
template <typename T, int VEC, int W>
__device__ __noinline__ void copy_edge(T *dst, const T *src, int s, int64_t D, int64_t d)
{
    if (dst == nullptr) return;
    for (int j = 0; j < W - 1; ++j)
        store_lanes<T, VEC>(dst + (int64_t(s) * (W - 1) + j) * D + d, load_edge<T, VEC, W>(src, s, j, D, d));
}

// The thread's taps and bias.
template <int VEC, int W, typename Args>
__device__ __forceinline__ void load_taps(const Args &p, int64_t d, Lanes<VEC> (&w)[W], Lanes<VEC> &bias)
{
    float f[VEC], all[VEC * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        load_vec<VEC>(p.w + d * W + i * VEC, f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) all[i * VEC + v] = f[v];
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) f[v] = all[v * W + k];
        w[k] = vfrom<VEC>(f);
    }
    bias = vset<VEC>(0.f);
    if (p.bias != nullptr) {
        load_vec<VEC>(p.bias + d, f);
        bias = vfrom<VEC>(f);
    }
}

// The inputs of rows r0-W+1 .. r0-1 into win[1 ..].
template <typename T, int VEC, int W>
__device__ __forceinline__ void first_window(const T *x, const T *x0, const ConvArgs &p, const Walk &k, int64_t r0,
                                             int64_t d, Lanes<VEC> (&win)[W])
{
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int i = j - (W - 1);
        win[j + 1] = i >= k.lo ? load_lanes<T, VEC>(x + (r0 + i) * p.ldx + d)
                               : load_edge<T, VEC, W>(x0, k.s, i - k.lo + W - 1, p.D, d);
    }
}

// Moves the walk to the sequence that begins at row i of the run; empty ones
// on the way hand their edge states on.
template <typename T, int VEC, int W>
__device__ __forceinline__ void next_sequence(const Seqs &q, Walk &k, int64_t r0, int i, T *dst, const T *src,
                                              int64_t D, int64_t d)
{
    const int s = q.of(r0 + i);
    for (++k.s; k.s < s; ++k.s) copy_edge<T, VEC, W>(dst, src, k.s, D, d);
    k.s = s;
    k.bounds(q, r0);
    k.lo = i;
}

// Empty sequences that lie at the run's first row, or at the batch's end,
// hand their edge states on.
template <typename T, int VEC, int W>
__device__ __forceinline__ void empty_before(const Seqs &q, const Walk &k, int64_t r0, T *dst, const T *src,
                                             int64_t D, int64_t d)
{
    if (k.lo == 0)
        for (int e = k.s - 1; e >= 0 && q.begin(e) == r0; --e) copy_edge<T, VEC, W>(dst, src, e, D, d);
}
template <typename T, int VEC, int W>
__device__ __forceinline__ void empty_after(const Seqs &q, int64_t r1, T *dst, const T *src, int64_t D, int64_t d)
{
    if (r1 != q.rows) return;
    for (int e = q.nseq - 1; e >= 0 && q.begin(e) >= q.rows; --e) copy_edge<T, VEC, W>(dst, src, e, D, d);
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kBlock, kFwdPerSm) conv_fwd_kernel(ConvArgs p, Seqs q, int64_t chan_blocks,
                                                       int64_t run)
{
    if (blockIdx.x == 0)
        check_cu(q, error_word(p.ws), threadIdx.y * blockDim.x + threadIdx.x,
                 blockDim.x * blockDim.y);
    const Place at = place(chan_blocks, VEC, p.D, q.rows, run);
    if (!at.live) return;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    const int64_t D = p.D, d = at.d;
    const T *x = static_cast<const T *>(p.x), *x0 = static_cast<const T *>(p.x0);
    T *y = static_cast<T *>(p.y), *x_last = static_cast<T *>(p.x_last);
    Lanes<VEC> w[W], bias, win[W];   // win: inputs r-W+1 .. r
    load_taps<VEC, W>(p, d, w, bias);
    Walk k;
    k.start(q, at.r0);
    empty_before<T, VEC, W>(q, k, at.r0, x_last, x0, D, d);
    first_window<T, VEC, W>(x, x0, p, k, at.r0, d, win);
    T *yp = y + at.r0 * D + d;
    const int n = int(at.r1 - at.r0);
    Ring<T, VEC> ring(ring_bytes, x + at.r0 * p.ldx + d, p.ldx);
#pragma unroll
    for (int g = 0; g < kGroups - 1; ++g) {
        ring.fetch(g, g * kUnroll, n);
        cp_async_commit();
    }
    auto row = [&](const Lanes<VEC> &in, T *to) {
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) win[j] = win[j + 1];
        win[W - 1] = in;
        Lanes<VEC> a = bias;
#pragma unroll
        for (int j = 0; j < W; ++j) a = vfma<VEC>(w[j], win[j], a);
        if (p.silu) a = vmul<VEC>(a, vsigmoid<VEC>(a));
        float o[VEC];
        vto<VEC>(a, o);
        store_out<VEC>(to, o);
    };
    int g = 0;
    for (int i0 = 0; i0 < n; i0 += kUnroll) {
        ring.fetch(g == 0 ? kGroups - 1 : g - 1, i0 + (kGroups - 1) * kUnroll, n);
        cp_async_commit();
        cp_async_wait<kGroups - 1>();
        if (i0 + kUnroll <= n && k.hi > i0 + kUnroll) {   // whole, inside one sequence
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                row(ring.get(g, i), yp);
                yp += D;
            }
        } else {
#pragma unroll 1
            for (int i = i0; i < i0 + kUnroll && i < n; ++i) {
                if (i == k.hi) {
                    next_sequence<T, VEC, W>(q, k, at.r0, i, x_last, x0, D, d);
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) win[j + 1] = load_edge<T, VEC, W>(x0, k.s, j, D, d);
                }
                row(ring.get(g, i - i0), yp);
                yp += D;
                if (i + 1 == k.hi && x_last != nullptr) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        store_lanes<T, VEC>(x_last + (int64_t(k.s) * (W - 1) + j) * D + d, win[j + 1]);
                }
            }
        }
        g = g + 1 == kGroups ? 0 : g + 1;
    }
    cp_async_wait<0>();
    empty_after<T, VEC, W>(q, at.r1, x_last, x0, D, d);
}

// Gradients.  The walk carries, next to the window, the sums that the rows
// r-W+2 .. r of dx have so far: row r sends w_k dv_r to row r-W+1+k, and the
// oldest of them is then complete.  A run goes W-1 rows past its end for its
// last rows' sums.  dw and dbias are summed over the run in registers, over
// the block in shared memory and over the blocks by sum_parts_kernel.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kBlock, kBwdPerSm) conv_bwd_kernel(ConvArgs p, Seqs q, int64_t chan_blocks,
                                                       int64_t run, float *part)
{
    // the rings, and after them the sums [blockDim.y][VEC * (W + 1)][blockDim.x]
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    float *sums = reinterpret_cast<float *>(ring_bytes);
    constexpr int NS = VEC * (W + 1);
    if (blockIdx.x == 0)
        check_cu(q, error_word(p.ws), threadIdx.y * blockDim.x + threadIdx.x,
                 blockDim.x * blockDim.y);
    const Place at = place(chan_blocks, VEC, p.D, q.rows, run);
    const int64_t D = p.D, d = at.d, rows_all = q.rows;
    Lanes<VEC> dw[W], db = vset<VEC>(0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = vset<VEC>(0.f);
    if (at.live) {
        const T *x = static_cast<const T *>(p.x), *x0 = static_cast<const T *>(p.x0);
        const T *dy = static_cast<const T *>(p.dy), *dx_last = static_cast<const T *>(p.dx_last);
        T *dx = static_cast<T *>(p.dx), *dx0 = static_cast<T *>(p.dx0);
        Lanes<VEC> w[W], bias, win[W], acc[W];
        load_taps<VEC, W>(p, d, w, bias);
        Walk k;
        k.start(q, at.r0);
        empty_before<T, VEC, W>(q, k, at.r0, dx0, dx_last, D, d);
        first_window<T, VEC, W>(x, x0, p, k, at.r0, d, win);
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = vset<VEC>(0.f);
        const int own = int(at.r1 - at.r0);   // rows, and those past the end for their sums
        const int n = int((at.r1 + W - 1 < rows_all ? at.r1 + W - 1 : rows_all) - at.r0);
        // dx of row i of the run, or of a row before the sequence, is complete.
        auto emit = [&](int i, const Lanes<VEC> &v) {
            if (i >= k.lo) {
                if (i >= 0 && i < own) store_lanes<T, VEC>(dx + (at.r0 + i) * D + d, v);
            } else if (dx0 != nullptr && k.lo >= 0 && k.lo < own && i >= k.lo - (W - 1)) {
                store_lanes<T, VEC>(dx0 + (int64_t(k.s) * (W - 1) + (i - k.lo + W - 1)) * D + d, v);
            }
        };
        bool done = false;
        Ring<T, VEC> ring(ring_bytes, x + at.r0 * p.ldx + d, p.ldx);
        Ring<T, VEC> ring_g(ring_bytes + Ring<T, VEC>::bytes(kBlock), dy + at.r0 * p.lddy + d, p.lddy);
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g) {
            ring.fetch(g, g * kUnroll, n);
            ring_g.fetch(g, g * kUnroll, n);
            cp_async_commit();
        }
        // row i of the run: acc[0] becomes what row i - (W - 1) of dx is
        auto row = [&](const Lanes<VEC> &in_row, Lanes<VEC> dv, bool mine) {
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) {
                win[j] = win[j + 1];
                acc[j] = acc[j + 1];
            }
            win[W - 1] = in_row;
            if (p.silu) {   // silu'(v) = s (1 + v (1 - s))
                Lanes<VEC> v = bias;
#pragma unroll
                for (int j = 0; j < W; ++j) v = vfma<VEC>(w[j], win[j], v);
                const Lanes<VEC> s = vsigmoid<VEC>(v), one = vset<VEC>(1.f);
                const Lanes<VEC> rest = vfma<VEC>(s, vset<VEC>(-1.f), one);
                dv = vmul<VEC>(dv, vmul<VEC>(s, vfma<VEC>(v, rest, one)));
            }
            if (mine) {
                db = vadd<VEC>(db, dv);
#pragma unroll
                for (int j = 0; j < W; ++j) dw[j] = vfma<VEC>(dv, win[j], dw[j]);
            }
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) acc[j] = vfma<VEC>(w[j], dv, acc[j]);
            acc[W - 1] = vmul<VEC>(w[W - 1], dv);
        };
        T *dxp = dx + (at.r0 - (W - 1)) * D + d;   // of the row that the next one completes
        int g = 0;
        for (int i0 = 0; i0 < n && !done; i0 += kUnroll) {
            ring.fetch(g == 0 ? kGroups - 1 : g - 1, i0 + (kGroups - 1) * kUnroll, n);
            ring_g.fetch(g == 0 ? kGroups - 1 : g - 1, i0 + (kGroups - 1) * kUnroll, n);
            cp_async_commit();
            cp_async_wait<kGroups - 1>();
            // whole, inside one sequence and the run, and no row before the
            // sequence is completed
            if (i0 + kUnroll <= own && k.hi > i0 + kUnroll && (k.lo < 0 || i0 - (W - 1) >= k.lo)) {
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    row(ring.get(g, i), ring_g.get(g, i), true);
                    if (i0 + i >= W - 1) {
                        float o[VEC];
                        vto<VEC>(acc[0], o);
                        store_out<VEC>(dxp, o);
                    }
                    dxp += D;
                }
            } else {
#pragma unroll 1
                for (int i = i0; i < i0 + kUnroll && i < n && !done; ++i) {
                    if (i == k.hi) {
                        next_sequence<T, VEC, W>(q, k, at.r0, i, dx0, dx_last, D, d);
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) {
                            win[j + 1] = load_edge<T, VEC, W>(x0, k.s, j, D, d);
                            acc[j + 1] = vset<VEC>(0.f);
                        }
                    }
                    row(ring.get(g, i - i0), ring_g.get(g, i - i0), i < own);
                    emit(i - (W - 1), acc[0]);
                    dxp += D;
                    if (i + 1 == k.hi) {   // the sequence ends: the rest is complete too
#pragma unroll
                        for (int j = 0; j < W - 1; ++j)
                            emit(i - (W - 2) + j, vadd<VEC>(acc[j + 1], load_edge<T, VEC, W>(dx_last, k.s, j, D, d)));
                        done = i + 1 >= own;
                    }
                }
            }
            g = g + 1 == kGroups ? 0 : g + 1;
        }
        cp_async_wait<0>();
        empty_after<T, VEC, W>(q, at.r1, dx0, dx_last, D, d);
    }
    __syncthreads();   // every thread is done with its rings
    // the block's sums over its runs, in order
    const int lanes = blockDim.x;
    float *mine = sums + threadIdx.y * lanes * NS + threadIdx.x;
    float f[VEC];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        vto<VEC>(dw[k], f);
#pragma unroll
        for (int v = 0; v < VEC; ++v) mine[(v * W + k) * lanes] = f[v];
    }
    vto<VEC>(db, f);
#pragma unroll
    for (int v = 0; v < VEC; ++v) mine[(VEC * W + v) * lanes] = f[v];
    __syncthreads();
    const int64_t d00 = blockIdx.x % chan_blocks * lanes * VEC, rb = blockIdx.x / chan_blocks;
    float *out = part + rb * D * (W + 1);
    for (int e = threadIdx.y * lanes + threadIdx.x; e < lanes * NS; e += lanes * blockDim.y) {
        const int lane = e % lanes, i = e / lanes;
        const int64_t dd = d00 + lane * VEC;
        if (dd >= D) continue;
        float a = 0.f;
        for (int yy = 0; yy < blockDim.y; ++yy) a += sums[(yy * NS + i) * lanes + lane];
        if (i < VEC * W) out[dd * W + i] = a;
        else out[D * W + dd + (i - VEC * W)] = a;
    }
}

// One token: the state's rows move up by one and x enters as the last.  A
// thread has kTokens rows of the batch and loads everything before the first
// of it is used, the taps once: 256 x 4096 bf16 channels take 5.8 us of which
// the bytes need 2.5 (one row a thread 6.3, eight 8.5; with a thread for each
// row and value-wise loads of the taps it was 10.2).
constexpr int kTokens = 4;
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvStepArgs p, unsigned chan_blocks)
{
    const int64_t d = (int64_t(blockIdx.x % chan_blocks) * blockDim.x + threadIdx.x) * VEC, D = p.D;
    if (d >= D) return;
    const int64_t b0 = int64_t(blockIdx.x / chan_blocks) * kTokens;
    const int rows = int(p.B - b0 < kTokens ? p.B - b0 : kTokens);
    T *st[kTokens];
    bool on[kTokens];   // a row whose slot is outside the pool gets 0
    Lanes<VEC> win[kTokens][W];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int64_t b = b0 + k, slot = k >= rows ? -1 : p.slots != nullptr ? __ldg(p.slots + b) : b;
        on[k] = slot >= 0 && slot < p.nslots;
        st[k] = static_cast<T *>(p.state) + (on[k] ? slot : 0) * (W - 1) * D + d;
        if (on[k]) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[k][j] = load_lanes<T, VEC>(st[k] + j * D);
            win[k][W - 1] = load_lanes<T, VEC>(static_cast<const T *>(p.x) + b * p.ldx + d);
        }
    }
    Lanes<VEC> w[W], bias;
    load_taps<VEC, W>(p, d, w, bias);
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        if (k >= rows) return;
        Lanes<VEC> a = vset<VEC>(0.f);
        if (on[k]) {
            a = bias;
#pragma unroll
            for (int j = 0; j < W; ++j) a = vfma<VEC>(w[j], win[k][j], a);
            if (p.silu) a = vmul<VEC>(a, vsigmoid<VEC>(a));
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_lanes<T, VEC>(st[k] + j * D, win[k][j + 1]);
        }
        store_lanes<T, VEC>(static_cast<T *>(p.y) + (b0 + k) * D + d, a);
    }
}

// Sums columns of part (see launch_sum_parts): 8 threads take every 8th part
// of a column, four at a time, and their sums are added in order.
struct SumOuts {
    SumOut o[3];
};
__global__ void __launch_bounds__(256) sum_parts_kernel(const float *part, int64_t parts, int64_t stride,
                                                        SumOuts outs)
{
    __shared__ float s[8][33];
    after_previous();
    const int64_t i = int64_t(blockIdx.x) * 32 + threadIdx.x;
    float a = 0.f;
    if (i < stride) {
        const float *c = part + i;
        int64_t j = threadIdx.y;
        for (; j + 24 < parts; j += 32) {
            const float v0 = c[j * stride], v1 = c[(j + 8) * stride], v2 = c[(j + 16) * stride], v3 = c[(j + 24) * stride];
            a += (v0 + v1) + (v2 + v3);
        }
        for (; j < parts; j += 8) a += c[j * stride];
    }
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && i < stride) {
        float t = 0.f;
        for (int k = 0; k < 8; ++k) t += s[k][threadIdx.x];
        int64_t at = i;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (at >= 0 && at < outs.o[k].n && outs.o[k].out != nullptr) outs.o[k].out[at] = t;
            at -= outs.o[k].n;
        }
    }
}

// How a launch cuts rows and channels.
struct Cut {
    dim3 block;
    int64_t chan_blocks, run, row_blocks;
};

// Lanes run over channels (a multiple of a warp), the rest of a block over
// runs; runs of `least` rows or more, long enough for about
// `blocks` blocks in all.
Cut cut(int64_t rows, int64_t D, int vec, int64_t least, int64_t blocks)
{
    Cut c;
    const int64_t lanes = ceil_div(D, vec);
    const int bx = lanes <= 32 ? 32 : lanes <= 64 ? 64 : kBlock, by = kBlock / bx;
    c.block = dim3(bx, by);
    c.chan_blocks = ceil_div(lanes, bx);
    const int64_t want = ceil_div(blocks, c.chan_blocks) * by;
    c.run = ceil_div(rows, want);
    c.run = c.run < least ? least : c.run;
    c.row_blocks = ceil_div(ceil_div(rows, c.run), by);
    return c;
}

constexpr int64_t kBwdBlocks = 152 * kBwdPerSm;

Cut cut_bwd(int64_t rows, int64_t D, int vec) { return cut(rows, D, vec, 16, kBwdBlocks); }

bool rows_aligned(int64_t D, int64_t ld1, int64_t ld2, int vec)
{
    return D % vec == 0 && ld1 % vec == 0 && ld2 % vec == 0;
}

template <typename T, int VEC, int W>
mg_status conv_fwd(const ConvArgs &p, cudaStream_t s)
{
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const Cut c = cut(q.rows, p.D, VEC, 16, 152 * kFwdPerSm);
    MG_TRY(check_grids("mg_causal_conv_fwd", {c.chan_blocks * c.row_blocks}));
    conv_fwd_kernel<T, VEC, W><<<unsigned(c.chan_blocks * c.row_blocks), c.block, Ring<T, VEC>::bytes(kBlock), s>>>(
        p, q, c.chan_blocks, c.run);
    return launched("mg_causal_conv_fwd");
}

template <typename T, int VEC, int W>
mg_status conv_bwd(const ConvArgs &p, cudaStream_t s)
{
    const Seqs q = make_seqs(p.cu, p.B, p.T, p.nseq);
    const Cut c = cut_bwd(q.rows, p.D, VEC);
    MG_TRY(check_grids("mg_causal_conv_bwd", {c.chan_blocks * c.row_blocks, sum_parts_blocks(p.D * (W + 1))}));
    float *part = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    constexpr size_t sums = kBlock * size_t(VEC * (W + 1)) * sizeof(float), rings = 2 * Ring<T, VEC>::bytes(kBlock);
    constexpr size_t smem = sums > rings ? sums : rings;
    MG_TRY(allow_shared<conv_bwd_kernel<T, VEC, W>>(smem));
    conv_bwd_kernel<T, VEC, W><<<unsigned(c.chan_blocks * c.row_blocks), c.block, smem, s>>>(
        p, q, c.chan_blocks, c.run, part);
    MG_TRY(launched("mg_causal_conv_bwd"));
    return launch_sum_parts(part, c.row_blocks, {{p.dw, p.D * W}, {p.dbias, p.D}}, s);
}

template <typename T, int VEC, int W>
mg_status conv_step(const ConvStepArgs &p, cudaStream_t s)
{
    const int64_t chan_blocks = ceil_div(ceil_div(p.D, VEC), 128), blocks = ceil_div(p.B, kTokens) * chan_blocks;
    MG_TRY(check_grids("mg_causal_conv_step", {blocks}));
    conv_step_kernel<T, VEC, W><<<unsigned(blocks), 128, 0, s>>>(p, unsigned(chan_blocks));
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
    // the most parts of any vector width
    size_t need = 0;
    for (int vec : {1, 2, 4}) {
        const Cut c = cut_bwd(B * T, D, vec);
        const size_t n = size_t(c.row_blocks) * D * (W + 1) * sizeof(float);
        need = n > need ? n : need;
    }
    return kControlBytes + need;
}

// The widest vectors, 4, 2 or 1 channels, that keep every row aligned.
#define MG_CONV_VEC(F, T, p, s, ld2)                                             \
    if (rows_aligned((p).D, (p).ldx, ld2, 4)) { MG_CONV_W(F, T, 4, p, s); }      \
    if (rows_aligned((p).D, (p).ldx, ld2, 2)) { MG_CONV_W(F, T, 2, p, s); }      \
    MG_CONV_W(F, T, 1, p, s)

mg_status launch_conv_fwd(const ConvArgs &p, mg_dtype dt, cudaStream_t s)
{
    if (dt == MG_F32) { MG_CONV_VEC(conv_fwd, float, p, s, p.ldx); }
    MG_CONV_VEC(conv_fwd, bf16_t, p, s, p.ldx);
}

mg_status launch_conv_bwd(const ConvArgs &p, mg_dtype dt, cudaStream_t s)
{
    if (dt == MG_F32) { MG_CONV_VEC(conv_bwd, float, p, s, p.lddy); }
    MG_CONV_VEC(conv_bwd, bf16_t, p, s, p.lddy);
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

mg_status launch_sum_parts(const float *part, int64_t parts, std::initializer_list<SumOut> outs, cudaStream_t s)
{
    SumOuts o{};
    int64_t stride = 0;
    int k = 0;
    for (const SumOut &x : outs) {
        o.o[k++] = x;
        stride += x.n;
    }
    return launch_next("sum over parts", sum_parts_kernel, sum_parts_blocks(stride), dim3(32, 8), 0, s, part, parts, stride, o);
}

}  // namespace mg
