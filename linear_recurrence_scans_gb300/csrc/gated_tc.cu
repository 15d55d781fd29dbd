// Gated recurrence in bf16: chunks of 128 rows as tensor-core products (the
// formulas are in gated_scan.cu).
//
// A call is three kernels.  A walk goes over the chunks of a segment (a few
// chunks of a sequence and head) and leaves, for each chunk, the state that
// the segment's earlier chunks give it; a pass over the segments adds up what
// comes to each of them; then all chunks' rows are computed at once, each with
// the state that it begins with: the walk's plus the decayed one of its segment.
// Backwards the same with the adjoints, from the last chunk on.
//
// Rounding.  q, k, v and dout are bf16 as they are given, so their products are
// exact in the tensor core's float32 sums.  What they are multiplied with (a
// chunk's weights, the state, its adjoint) goes in as a sum of bf16 pieces, two
// where the result is bf16 (to 2^-16, so that the rounding at the store is the
// only one that counts: with one piece o, dq, dk and dv were off by 2.3e-3 of
// their norm where that rounding alone is 1.7e-3), three where it is float32
// (states, their adjoints, the gates' gradients; to 2^-24).  There the smallest
// pieces are summed first: the tensor core's sums lose up to a last bit of the sum
// at each step, and the large piece first made dg's errors 1.2e-6 where they are
// 3e-7.
#include "gated_scan.cuh"
#include "umma.cuh"

namespace mg {
namespace {

constexpr int kRows = 128;   // of a chunk: the rows of a tensor-core product

// A chunk's gate sums as two floats.  The forward walk leaves them for the kernels
// behind it.
struct Gates128 {
    alignas(16) float hi[kRows], lo[kRows];   // copied as they lie
    __device__ __forceinline__ float span(float hi_i, float lo_i, int j) const { return exp_of((hi_i - hi[j]) + (lo_i - lo[j])); }
    // The four of j .. j + 3, j a multiple of 4, zeros from `count` of them on: the
    // exponent is what is selected, so that no element is a branch of its own (as
    // branches these took 3300 cycles of a block's 26000, and other pairs' 800).
    __device__ __forceinline__ void spans(float hi_i, float lo_i, int j, int count, float (&by)[4]) const
    {
        const float4 h = *reinterpret_cast<const float4 *>(hi + j), l = *reinterpret_cast<const float4 *>(lo + j);
        const float x[4] = {(hi_i - h.x) + (lo_i - l.x), (hi_i - h.y) + (lo_i - l.y), (hi_i - h.z) + (lo_i - l.z), (hi_i - h.w) + (lo_i - l.w)};
#pragma unroll
        for (int e = 0; e < 4; ++e) by[e] = exp_of(e < count ? x[e] : -INFINITY);
    }
    // e^x in two instructions.  The rounding of x log2 e costs a relative |x|
    // 2^-24 of a weight that is e^x itself.
    static __device__ __forceinline__ float exp_of(float x) { return ex2_ftz(x * kLog2eF); }
};

// One warp: a lane has the gates of rows 4 lane .. 4 lane + 3, and gets the sums
// up to each of them.
__device__ __forceinline__ void sum_gates(const float (&g)[4], float (&h)[4], float (&l)[4])
{
    const int lane = threadIdx.x & 31;
    h[0] = g[0], l[0] = 0.f;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        h[i] = h[i - 1], l[i] = l[i - 1];
        add_two(h[i], l[i], g[i], 0.f);
    }
    float th = h[3], tl = l[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float uh = __shfl_up_sync(~0u, th, o), ul = __shfl_up_sync(~0u, tl, o);
        if (lane >= o) add_two(th, tl, uh, ul);
    }
    const float bh = __shfl_up_sync(~0u, th, 1), bl = __shfl_up_sync(~0u, tl, 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane > 0) add_two(h[i], l[i], bh, bl);
}
__device__ __forceinline__ void fetch_gates(float (&g)[8], const float *from, int64_t ld, int len)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * (threadIdx.x & 31) + i;
        g[i] = r < len ? __ldg(from + r * ld) : 0.f;   // as they are: nothing waits for them yet
    }
}

// The 8 values of a row from column 8 piece on, zeros beyond `cols`; where rows
// are not aligned, value by value.
template <bool VEC>
__device__ __forceinline__ uint4 fetch_piece(const bf16_t *row, int piece, int cols, bool on)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    const int c = piece * 8;
    if (!on || c >= cols) return v;
    if constexpr (VEC) {
        v = __ldg(reinterpret_cast<const uint4 *>(row + c));
    } else {
        unsigned w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = c + e < cols ? __ldg(&row[c + e].bits) : 0;
        v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
    return v;
}

// `len` rows of `cols` values into a tile of 128 rows, value by value, zeros
// beside and below.
template <int PANELS, int THREADS>
__device__ __forceinline__ void load_rows(unsigned tile, const bf16_t *from, int64_t ld, int len, int cols)
{
    constexpr int kPieces = PANELS * 8;
#pragma unroll
    for (int u = 0; u < kRows * kPieces / THREADS; ++u) {
        const int id = threadIdx.x + THREADS * u, row = id / kPieces, piece = id % kPieces;
        st_tile(tile, tile_at(kRows, row, piece), fetch_piece<false>(from + row * ld, piece, cols, row < len));
    }
}

// Zeros in a tile's rows from `len` on: a copy takes 128 rows, whoever's they are.
template <int PANELS, int THREADS>
__device__ __forceinline__ void clear_rows(unsigned tile, int len)
{
    for (int i = threadIdx.x; i < (kRows - len) * PANELS * 8; i += THREADS)
        st_tile(tile, tile_at(kRows, len + i / (PANELS * 8), i % (PANELS * 8)), make_uint4(0, 0, 0, 0));
}

// Asks for memory (16-byte multiples) to be brought to L2.
__device__ __forceinline__ void to_l2(const void *from, unsigned bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" : : "l"(from), "r"(bytes) : "memory");
}

// A tile's rows to global memory, `cols` of each.
template <int PANELS, int THREADS, bool VEC>
__device__ __forceinline__ void store_rows(bf16_t *to, int64_t ld, unsigned tile, int len, int cols)
{
    constexpr int kPieces = PANELS * 8;
#pragma unroll
    for (int u = 0; u < kRows * kPieces / THREADS; ++u) {
        const int id = threadIdx.x + THREADS * u, row = id / kPieces, piece = id % kPieces;
        if (row >= len || piece * 8 >= cols) continue;
        const uint4 v = ld_tile(tile, tile_at(kRows, row, piece));
        bf16_t *o = to + row * ld + piece * 8;
        if constexpr (VEC) {
            __stcs(reinterpret_cast<uint4 *>(o), v);
        } else {
            const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (piece * 8 + e < cols) o[e].bits = (unsigned short)(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu);
        }
    }
}

// V values of one row, rounded, into a tile from column 8 piece on.
template <int V>
__device__ __forceinline__ void put(unsigned tile, int row, int piece, const float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V / 8; ++i)
        st_tile(tile, tile_at(kRows, row, piece + i),
                make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7])));
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8])
{
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

// States between the kernels lie as [P / 4][N][4] (zeros beyond P): a lane a
// row of the accumulators, neighbouring lanes 16 bytes apart.
__host__ __device__ constexpr int state_size(int N, int P) { return (P + 3) / 4 * N * 4; }

// A walk's results, for the states or for their adjoints.
struct Walked {
    float *local;    // [chunks][H][state]: of the segment's other chunks before (behind) the chunk
    float *carry;    // [segments][H][state]: before (behind) the segment
    float *reach;    // [chunks][H]: sum of the gates between the chunk and that end of its segment
    float *totals;   // [segments][H]: of the segment's gates
    float *sums;     // [chunks][H]: a chunk's Gates128
};

struct TcCall {
    CUtensorMap q, k, v, dout, o, dq, dk, dv;   // where rows are aligned
    GatedArgs a;
    Chunks c, seg;   // chunks, and segments of m of them
    int m;
    Walked s, d;
    float *partial;
    int splits, heads;
    bool starts;     // the first segments' carries may hold start states
    int state;       // values of a state
    int next_c, next_h;   // chunks and heads from a block to the one that follows on its SM
    unsigned *error;
};

// Where a chunk's states come from, local + e^reach carry, but for the head.
struct Place {
    int c, seg;          // chunk, its segment
    bool local, carry;   // whether there is anything
};
template <bool BACK>
__device__ __forceinline__ Place place_of(const TcCall &p, const Chunks::One &ch, int c)
{
    const int begin = p.c.begin(ch.seq), count = p.c.end(ch.seq) - begin, seg = int(unsigned(ch.idx) / unsigned(p.m)), in = ch.idx - seg * p.m;
    Place o;
    o.c = c, o.seg = p.seg.begin(ch.seq) + seg;
    o.local = BACK ? ch.idx != count - 1 && in != p.m - 1 : in != 0;
    o.carry = BACK ? p.a.dS_last != nullptr || (seg + 1) * p.m < count : p.starts || seg > 0;
    return o;
}
struct Source {
    const float *local, *carry;   // NULL: nothing from there
    const float *reach;
};
template <bool BACK>
__device__ __forceinline__ Source source_of(const TcCall &p, const Place &o, int h)
{
    const Walked &w = BACK ? p.d : p.s;
    const int64_t at = int64_t(o.c) * p.a.H + h;
    return Source{o.local ? w.local + at * p.state : nullptr,
                  o.carry ? w.carry + (int64_t(o.seg) * p.a.H + h) * p.state : nullptr, w.reach + at};
}

// A thread's pieces of a state, 8 values each: rows and columns of a tile of NB
// rows, THREADS pieces on in each step (neighbouring lanes, neighbouring rows).
template <int NB, int PP, int THREADS>
struct Pieces8 {
    static constexpr int kAll = NB * PP * 8, kMine = (kAll + THREADS - 1) / THREADS;
    static __device__ __forceinline__ int row(int u) { return (threadIdx.x + THREADS * u) % NB; }
    static __device__ __forceinline__ int piece(int u) { return (threadIdx.x + THREADS * u) / NB; }
    static __device__ __forceinline__ bool mine(int u) { return kAll % THREADS == 0 || threadIdx.x + THREADS * u < kAll; }
};

// A thread's pieces of local + e^reach carry, zeros beside N and P.
template <typename S>
__device__ __forceinline__ void fetch_states(const Source &from, float by, int N, int P, float (&v)[S::kMine][8])
{
#pragma unroll
    for (int u = 0; u < S::kMine; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
    const auto each = [&](const float *base, auto f) {
#pragma unroll
        for (int u = 0; u < S::kMine; ++u) {
            const int n = S::row(u), col = S::piece(u) * 8, at = (2 * S::piece(u) * N + n) * 4;
            if (S::mine(u) && n < N) {
                if (col < P) f(*reinterpret_cast<const float4 *>(base + at), v[u], 0);
                if (col + 4 < P) f(*reinterpret_cast<const float4 *>(base + at + 4 * N), v[u], 4);
            }
        }
    };
    if (from.local != nullptr)
        each(from.local, [](const float4 x, float (&o)[8], int e) { o[e] = x.x, o[e + 1] = x.y, o[e + 2] = x.z, o[e + 3] = x.w; });
    if (from.carry == nullptr) return;
    each(from.carry, [by](const float4 x, float (&o)[8], int e) {
        o[e] = fmaf(by, x.x, o[e]), o[e + 1] = fmaf(by, x.y, o[e + 1]), o[e + 2] = fmaf(by, x.z, o[e + 2]), o[e + 3] = fmaf(by, x.w, o[e + 3]);
    });
}
__device__ __forceinline__ float reach_of(const Source &s) { return s.carry != nullptr ? __ldg(s.reach) : 0.f; }

__device__ __forceinline__ void wait_or_tell(uint64_t *bar, unsigned phase, unsigned *error)
{
    if (!bar_wait(bar, phase)) atomicOr(error, kErrLookbackTimeout);
}

// ------------------------------------------------------------------- walk
// A block: a segment, a head, 64 columns of its state, which stay in registers
// (row n a lane, 16 columns a thread).  Each chunk adds K^T V~, the row weights
// in V~'s three pieces; the next chunk's rows arrive meanwhile.
//
// 62 us at 4x4096x16x128x128 (264 MB, 4.3 TB/s; tensor pipe 21%).  A step, V into
// pieces, products, the state, is about 7000 cycles, the same with one block on an
// SM as with two.  Only the state itself needs the step before; what makes the
// steps a chain is that V's pieces have one place and each step two barriers.  Two
// blocks hide half of each other's.  Segments cut the walks (of 32 chunks here, into
// 256 blocks) so that most SMs have two: with whole sequences 107 us where segments
// took 67.

constexpr int kWalkThreads = 512, kGateWarp = 4;

struct WalkSmall {
    float by[kRows];         // the weights of the chunk's rows
    float whole, whole_lo;   // the sum of its gates
    uint64_t bar, full[2];
    unsigned tmem;
};

template <int PN, bool VEC, bool BACK>
__global__ void __launch_bounds__(kWalkThreads, 2) gated_walk_kernel(const __grid_constant__ TcCall p, int tiles)
{
    after_previous();
    extern __shared__ __align__(1024) char sm[];
    constexpr unsigned kK = PN * kRows * 128, kV = kRows * 128;
    const GatedArgs &a = p.a;
    const unsigned base = smem_addr(sm), tv = base + 2 * kK;
    using Small = WalkSmall;
    Small &sh = *reinterpret_cast<Small *>(sm + 2 * kK + 3 * kV);

    const unsigned of = blockIdx.x / unsigned(tiles);
    const int tile = int(blockIdx.x % unsigned(tiles)), h = int(of % unsigned(a.H)), grp = h / (a.H / a.G), sg = int(of / unsigned(a.H));
    const Chunks::One s = p.seg.get(sg);
    if (s.len == 0) return;
    const Walked &w = BACK ? p.d : p.s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int p0 = tile * 64, cols = a.P - p0 < 64 ? a.P - p0 : 64;
    const int count = (s.len + kRows - 1) / kRows;
    const int c0 = p.c.begin(s.seq) + s.idx * p.m, size = p.state;
    const bf16_t *kk = static_cast<const bf16_t *>(BACK ? a.q : a.k) + grp * a.N;   // where K is loaded value by value
    const bf16_t *vv = static_cast<const bf16_t *>(BACK ? a.dout : a.v) + h * a.P + p0;
    const int64_t ldk = BACK ? a.ldq : a.ldk, ldv = BACK ? a.lddo : a.ldv;

    if (warp == 0) tmem_take(&sh.tmem, 64);
    if (tid == 0) bar_init(&sh.bar), bar_init(&sh.full[0]), bar_init(&sh.full[1]);
    fence_tiles();
    __syncthreads();
    uint4 v[2];
    const auto chunk_at = [&](int i) { return BACK ? count - 1 - i : i; };
    // chunk i of the walk: K into its buffer, and what comes kFar chunks later to
    // L2; V into registers
    constexpr int kFar = 3;
    const auto copy_k = [&](int i) {
        if (i >= count) return;
        const int ci = chunk_at(i);
        const int64_t row = s.row + int64_t(ci) * kRows;
        if constexpr (VEC) {
            if (tid == kWalkThreads - 32) {
                bar_expect(&sh.full[i & 1], PN * kPanelBytes);
                copy_tile<PN>(base + (i & 1) * kK, BACK ? p.q : p.k, grp, int(row), &sh.full[i & 1]);
                if (i + kFar < count) {
                    const int far = int(s.row) + chunk_at(i + kFar) * kRows;
                    tile_to_l2<PN>(BACK ? p.q : p.k, grp, far);
                    tile_to_l2<1>(BACK ? p.dout : p.v, h, far, p0);
                }
            }
        } else {
            load_rows<PN, kWalkThreads>(base + (i & 1) * kK, kk + row * ldk, ldk, s.len - ci * kRows < kRows ? s.len - ci * kRows : kRows, a.N);
        }
    };
    const auto fetch_v = [&](int i) {
        if (i >= count) return;
        const int ci = chunk_at(i), len = s.len - ci * kRows < kRows ? s.len - ci * kRows : kRows;
        const bf16_t *from = vv + (s.row + int64_t(ci) * kRows) * ldv;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (tid >> 3) + 64 * u;
            v[u] = fetch_piece<VEC>(from + r * ldv, tid & 7, cols, r < len);
        }
    };
    // Two warps, not the one that begins the products, take the chunks' gates in
    // turn: one adds up those of the chunk after the next, while the other turns
    // the next one's sums into weights and asks for the gates of its chunk behind
    // (one warp with both took longer than the products: walks of 64 and 60 us at
    // 4x4096x16x128x128, now 62 and 57).  Backwards the forward walk's sums are there.
    const int turn = warp - kGateWarp;   // chunks of this parity, if 0 or 1
    float gates[8];
    const auto next_gates = [&](int i) {
        if (i >= count) return;
        const int ci = chunk_at(i), len = s.len - ci * kRows < kRows ? s.len - ci * kRows : kRows;
        if constexpr (BACK) {
            const float *from = p.s.sums + (int64_t(c0 + ci) * a.H + h) * (2 * kRows) + 4 * lane;
            const float4 x = __ldg(reinterpret_cast<const float4 *>(from)), y = __ldg(reinterpret_cast<const float4 *>(from + kRows));
            gates[0] = x.x, gates[1] = x.y, gates[2] = x.z, gates[3] = x.w, gates[4] = y.x, gates[5] = y.y, gates[6] = y.z, gates[7] = y.w;
        } else {
            fetch_gates(gates, a.g + (s.row + int64_t(ci) * kRows) * a.ldg + h, a.ldg, len);
        }
    };
    const auto add_gates = [&]() {
        if constexpr (!BACK) {
            const float g[4] = {gate_of(gates[0]), gate_of(gates[1]), gate_of(gates[2]), gate_of(gates[3])};
            float hi[4], lo[4];
            sum_gates(g, hi, lo);
#pragma unroll
            for (int e = 0; e < 4; ++e) gates[e] = hi[e], gates[4 + e] = lo[e];
        }
    };
    const auto weigh = [&](int i) {
        if (i >= count) return;
        if (!BACK && tile == 0) {
            float *to = w.sums + (int64_t(c0 + chunk_at(i)) * a.H + h) * (2 * kRows) + 4 * lane;
            *reinterpret_cast<float4 *>(to) = make_float4(gates[0], gates[1], gates[2], gates[3]);
            *reinterpret_cast<float4 *>(to + kRows) = make_float4(gates[4], gates[5], gates[6], gates[7]);
        }
        const float th = __shfl_sync(~0u, gates[3], 31), tl = __shfl_sync(~0u, gates[7], 31);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sh.by[4 * lane + e] = BACK ? a.scale * Gates128::exp_of(gates[e] + gates[4 + e]) : Gates128::exp_of((th - gates[e]) + (tl - gates[4 + e]));
        if (lane == 0) sh.whole = th, sh.whole_lo = tl;
    };
    copy_k(0);
    fetch_v(0);
    if (turn == 0 || turn == 1) {
        next_gates(turn);
        if (turn < count) add_gates();
        if (turn == 0) weigh(0), next_gates(2);
    }
    float S[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) S[i] = 0.f;
    const int n = 32 * (warp & 3) + lane, quad0 = p0 / 4 + 4 * (warp >> 2);
    const auto put = [&](float *to) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (n < a.N && (quad0 + q) * 4 < a.P)
                *reinterpret_cast<float4 *>(to + ((quad0 + q) * a.N + n) * 4) = make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
    };
    float reach = 0.f;
    for (int i = 0; i < count; ++i) {
        __syncthreads();   // the weights; the other buffer's products are done
        copy_k(i + 1);
        if constexpr (VEC) {
            const int left = s.len - chunk_at(i) * kRows;
            wait_or_tell(&sh.full[i & 1], (i >> 1) & 1, p.error);
            if (left < kRows) clear_rows<PN, kWalkThreads>(base + (i & 1) * kK, left);
        }
        const int64_t ch = int64_t(c0 + chunk_at(i)) * a.H + h;
        const float whole = sh.whole, whole_lo = sh.whole_lo;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = (tid >> 3) + 64 * u;
            const float by = sh.by[r];
            float f[8];
            unpack8(v[u], f);
            unsigned x[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Pieces q = split3(f[2 * e] * by, f[2 * e + 1] * by);
                x[0][e] = q.a, x[1][e] = q.b, x[2][e] = q.c;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
                st_tile(tv + k * kV, tile_at(kRows, r, tid & 7), make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]));
        }
        fetch_v(i + 1);
        fence_tiles();
        tmem_before_sync();
        __syncthreads();
        const unsigned acc = sh.tmem;
        if (tid == 0) {
            tmem_after_sync();
            for (int k = 2; k >= 0; --k)
                multiply(acc, Tile<kRows, true>{base + (i & 1) * kK}, Tile<kRows, true>{tv + k * kV}, 64, kRows / 16, k < 2);
            bar_after_products(&sh.bar);
        }
        if (turn == ((i + 1) & 1)) {   // everyone has read this chunk's
            weigh(i + 1);
            next_gates(i + 3);
        } else if (turn == (i & 1) && i + 2 < count) {
            add_gates();
        }
        // while the products run: the state that came to the chunk
        if (tid == 0 && tile == 0) w.reach[ch] = reach;
        if (i > 0) put(w.local + ch * size);
        reach += whole + whole_lo;
        const float decay = expf(whole) * (1.f + whole_lo);
        wait_or_tell(&sh.bar, i & 1, p.error);
        tmem_after_sync();
        float add[16];
        tmem_load(acc + (unsigned(32 * (warp & 3)) << 16) + 16 * (warp >> 2), add);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[e] = fmaf(decay, S[e], add[e]);
    }
    put(w.carry + (int64_t(sg) * a.H + h) * size);
    if (tid == 0 && tile == 0) w.totals[int64_t(sg) * a.H + h] = reach;
    tmem_before_sync();
    __syncthreads();
    if (warp == 0) tmem_free(sh.tmem, 64);
}

// ----------------------------------------------------- pass over segments
// In place: carry holds what each segment leaves, and is left with what comes
// to it, from `from` (N x P each; NULL: zero) and on to `to` (may be NULL).  A
// thread a quad of a state's row.

template <bool BACK>
__global__ void __launch_bounds__(256) over_segments_kernel(const Chunks seg, const Walked w, const float *from, float *to,
                                                            int H, int N, int P, int blocks_per)
{
    after_previous();
    constexpr int kAhead = 8;
    const unsigned su = blockIdx.x / unsigned(blocks_per);   // sequence and head
    const int seq = int(su / unsigned(H)), h = int(su % unsigned(H));
    const int64_t sh = su;
    const int at = int(blockIdx.x % unsigned(blocks_per)) * 256 + threadIdx.x, quads = (P + 3) / 4;
    if (at >= quads * N) return;
    const int n = at % N, p0 = at / N * 4, cols = P - p0 < 4 ? P - p0 : 4;
    const int64_t size = state_size(N, P), out = (sh * N + n) * P + p0;
    const int64_t lo = seg.begin(seq), hi = seg.end(seq);
    float s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = 0.f;
    if (from != nullptr) {
        if (P % 4 == 0) {
            load_vec<4>(from + out, s);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < cols) s[e] = __ldg(from + out + e);
        }
        // + 0: a caller's signalling NaN must not get into the workspace as it is
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += 0.f;
    }
    for (int64_t i0 = 0; i0 < hi - lo; i0 += kAhead) {
        float add[kAhead][4], gate[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i0 + u >= hi - lo) continue;
            const int64_t g = (BACK ? hi - 1 - i0 - u : lo + i0 + u) * H + h;
            load_vec<4>(w.carry + g * size + int64_t(at) * 4, add[u]);
            gate[u] = w.totals[g];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (i0 + u >= hi - lo) continue;
            const int64_t g = (BACK ? hi - 1 - i0 - u : lo + i0 + u) * H + h;
            store_vec<4>(w.carry + g * size + int64_t(at) * 4, s);
            const float d = expf(gate[u]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = fmaf(d, s[e], add[u][e]);
        }
    }
    if (to == nullptr) return;
    if (P % 4 == 0) {
        store_vec<4>(to + out, s);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < cols) to[out + e] = s[e];
    }
}

// Within a chunk, weights e^{G_i - G_j}: pairs of rows in the same 32 take the
// exponential; the others the product of e^{G_i - G_r} and e^{G_r - G_j}, r the
// last of j's 32 rows, both at most 1: one exponential a row and block instead
// of one a pair.
struct Weights {
    Gates128 g;
    float to_end[kRows];   // e^{G_r - G_j}
    // One warp, once the sums are there.
    __device__ __forceinline__ void fill()
    {
        for (int b = 0; b < 4; ++b) {
            const int j = 32 * b + (threadIdx.x & 31);
            to_end[j] = g.span(g.hi[32 * b + 31], g.lo[32 * b + 31], j);
        }
    }
};

// ------------------------------------------------------------------- rows
// A block: o of a chunk and head.  Q K^T, weights, times V, and Q S beside it;
// the weights take Q's and the state's places in shared memory and V takes K's, so
// that two blocks fit an SM and one's products run under the other's loads and
// exponentials.  A state of 128 x 128 has room for one piece at a time.
//
// 82 us at 4x4096x16x128x128 (403 MB, 4.9 TB/s of 6.8; 77 us with one piece of each
// factor): memory, and a block's chain of set-up, state, products, weights,
// products and output, of which two blocks hide half.

constexpr int kRowThreads = 512;
constexpr unsigned kRowsS = 2 * kPanelBytes;   // the state's place, then the weights' second pieces'

struct RowsSmall {
    Weights w;
    uint64_t full[2], done[2], gates;
    unsigned tmem;
};

template <int PN, int PP, bool VEC>
__global__ void __launch_bounds__(kRowThreads, 2) gated_rows_kernel(const __grid_constant__ TcCall p)
{
    after_previous();
    extern __shared__ __align__(1024) char sm[];
    constexpr int NB = 64 * PN, PB = 64 * PP;
    constexpr unsigned kQ = 2 * kPanelBytes, kK = (PN > PP ? PN : PP) * kPanelBytes, kS = kRowsS;
    const GatedArgs &a = p.a;
    const unsigned tq = smem_addr(sm), tk = tq + kQ, ts = tk + kK;
    using Small = RowsSmall;
    Small &sh = *reinterpret_cast<Small *>(sm + kQ + kK + kS);
    const int c = int(blockIdx.x / unsigned(a.H)), h = int(blockIdx.x % unsigned(a.H)), grp = h / (a.H / a.G);
    const Chunks::One ch = p.c.get(c);
    if (ch.len == 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rb = warp & 3, cb = warp >> 2, row = 32 * rb + lane;
    if (tid == 32) {
        bar_init(&sh.done[0]), bar_init(&sh.done[1]), bar_init(&sh.full[0]), bar_init(&sh.full[1]), bar_init(&sh.gates);
        fence_tiles();
        bar_expect(&sh.gates, sizeof(Gates128));
        copy_bytes(smem_addr(&sh.w.g), p.s.sums + (int64_t(c) * a.H + h) * (2 * kRows), sizeof(Gates128), &sh.gates);
        if constexpr (VEC) {
            bar_expect(&sh.full[0], 2 * PN * kPanelBytes);
            copy_tile<PN>(tq, p.q, grp, int(ch.row), &sh.full[0]);
            copy_tile<PN>(tk, p.k, grp, int(ch.row), &sh.full[0]);
        }
    }
    __syncthreads();   // the barriers are set up
    if (warp == 12) {  // a warp without weights
        wait_or_tell(&sh.gates, 0, p.error);
        sh.w.fill();
    }
    if (warp == 0) tmem_take(&sh.tmem, 256);
    if constexpr (!VEC) {
        load_rows<PN, kRowThreads>(tq, static_cast<const bf16_t *>(a.q) + ch.row * a.ldq + grp * a.N, a.ldq, ch.len, a.N);
        load_rows<PN, kRowThreads>(tk, static_cast<const bf16_t *>(a.k) + ch.row * a.ldk + grp * a.N, a.ldk, ch.len, a.N);
    }
    using Mine = Pieces8<NB, PP, kRowThreads>;
    constexpr unsigned kState = PP * NB * 128;
    constexpr bool kBoth = 2 * kState <= kS;   // both pieces of the state have room at once
    uint4 rest[Mine::kMine];   // else the second ones wait until the first ones are read
    {
        const Source s = source_of<false>(p, place_of<false>(p, ch, c), h);
        float f[Mine::kMine][8];
        fetch_states<Mine>(s, expf(reach_of(s)), a.N, a.P, f);
#pragma unroll
        for (int u = 0; u < Mine::kMine; ++u) {
            uint4 v;
            split2(f[u], v, rest[u]);
            if (!Mine::mine(u)) continue;
            st_tile(ts, tile_at(NB, Mine::row(u), Mine::piece(u)), v);
            if constexpr (kBoth) st_tile(ts + kState, tile_at(NB, Mine::row(u), Mine::piece(u)), rest[u]);
        }
    }
    if (VEC && tid == 64) {   // what the block that follows on this SM will read
        const int wrap = h + p.next_h >= a.H, cn = c + p.next_c + wrap, hn = h + p.next_h - (wrap ? a.H : 0);
        const Chunks::One n = cn < p.c.most ? p.c.get(cn) : Chunks::One{0, 0, 0, 0};
        if (n.len > 0) {
            const int gn = hn / (a.H / a.G);
            tile_to_l2<PN>(p.q, gn, int(n.row));
            tile_to_l2<PN>(p.k, gn, int(n.row));
            tile_to_l2<PP>(p.v, hn, int(n.row));
            const Source f = source_of<false>(p, place_of<false>(p, n, cn), hn);
            if (f.local != nullptr) to_l2(f.local, unsigned(p.state) * 4);
        }
    }
    fence_tiles();
    tmem_before_sync();
    __syncthreads();
    tmem_after_sync();
    const unsigned acc = sh.tmem, acc_s = acc + 128, mine = unsigned(32 * rb) << 16;
    if (tid == 0) {
        const int steps = (a.N + 15) / 16;
        // rows of K and Q behind the chunk only reach rows and columns that are not used
        if constexpr (VEC) wait_or_tell(&sh.full[0], 0, p.error);
        multiply(acc, Tile<kRows, false>{tq}, Tile<kRows, false>{tk}, kRows, steps, false);
        bar_after_products(&sh.done[0]);
        if constexpr (kBoth) multiply(acc_s, Tile<kRows, false>{tq}, Tile<NB, true>{ts + kState}, PB, steps, false);
        multiply(acc_s, Tile<kRows, false>{tq}, Tile<NB, true>{ts}, PB, steps, kBoth);
        bar_after_products(&sh.done[1]);
    }
    wait_or_tell(&sh.gates, 0, p.error);
    const float hi = sh.w.g.hi[row], lo = sh.w.g.lo[row];
    wait_or_tell(&sh.done[0], 0, p.error);
    if constexpr (VEC) {
        if (tid == 32) {   // K is read
            bar_expect(&sh.full[1], PP * kPanelBytes);
            copy_tile<PP>(tk, p.v, h, int(ch.row), &sh.full[1]);
        }
    } else {
        load_rows<PP, kRowThreads>(tk, static_cast<const bf16_t *>(a.v) + ch.row * a.ldv + h * a.P, a.ldv, ch.len, a.P);
    }
    if constexpr (!kBoth) {
        wait_or_tell(&sh.done[1], 0, p.error);   // the first pieces are read
#pragma unroll
        for (int u = 0; u < Mine::kMine; ++u)
            if (Mine::mine(u)) st_tile(ts, tile_at(NB, Mine::row(u), Mine::piece(u)), rest[u]);
        fence_tiles();
        __syncthreads();
        if (tid == 0) {
            multiply(acc_s, Tile<kRows, false>{tq}, Tile<NB, true>{ts}, PB, (a.N + 15) / 16, true);
            bar_after_products(&sh.done[1]);
        }
    }
    tmem_after_sync();
    {   // a block of 32 columns a warp; those above the diagonal are zeros
        float w[32];
        if (cb < rb) {
            const float from = sh.w.g.span(hi, lo, 32 * cb + 31);
            tmem_load(acc + mine + 32 * cb, w);
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] *= from * sh.w.to_end[32 * cb + e];
        } else if (cb == rb) {
            tmem_load(acc + mine + 32 * cb, w);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float by[4];
                sh.w.g.spans(hi, lo, 32 * cb + e, lane + 1 - e, by);
#pragma unroll
                for (int u = 0; u < 4; ++u) w[e + u] = (e + u <= lane ? w[e + u] : 0.f) * by[u];
            }
        }
        wait_or_tell(&sh.done[1], kBoth ? 0 : 1, p.error);   // Q and the state are read: the weights may take their places
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0), more = v;
            if (cb <= rb) split2(w + 8 * i, v, more);
            st_tile(tq, tile_at(kRows, row, 4 * cb + i), v);
            st_tile(ts, tile_at(kRows, row, 4 * cb + i), more);
        }
    }
    if constexpr (VEC) {
        wait_or_tell(&sh.full[1], 0, p.error);
        if (ch.len < kRows) clear_rows<PP, kRowThreads>(tk, ch.len);
    }
    fence_tiles();
    tmem_before_sync();
    __syncthreads();
    if (tid == 0) {
        tmem_after_sync();
        multiply(acc, Tile<kRows, false>{ts}, Tile<kRows, true>{tk}, PB, (ch.len + 15) / 16, false);
        multiply(acc, Tile<kRows, false>{tq}, Tile<kRows, true>{tk}, PB, (ch.len + 15) / 16, true);
        bar_after_products(&sh.done[0]);
    }
    const float up = Gates128::exp_of(hi + lo);
    wait_or_tell(&sh.done[0], 1, p.error);
    tmem_after_sync();
    if (cb < PB / 32) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[16], y[16];
            tmem_load(acc + mine + 32 * cb + 16 * half, x);
            tmem_load(acc_s + mine + 32 * cb + 16 * half, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = a.scale * fmaf(up, y[e], x[e]);
            put<16>(tk, row, 4 * cb + 2 * half, x);
        }
    }
    fence_tiles();
    tmem_before_sync();
    __syncthreads();
    if (VEC && ch.len == kRows) {
        if (tid == 32) {
            put_tile<PP>(p.o, tk, h, int(ch.row));
            tiles_put();
        }
    } else {
        store_rows<PP, kRowThreads, VEC>(static_cast<bf16_t *>(a.o) + (ch.row * a.H + h) * a.P, int64_t(a.H) * a.P, tk, ch.len, a.P);
    }
    if (warp == 0) tmem_free(acc, 256);
}

// -------------------------------------------------------------- gradients
// A block: a chunk, a group's heads (or a part of them), one after another: dv
// and dg of each, dq and dk summed over them in tensor memory.  One block fits an
// SM; the adjoint's and the state's pieces share a place (kX), which for N and
// P above 64 is the weights' too, with V's for what is left of them.  Else the
// weights have a place for one piece at a time, and the second pieces' products
// come between the first ones' and the state's.
//
// 258 us at 4x4096x16x128x128 (738 MB, 2.9 TB/s), 182 us at 2x4096x32x128x64 with
// shared q and k (with one piece of the weights 237 and 155): 18.4 and 12.5 us a
// head, of which the products' steps are 8200 and 5400 cycles; the rest is loads
// of states (the next head's adjoint is copied ahead), weights, pieces and sums
// over rows between barriers; shared memory is full with one block, so that
// nothing else runs beside them.

constexpr int kGradThreads = 1024;
// The warp that begins the products: rows 0 to 31 and columns 112 on, which have
// no weights.
constexpr int kMmaWarp = 28;

template <int PN, int PP>
struct Grad {
    static constexpr int NB = 64 * PN, PB = 64 * PP;
    // N and P above 64: the adjoint's products come before the weights', straight
    // into dk's sums, for a single head; else beside the weights' products.
    static constexpr bool kFirst = PN == 2 && PP == 2;
    static constexpr unsigned kQ = PN * kPanelBytes, kV = PP * kPanelBytes, kState = PP * NB * 128, kW = 2 * kPanelBytes;
    static constexpr unsigned kX = 3 * kState;
    static constexpr unsigned kTiles = 2 * kQ + 2 * kV + (kFirst ? kX : 2 * kW + kX);
    struct Small {
        Weights w;
        float after[kRows], key[kRows], dots[32], end[2];
        uint64_t full[2], done[2], gates, adjoint;
        unsigned tmem;
        float parts[kFirst ? 1 : 12 * kRows];   // sums by blocks of 16 columns and of 32 rows
    };
    static constexpr size_t bytes = kTiles + sizeof(Small);
};

// Sums over a warp's 32 rows: lanes l and l + 16 get column l's.
__device__ __forceinline__ float column_sums(float (&w)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] += __shfl_xor_sync(~0u, w[k], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const bool up = lane & o;
            const float send = up ? w[k] : w[k + o], keep = up ? w[k + o] : w[k];
            w[k] = keep + __shfl_xor_sync(~0u, send, o);
        }
    return w[0];
}

template <int PN, int PP, bool VEC>
__global__ void __launch_bounds__(kGradThreads, 1) gated_grads_kernel(const __grid_constant__ TcCall p)
{
    after_previous();
    extern __shared__ __align__(1024) char sm[];
    using M = Grad<PN, PP>;
    constexpr int NB = M::NB, PB = M::PB;
    const GatedArgs &a = p.a;
    const unsigned tq = smem_addr(sm), tk = tq + M::kQ, tv = tk + M::kQ, to = tv + M::kV, tw = to + M::kV, tdw = tw + M::kW;
    const unsigned tx = M::kFirst ? tw : tdw + M::kW;
    auto &sh = *reinterpret_cast<typename M::Small *>(sm + M::kTiles);
    // beside the weights where they share their place with the pieces
    float *row_part = M::kFirst ? reinterpret_cast<float *>(sm + 2 * M::kQ + 2 * M::kV + 2 * M::kW) : sh.parts, *col_part = row_part + 8 * kRows;
    float *key_part = M::kFirst ? col_part + 4 * kRows : row_part;

    // the parts of a group's heads one after another: the last, maybe smaller, ones fill up the SMs
    const unsigned all = unsigned(p.c.most) * unsigned(a.G), of_c = blockIdx.x % all;
    const int split = int(blockIdx.x / all), grp = int(of_c % unsigned(a.G)), c = int(of_c / unsigned(a.G));
    const Chunks::One ch = p.c.get(c);
    if (ch.len == 0) return;
    const Place place_d = place_of<true>(p, ch, c), place_s = place_of<false>(p, ch, c);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rb = warp & 3, cb = warp >> 2, row = 32 * rb + lane;
    const int per_group = a.H / a.G, h0 = split * p.heads, h1 = M::kFirst ? h0 + 1 : h0 + p.heads < per_group ? h0 + p.heads : per_group;
    // V, dO, gate sums and (into the weights' place) the adjoint's two parts
    const auto copy_head = [&](int h) {
        if constexpr (VEC) {
            bar_expect(&sh.full[1], 2 * PP * kPanelBytes);
            copy_tile<PP>(tv, p.v, h, int(ch.row), &sh.full[1]);
            copy_tile<PP>(to, p.dout, h, int(ch.row), &sh.full[1]);
        }
        bar_expect(&sh.gates, sizeof(Gates128));
        copy_bytes(smem_addr(&sh.w.g), p.s.sums + (int64_t(c) * a.H + h) * (2 * kRows), sizeof(Gates128), &sh.gates);
        if constexpr (!M::kFirst) {
            const Source d = source_of<true>(p, place_d, h);
            const unsigned bytes = unsigned(p.state) * 4;
            if (place_d.local || place_d.carry) bar_expect(&sh.adjoint, bytes * (unsigned(place_d.local) + unsigned(place_d.carry)));
            if (place_d.local) copy_bytes(tw, d.local, bytes, &sh.adjoint);
            if (place_d.carry) copy_bytes(tdw, d.carry, bytes, &sh.adjoint);
        }
    };
    if (tid == 32) {
        bar_init(&sh.done[0]), bar_init(&sh.done[1]), bar_init(&sh.full[0]), bar_init(&sh.full[1]), bar_init(&sh.gates), bar_init(&sh.adjoint);
        fence_tiles();
        copy_head(grp * per_group + h0);
        if constexpr (VEC) {
            bar_expect(&sh.full[0], 2 * PN * kPanelBytes);
            copy_tile<PN>(tq, p.q, grp, int(ch.row), &sh.full[0]);
            copy_tile<PN>(tk, p.k, grp, int(ch.row), &sh.full[0]);
        }
    }
    if (warp == 0) tmem_take(&sh.tmem, 512);
    __syncthreads();   // the barriers are set up
    if constexpr (!VEC) {
        load_rows<PN, kGradThreads>(tq, static_cast<const bf16_t *>(a.q) + ch.row * a.ldq + grp * a.N, a.ldq, ch.len, a.N);
        load_rows<PN, kGradThreads>(tk, static_cast<const bf16_t *>(a.k) + ch.row * a.ldk + grp * a.N, a.ldk, ch.len, a.N);
    }
    const int nsteps = (a.N + 15) / 16, psteps = (a.P + 15) / 16;
    const unsigned mine = unsigned(32 * rb) << 16;
    unsigned phase[2] = {0, 0}, acc0 = 0, acc1 = 0, acc_q = 0, acc_k = 0, acc_d = 0;
    const auto products_done = [&](int b) {
        wait_or_tell(&sh.done[b], phase[b], p.error);
        phase[b] ^= 1;
        tmem_after_sync();
    };
    // writes of tiles and reads of accumulators before the next products
    const auto before_products = [&]() {
        fence_tiles();
        tmem_before_sync();
        __syncthreads();
        tmem_after_sync();
    };
    // the sum of a row's parts, block after block
    const auto of_blocks = [&](const float *part, int blocks) {
        float v = 0.f;
        for (int b = 0; b < blocks; ++b) v += part[b * kRows + tid];
        return v;
    };
    using Mine = Pieces8<NB, PP, kGradThreads>;
    float st[Mine::kMine][8];
    float reach_d = reach_of(source_of<true>(p, place_d, grp * per_group + h0)), reach_s = reach_of(source_of<false>(p, place_s, grp * per_group + h0));
    const auto put_states = [&]() {   // as three pieces
#pragma unroll
        for (int u = 0; u < Mine::kMine; ++u) {
            if (!Mine::mine(u)) continue;
            unsigned x[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const Pieces q = split3(st[u][2 * e], st[u][2 * e + 1]);
                x[0][e] = q.a, x[1][e] = q.b, x[2][e] = q.c;
            }
            const unsigned at = tile_at(NB, Mine::row(u), Mine::piece(u));
#pragma unroll
            for (int k = 0; k < 3; ++k) st_tile(tx + k * M::kState, at, make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]));
        }
    };
    const auto with_pieces = [&](unsigned acc, unsigned tile) {   // acc = tile (S or D)^T, the small pieces first
        for (int k = 2; k >= 0; --k)
            multiply(acc, Tile<kRows, false>{tile}, Tile<NB, false>{tx + k * M::kState}, NB, psteps, k < 2);
    };
    // Rows of `from` times `by`, added to those of `sums` (or in their place); their products with the tile's rows.
    const auto take = [&](unsigned from, unsigned sums, float by, unsigned tile, bool add) {
        float x[16], of = 0.f;
        tmem_load(from + mine + 16 * cb, x);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float f[8];
            unpack8(ld_tile(tile, tile_at(kRows, row, 2 * cb + i)), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[8 * i + e] *= by;
                of = fmaf(x[8 * i + e], f[e], of);
            }
        }
        if (add) {
            float t[16];
            tmem_load(sums + mine + 16 * cb, t);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] += t[e];
        }
        tmem_store(sums + mine + 16 * cb, x);
        return of;
    };
    for (int hh = h0; hh < h1; ++hh) {
        const int h = grp * per_group + hh;
        if constexpr (!VEC) {   // the head before is done with its tiles
            load_rows<PP, kGradThreads>(tv, static_cast<const bf16_t *>(a.v) + ch.row * a.ldv + h * a.P, a.ldv, ch.len, a.P);
            load_rows<PP, kGradThreads>(to, static_cast<const bf16_t *>(a.dout) + ch.row * a.lddo + h * a.P, a.lddo, ch.len, a.P);
        }
        const Source from_d = source_of<true>(p, place_d, h), from_s = source_of<false>(p, place_s, h);
        const float by_d = expf(reach_d), by_s = expf(reach_s);
        if constexpr (M::kFirst) {
            fetch_states<Mine>(from_d, by_d, a.N, a.P, st);
        } else {
            if (place_d.local || place_d.carry) wait_or_tell(&sh.adjoint, (hh - h0) & 1, p.error);
            const float *copied = reinterpret_cast<const float *>(sm + (tw - tq));
            fetch_states<Mine>(Source{place_d.local ? copied : nullptr, place_d.carry ? copied + M::kW / 4 : nullptr, nullptr}, by_d, a.N, a.P, st);
        }
        float dot = 0.f;   // <S, D>
        const auto put_dot = [&]() {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
            if (lane == 0) sh.dots[warp] = dot;
        };
        if constexpr (M::kFirst) {   // D's pieces make room before S comes for good
            float other[Mine::kMine][8];
            fetch_states<Mine>(from_s, by_s, a.N, a.P, other);
#pragma unroll
            for (int u = 0; u < Mine::kMine; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(other[u][e], st[u][e], dot);
            put_dot();
        }
        if (VEC && tid == 64) {   // what comes after this head: the block's next one, or the block that follows on the SM
            if (hh + 1 < h1) {
                tile_to_l2<PP>(p.v, h + 1, int(ch.row));
                tile_to_l2<PP>(p.dout, h + 1, int(ch.row));
                if (place_d.local) to_l2(from_d.local + p.state, unsigned(p.state) * 4);
                if (place_s.local) to_l2(from_s.local + p.state, unsigned(p.state) * 4);
            } else {
                const unsigned next = blockIdx.x + 152, of_n = next % all;
                const int gn = int(of_n % unsigned(a.G)), cn = int(of_n / unsigned(a.G)), hn = gn * per_group + int(next / all) * p.heads;
                const Chunks::One n = next < gridDim.x ? p.c.get(cn) : Chunks::One{0, 0, 0, 0};
                if (n.len > 0) {
                    tile_to_l2<PN>(p.q, gn, int(n.row));
                    tile_to_l2<PN>(p.k, gn, int(n.row));
                    tile_to_l2<PP>(p.v, hn, int(n.row));
                    tile_to_l2<PP>(p.dout, hn, int(n.row));
                    const Source d = source_of<true>(p, place_of<true>(p, n, cn), hn), f = source_of<false>(p, place_of<false>(p, n, cn), hn);
                    if (d.local != nullptr) to_l2(d.local, unsigned(p.state) * 4);
                    if (f.local != nullptr) to_l2(f.local, unsigned(p.state) * 4);
                }
            }
        }
        if (warp == kMmaWarp) {
            wait_or_tell(&sh.gates, (hh - h0) & 1, p.error);
            sh.w.fill();
            if (lane == 0) sh.end[(hh - h0) & 1] = Gates128::exp_of(sh.w.g.hi[kRows - 1] + sh.w.g.lo[kRows - 1]);
        }
        put_states();
        if constexpr (VEC) {
            if (hh == h0) wait_or_tell(&sh.full[0], 0, p.error);
            wait_or_tell(&sh.full[1], (hh - h0) & 1, p.error);
            if (ch.len < kRows) {   // rows of other chunks that came along
                if (hh == h0) clear_rows<PN, kGradThreads>(tq, ch.len), clear_rows<PN, kGradThreads>(tk, ch.len);
                clear_rows<PP, kGradThreads>(tv, ch.len), clear_rows<PP, kGradThreads>(to, ch.len);
            }
        }
        before_products();
        acc0 = sh.tmem, acc1 = acc0 + 128, acc_q = acc0 + 256, acc_k = acc_q + NB;
        acc_d = M::kFirst ? acc_q : PB == 64 ? acc0 + 64 : acc_k + NB;   // K D
        if (tid == 32 * kMmaWarp) {
            multiply(acc0, Tile<kRows, false>{tq}, Tile<kRows, false>{tk}, kRows, nsteps, false);
            multiply(acc1, Tile<kRows, false>{to}, Tile<kRows, false>{tv}, kRows, psteps, false);
            bar_after_products(&sh.done[0]);
            if constexpr (M::kFirst) {
                with_pieces(acc_k, tv);
                for (int k = 1; k >= 0; --k)
                    multiply(acc_d, Tile<kRows, false>{tk}, Tile<NB, true>{tx + k * M::kState}, PB, nsteps, k < 1);
                bar_after_products(&sh.done[1]);
            }
        }
        wait_or_tell(&sh.gates, (hh - h0) & 1, p.error);
        const float hi = sh.w.g.hi[row], lo = sh.w.g.lo[row];
        const float tail = sh.w.g.span(sh.w.g.hi[kRows - 1], sh.w.g.lo[kRows - 1], row), up = Gates128::exp_of(hi + lo);
        products_done(0);
        // weights, and what each pair of rows gives to the gates between them: rows
        // from 32 rb, columns from 16 cb
        float of_row = 0.f, of_col = 0.f, w[16], d[16];
        if (cb <= 2 * rb + 1) {
            float s[16];
            tmem_load(acc0 + mine + 16 * cb, s);
            tmem_load(acc1 + mine + 16 * cb, d);
            const int first = 16 * cb - 32 * rb;   // columns up to lane - first reach the row
            if (first < 0) {   // all of them
                const float from = a.scale * sh.w.g.span(hi, lo, 32 * (cb >> 1) + 31);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float by = from * sh.w.to_end[16 * cb + j];
                    w[j] = s[j] * by, d[j] *= by, s[j] *= d[j], of_row += s[j];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float by[4];
                    sh.w.g.spans(hi, lo, 16 * cb + e, lane + 1 - first - e, by);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int j = e + u;
                        const bool in = first + j <= lane;   // what is behind may be a NaN
                        by[u] *= a.scale;
                        w[j] = (in ? s[j] : 0.f) * by[u];
                        d[j] = (in ? d[j] : 0.f) * by[u], s[j] = (first + j < lane ? s[j] : 0.f) * d[j], of_row += s[j];
                    }
                }
            }
            of_col = column_sums(s);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = d[e] = 0.f;
        }
        // the weights' two pieces, the second ones kept for later
        uint4 w_rest[2], d_rest[2];
        const auto put_weights = [&]() {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 v;
                split2(w + 8 * i, v, w_rest[i]);
                st_tile(tw, tile_at(kRows, row, 2 * cb + i), v);
                split2(d + 8 * i, v, d_rest[i]);
                st_tile(tdw, tile_at(kRows, row, 2 * cb + i), v);
            }
            row_part[cb * kRows + row] = of_row;
            if (lane < 16) col_part[rb * kRows + 16 * cb + lane] = of_col;
        };
        const auto put_rest = [&](unsigned tile, const uint4 (&v)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) st_tile(tile, tile_at(kRows, row, 2 * cb + i), v[i]);
        };
        float dv[16];   // K D's part of dv
        // where the weights' second pieces lie
        const unsigned tw2 = M::kFirst ? tv : tw, tdw2 = M::kFirst ? tdw + M::kW : tdw;
        const auto sum_parts = [&]() {
            if (tid < kRows) sh.after[tid] = of_blocks(row_part, 8) - of_blocks(col_part, 4);
            if (M::kFirst && tid < kRows) sh.key[tid] = of_blocks(key_part, 8);
        };
        if constexpr (M::kFirst) {
            products_done(1);
            put_weights();   // the adjoint's pieces are read, and V
            put_rest(tw2, w_rest);
            key_part[cb * kRows + row] = take(acc_k, acc_k, tail, tk, false);
            tmem_load(acc_d + mine + 16 * cb, dv);
            __syncthreads();
            sum_parts();
            __syncthreads();
            put_rest(tdw2, d_rest);
        } else {
            put_weights();
        }
        before_products();
        if (tid == 32 * kMmaWarp) {
            const bool add = hh > h0;
            if constexpr (M::kFirst) {
                multiply(acc0, Tile<kRows, true>{tw2}, Tile<kRows, true>{to}, PB, kRows / 16, false);
                multiply(acc_q, Tile<kRows, false>{tdw2}, Tile<kRows, true>{tk}, NB, kRows / 16, false);
                multiply(acc_k, Tile<kRows, true>{tdw2}, Tile<kRows, true>{tq}, NB, kRows / 16, true);
            }
            multiply(acc0, Tile<kRows, true>{tw}, Tile<kRows, true>{to}, PB, kRows / 16, M::kFirst);
            multiply(acc_q, Tile<kRows, false>{tdw}, Tile<kRows, true>{tk}, NB, kRows / 16, add || M::kFirst);
            multiply(acc_k, Tile<kRows, true>{tdw}, Tile<kRows, true>{tq}, NB, kRows / 16, add || M::kFirst);
            if constexpr (!M::kFirst) {
                for (int k = 1; k >= 0; --k)
                    multiply(acc_d, Tile<kRows, false>{tk}, Tile<NB, true>{tx + k * M::kState}, PB, nsteps, k < 1);
                with_pieces(acc1, tv);
            }
            bar_after_products(&sh.done[0]);
        }
        if constexpr (!M::kFirst) sum_parts();
        fetch_states<Mine>(from_s, by_s, a.N, a.P, st);
        if constexpr (!M::kFirst) {   // D is the sum of its pieces
#pragma unroll
            for (int u = 0; u < Mine::kMine; ++u) {
                if (!Mine::mine(u)) continue;
                float x[3][8];
#pragma unroll
                for (int k = 0; k < 3; ++k) unpack8(ld_tile(tx + k * M::kState, tile_at(NB, Mine::row(u), Mine::piece(u))), x[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(st[u][e], x[0][e] + (x[1][e] + x[2][e]), dot);
            }
            put_dot();
        }
        products_done(0);
        if constexpr (!M::kFirst) {   // the weights' second pieces: in the first ones' places, where zeros stay
            if (cb <= 2 * rb + 1) put_rest(tw2, w_rest), put_rest(tdw2, d_rest);
            put_states();   // the adjoint's pieces are read
            before_products();
            if (tid == 32 * kMmaWarp) {
                multiply(acc0, Tile<kRows, true>{tw2}, Tile<kRows, true>{to}, PB, kRows / 16, true);
                multiply(acc_k, Tile<kRows, true>{tdw2}, Tile<kRows, true>{tq}, NB, kRows / 16, true);
                bar_after_products(&sh.done[0]);
            }
            if (hh + 1 < h1) {   // of the next head
                if (place_d.carry) reach_d = __ldg(from_d.reach + 1);
                if (place_s.carry) reach_s = __ldg(from_s.reach + 1);
            }
            products_done(0);
        }
        if (cb < PB / 16) {
            float x[16];
            tmem_load(acc0 + mine + 16 * cb, x);
            if constexpr (!M::kFirst) tmem_load(acc_d + mine + 16 * cb, dv);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fmaf(tail, dv[e], x[e]);
            put<16>(tv, row, 2 * cb, x);   // V is read
        }
        if constexpr (M::kFirst) put_states();   // the adjoint's pieces and the weights are read
        before_products();
        if (tid == 32 * kMmaWarp) {
            with_pieces(M::kFirst ? acc1 : acc0, to);   // what was in these is read
            if constexpr (!M::kFirst) multiply(acc_q, Tile<kRows, false>{tdw2}, Tile<kRows, true>{tk}, NB, kRows / 16, true);
            bar_after_products(&sh.done[0]);
        }
        if constexpr (!M::kFirst) {
            if (cb < NB / 16) key_part[cb * kRows + row] = take(acc1, acc_k, tail, tk, true);
        }
        if (VEC && ch.len == kRows) {
            if (tid == 32) put_tile<PP>(p.dv, tv, h, int(ch.row));
        } else {
            store_rows<PP, kGradThreads, VEC>(static_cast<bf16_t *>(a.dv) + (ch.row * a.H + h) * a.P, int64_t(a.H) * a.P, tv, ch.len, a.P);
        }
        products_done(0);
        if constexpr (!M::kFirst) {
            fence_tiles();
            __syncthreads();
            if (tid == 32 && hh + 1 < h1) {   // all places are free but Q's and K's
                tiles_put();
                copy_head(h + 1);
            }
            if (tid < kRows) sh.key[tid] = of_blocks(key_part, NB / 16);
            __syncthreads();
        }
        if (cb < NB / 16) row_part[cb * kRows + row] = take(M::kFirst ? acc1 : acc0, acc_q, a.scale * up, tq, true);
        __syncthreads();
        if (tid < kRows) sh.after[tid] += of_blocks(row_part, NB / 16);
        __syncthreads();
        if (warp == 0) {   // dg: four rows a lane
            float x[4], z[4], after = 0.f, before = 0.f, whole = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = sh.after[4 * lane + i], z[i] = sh.key[4 * lane + i], after += x[i], before += z[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_down_sync(~0u, after, o), v = __shfl_up_sync(~0u, before, o);
                if (lane + o < 32) after += u;
                if (lane >= o) before += v;
            }
            const float right = __shfl_down_sync(~0u, after, 1), left = __shfl_up_sync(~0u, before, 1);
            after = lane < 31 ? right : 0.f, before = lane > 0 ? left : 0.f;   // of the lanes behind and before
            for (int w = 0; w < 32; ++w) whole += sh.dots[w];
            whole *= sh.end[(hh - h0) & 1];
            float suffix[4];
#pragma unroll
            for (int i = 3; i >= 0; --i) suffix[i] = after += x[i];
            float *dg = a.dg + ch.row * a.H + h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * lane + i;
                if (r < ch.len) dg[int64_t(r) * a.H] = suffix[i] + before + whole;
                before += z[i];
            }
        }
    }
    // dq and dk: through the weights' place
    __syncthreads();
    tmem_after_sync();
    if (cb < NB / 16) {
        float x[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            tmem_load((k == 0 ? acc_q : acc_k) + mine + 16 * cb, x);
            if (p.splits == 1) {
                put<16>(tw + k * M::kW, row, 2 * cb, x);
            } else {
                const int quads = (a.N + 3) / 4;
                float *to_part = p.partial + (((int64_t(split) * p.c.most + c) * a.G + grp) * 2 + k) * quads * kRows * 4;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (4 * cb + q < quads)
                        *reinterpret_cast<float4 *>(to_part + (int64_t(4 * cb + q) * kRows + row) * 4) = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
        }
    }
    fence_tiles();
    tmem_before_sync();
    __syncthreads();
    if (p.splits == 1 && VEC && ch.len == kRows) {
        if (tid == 32) {
            put_tile<PN>(p.dq, tw, grp, int(ch.row));
            put_tile<PN>(p.dk, tw + M::kW, grp, int(ch.row));
        }
    } else if (p.splits == 1) {
        store_rows<PN, kGradThreads, VEC>(static_cast<bf16_t *>(a.dq) + (ch.row * a.G + grp) * a.N, int64_t(a.G) * a.N, tw, ch.len, a.N);
        store_rows<PN, kGradThreads, VEC>(static_cast<bf16_t *>(a.dk) + (ch.row * a.G + grp) * a.N, int64_t(a.G) * a.N, tw + M::kW, ch.len, a.N);
    }
    if (tid == 32) tiles_put();
    if (warp == 0) tmem_free(acc0, 512);
}

// dq and dk of a chunk and group from the parts of its heads: a thread a row's
// quad, in the parts' order.
constexpr int kJoinBlocks = 8;   // for a chunk and group
__global__ void __launch_bounds__(256) gated_join_rows_kernel(const __grid_constant__ TcCall p)
{
    after_previous();
    const GatedArgs &a = p.a;
    const int quads = (a.N + 3) / 4, grp = int(blockIdx.x / kJoinBlocks % unsigned(a.G)), c = int(blockIdx.x / kJoinBlocks / unsigned(a.G));
    const Chunks::One ch = p.c.get(c);
    for (int id = int(blockIdx.x % kJoinBlocks) * 256 + threadIdx.x; id < 2 * quads * kRows; id += kJoinBlocks * 256) {
        const int k = id / (quads * kRows), quad = id / kRows % quads, row = id % kRows;
        if (row >= ch.len) continue;
        float v[4] = {};
        for (int s = 0; s < p.splits; ++s) {
            float x[4];
            load_vec<4>(p.partial + (((int64_t(s) * p.c.most + c) * a.G + grp) * 2 + k) * quads * kRows * 4 + int64_t(id % (quads * kRows)) * 4, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += x[e];
        }
        bf16_t *o = static_cast<bf16_t *>(k == 0 ? a.dq : a.dk) + ((ch.row + row) * a.G + grp) * a.N + quad * 4;
        if (a.N % 4 == 0) {
            store_vec<4>(o, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (quad * 4 + e < a.N) store1(o + e, v[e]);
        }
    }
}

// ------------------------------------------------------------------- host

// Chunks of a segment.  Two walks run on an SM, in rounds of a segment's chunks
// and about one and a half more for a block's beginning and end.
int segment_chunks(int64_t chunks, int64_t nseq, int H, int P)
{
    const int64_t blocks = H * ceil_div(P, 64), each = ceil_div(chunks, nseq > 0 ? nseq : 1);
    int best = 1;
    double least = 1e300;
    for (int m = 1; m <= 64; ++m) {
        const double t = double(ceil_div(nseq * ceil_div(each, m) * blocks, 2 * 152)) * (m + 1.5);
        if (t < least * 0.999) least = t, best = m;
    }
    return best;
}

// Heads of a block of the gradients, of a group's: such blocks run one on an SM,
// each for its heads' time and about half a head's for the group's own tiles.  A
// group's last block may have fewer heads; those come after all others and run
// where the others' last round leaves SMs (2x4096 rows, a group of 32 heads of
// 128 x 64: parts of 14, 14 and 4 heads 155 us and 12 for joining them, two of 16
// 174 and 10).  Above 64 values of both kinds a block takes one head.
int grad_heads(int64_t chunks, int H, int G, int N, int P)
{
    const int per = H / G;
    if (N > 64 && P > 64) return 1;
    const int64_t groups = chunks * G;
    int best = per;
    double least = 1e300;
    for (int heads = per; heads >= 1; --heads) {
        const int rest = per % heads;
        const int64_t full = groups * (per / heads), rounds = full / 152, last = full % 152;
        double t = double(rounds + (last > 0)) * (heads + 0.5);
        if (rest > 0) {
            const int64_t fit = last > 0 ? (152 - last) * int64_t((heads + 0.5) / (rest + 0.5)) : 0;
            if (groups > fit) t += double(ceil_div(groups - fit, 152)) * (rest + 0.5);
        }
        if (t < least * 0.999) least = t, best = heads;
    }
    return best;
}

struct Plan {
    int64_t chunks, segments;
    int m, heads, splits;
    size_t first, seg_first, local, carry, reach, totals, sums, partial, end;   // of the workspace
    size_t s_carry, s_reach, s_sums, saved;                                       // of `saved`, whose local states come first
};
Plan plan_of(int64_t B, int64_t T, int H, int G, int N, int P, int64_t nseq, bool packed, bool bwd)
{
    Plan w{};
    const size_t state = size_t(state_size(N, P)) * 4;
    w.chunks = chunks_most(B, T, nseq, packed, kRows);
    w.m = segment_chunks(w.chunks, nseq, H, P);
    w.segments = chunks_most(B, T, nseq, packed, kRows * w.m);
    w.heads = bwd ? grad_heads(w.chunks, H, G, N, P) : H / G;
    w.splits = int(ceil_div(H / G, w.heads));
    const size_t table = packed ? align_up(size_t(nseq + 1) * 4, 256) : 0;
    w.first = kControlBytes, w.seg_first = w.first + table;
    w.totals = w.seg_first + table;
    w.local = w.totals + align_up(size_t(w.segments) * H * 4, 256);
    w.carry = w.local + align_up(size_t(w.chunks) * H * state, 256);
    w.reach = w.carry + align_up(size_t(w.segments) * H * state, 256);
    w.sums = w.reach + align_up(size_t(w.chunks) * H * 4, 256);
    w.partial = w.sums + size_t(w.chunks) * H * sizeof(Gates128);
    w.end = w.partial + (w.splits > 1 ? size_t(w.splits) * w.chunks * G * 2 * ((N + 3) / 4) * kRows * 16 : 0);
    w.s_carry = size_t(w.chunks) * H * state;
    w.s_reach = w.s_carry + size_t(w.segments) * H * state;
    w.s_sums = w.s_reach + align_up(size_t(w.chunks) * H * 4, 16);
    w.saved = w.s_sums + size_t(w.chunks) * H * sizeof(Gates128);
    return w;
}

template <bool BACK>
mg_status over_segments(const TcCall &p, const float *from, float *to, cudaStream_t s)
{
    const GatedArgs &a = p.a;
    const int per = int(ceil_div(int64_t((a.P + 3) / 4) * a.N, 256));
    return launch_next("pass over segments", over_segments_kernel<BACK>, a.nseq * a.H * per, dim3(256), 0, s, p.seg, BACK ? p.d : p.s, from, to,
                       a.H, a.N, a.P, per);
}

template <int PN, bool VEC, bool BACK>
mg_status walk(const TcCall &p, cudaStream_t s)
{
    constexpr size_t smem = 2 * PN * kRows * 128 + 3 * kRows * 128 + sizeof(WalkSmall);
    static_assert(2 * (smem + 1024) <= 228 * 1024 || PN == 1, "two blocks an SM");
    MG_TRY((allow_shared<gated_walk_kernel<PN, VEC, BACK>>(smem)));
    const int tiles = int(ceil_div(p.a.P, 64));
    const int64_t blocks = int64_t(p.seg.most) * p.a.H * tiles;
    if (p.a.cu != nullptr) return launch_next("mg_gated_scan", gated_walk_kernel<PN, VEC, BACK>, blocks, dim3(kWalkThreads), smem, s, p, tiles);
    gated_walk_kernel<PN, VEC, BACK><<<unsigned(blocks), kWalkThreads, smem, s>>>(p, tiles);   // the call's first kernel
    return launched("mg_gated_scan");
}

template <int PN, int PP, bool VEC>
mg_status forward(const TcCall &p, cudaStream_t s)
{
    MG_TRY((walk<PN, VEC, false>(p, s)));
    MG_TRY(over_segments<false>(p, p.a.S0, p.a.S_last, s));
    constexpr size_t smem = 2 * kPanelBytes + (PN > PP ? PN : PP) * kPanelBytes + kRowsS + sizeof(RowsSmall);
    static_assert(2 * (smem + 1024) <= 228 * 1024, "two blocks an SM");
    MG_TRY((allow_shared<gated_rows_kernel<PN, PP, VEC>>(smem)));
    return launch_next("mg_gated_scan_fwd", gated_rows_kernel<PN, PP, VEC>, int64_t(p.c.most) * p.a.H, dim3(kRowThreads), smem, s, p);
}

template <int PN, int PP, bool VEC>
mg_status backward(const TcCall &p, cudaStream_t s)
{
    MG_TRY((walk<PN, VEC, true>(p, s)));
    MG_TRY(over_segments<true>(p, p.a.dS_last, p.a.dS0, s));
    constexpr size_t smem = Grad<PN, PP>::bytes;
    static_assert(smem <= 227 * 1024, "one block an SM");
    MG_TRY((allow_shared<gated_grads_kernel<PN, PP, VEC>, 227 * 1024>(smem)));
    MG_TRY(launch_next("mg_gated_scan_bwd", gated_grads_kernel<PN, PP, VEC>, int64_t(p.c.most) * p.a.G * p.splits, dim3(kGradThreads), smem, s, p));
    if (p.splits == 1) return MG_OK;
    return launch_next("mg_gated_scan_bwd", gated_join_rows_kernel, int64_t(p.c.most) * p.a.G * kJoinBlocks, dim3(256), 0, s, p);
}

// Whole 16-byte pieces where every row and head begins and ends on such a
// boundary; row numbers of copies are 32-bit.
bool by_pieces(const GatedArgs &a)
{
    const int64_t all = a.N | a.P | a.ldq | a.ldk | a.ldv | (a.dout != nullptr ? a.lddo : 0);
    return all % 8 == 0 && a.B * a.T <= INT32_MAX - kRows;
}

mg_status make_call(const GatedArgs &a, bool bwd, TcCall &p, cudaStream_t s)
{
    const bool packed = a.cu != nullptr;
    const Plan w = plan_of(a.B, a.T, a.H, a.G, a.N, a.P, a.nseq, packed, bwd);
    char *ws = static_cast<char *>(a.ws);
    const auto at = [&](size_t o) { return reinterpret_cast<float *>(ws + o); };
    p.a = a, p.m = w.m;
    p.c.q = p.seg.q = make_seqs(a.cu, a.B, a.T, a.nseq);
    p.c.L = kRows, p.seg.L = kRows * w.m;
    p.c.per = int(ceil_div(a.T, p.c.L)), p.seg.per = int(ceil_div(a.T, p.seg.L));
    p.c.most = int(w.chunks), p.seg.most = int(w.segments);
    p.state = state_size(a.N, a.P);
    p.next_c = 2 * 152 / a.H, p.next_h = 2 * 152 % a.H;   // two blocks of rows on an SM
    p.c.first = reinterpret_cast<const int *>(ws + w.first), p.seg.first = reinterpret_cast<const int *>(ws + w.seg_first);
    const Walked in_ws{at(w.local), at(w.carry), at(w.reach), at(w.totals), at(w.sums)};
    float *saved = bwd ? const_cast<float *>(a.saved_in) : a.saved;
    if (saved != nullptr) p.s = Walked{saved, saved + w.s_carry / 4, saved + w.s_reach / 4, at(w.totals), saved + w.s_sums / 4};
    else p.s = in_ws;
    p.d = in_ws;
    p.starts = bwd || a.S0 != nullptr;
    p.partial = at(w.partial);
    p.splits = w.splits, p.heads = w.heads;
    p.error = &reinterpret_cast<Control *>(a.ws)->error;
    MG_TRY(check_grids(bwd ? "mg_gated_scan_bwd" : "mg_gated_scan_fwd",
                       {w.chunks * a.H, w.segments * a.H * ceil_div(a.P, 64), w.chunks * a.G * (w.splits > 1 && w.splits < kJoinBlocks ? kJoinBlocks : w.splits),
                        a.nseq * a.H * ceil_div(int64_t((a.P + 3) / 4) * a.N, 256)}));
    if (by_pieces(a)) {
        const int64_t rows = a.B * a.T;
        MG_TRY(rows_map(&p.q, a.q, rows, a.G, a.N, a.ldq));
        MG_TRY(rows_map(&p.k, a.k, rows, a.G, a.N, a.ldk));
        MG_TRY(rows_map(&p.v, a.v, rows, a.H, a.P, a.ldv));
        if (bwd) {
            MG_TRY(rows_map(&p.dout, a.dout, rows, a.H, a.P, a.lddo));
            MG_TRY(rows_map(&p.dq, a.dq, rows, a.G, a.N, int64_t(a.G) * a.N));
            MG_TRY(rows_map(&p.dk, a.dk, rows, a.G, a.N, int64_t(a.G) * a.N));
            MG_TRY(rows_map(&p.dv, a.dv, rows, a.H, a.P, int64_t(a.H) * a.P));
        } else {
            MG_TRY(rows_map(&p.o, a.o, rows, a.H, a.P, int64_t(a.H) * a.P));
        }
    }
    if (!packed) return MG_OK;
    return launch_chunk_tables(p.c, p.seg, a.ws, s);
}

#define MG_GATED_TC(F)                                                  \
    const bool vec = by_pieces(a);                                      \
    if (a.N <= 64) {                                                    \
        if (a.P <= 64) return vec ? F<1, 1, true>(p, s) : F<1, 1, false>(p, s); \
        return vec ? F<1, 2, true>(p, s) : F<1, 2, false>(p, s);        \
    }                                                                   \
    if (a.P <= 64) return vec ? F<2, 1, true>(p, s) : F<2, 1, false>(p, s); \
    return vec ? F<2, 2, true>(p, s) : F<2, 2, false>(p, s);

}  // namespace

size_t gated_tc_saved_bytes(int64_t B, int64_t T, int H, int N, int P, int64_t nseq, bool packed)
{
    return plan_of(B, T, H, 1, N, P, nseq, packed, false).saved;
}

size_t gated_tc_ws_bytes(int64_t B, int64_t T, int H, int G, int N, int P, int64_t nseq, bool packed, bool bwd)
{
    return plan_of(B, T, H, G, N, P, nseq, packed, bwd).end;
}

mg_status launch_gated_tc_fwd(const GatedArgs &a, cudaStream_t s)
{
    TcCall p{};
    MG_TRY(make_call(a, false, p, s));
    MG_GATED_TC(forward)
}

mg_status launch_gated_tc_bwd(const GatedArgs &a, cudaStream_t s)
{
    TcCall p{};
    MG_TRY(make_call(a, true, p, s));
    MG_GATED_TC(backward)
}

}  // namespace mg
