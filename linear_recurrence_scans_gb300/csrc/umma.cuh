// Tensor-core products with operands in shared memory and accumulators in
// tensor memory (tcgen05): tiles, descriptors, waits.
#pragma once

#include <cuda.h>

#include "ssm.cuh"

namespace mg {

// ------------------------------------------------------------------- tiles
// A tile of R rows of bf16 in panels of 64 columns: row r of a panel is 128
// bytes at r * 128, its 16-byte piece c at place c ^ (r & 7) (the 128-byte
// swizzle of the matrix descriptors).  The same tile serves as an operand
// whose rows are the product's rows ("k-major": a row's values are summed
// over) and as one whose rows are summed over ("mn-major").
__device__ __forceinline__ unsigned tile_at(int rows, int row, int piece)   // piece: column / 8
{
    return unsigned((piece >> 3) * rows * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void st_tile(unsigned base, unsigned at, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" : : "r"(base + at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_tile(unsigned base, unsigned at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(base + at) : "memory");
    return v;
}
// A tensor of rows, heads of `cols` bf16 values in each, rows `ld` values apart,
// for copies of a head's 64 columns of 128 rows: a panel of a tile, zeros where
// columns or rows lie outside the tensor.  The address and all strides are
// multiples of 16 bytes.
mg_status rows_map(CUtensorMap *map, const void *base, int64_t rows, int64_t heads, int64_t cols, int64_t ld);

constexpr unsigned kPanelBytes = 128 * 128;

__device__ __forceinline__ void copy_panel(unsigned to, const CUtensorMap &map, int col, int head, int row, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 : : "r"(to), "l"(&map), "r"(col), "r"(head), "r"(row), "r"(smem_addr(bar)) : "memory");
}
template <int PANELS>
__device__ __forceinline__ void copy_tile(unsigned to, const CUtensorMap &map, int head, int row, uint64_t *bar)
{
#pragma unroll
    for (int i = 0; i < PANELS; ++i) copy_panel(to + i * kPanelBytes, map, 64 * i, head, row, bar);
}
// `bytes` of it (a multiple of 16) as they lie.
__device__ __forceinline__ void copy_bytes(unsigned to, const void *from, unsigned bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 : : "r"(to), "l"(from), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}
// A tile to L2 alone.
template <int PANELS>
__device__ __forceinline__ void tile_to_l2(const CUtensorMap &map, int head, int row, int col = 0)
{
#pragma unroll
    for (int i = 0; i < PANELS; ++i)
        asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                     : : "l"(&map), "r"(col + 64 * i), "r"(head), "r"(row) : "memory");
}
// A tile's 128 rows to the tensor; columns beyond it are left out.
template <int PANELS>
__device__ __forceinline__ void put_tile(const CUtensorMap &map, unsigned from, int head, int row)
{
#pragma unroll
    for (int i = 0; i < PANELS; ++i)
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                     : : "l"(&map), "r"(64 * i), "r"(head), "r"(row), "r"(from + i * kPanelBytes) : "memory");
    asm volatile("cp.async.bulk.commit_group;" : : : "memory");
}
// Until this thread's put_tile have read shared memory.
__device__ __forceinline__ void tiles_put() { asm volatile("cp.async.bulk.wait_group.read 0;" : : : "memory"); }

// The one arrival of a barrier's phase, which ends when the bytes have come too.
__device__ __forceinline__ void bar_expect(uint64_t *bar, unsigned bytes)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" : : "r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// Makes this thread's writes to shared memory seen by the tensor core.
__device__ __forceinline__ void fence_tiles() { asm volatile("fence.proxy.async.shared::cta;" : : : "memory"); }

// ------------------------------------------------------------- descriptors

// An operand's place.  Both kinds: rows 128 bytes apart, groups of 8 rows
// 1024.  An mn-major operand of more than 64 columns has its panels `panel`
// bytes apart; a k-major one names one panel at a time.
__device__ __forceinline__ uint64_t operand(unsigned addr, unsigned panel = 16)
{
    return uint64_t((addr >> 4) & 0x3fff) | uint64_t(panel >> 4) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}

// bf16 operands, float32 accumulator of 128 rows and n columns.
__device__ __forceinline__ constexpr unsigned product(int n, bool a_mn, bool b_mn)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | unsigned(a_mn) << 15 | unsigned(b_mn) << 16 | unsigned(n >> 3) << 17 | 8u << 24;
}

__device__ __forceinline__ void mma(unsigned acc, uint64_t a, uint64_t b, unsigned what)   // adds
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, 1, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 : : "r"(acc), "l"(a), "l"(b), "r"(what) : "memory");
}
__device__ __forceinline__ void mma(unsigned acc, uint64_t a, uint64_t b, unsigned what, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 : : "r"(acc), "l"(a), "l"(b), "r"(what), "r"(unsigned(add)) : "memory");
}

// An operand tile of R rows (all of its panels) for the steps of a product, 16
// summed values each.
template <int R, bool MN>
struct Tile {
    static constexpr bool mn = MN;
    unsigned base;
    __device__ __forceinline__ uint64_t first() const { return MN ? operand(base, R * 128) : operand(base); }
    // What step k adds: k-major, 32 bytes in a panel of 4 steps; mn-major, 16 rows.
    static __device__ __forceinline__ constexpr unsigned step(int k) { return (MN ? k * 2048 : (k >> 2) * R * 128 + (k & 3) * 32) >> 4; }
};

// acc (128 x n) (+)= A B over `steps` steps, 8 at most; one thread calls it.  A
// step runs 32 cycles for each 64 columns, so its set-up is two additions (with
// descriptors built anew for each, products took twice their time).
template <typename A, typename B>
__device__ __forceinline__ void multiply(unsigned acc, A a, B b, int n, int steps, bool add)
{
    const unsigned what = product(n, A::mn, B::mn);
    const uint64_t x = a.first(), y = b.first();
    mma(acc, x, y, what, add);
#pragma unroll
    for (int k = 1; k < 8; ++k)
        if (k < steps) mma(acc, x + A::step(k), y + B::step(k), what);
}

// ---------------------------------------------------- tensor memory, waits

// A warp takes `columns` (a power of two, 32 or more) and leaves their address.
__device__ __forceinline__ void tmem_take(unsigned *where, int columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" : : "r"(smem_addr(where)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" : : : "memory");
}
__device__ __forceinline__ void tmem_free(unsigned at, int columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" : : "r"(at), "r"(columns) : "memory");
}

// Around a block's barrier that orders one thread's products and all threads'
// reads of their results.
__device__ __forceinline__ void tmem_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" : : : "memory"); }
__device__ __forceinline__ void tmem_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" : : : "memory"); }

__device__ __forceinline__ void bar_init(uint64_t *bar)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" : : "r"(smem_addr(bar)) : "memory");
}
// Completes the barrier's phase when all products issued so far are done.
__device__ __forceinline__ void bar_after_products(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" : : "r"(smem_addr(bar)) : "memory");
}
// Waits for a phase, with a limit far beyond any product's time (each try waits
// itself, for a hardware limit).  False: it ran out.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, unsigned phase)
{
    for (int i = 0; i < 1 << 16; ++i) {
        unsigned done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(smem_addr(bar)), "r"(phase) : "memory");
        if (done) return true;
    }
    return false;
}

// 32 columns of the 32 accumulator rows that belong to the warp (warp % 4): a
// row a thread.
__device__ __forceinline__ void tmem_load(unsigned at, float (&v)[32])
{
    unsigned r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" : : : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load(unsigned at, float (&v)[16])
{
    unsigned r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" : : : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_store(unsigned at, const float (&v)[16])
{
    unsigned r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
                 : : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
                 : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" : : : "memory");
}

// -------------------------------------------------------- bf16 in pieces

// v = a + b with bf16 a, b to 2^-16 of v, two values at a time.
struct Halves {
    unsigned a, b;
};
__device__ __forceinline__ Halves split2(float x, float y)
{
    Halves p;
    p.a = pack_bf16x2(x, y);
    p.b = pack_bf16x2(x - __uint_as_float(p.a << 16), y - __uint_as_float(p.a & 0xffff0000u));
    return p;
}
// Eight of them.
__device__ __forceinline__ void split2(const float *v, uint4 &a, uint4 &b)
{
    const Halves p = split2(v[0], v[1]), q = split2(v[2], v[3]), r = split2(v[4], v[5]), s = split2(v[6], v[7]);
    a = make_uint4(p.a, q.a, r.a, s.a), b = make_uint4(p.b, q.b, r.b, s.b);
}

// v = a + b + c with bf16 a, b, c to 2^-24 of v, two values at a time.
struct Pieces {
    unsigned a, b, c;
};
__device__ __forceinline__ Pieces split3(float x, float y)
{
    Pieces p;
    p.a = pack_bf16x2(x, y);
    x -= __uint_as_float(p.a << 16), y -= __uint_as_float(p.a & 0xffff0000u);
    p.b = pack_bf16x2(x, y);
    x -= __uint_as_float(p.b << 16), y -= __uint_as_float(p.b & 0xffff0000u);
    p.c = pack_bf16x2(x, y);
    return p;
}

}  // namespace mg
