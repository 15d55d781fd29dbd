// Group norm with an activation, channels last: each row's channels in G
// groups, each group normalised by itself, with a gate before or behind the
// norm (forward and gradients).
//
// A team of `tpg` neighbouring threads (a power of two) holds one row's
// group in registers: NV vectors of VEC channels a thread, read once.  The
// mean is taken first and the variance from the differences, both in
// registers, so there is no second pass over memory and no cancellation of
// E[p^2] against E[p]^2.
//
// A team keeps its group and walks over rows: its weights stay in registers,
// and its next rows arrive by asynchronous copies into each thread's own slots
// of shared memory, kAhead rows ahead.  Memory bounds the forward, 32768 x 4096
// bf16 channels in one group in 133 us with a cold L2, 6.1 TB/s, and nearly the
// gradients of groups that a warp holds (the same in 16 groups: 258 us, 5.2
// TB/s); in wider groups they wait at the row's barriers (one group of 4096:
// 359 us, 3.7 TB/s).
#include "ssm.cuh"

namespace mg {
namespace {

constexpr int kMaxTeam = 512;

constexpr int kAhead = 3;   // rows in flight for a thread

// Sum of v over each team; every thread of the team gets it.  TEAM: the team's
// size where it is known when compiled, kAny for any size, kBlock for whole
// warps.  buf: one float for each warp of the block, and not the one of the
// call before (whose readers this call's barrier waits for).  All threads of
// the block call it.  (With the size as an argument alone, the two sums of a
// row took 100 of its 290 instructions.)
constexpr int kAny = 0, kBlock = -1;
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, int tpg, float *buf)
{
    if constexpr (TEAM > 0) {
#pragma unroll
        for (int o = TEAM / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        return v;
    }
    const int in_warp = TEAM == kBlock || tpg > 32 ? 32 : tpg;
    for (int o = in_warp / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    if (TEAM == kAny && tpg <= 32) return v;
    const int warp = threadIdx.x >> 5, per = tpg >> 5, first = warp / per * per;
    if ((threadIdx.x & 31) == 0) buf[warp] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < per; ++i) v += buf[first + i];
    return v;
}

// The sum of a's values, and of a's values times b's.
template <int VEC>
__device__ __forceinline__ float vsum(const Lanes<VEC> &a)
{
    pair_t t = a.p[0];
#pragma unroll
    for (int i = 1; i < VEC / 2; ++i) t = add2(t, a.p[i]);
    float x, y;
    unpack2(t, x, y);
    return x + y;
}
template <int VEC>
__device__ __forceinline__ float vdot(const Lanes<VEC> &a, const Lanes<VEC> &b)
{
    pair_t t = mul2(a.p[0], b.p[0]);
#pragma unroll
    for (int i = 1; i < VEC / 2; ++i) t = fma2(a.p[i], b.p[i], t);
    float x, y;
    unpack2(t, x, y);
    return x + y;
}

// act(v) and, if grad, its derivative; sigmoid s: v s and s (1 + v (1 - s)).
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vact(const Lanes<VEC> &v, int silu)
{
    return silu ? vmul<VEC>(v, vsigmoid<VEC>(v)) : v;
}
template <int VEC>
__device__ __forceinline__ Lanes<VEC> vact(const Lanes<VEC> &v, int silu, Lanes<VEC> &grad)
{
    const Lanes<VEC> one = vset<VEC>(1.f);
    if (!silu) {
        grad = one;
        return v;
    }
    const Lanes<VEC> s = vsigmoid<VEC>(v);
    grad = vmul<VEC>(s, vfma<VEC>(v, vfma<VEC>(s, vset<VEC>(-1.f), one), one));
    return vmul<VEC>(v, s);
}

// Vectors of half that (4 bf16, 2 float32) stand for groups and rows that
// 16-byte vectors do not fit: they start at any value, and a group's last one
// may hold fewer (`count`; the others read as 0 and are not written).
template <typename T, int VEC>
constexpr bool kRagged = VEC * sizeof(T) < 16;
template <int VEC, typename T>
__device__ __forceinline__ Lanes<VEC> vload_any(const T *from, int count)
{
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = e < count ? load1(from + e) : 0.f;
    return vfrom<VEC>(f);
}
template <int VEC, typename T>
__device__ __forceinline__ void vstore_any(T *to, const Lanes<VEC> &v, int count)
{
    float f[VEC];
    vto<VEC>(v, f);
    const int lead = int(reinterpret_cast<uintptr_t>(to) / sizeof(T) % 2);   // a value before the first whole pair
    if (count >= VEC) {
        if (lead == 0) {
#pragma unroll
            for (int e = 0; e < VEC; e += 2) store_vec<2>(to + e, reinterpret_cast<const float (&)[2]>(f[e]));
        } else {
            store1(to, f[0]);
#pragma unroll
            for (int e = 1; e + 1 < VEC; e += 2) store_vec<2>(to + e, reinterpret_cast<const float (&)[2]>(f[e]));
            store1(to + VEC - 1, f[VEC - 1]);
        }
    } else {
#pragma unroll
        for (int e = 0; e + 1 < VEC; ++e)
            if (e < count) store1(to + e, f[e]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void vstore(T *to, const Lanes<VEC> &v, int count)
{
    if constexpr (kRagged<T, VEC>) {
        vstore_any<VEC>(to, v, count);
    } else {
        float f[VEC];
        vto<VEC>(v, f);
        store_out<VEC>(to, f);
    }
}
// The values of a parameter, or sums, that go with a vector of T.
template <typename T, int VEC>
__device__ __forceinline__ Lanes<VEC> pload(const float *from, int count)
{
    if constexpr (kRagged<T, VEC>) return vload_any<VEC>(from, count);
    float f[VEC];
    load_vec<VEC>(from, f);
    return vfrom<VEC>(f);
}
template <typename T, int VEC>
__device__ __forceinline__ void pstore(float *to, const Lanes<VEC> &v, int count)
{
    if constexpr (kRagged<T, VEC>) {
        vstore_any<VEC>(to, v, count);
    } else {
        float f[VEC];
        vto<VEC>(v, f);
        store_vec<VEC>(to, f);
    }
}

// A thread's vectors of the rows to come, K tensors of them: slots of shared
// memory that only the thread's own copies fill.  Ragged vectors come as the
// 4-byte words that hold them: 4 bf16 that start in the middle of a word as
// three, of which the value before them (never the first of a tensor) is
// dropped.  8192 rows of 1001 bf16 channels in one group take 56 us, the
// gradients 75, in 7 groups 65 and 87 (as pairs 62 and 86, 68 and 93; single
// values loaded where they are used 136 and 157, 63 and 192).  Instructions
// bound these.
template <typename T, int VEC, int NV, int K>
struct Ahead {
    static constexpr bool kRag = kRagged<T, VEC>;
    static constexpr int kBytes = kRag && sizeof(T) == 4 ? 8 : 16;
    static constexpr bool kAsync = NV * kBytes <= 32;
    static size_t bytes(int threads) { return kAsync ? size_t(kAhead) * K * NV * threads * kBytes : 0; }
    unsigned char *mine;
    __device__ __forceinline__ unsigned char *at(int slot, int k, int i) const
    {
        return mine + size_t((slot * K + k) * NV + i) * blockDim.x * kBytes;
    }
    static __device__ __forceinline__ bool odd(const T *from) { return reinterpret_cast<uintptr_t>(from) % 4 != 0; }
    __device__ __forceinline__ void fetch(int slot, int k, int i, const T *from, int count) const
    {
        const unsigned to = smem_addr(at(slot, k, i));
        if constexpr (!kAsync) {
            return;
        } else if constexpr (!kRag) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" : : "r"(to), "l"(from) : "memory");
        } else {
            // the vector's bytes from the start of its first word
            const int lead = odd(from) ? 2 : 0, all = lead + (count < VEC ? count : VEC) * int(sizeof(T));
            const char *first = reinterpret_cast<const char *>(from) - lead;
#pragma unroll
            for (int b = 0; b < VEC * int(sizeof(T)) + (sizeof(T) == 2 ? 4 : 0); b += 4) {
                const int n = all - b > 4 ? 4 : all - b;
                if (b < VEC * int(sizeof(T)) || lead != 0)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" : : "r"(to + b),
                                 "l"(n > 0 ? first + b : first), "r"(n > 0 ? n : 0) : "memory");
            }
        }
    }
    __device__ __forceinline__ Lanes<VEC> get(int slot, int k, int i, const T *from, int count) const
    {
        if constexpr (!kAsync && kRag) {
            return vload_any<VEC>(from, count);
        } else if constexpr (kRag && sizeof(T) == 2) {
            const uint4 w = *reinterpret_cast<const uint4 *>(at(slot, k, i));
            const bool mid = odd(from);
            const unsigned a = mid ? __funnelshift_r(w.x, w.y, 16) : w.x, b = mid ? __funnelshift_r(w.y, w.z, 16) : w.y;
            Lanes<VEC> v;
            v.p[0] = pack2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
            v.p[1] = pack2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
            return v;
        } else {
            float o[VEC];
            load_vec<VEC>(kAsync ? reinterpret_cast<const T *>(at(slot, k, i)) : from, o);
            return vfrom<VEC>(o);
        }
    }
};

// The team's place: its group, its first row, and its thread's channels.
struct Team {
    int lane, g, slot;
    int64_t d0;
    bool live;
    __device__ __forceinline__ Team(const NormArgs &p, int tpg, int row_teams)
    {
        const unsigned t = blockIdx.x * (blockDim.x / tpg) + threadIdx.x / tpg, G = unsigned(p.G);
        lane = threadIdx.x & (tpg - 1);
        g = int(t % G);
        slot = int(t / G);
        d0 = int64_t(g) * (p.D / p.G);
        live = slot < row_teams;
    }
};

// SILU: 1 where the activation is known to be SiLU when compiled, else -1.
template <typename T, int VEC, int NV, mg_gate GATE, int TEAM, int SILU>
__global__ void __launch_bounds__(512, NV == 1 || (kRagged<T, VEC> && NV <= 4) ? 2 : 1)
norm_fwd_kernel(NormArgs p, int team_size, int row_teams)
{
    const int tpg = TEAM > 0 ? TEAM : team_size, silu = SILU == 1 ? 1 : p.silu;
    constexpr int K = GATE == MG_GATE_NONE ? 1 : 2;
    __shared__ float buf[2][32];
    extern __shared__ __align__(16) unsigned char ring[];
    const Team team(p, tpg, row_teams);
    const int gs = int(p.D / p.G);
    const Ahead<T, VEC, NV, K> ahead{ring + threadIdx.x * Ahead<T, VEC, NV, K>::kBytes};
    const T *x = static_cast<const T *>(p.x) + int64_t(team.slot) * p.ldx + team.d0;
    const T *z = static_cast<const T *>(p.z) + int64_t(team.slot) * p.ldz + team.d0;
    T *y = static_cast<T *>(p.y) + int64_t(team.slot) * p.D + team.d0;
    Lanes<VEC> w[NV], b[NV];
    int c[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = (i * tpg + team.lane) * VEC;
        in[i] = team.live && c[i] < gs;
        w[i] = b[i] = vset<VEC>(0.f);
        if (in[i]) {
            w[i] = pload<T, VEC>(p.w + team.d0 + c[i], gs - c[i]);
            if (p.bias != nullptr) b[i] = pload<T, VEC>(p.bias + team.d0 + c[i], gs - c[i]);
        }
    }
    const int64_t xs = row_teams * p.ldx, zs = row_teams * p.ldz, ys = row_teams * p.D;
    const T *xn = x, *zn = z;   // of the next row to be fetched
    const int M = int(p.M);   // M G < 2^31
    int64_t row_next = team.slot;
    auto fetch = [&](int slot) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i] && row_next < M) {
                ahead.fetch(slot, 0, i, xn + c[i], gs - c[i]);
                if (K == 2) ahead.fetch(slot, 1, i, zn + c[i], gs - c[i]);
            }
        xn += xs;
        zn += zs;
        row_next += row_teams;
        cp_async_commit();
    };
    const float inv = 1.f / float(gs);
    const bool writes_stats = team.lane == 0 && p.stats != nullptr;
    float2 *stats = reinterpret_cast<float2 *>(p.stats) + (int64_t(team.slot) * p.G + team.g);
    const int64_t ss = row_teams * p.G;
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) fetch(k);
    const int rounds = (M - 1) / row_teams + 1;   // the same for every team
    int slot = 0;
    int64_t row = team.slot;
    for (int k = 0; k < rounds; ++k, row += row_teams, stats += ss) {
        fetch(slot == 0 ? kAhead - 1 : slot - 1);
        cp_async_wait<kAhead - 1>();
        const bool live = row < M;
        Lanes<VEC> f[NV], gate[NV];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f[i] = vset<VEC>(0.f);
            if (in[i] && live) {
                f[i] = ahead.get(slot, 0, i, x + c[i], gs - c[i]);
                if (K == 2) gate[i] = vact<VEC>(ahead.get(slot, 1, i, z + c[i], gs - c[i]), silu);
                if (GATE == MG_GATE_FIRST) f[i] = vmul<VEC>(f[i], gate[i]);
                sum += vsum<VEC>(f[i]);
            }
        }
        float mean = 0.f;
        if (!p.rms) mean = team_sum<TEAM>(sum, tpg, buf[0]) * inv;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i] && live) {
                f[i] = vadd<VEC>(f[i], vset<VEC>(-mean));
                if (kRagged<T, VEC> && c[i] + VEC > gs) {   // no difference where there is no channel
                    float v[VEC];
                    vto<VEC>(f[i], v);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[e] = c[i] + e < gs ? v[e] : 0.f;
                    f[i] = vfrom<VEC>(v);
                }
                sq += vdot<VEC>(f[i], f[i]);
            }
        // (one sum a row: the buffers take turns)
        const float rstd = rsqrtf(fmaf(team_sum<TEAM>(sq, tpg, buf[p.rms ? k & 1 : 1]), inv, p.eps));
        if (live && team.live) {
            if (writes_stats) *stats = make_float2(mean, rstd);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i]) {
                    Lanes<VEC> o = vfma<VEC>(vmul<VEC>(f[i], vset<VEC>(rstd)), w[i], b[i]);
                    if (GATE == MG_GATE_AFTER) o = vmul<VEC>(o, gate[i]);
                    if (GATE == MG_GATE_NONE) o = vact<VEC>(o, silu);
                    vstore<T, VEC>(y + c[i], o, gs - c[i]);
                }
        }
        x += xs;
        z += zs;
        y += ys;
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    cp_async_wait<0>();
}

// Gradients.  With n = (p - mean) rstd and dn = do w, over a group
//   dp = rstd (dn - mean(dn) - n mean(dn n))    (rms: without mean(dn))
// and the gate's chain rule around it.  dw and dbias are summed over a team's
// rows in registers; the teams' sums are added in order by sum_parts_kernel.
template <typename T, int VEC, int NV, mg_gate GATE, int TEAM, int SILU>
__global__ void __launch_bounds__(512)
norm_bwd_kernel(NormArgs p, int team_size, int row_teams, float *part)
{
    const int tpg = TEAM > 0 ? TEAM : team_size, silu = SILU == 1 ? 1 : p.silu;
    constexpr int K = GATE == MG_GATE_NONE ? 2 : 3;
    __shared__ float buf[2][32];
    extern __shared__ __align__(16) unsigned char ring[];
    const Team team(p, tpg, row_teams);
    const int gs = int(p.D / p.G);
    const Ahead<T, VEC, NV, K> ahead{ring + threadIdx.x * Ahead<T, VEC, NV, K>::kBytes};
    const T *x = static_cast<const T *>(p.x) + int64_t(team.slot) * p.ldx + team.d0;
    const T *z = static_cast<const T *>(p.z) + int64_t(team.slot) * p.ldz + team.d0;
    const T *dy = static_cast<const T *>(p.dy) + int64_t(team.slot) * p.lddy + team.d0;
    int64_t out = int64_t(team.slot) * p.D + team.d0;
    Lanes<VEC> w[NV], b[NV], dw[NV], db[NV];
    int c[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = (i * tpg + team.lane) * VEC;
        in[i] = team.live && c[i] < gs;
        w[i] = b[i] = dw[i] = db[i] = vset<VEC>(0.f);
        if (in[i]) {
            w[i] = pload<T, VEC>(p.w + team.d0 + c[i], gs - c[i]);
            if (GATE != MG_GATE_FIRST && p.bias != nullptr) b[i] = pload<T, VEC>(p.bias + team.d0 + c[i], gs - c[i]);
        }
    }
    const int64_t xs = row_teams * p.ldx, zs = row_teams * p.ldz, gst = row_teams * p.lddy, os = row_teams * p.D;
    const T *xn = x, *zn = z, *gn = dy;   // of the next row to be fetched
    const int M = int(p.M);   // M G < 2^31
    int64_t row_next = team.slot;
    auto fetch = [&](int slot) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in[i] && row_next < M) {
                ahead.fetch(slot, 0, i, xn + c[i], gs - c[i]);
                ahead.fetch(slot, 1, i, gn + c[i], gs - c[i]);
                if (K == 3) ahead.fetch(slot, K - 1, i, zn + c[i], gs - c[i]);
            }
        xn += xs;
        zn += zs;
        gn += gst;
        row_next += row_teams;
        cp_async_commit();
    };
    const float inv = 1.f / float(gs);
#pragma unroll
    for (int k = 0; k < kAhead - 1; ++k) fetch(k);
    const int rounds = (M - 1) / row_teams + 1;   // the same for every team
    const float2 *stats = reinterpret_cast<const float2 *>(p.stats_in) + (int64_t(team.slot) * p.G + team.g);
    const int64_t ss = row_teams * p.G;
    int slot = 0;
    int64_t row = team.slot;
    for (int k = 0; k < rounds; ++k, row += row_teams, stats += ss) {
        fetch(slot == 0 ? kAhead - 1 : slot - 1);
        const bool live = team.live && row < M;
        float2 st = make_float2(0.f, 0.f);
        if (live) st = *stats;
        cp_async_wait<kAhead - 1>();
        const Lanes<VEC> rstd = vset<VEC>(st.y);
        Lanes<VEC> n[NV], dn[NV], ga[NV], gg[NV];
        float m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in[i]) {
                Lanes<VEC> pv = ahead.get(slot, 0, i, x + c[i], gs - c[i]), dov = ahead.get(slot, 1, i, dy + c[i], gs - c[i]);
                if (K == 3) ga[i] = vact<VEC>(ahead.get(slot, K - 1, i, z + c[i], gs - c[i]), silu, gg[i]);
                if (GATE == MG_GATE_FIRST) {
                    gg[i] = vmul<VEC>(gg[i], pv);
                    pv = vmul<VEC>(pv, ga[i]);
                }
                // (p - mean) rstd: the difference first where the mean is not 0
                n[i] = p.rms ? vmul<VEC>(pv, rstd) : vmul<VEC>(vadd<VEC>(pv, vset<VEC>(-st.x)), rstd);
                if (GATE != MG_GATE_FIRST) {
                    const Lanes<VEC> o = vfma<VEC>(n[i], w[i], b[i]);
                    if (GATE == MG_GATE_AFTER) {
                        vstore<T, VEC>(static_cast<T *>(p.dz) + out + c[i], vmul<VEC>(vmul<VEC>(dov, o), gg[i]), gs - c[i]);
                        dov = vmul<VEC>(dov, ga[i]);
                    } else {
                        Lanes<VEC> grad;
                        vact<VEC>(o, silu, grad);
                        dov = vmul<VEC>(dov, grad);
                    }
                }
                dw[i] = vfma<VEC>(dov, n[i], dw[i]);
                db[i] = vadd<VEC>(db[i], dov);
                dn[i] = vmul<VEC>(dov, w[i]);
                m1 += vsum<VEC>(dn[i]);
                m2 += vdot<VEC>(dn[i], n[i]);
            }
        m1 = p.rms ? 0.f : team_sum<TEAM>(m1, tpg, buf[0]) * inv;
        m2 = team_sum<TEAM>(m2, tpg, buf[p.rms ? k & 1 : 1]) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && in[i]) {
                Lanes<VEC> dp = vadd<VEC>(vfma<VEC>(n[i], vset<VEC>(-m2), dn[i]), vset<VEC>(-m1));
                dp = vmul<VEC>(dp, rstd);
                if (GATE == MG_GATE_FIRST) {
                    vstore<T, VEC>(static_cast<T *>(p.dz) + out + c[i], vmul<VEC>(dp, gg[i]), gs - c[i]);
                    dp = vmul<VEC>(dp, ga[i]);
                }
                vstore<T, VEC>(static_cast<T *>(p.dx) + out + c[i], dp, gs - c[i]);
            }
        x += xs;
        z += zs;
        dy += gst;
        out += os;
        slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    // part: row_teams rows of dw (D) and then of dbias (D)
    float *to = part + int64_t(team.slot) * 2 * p.D + team.d0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in[i]) {
            pstore<T, VEC>(to + c[i], dw[i], gs - c[i]);
            pstore<T, VEC>(to + p.D + c[i], db[i], gs - c[i]);
        }
}

// The team for groups of gs channels: the smallest power of two that covers
// it with NV vectors of vec channels a thread.
int team_for(int64_t gs, int vec, int nv)
{
    int t = 1;
    while (int64_t(t) * vec * nv < gs) t *= 2;
    return t;
}

// A team of several warps has its block to itself, for its barriers.
// (32768 rows of 4 groups of 1024 bf16: 158 -> 146 us, gradients 376 -> 333.)
int block_for(int tpg) { return tpg > 32 ? tpg : 256; }

// (vector width, vectors a thread, team) of a call.  Vectors are 16 bytes
// where the group's width and the rows allow, else half that, ragged.
//
// A thread takes two vectors where a group has more than 8 of them, which
// leaves fewer threads to meet over its sums, and more only where 512 threads
// do not cover it.  Of 32768 x 4096 bf16 channels gated first, one vector
// against two: one group 175 us to 134, 4 groups 164 to 131, 32 groups 144 to
// 136.  The gradients hold more of a row in registers and begin later, at more
// than 256 (128 float32) channels: one group 397 to 366 us, 8 groups 297 to
// 278, but 16 groups 256 to 276; 8192 rows of 32 float32 groups 135 to 118.
//
// Ragged vectors take the fewest a thread whose team fits a warp, else at most
// kRaggedTeam threads (8192 rows of 1001 bf16 channels: 56 us; with up to 64
// 62; of float32 65 and 90).  512 threads of 8 vectors (float32 pairs: 16)
// hold the widest group, 16384 channels.
constexpr int kRaggedTeam = 128;
struct Shape {
    int vec, nv, tpg;
};
Shape shape_for(mg_dtype dt, int64_t gs, bool aligned, bool backward)
{
    const int full = dt == MG_F32 ? 4 : 8;
    Shape c;
    const bool whole = aligned && gs % full == 0;
    c.vec = whole ? full : full / 2;
    const int most = c.vec == 2 ? 16 : 8, warp = 32, one = backward ? 4 * full : 8;
    auto fits = [&](int nv, int limit) {
        c.nv = nv;
        c.tpg = team_for(gs, c.vec, nv);
        return c.tpg <= limit;
    };
    if (!whole) {
        for (int limit : {warp, kRaggedTeam, kMaxTeam})
            if (fits(1, limit) || fits(2, limit) || (c.vec == 2 && fits(4, limit))) return c;
        if (fits(4, kMaxTeam)) return c;
    } else if (fits(1, one) || fits(2, kMaxTeam) || fits(4, kMaxTeam)) {
        return c;
    }
    if (!fits(most, kMaxTeam)) c.tpg = 0;
    return c;
}

// Row teams: so many that the teams of all groups fill the SMs with `warps`
// warps each, at most one for each row.
int64_t row_teams_for(int64_t M, int64_t G, int tpg, int warps)
{
    const int block = block_for(tpg);
    const int64_t all = int64_t(152) * (warps * 32 / block > 0 ? warps * 32 / block : 1) * (block / tpg);
    int64_t n = all / G;
    n = n < 1 ? 1 : n;
    return n < M ? n : M;
}
constexpr int kFwdWarps = 32, kBwdWarps = 16;   // what an SM holds by the kernels' registers

template <typename T, int VEC, int NV, mg_gate GATE, int TEAM, int SILU>
mg_status norm_fwd_team(const NormArgs &p, int tpg, cudaStream_t s)
{
    const int block = block_for(tpg);
    const int64_t rt = row_teams_for(p.M, p.G, tpg, kFwdWarps);
    MG_TRY(check_grids("mg_group_norm_fwd", {ceil_div(rt * p.G, block / tpg)}));
    const size_t smem = Ahead<T, VEC, NV, GATE == MG_GATE_NONE ? 1 : 2>::bytes(block);
    MG_TRY(allow_shared<norm_fwd_kernel<T, VEC, NV, GATE, TEAM, SILU>>(smem));
    norm_fwd_kernel<T, VEC, NV, GATE, TEAM, SILU><<<unsigned(ceil_div(rt * p.G, block / tpg)), block, smem, s>>>(
        p, tpg, int(rt));
    return launched("mg_group_norm_fwd");
}

template <typename T, int VEC, int NV, mg_gate GATE, int TEAM, int SILU>
mg_status norm_bwd_team(const NormArgs &p, int tpg, cudaStream_t s)
{
    const int block = block_for(tpg);
    const int64_t rt = row_teams_for(p.M, p.G, tpg, kBwdWarps);
    MG_TRY(check_grids("mg_group_norm_bwd", {ceil_div(rt * p.G, block / tpg), sum_parts_blocks(2 * p.D)}));
    float *part = reinterpret_cast<float *>(static_cast<char *>(p.ws) + kControlBytes);
    const size_t smem = Ahead<T, VEC, NV, GATE == MG_GATE_NONE ? 2 : 3>::bytes(block);
    MG_TRY(allow_shared<norm_bwd_kernel<T, VEC, NV, GATE, TEAM, SILU>>(smem));
    norm_bwd_kernel<T, VEC, NV, GATE, TEAM, SILU><<<unsigned(ceil_div(rt * p.G, block / tpg)), block, smem, s>>>(
        p, tpg, int(rt), part);
    MG_TRY(launched("mg_group_norm_bwd"));
    return launch_sum_parts(part, rt, {{p.dw, p.D}, {p.dbias, p.D}}, s);
}

// Groups of one or two 16-byte vectors a thread, gated or activated by SiLU,
// have kernels for their team's size; the rest share one for any size.
#define MG_NORM_TEAM(F)                                                              \
    if constexpr (NV <= 2 && !kRagged<T, VEC>) {                                     \
        if (p.silu) {                                                                \
            if (tpg == 8) return F<T, VEC, NV, GATE, 8, 1>(p, tpg, s);               \
            if (tpg == 16) return F<T, VEC, NV, GATE, 16, 1>(p, tpg, s);             \
            if (tpg == 32) return F<T, VEC, NV, GATE, 32, 1>(p, tpg, s);             \
            if (tpg > 32) return F<T, VEC, NV, GATE, kBlock, 1>(p, tpg, s);          \
        }                                                                            \
    }                                                                                \
    return F<T, VEC, NV, GATE, kAny, -1>(p, tpg, s);
template <typename T, int VEC, int NV, mg_gate GATE>
mg_status norm_fwd_gate(const NormArgs &p, int tpg, cudaStream_t s)
{
    MG_NORM_TEAM(norm_fwd_team)
}
template <typename T, int VEC, int NV, mg_gate GATE>
mg_status norm_bwd_gate(const NormArgs &p, int tpg, cudaStream_t s)
{
    MG_NORM_TEAM(norm_bwd_team)
}

template <typename T, int VEC, int NV>
mg_status norm_fwd(const NormArgs &p, int tpg, cudaStream_t s)
{
    switch (p.gate) {
    case MG_GATE_NONE: return norm_fwd_gate<T, VEC, NV, MG_GATE_NONE>(p, tpg, s);
    case MG_GATE_AFTER: return norm_fwd_gate<T, VEC, NV, MG_GATE_AFTER>(p, tpg, s);
    default: return norm_fwd_gate<T, VEC, NV, MG_GATE_FIRST>(p, tpg, s);
    }
}
template <typename T, int VEC, int NV>
mg_status norm_bwd(const NormArgs &p, int tpg, cudaStream_t s)
{
    switch (p.gate) {
    case MG_GATE_NONE: return norm_bwd_gate<T, VEC, NV, MG_GATE_NONE>(p, tpg, s);
    case MG_GATE_AFTER: return norm_bwd_gate<T, VEC, NV, MG_GATE_AFTER>(p, tpg, s);
    default: return norm_bwd_gate<T, VEC, NV, MG_GATE_FIRST>(p, tpg, s);
    }
}

// Calls F<T, VEC, NV> for the call's shape.
#define MG_NORM_NV(F, T, VEC)                      \
    switch (c.nv) {                                \
    case 1: return F<T, VEC, 1>(p, c.tpg, s);      \
    case 2: return F<T, VEC, 2>(p, c.tpg, s);      \
    case 4: return F<T, VEC, 4>(p, c.tpg, s);      \
    }
#define MG_NORM(F)                                                                       \
    const int vec = dt == MG_F32 ? 4 : 8;                                                \
    const bool al = p.D % vec == 0 && p.ldx % vec == 0 &&                                \
                    (p.z == nullptr || p.ldz % vec == 0) &&                              \
                    (p.dy == nullptr || p.lddy % vec == 0);                              \
    const Shape c = shape_for(dt, p.D / p.G, al, p.dy != nullptr);                       \
    if (c.tpg == 0)                                                                      \
        return fail(MG_ERR_UNSUPPORTED, "group of %lld channels too wide",               \
                    (long long)(p.D / p.G));                                             \
    if (dt == MG_F32) {                                                                  \
        if (c.vec == 4) {                                                                \
            MG_NORM_NV(F, float, 4)                                                      \
            return F<float, 4, 8>(p, c.tpg, s);                                          \
        }                                                                                \
        MG_NORM_NV(F, float, 2)                                                          \
        return F<float, 2, 16>(p, c.tpg, s);                                             \
    }                                                                                    \
    if (c.vec == 8) {                                                                    \
        MG_NORM_NV(F, bf16_t, 8)                                                         \
        return fail(MG_ERR_UNSUPPORTED, "group too wide");                               \
    }                                                                                    \
    MG_NORM_NV(F, bf16_t, 4)                                                             \
    return F<bf16_t, 4, 8>(p, c.tpg, s);

}  // namespace

size_t norm_ws_bytes(int64_t M, int64_t D, int64_t G)
{
    // the largest over the shapes that the call's type and strides may give
    size_t need = 0;
    for (mg_dtype dt : {MG_F32, MG_BF16})
        for (bool al : {false, true}) {
            const Shape c = shape_for(dt, D / G, al, true);
            if (c.tpg == 0) continue;
            const size_t n = size_t(row_teams_for(M, G, c.tpg, kBwdWarps)) * 2 * D * sizeof(float);
            need = n > need ? n : need;
        }
    return kControlBytes + need;
}

mg_status launch_norm_fwd(const NormArgs &p, mg_dtype dt, cudaStream_t s) { MG_NORM(norm_fwd) }
mg_status launch_norm_bwd(const NormArgs &p, mg_dtype dt, cudaStream_t s) { MG_NORM(norm_bwd) }

}  // namespace mg
