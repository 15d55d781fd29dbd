// Shared by the gated recurrence's kernels: chunks of rows, gates within a
// chunk, the passes over chunks.
#pragma once

#include "block.cuh"

namespace mg {

// Gates below this count as this: exp(-128) is 0 in float32, and sums of a
// chunk's gates keep their precision.  (+ 0: a caller's signalling NaN must not
// get into the workspace as it is.)
constexpr float kLeastGate = -128.f;
__device__ __forceinline__ float gate_of(float g) { return (g < kLeastGate ? kLeastGate : g) + 0.f; }

// x + y as two floats, exact but for the last bits of the lower ones.
__device__ __forceinline__ void add_two(float &xh, float &xl, float yh, float yl)
{
    const float s = xh + yh, b = s - xh;
    const float e = (xh - (s - b)) + (yh - b) + (xl + yl);
    xh = s + e;
    xl = e - (xh - s);
}

// A batch's chunks of up to L rows, none of them across two sequences.  Dense:
// `per` in each sequence.  Packed: sequence s has the chunks first[s] ..
// first[s+1]-1, a table that launch_chunk_tables leaves in the workspace; of a
// cu that breaks the rules there are none.
struct Chunks {
    Seqs q;
    const int *first;
    int per, L;
    int most;   // chunks that buffers have room for

    struct One {
        long long row;
        int len, seq, idx;   // rows, sequence, place in it
    };
    // Chunk c; len 0: there is none.
    __device__ __forceinline__ One get(int c) const
    {
        One o{0, 0, 0, 0};
        if (q.cu == nullptr) {
            o.seq = int(unsigned(c) / unsigned(per));
            o.idx = c - o.seq * per;
            const long long at = (long long)o.idx * L;
            o.row = (long long)o.seq * q.T + at;
            o.len = int(q.T - at < L ? q.T - at : L);
            return o;
        }
        if (c >= __ldg(first + q.nseq)) return o;
        int lo = 0, hi = q.nseq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(first + mid) <= c) lo = mid; else hi = mid;
        }
        o.seq = lo;
        o.idx = c - __ldg(first + lo);
        o.row = __ldg(q.cu + lo) + (long long)o.idx * L;
        const long long left = __ldg(q.cu + lo + 1) - o.row;
        o.len = int(left < L ? left : L);
        return o;
    }
    __device__ __forceinline__ int begin(int s) const { return q.cu == nullptr ? s * per : __ldg(first + s); }
    __device__ __forceinline__ int end(int s) const { return begin(s + 1); }
};

// The most chunks that a batch can have.
inline int64_t chunks_most(int64_t B, int64_t T, int64_t nseq, bool packed, int L)
{
    return packed ? T / L + (nseq < T ? nseq : T) : B * ceil_div(T, L);
}

// The workspace's parts: [control][first][totals][states][more].
struct GatedWs {
    int64_t chunks;
    size_t first, totals, states, more;   // offsets
};
inline GatedWs gated_ws(int64_t B, int64_t T, int64_t H, int64_t N, int64_t P, int64_t nseq, bool packed, int L,
                        bool states)
{
    GatedWs w{};
    w.chunks = chunks_most(B, T, nseq, packed, L);
    w.first = kControlBytes;
    w.totals = w.first + align_up(packed ? size_t(nseq + 1) * 4 : 0, 256);
    w.states = w.totals + align_up(size_t(w.chunks) * H * 4, 256);
    w.more = w.states + (states ? align_up(size_t(w.chunks) * H * N * P * 4, 256) : 0);
    return w;
}

// Packed batches: checks cu and fills the tables of two cuts of the batch.
mg_status launch_chunk_tables(const Chunks &c, const Chunks &d, void *ws, cudaStream_t s);

// Over the chunks of every sequence and head, in place: states[c] holds what
// chunk c adds, and is left with what comes to it: the state before it
// (forward), or the adjoint of the state behind it (backward = true), from
// `from` (NULL: zero); `to` (may be NULL) gets what comes out at the end.
// totals[c] is the sum of a chunk's gates.
mg_status launch_over_chunks(const Chunks &c, float *states, const float *totals, const float *from, float *to, int H,
                             int64_t NP, bool backward, cudaStream_t s);

// bf16: tensor-core kernels (gated_tc.cu).
size_t gated_tc_saved_bytes(int64_t B, int64_t T, int H, int N, int P, int64_t nseq, bool packed);
size_t gated_tc_ws_bytes(int64_t B, int64_t T, int H, int G, int N, int P, int64_t nseq, bool packed, bool bwd);
mg_status launch_gated_tc_fwd(const GatedArgs &a, cudaStream_t s);
mg_status launch_gated_tc_bwd(const GatedArgs &a, cudaStream_t s);

// The float32 kernels' arguments.
struct GatedCall {
    GatedArgs a;
    Chunks c;
    float *totals, *states;      // states before each chunk
    float *adjoints;             // of the states behind each chunk
    float *partial;              // sums over some of a group's heads: dq, dk
    int splits, heads;           // blocks for a group's heads, heads of each
};

}  // namespace mg
