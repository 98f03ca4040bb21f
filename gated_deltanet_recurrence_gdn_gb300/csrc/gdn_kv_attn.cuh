// gdn_kv_attn.cuh -- what the attention kernels over the 4-bit cache share: the
// call's arguments, what each row sees, and the division of the work.
#pragma once

#include "gdn_kv.cuh"

namespace gdn {
namespace kv {

struct AttnArgs {
    Kv kv;
    const void *q;             // rows of the I/O dtype, strides below
    void *o;
    float *lse;                // [n_tokens][Hq] or nullptr
    long long q_head, q_tok, o_head, o_tok;
    int Hq, G;                 // query heads; of one key/value head
    int max_len, max_new;
    float scale_log2;          // scale * log2(e)
    int window;                // 0: none
    bool causal;
    float *part_o;             // [2 * grid][rows][d], sums that a join still divides
    float2 *part_ml;           // [2 * grid][rows]: what scores lost (log2 units) and sum
    struct Cut *cuts;          // [grid], nullptr where nothing is cut
    int *err;
    uint32_t wait_limit;       // polls of a wait before it gives up
};

// A (sequence, key/value head, row tile) that is cut, written by the CTA with its
// first piece: pieces are slot0 of that CTA i, then slots 2 (i + 1), 2 (i + 2), ...
struct Cut {
    int pieces;                // 0: the CTA's last piece is whole
    int slot0, first, h, row0, rows;
};

// Tokens of one sequence and what its rows see.  Row r of a (sequence,
// key/value head) is query head h G + r % G of new token r / G.
struct Seq {
    int first, n, len;
    int lo;                    // first place that any row sees, rounded down to a page or
                               // to 128, whichever is less
    int span;                  // places [lo, lo + span) cover what any row sees

    __device__ __forceinline__ void get(const AttnArgs &a, int b) {
        a.kv.tokens(b, first, n, len, a.err);
        if (len > a.max_len || n > a.max_new) {
            atomicCAS(a.err, 0, kErrBadIndex);
            if (len > a.max_len) len = 0;
            if (n > a.max_new) n = 0;
        }
        lo = 0;
        if (a.window > 0) lo = max(0, len - n + 1 - a.window) & -min(a.kv.page_size(), 128);
        span = max(0, len - lo);
    }
    // Places [from, to) that new token j sees.
    __device__ __forceinline__ void sees(const AttnArgs &a, int j, int &from, int &to) const {
        const int p = len - n + j;
        to = p < 0 ? 0 : a.causal ? p + 1 : len;
        from = a.window > 0 ? max(0, p + 1 - a.window) : 0;
    }
};

// The work of a call is a list of tiles of `kTile` places: of every sequence in
// turn, of its key/value heads, of the head's row tiles (kRows rows each), of
// what the sequence's rows see (one tile where they see nothing: its rows are
// written as zero).  CTA i of `grid` takes the tiles [total i / g, total (i + 1)
// / g), g = min(grid, total): every CTA has the same number of tiles to within
// one whatever the lengths, and a (sequence, head, row tile) is cut only where
// one of the g - 1 borders falls inside it.
template <int kTile, int kRows, int kThreads>
struct Plan {
    long long prefix[kThreads];   // tiles before the sequences of each thread's share
    long long total;

    __device__ static __forceinline__ int tiles(const Seq &s) {
        return max(1, (s.span + kTile - 1) / kTile);
    }
    __device__ static __forceinline__ int row_tiles(const AttnArgs &a, const Seq &s) {
        return (int)(((long long)s.n * a.G + kRows - 1) / kRows);
    }
    __device__ static __forceinline__ long long weight(const AttnArgs &a, const Seq &s) {
        return (long long)row_tiles(a, s) * a.kv.H * tiles(s);
    }
    // Whole CTA; `this` in shared memory.
    __device__ void build(const AttnArgs &a) {
        __shared__ long long warp_sum[kThreads / 32];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int share = (a.kv.N + kThreads - 1) / kThreads;
        long long mine = 0;
        for (int i = 0; i < share; ++i) {
            const int b = threadIdx.x * share + i;
            if (b < a.kv.N) {
                Seq s;
                s.get(a, b);
                mine += weight(a, s);
            }
        }
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        long long before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            all += warp_sum[w];
        }
        prefix[threadIdx.x] = before + x - mine;
        if (threadIdx.x == 0) total = all;
        __syncthreads();
    }
    // The sequence that tile `at` belongs to, and the tiles before that sequence.
    __device__ void find(const AttnArgs &a, long long at, int &b, long long &start, Seq &s) const {
        int lo = 0, hi = kThreads;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (prefix[m] <= at) lo = m;
            else hi = m;
        }
        const int share = (a.kv.N + kThreads - 1) / kThreads;
        b = lo * share;
        start = prefix[lo];
        for (;; ++b) {
            s.get(a, b);
            const long long w = weight(a, s);
            if (at < start + w) return;
            start += w;
        }
    }
};

}  // namespace kv
}  // namespace gdn
