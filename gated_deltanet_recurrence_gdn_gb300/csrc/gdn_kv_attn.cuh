// gdn_kv_attn.cuh -- what the attention kernels over a paged cache (4 or 8 bits) share:
// the call's arguments, what each row sees, and the division of the work.
#pragma once

#include <cmath>

#include "gdn_kv.cuh"
#include "tc_ptx.cuh"

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
    int end_tiles;             // what the end of a piece costs, in tiles (Plan, where it counts it)

    // The bounds-check build: a row of q, o and lse; one of the pieces' rows, of `rows` each
    // in two slots a CTA.
    __device__ __forceinline__ bool row_ok(long long tok, int hq) const {
        return GDN_IDX_OK(tok, 1, kv.n_tokens) && GDN_IDX_OK(hq, 1, Hq);
    }
    __device__ __forceinline__ bool part_ok(long long row, int rows) const {
        return GDN_IDX_OK(row, 1, 2ll * gridDim.x * rows);
    }
};

// A (sequence, key/value head, row tile) that is cut, written by the CTA with its
// first piece: pieces are slot0 of that CTA i, then slots 2 (i + 1), 2 (i + 2), ...
struct Cut {
    int pieces;                // 0: the CTA's last piece is whole
    int slot0, first, h, row0, rows;
};

// Quotients of counts, which seldom need 64 bits (a division in 64 takes about 500
// cycles when its code is met for the first time).
__device__ __forceinline__ long long quot(long long a, long long b) {
    if (__builtin_expect((a | b) >> 32 != 0, 0)) return a / b;
    return (unsigned)a / (unsigned)b;
}

// Tokens of one sequence and what its rows see.  Row r of a (sequence,
// key/value head) is query head h G + r % G of new token r / G.
struct Seq {
    int first, n, len;

    __device__ __forceinline__ void get(const AttnArgs &a, int b) {
        a.kv.tokens(b, first, n, len, a.err);
        if (len > a.max_len || n > a.max_new) {
            atomicCAS(a.err, 0, kErrBadIndex);
            if (len > a.max_len) len = 0;
            if (n > a.max_new) n = 0;
        }
    }
    // Places [from, to) that new token j sees.  (p may be far below 0 and the window as
    // large as an int: their difference is formed only where it is not negative.)
    __device__ __forceinline__ void sees(const AttnArgs &a, int j, int &from, int &to) const {
        const int p = len - n + j;
        to = p < 0 ? 0 : a.causal ? p + 1 : len;
        from = a.window > 0 && p >= a.window ? p + 1 - a.window : 0;
    }
};

// The work of a call is a list of tiles of `kTile` places: of every sequence in
// turn, of its key/value heads, of the head's row tiles (kRows rows each), of
// what the row tile's rows see (one tile where they see nothing: its rows are
// written as zero).  CTA i of `grid` takes the tiles [total i / g, total (i + 1)
// / g), g = min(grid, total): every CTA has the same number of tiles to within
// one whatever the lengths, and a (sequence, head, row tile) is cut only where
// one of the g - 1 borders falls inside it.  With kEnds each (sequence, head, row tile)
// counts `end_tiles` tiles more, behind its own and with nothing in them, for the time
// that its end takes: a share of many short ones has fewer tiles.
template <int kTile, int kRows, int kThreads, bool kEnds = false>
struct Plan {
    long long prefix[kThreads];   // tiles before the sequences of each thread's share
    long long total;

    __device__ static __forceinline__ int row_tiles(const AttnArgs &a, const Seq &s) {
        return (int)(((unsigned)s.n * (unsigned)a.G + kRows - 1) / kRows);   // (below 2^31 rows)
    }
    // Places [lo, lo + span) cover what any row of row tile rt sees; lo is rounded
    // down to a page or to 128, whichever is less.
    __device__ static __forceinline__ void range(const AttnArgs &a, const Seq &s, int rt, int &lo,
                                                 int &span) {
        int none, to;
        const unsigned r0 = (unsigned)rt * kRows, G = a.G;
        s.sees(a, (int)(r0 / G), lo, none);
        s.sees(a, min(s.n - 1, (int)((r0 + kRows - 1) / G)), none, to);
        lo &= -min(a.kv.page_size(), 128);
        span = max(0, to - lo);
    }
    __device__ static __forceinline__ int tiles(int span) {
        return max(1, (span + kTile - 1) / kTile);
    }
    __device__ static __forceinline__ int counted(const AttnArgs &a, int span) {
        return tiles(span) + (kEnds ? a.end_tiles : 0);
    }
    // Tiles of row tiles [r0, r1) of one key/value head of the sequence.
    __device__ static __forceinline__ long long tiles_of(const AttnArgs &a, const Seq &s, int r0,
                                                         int r1) {
        long long sum = 0;
        for (int rt = r0; rt < r1; ++rt) {
            int lo, span;
            range(a, s, rt, lo, span);
            sum += counted(a, span);
        }
        return sum;
    }
    // The same of all row tiles by a warp, a run of `per` of them a lane: the sum up to
    // and with this lane's in `upto`.
    __device__ static __forceinline__ long long tiles_by_lane(const AttnArgs &a, const Seq &s,
                                                              int &per, long long &upto) {
        const int n = row_tiles(a, s), lane = threadIdx.x & 31;
        per = (n + 31) / 32;
        if (n <= 1) {
            upto = tiles_of(a, s, 0, n);
            return lane == 0 ? upto : 0;
        }
        const long long own = tiles_of(a, s, min(n, lane * per), min(n, lane * per + per));
        upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        return own;
    }
    // Whole CTA; `this` in shared memory.
    __device__ void build(const AttnArgs &a) {
        __shared__ long long warp_sum[kThreads / 32];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int share = (a.kv.N + kThreads - 1) / kThreads;
        long long mine = 0;
        Seq s;
        if (a.kv.N <= kThreads / 32) {      // a warp a sequence: few may have many row tiles
            if (warp < a.kv.N) {
                int per;
                long long upto;
                s.get(a, warp);
                tiles_by_lane(a, s, per, upto);
                if (lane == 31) prefix[warp] = a.kv.H * upto;
            }
            __syncthreads();
            if (threadIdx.x < a.kv.N) mine = prefix[threadIdx.x];
        } else {
            for (int i = 0; i < share; ++i) {
                const int b = threadIdx.x * share + i;
                if (b >= a.kv.N) break;
                s.get(a, b);
                mine += a.kv.H * tiles_of(a, s, 0, row_tiles(a, s));
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
};

// One CTA's walk over its pieces: the part of its tiles that belongs to one
// (sequence, head, row tile).
template <int kTile, int kRows, int kThreads, bool kEnds = false>
struct Walk {
    using P = Plan<kTile, kRows, kThreads, kEnds>;
    Seq sq;
    int b, h, rt, n_rt, lo, span, n_tiles;
    int tile0, tile1;             // the piece: tiles [tile0, tile1) of n_tiles
    long long cur, end;           // first tile of the piece, end of the CTA's tiles

    __device__ __forceinline__ int row0() const { return rt * kRows; }
    __device__ __forceinline__ int rows(const AttnArgs &a) const {
        return min(kRows, sq.n * a.G - rt * kRows);
    }
    __device__ __forceinline__ bool complete() const { return tile0 == 0 && tile1 == n_tiles; }
    __device__ __forceinline__ int place0() const { return lo + tile0 * kTile; }
    // Tiles of the piece that hold anything.
    __device__ __forceinline__ int count() const {
        if (span <= 0) return 0;
        if constexpr (!kEnds) return tile1 - tile0;
        const int real = P::tiles(span);
        return min(tile1, real) - min(tile0, real);
    }

    __device__ __forceinline__ void piece(const AttnArgs &a, int from) {
        P::range(a, sq, rt, lo, span);
        n_tiles = P::counted(a, span);
        tile0 = from;
        tile1 = (int)min((long long)n_tiles, tile0 + (end - cur));
    }
    // Of a call whose pieces are one tile each (nothing is cut and no end counted), the same
    // number in every sequence: without a plan.
    __device__ static __forceinline__ long long alike_total(const AttnArgs &a) {
        return (long long)a.kv.N * a.kv.H * P::row_tiles(a, Seq{0, a.kv.n_tokens / a.kv.N, 0});
    }
    __device__ __forceinline__ void start_alike(const AttnArgs &a, long long at, long long until) {
        cur = at;
        end = until;
        n_rt = P::row_tiles(a, Seq{0, a.kv.n_tokens / a.kv.N, 0});
        const long long head = quot(at, n_rt);
        rt = (int)(at - head * n_rt);
        b = (int)quot(head, a.kv.H);
        h = (int)(head - (long long)b * a.kv.H);
        sq.get(a, b);
        piece(a, 0);
    }
    // By whole warps.
    __device__ void start(const AttnArgs &a, const P &plan, long long at, long long until) {
        cur = at;
        end = until;
        int i = 0, j = kThreads;
        while (j - i > 1) {
            const int m = (i + j) >> 1;
            if (plan.prefix[m] <= at) i = m;
            else j = m;
        }
        b = i * ((a.kv.N + kThreads - 1) / kThreads);
        long long left = at - plan.prefix[i], per_head, own, upto;
        int per;
        for (;; ++b) {
            sq.get(a, b);
            own = P::tiles_by_lane(a, sq, per, upto);
            per_head = __shfl_sync(0xffffffffu, upto, 31);
            if (left < per_head * a.kv.H) break;
            left -= per_head * a.kv.H;
        }
        h = (int)quot(left, per_head);
        left -= h * per_head;
        n_rt = P::row_tiles(a, sq);
        // the lane that has the tile, then the row tile
        const int lane = __ffs(__ballot_sync(0xffffffffu, upto > left)) - 1;
        left -= __shfl_sync(0xffffffffu, upto - own, lane);
        for (rt = lane * per;; ++rt) {
            P::range(a, sq, rt, lo, span);
            const int n = P::counted(a, span);
            if (left < n) break;
            left -= n;
        }
        piece(a, (int)left);
    }
    // The next piece; false at the end of the CTA's tiles.
    __device__ __forceinline__ bool next(const AttnArgs &a) {
        cur += tile1 - tile0;
        if (cur >= end) return false;
        if (++rt == n_rt) {
            rt = 0;
            if (++h == a.kv.H) {
                h = 0;
                do {
                    sq.get(a, ++b);
                    n_rt = P::row_tiles(a, sq);
                } while (n_rt == 0);
            }
        }
        piece(a, 0);
        return true;
    }
};

// Copy of `bytes` (a multiple of 16, both sides 16-byte aligned) into shared
// memory, counted on the mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
    if (!GDN_SMEM_OK(dst, bytes) || !GDN_SMEM_OK(ptx::smem_u32(bar), 8)) return;
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
        : "memory");
}

// Waits, in one warp, for the copies still on their way into a ring: armed[s] is the number
// of phases of full[s] that copies have been counted on, the last one's may be in flight.
template <int kStages>
__device__ __forceinline__ void drain_ring(uint64_t *full, const uint32_t *armed) {
    for (int s = 0; s < kStages; ++s)
        if (armed[s] > 0) ptx::mbar_wait(full + s, (armed[s] - 1) & 1, ptx::kDrainLimit);
}

// The waits of a CTA: bounded, and over at once when one of them has given up
// (the error is recorded, and the CTA runs to its end without computing).
struct Waits {
    volatile int *abort;
    int *err;
    uint32_t limit;
    // By a whole warp, all lanes of which learn the same: lanes poll the barrier and the
    // CTA's flag one by one, so they vote.  What follows may be for the whole warp.
    __device__ __forceinline__ bool on(uint64_t *bar, uint32_t parity) const {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        for (uint32_t i = 0; i < limit; ++i) {
            if (__any_sync(0xffffffffu, *abort != 0)) return false;
            if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
        }
        *abort = 1;
        atomicCAS(err, 0, kErrTimeout);
        return false;
    }
    // A lane's own: lanes may learn different things when it gives up, so that nothing
    // which the whole warp takes part in may depend on the result.
    __device__ __forceinline__ bool on_lane(uint64_t *bar, uint32_t parity) const {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        for (uint32_t i = 0; i < limit; ++i) {
            if (*abort) return false;
            if (ptx::mbar_try_wait(bar, parity)) return true;
        }
        *abort = 1;
        atomicCAS(err, 0, kErrTimeout);
        return false;
    }
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, __half2 b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The power of two that brings a row whose largest magnitude is m to [2^13, 2^14)
// (fp16's upper range; rows below 2^-100 stay smaller), and what undoes it.
__device__ __forceinline__ float row_up(float m, float &down) {
    const uint32_t ex = max(27u, __float_as_uint(m) >> 23);
    down = __uint_as_float((ex - 13u) << 23);
    return __uint_as_float((267u - ex) << 23);
}

__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(a, b), pack2(c, d));
}
// A row's logarithm of the sum of its exponentials, from what its scores lost.
__device__ __forceinline__ float lse_of(float sub, float sum) {
    return sum == 0.f ? -INFINITY : (sub + log2f(sum)) * 0.69314718055994531f;
}

// Adds the pieces of what was cut, in order.  CTA (i, y): kJoin / kStripes rows of
// the one whose first piece CTA i of the attention kernel had; kStripes of its kJoin
// warps share a row's pieces (many pieces of few rows, or the other way round).
template <typename T, int D, int kRows, int kJoin, int kStripes>
__global__ void __launch_bounds__(kJoin * 32) k_kv_join(const AttnArgs a) {
    constexpr int kVec = D / 32, kCtaRows = kJoin / kStripes;
    __shared__ float sums[kJoin][D];
    __shared__ float2 warp_ml[kJoin];
    ptx::griddep_wait();
    const Cut c = a.cuts[blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int local = warp / kStripes, stripe = warp - local * kStripes;
    if (blockIdx.y * kCtaRows >= c.rows || c.pieces == 0) return;
    const int r = min((int)blockIdx.y * kCtaRows + local, c.rows - 1);   // (the last row again)
    auto slot = [&](int k) {
        return (k == 0 ? (long long)c.slot0 : 2ll * (blockIdx.x + k)) * kRows + r;
    };
    // (a row's first pieces are on their way while its maximum is found)
    constexpr int kFirst = 2;
    struct Piece {
        float2 ml;
        float v[kVec];
        __device__ __forceinline__ void load(const AttnArgs &a, long long at, int lane) {
            if (!a.part_ok(at, kRows)) return;
            const float *p = a.part_o + at * D + lane * kVec;
            ml = a.part_ml[at];
            if constexpr (kVec == 2) {
                const float2 x = *reinterpret_cast<const float2 *>(p);
                v[0] = x.x; v[1] = x.y;
            } else {
#pragma unroll
                for (int e = 0; e < kVec; e += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(p + e);
                    v[e] = x.x; v[e + 1] = x.y; v[e + 2] = x.z; v[e + 3] = x.w;
                }
            }
        }
    } first[kFirst];
#pragma unroll
    for (int u = 0; u < kFirst; ++u)
        if (stripe + u * kStripes < c.pieces) first[u].load(a, slot(stripe + u * kStripes), lane);
    float m = -INFINITY;
    for (int k = lane; k < c.pieces; k += 32)
        if (a.part_ok(slot(k), kRows)) m = fmaxf(m, a.part_ml[slot(k)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float v[kVec] = {}, l = 0.f;
    auto add = [&](const Piece &x) {
        const float f = m == -INFINITY ? 1.f : ex2(x.ml.x - m);
        l += x.ml.y * f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] += x.v[e] * f;
    };
#pragma unroll
    for (int u = 0; u < kFirst; ++u)
        if (stripe + u * kStripes < c.pieces) add(first[u]);
#pragma unroll 4
    for (int k = stripe + kFirst * kStripes; k < c.pieces; k += kStripes) {
        Piece x;
        x.load(a, slot(k), lane);
        add(x);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sums[warp][lane * kVec + e] = v[e];
    if (lane == 0) warp_ml[warp].y = l;
    __syncthreads();
    if (stripe != 0) return;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kStripes; ++w) l += warp_ml[warp + w].y;
    const int rr = c.row0 + r, j = rr / a.G, hq = c.h * a.G + rr - j * a.G;
    const float gv = a.kv.head_scale ? __ldg(a.kv.head_scale + a.kv.H + c.h) : 1.f;
    const float inv = l == 0.f ? 0.f : gv / l;
    T *p = static_cast<T *>(a.o) + (c.first + j) * a.o_tok + hq * a.o_head;
    if (!a.row_ok((long long)c.first + j, hq)) return;
    for (int d = 4 * lane; d < D; d += 128) {
        float x[4] = {};
#pragma unroll
        for (int w = 0; w < kStripes; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += sums[warp + w][d + e];
        store4(p + d, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    }
    if (a.lse && lane == 0) a.lse[(long long)(c.first + j) * a.Hq + hq] = lse_of(m, l);
}

// Scratch for the pieces of a launch of `grid` CTAs with kRows rows, into `a`.
template <int D, int kRows>
inline cudaError_t alloc_pieces(AttnArgs &a, int grid, void **scratch, cudaStream_t st) {
    const size_t po = (size_t)2 * grid * kRows * D * 4, pm = (size_t)2 * grid * kRows * 8;
    const cudaError_t e = scratch_alloc(scratch, po + pm + grid * sizeof(Cut), st);
    if (e != cudaSuccess) return e;
    a.part_o = static_cast<float *>(*scratch);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(*scratch) + po);
    a.cuts = reinterpret_cast<Cut *>(static_cast<uint8_t *>(*scratch) + po + pm);
    return cudaSuccess;
}
// The join after such a launch: started while that runs, it waits for its end.
template <typename T, int D, int kRows, int kJoin, int kStripes>
inline cudaError_t launch_join(const AttnArgs &a, int grid, cudaStream_t st) {
    const long long most = (long long)a.max_new * a.G;
    const int rows = (int)(most < kRows ? most : kRows), per = kJoin / kStripes;
    if (grid < 2 || rows < 1) return cudaSuccess;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid, (rows + per - 1) / per);
    cfg.blockDim = dim3(kJoin * 32);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, k_kv_join<T, D, kRows, kJoin, kStripes>, a);
}

// Many rows (gdn_kv_attn_tc.cu): bf16 rows, d = 64 or 128; F: Fmt4 or Fmt8.
template <typename F>
gdn_status attn_many(AttnArgs &a, cudaStream_t st);

}  // namespace kv
}  // namespace gdn
