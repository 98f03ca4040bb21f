// gdn_kv_attn_tc.cu -- attention over the 4-bit paged cache for many rows (a
// chunk of a prompt): tcgen05 products, bf16 rows, d = 64 or 128.
//
// A CTA takes 256 rows of a (sequence, key/value head), row r being query head
// r % G of token r / G, as two tiles of 128, over 128 tokens at a time:
//     S = Q K^T (TMEM),  P = 2^(S - sub) (fp16, into S's columns),  O += P V (TMEM).
// Four roles, 16 warps:
//   warps 0-3, 4-7   softmax of row tile 0 and 1, a thread a row: no exchange
//                    between threads, the row's sum and `sub` in registers;
//   warps 8-11       turn the next 128 tokens' 4-bit numbers into fp16 operand
//                    tiles (128-byte swizzle), a thread a token, its codes
//                    loaded straight into registers one tile ahead;
//   warps 12, 13     issue the products of row tile 0 and 1.  Scores and
//                    probabilities go by halves of 64 tokens with columns of their
//                    own: while the softmax works on one half, PV of the other and
//                    QK of the next tile's follow.
// The products bound it (2 x 2 x 128^3 multiply-adds a tile at d = 128), and next
// to them the exponentials; turning a tile into fp16 costs 1/4 of that time in
// issue slots because 256 rows share it.  Fetching instructions is what a role
// waits for most, so what runs once a tile is kept short: one copy of the
// softmax's code, masks written into the scores before it, issuing loops rolled.
//
// e2m1 * e4m3 is exact in fp16, queries are scaled by a power of two per row, and
// probabilities are fp16 numbers.  `sub` is set so that the first scores' maximum
// is 2^kLift; it moves only when a tile's sum passes 2^15, which any number near
// fp16's end brings about, so no maximum is taken otherwise.  A weight keeps its
// 11 bits down to 2^-22 of the row's largest.  Sums are fp32.
//
// Measured, join included (bf16, d = 128, 16 query and 4 key/value heads): chunks of
// 2048 tokens over 12001 to 16384, two sequences: 350 us, 1.25 PFLOP/s (65 % of a
// dense bf16 product's rate; 3300 cycles a tile where its products alone take
// 2560: scores by halves, n = 64, take 48 cycles a product instead of 32, but
// let products and softmax overlap: with whole tiles 10 % more).  Drafts of 5
// tokens in a window of 4096, 16 sequences: 34 us, in 20 rows of the 256: a tile takes
// 3000 to 3500 cycles there too, bound by the chain from scores to probabilities to
// the next scores.
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace kv {
namespace {

using namespace ptx;

constexpr int kTile = 128;                  // tokens
constexpr int kHalf = kTile / 2;
constexpr int kRowTile = 128;
constexpr int kRows = 2 * kRowTile;
constexpr int kThreads = 512;
constexpr int kConvert = 256;               // first thread of the converting warps
constexpr int kIssuer = 384;                // first thread of the issuing warps
// Registers a thread of each role; together no more than the launch's 512 x 128.
constexpr int kSoftmaxRegs = 168, kConvertRegs = 96, kIssuerRegs = 64;
static_assert(256 * kSoftmaxRegs + 128 * kConvertRegs + 128 * kIssuerRegs <= 512 * 128, "registers");
constexpr float kLift = 8.f;                // log2 of the first maximum's probability
constexpr float kMostSum = 32768.f;         // of a tile: above it `sub` moves

// mbarriers
enum : int {
    B_K_FULL = 0,             // [2] converted keys; 4 warps
    B_K_FREE = 2,             // [2] their products are done; 2 issuing warps
    B_V_FULL = 4,             // [2]
    B_V_FREE = 6,             // [2]
    B_Q_FULL = 8,             // [2] a row tile's queries; 4 warps
    B_S_FULL = 10,            // [2][2] scores of a row tile with each half of the tokens
    B_P_FULL = 14,            // [2][2] probabilities; 4 warps
    B_O_FULL = 18,            // [2][2] their PV is done
    B_SEEN = 22,              // row tile 1 has read a piece's last NaN blocks; 4 warps
    B_DRAIN = 23,             // [2]
    B_COUNT = 25
};

template <int D>
struct Lay {
    static constexpr int kOperand = 128 * D * 2;                 // Q row tile, K tile, V tile
    static constexpr int OFF_Q = 0;                              // [2]
    static constexpr int OFF_K = 2 * kOperand;                   // [2]
    static constexpr int OFF_V = 4 * kOperand;                   // [2]
    static constexpr int OFF_BAR = 6 * kOperand;                 // mbarriers
    static constexpr int SIZE = OFF_BAR + B_COUNT * 8 + 1024;    // (aligned up to 1024)
    static constexpr uint32_t TM_S = 0, TM_O = 256;              // TMEM columns, 128 a row tile
};

__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn) {
    // kind::f16 with fp16 A and B, fp32 accumulation, M = 128
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    if (!GDN_TMEM_OK(d, 128) || !GDN_TMEM_OK(a, 8)) return;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    if (!GDN_TMEM_OK(taddr, 32)) return;   // the address is warp-uniform
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " GDN_OPS32 ";" ::"r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                 "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
                 "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
                 "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
    if (!GDN_SMEM_OK(at, 16)) return;
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// 16-byte chunk c (8 numbers) of row `row` of an operand tile: 64-column blocks
// of 128 rows of 128 bytes, 128-byte swizzled.
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int c) {
    return tile + (c >> 3) * 16384 + sw128_offset(row, c & 7);
}

template <int N>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Pairs of fp32 numbers in one register pair.
__device__ __forceinline__ uint64_t pack64(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack64(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void unpack64(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// One token's codes and scales of K or V of a head, in registers.
template <int D>
struct Token {
    uint4 w[D / 32];
    uint32_t s[D / 64];       // D / 16 scale bytes
    __device__ __forceinline__ void load(const uint8_t *code, const uint8_t *scale) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(code) + i);
        if constexpr (D == 128) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(scale));
            s[0] = x.x; s[1] = x.y;
        } else {
            s[0] = __ldg(reinterpret_cast<const uint32_t *>(scale));
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) s[i] = 0;
    }
    // Zeroes the scales that are NaN; the mask of their blocks.
    __device__ __forceinline__ uint32_t take_nan() {
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            if (((s[i / 4] >> (8 * (i & 3))) & 0x7f) == 0x7f) {
                bad |= 1u << i;
                s[i / 4] &= ~(0xffu << (8 * (i & 3)));
            }
        return bad;
    }
    // Its D numbers as fp16 into row `row` of an operand tile.
    __device__ __forceinline__ void convert(uint32_t tile, int row) const {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {     // 32 numbers: two blocks
            const uint32_t two = e4m3x2_f16(s[i / 2] >> (16 * (i & 1)));
            const __half2 h = *reinterpret_cast<const __half2 *>(&two);
            const __half2 lo = __low2half2(h), hi = __high2half2(h);
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t r[4];
                e2m1x8_f16(x[k], r);
                const __half2 f = k < 2 ? lo : hi;
                st_shared16(chunk_at(tile, row, 4 * i + k), mul2(r[0], f), mul2(r[1], f),
                            mul2(r[2], f), mul2(r[3], f));
            }
        }
    }
};

// One lane of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// The issuing warp of row tile m.  Every lane walks along, so that the descriptors
// stay in uniform registers, and an elected one issues; while one of the two warps
// waits, the other keeps the tensor cores fed (their queue is a few products
// deep).  The loops are kept rolled: a warp runs each instruction once a tile, and
// fetches what is long from far away.
template <int D, typename W>
__device__ __forceinline__ void issue(const AttnArgs &a, const typename W::P &plan, W &w,
                                      long long beg, long long end, uint32_t base, uint32_t tmem,
                                      uint64_t *bar, const Waits &waits, int m) {
    using L = Lay<D>;
    constexpr uint32_t id_qk = idesc_f16(kHalf, false), id_pv = idesc_f16(D, true);
    const uint64_t dQ = make_sdesc(base + L::OFF_Q, 16, 1024, kSwizzle128B) +
                        ((m * L::kOperand) >> 4);
    const uint64_t dK = make_sdesc(base + L::OFF_K, 16, 1024, kSwizzle128B);
    const uint64_t dV = make_sdesc(base + L::OFF_V, 16384, 1024, kSwizzle128B);
    const uint32_t tS = tmem + L::TM_S + 128 * m, tO = tmem + L::TM_O + 128 * m;
    uint32_t n = 0, done = 0, pieces = 0;
    bool alive = true;            // (a lane's: only the elected one's counts)
    // Q K^T with half of the token tile in `buf`; the second half's frees the keys
    auto scores = [&](int half, int buf) {
        if (elect_one()) {
            if (alive) {
#pragma unroll 1
                for (int s = 0; s < D / 64; ++s) {
                    const uint64_t q = dQ + ((s * 16384) >> 4);
                    const uint32_t at = buf * L::kOperand + s * 16384 + half * kHalf * 128;
                    if (!GDN_SMEM_OK(base + L::OFF_K + at, kHalf * 128)) break;
                    const uint64_t k = dK + (at >> 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mma_bf16(tS + kHalf * half, q + 2 * e, k + 2 * e, id_qk, (s | e) != 0);
                }
            }
            mma_commit(bar + B_S_FULL + 2 * m + half);
            if (half == 1) mma_commit(bar + B_K_FREE + buf);
        }
        __syncwarp();
    };
    w.start(a, plan, beg, end);
    do {
        const int count = w.count();
        if (count == 0) continue;
        if (w.rows(a) <= m * kRowTile) {
            // no rows: the tiles go by, in step with the other warp's, once the softmax's warps
            // are done with the last piece that had some
            if (pieces > 0) waits.on_lane(bar + B_SEEN, (pieces - 1) & 1);
#pragma unroll 1
            for (int i = 0; i < count; ++i, ++n) {
                waits.on_lane(bar + B_K_FULL + (n & 1), (n >> 1) & 1);
                waits.on_lane(bar + B_V_FULL + (n & 1), (n >> 1) & 1);
                if (elect_one()) {
                    mbar_arrive(bar + B_K_FREE + (n & 1));
                    mbar_arrive(bar + B_V_FREE + (n & 1));
                }
                __syncwarp();
            }
            continue;
        }
        alive &= waits.on_lane(bar + B_Q_FULL + m, pieces++ & 1);
        alive &= waits.on_lane(bar + B_K_FULL + (n & 1), (n >> 1) & 1);
        tc_fence_after();
        scores(0, n & 1);
        scores(1, n & 1);
#pragma unroll 1
        for (int i = 0; i < count; ++i, ++n, ++done) {
            const int buf = n & 1;
            const bool more = i + 1 < count;
            if (more) alive &= waits.on_lane(bar + B_K_FULL + (buf ^ 1), ((n + 1) >> 1) & 1);
            alive &= waits.on_lane(bar + B_V_FULL + buf, (n >> 1) & 1);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                alive &= waits.on_lane(bar + B_P_FULL + 2 * m + half, done & 1);
                tc_fence_after();
                if (elect_one()) {
                    if (alive) {
                        const uint32_t at = buf * L::kOperand + half * kHalf * 128;
                        const uint64_t v = dV + (at >> 4);
#pragma unroll
                        for (int s = 0; s < kHalf / 16; ++s)
                            if (GDN_SMEM_OK(base + L::OFF_V + at + s * 2048,
                                            (D / 64 - 1) * 16384 + 2048))
                                mma_ts(tO, tS + kHalf * half + 8 * s, v + s * (2048 >> 4), id_pv,
                                       (i | half | s) != 0);
                    }
                    mma_commit(bar + B_O_FULL + 2 * m + half);
                    if (half == 1) mma_commit(bar + B_V_FREE + buf);
                }
                __syncwarp();
                if (more) scores(half, buf ^ 1);
            }
        }
    } while (w.next(a));
    // before tensor memory is given back, whatever happened
    if (elect_one()) mma_commit(bar + B_DRAIN + m);
    __syncwarp();
    mbar_wait(bar + B_DRAIN + m, 0, kDrainLimit);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) k_kv_attn_tc(const AttnArgs a) {
    using L = Lay<D>;
    using W = Walk<kTile, kRows, kThreads>;
    using T = __nv_bfloat16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ typename W::P plan;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    // NaN blocks of V of the last four tiles' tokens, and whether a warp found any.  A tile's
    // are read by a row tile's softmax before its probabilities of the next tile are stored,
    // and the values of the fourth next tile are converted behind the products of the second
    // next.  A piece's last ones are read by row tile 0 before its next piece's first
    // probabilities; row tile 1 may have none in the next pieces, whose tiles then go by only
    // behind B_SEEN.
    __shared__ uint8_t nan_of[4][kTile];
    __shared__ uint32_t nan_any[4][4];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint64_t *bar =
        reinterpret_cast<uint64_t *>(smem_raw + (base - smem_u32(smem_raw)) + L::OFF_BAR);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kIssuer / 32) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            const bool warps = i < B_K_FREE || i == B_V_FULL || i == B_V_FULL + 1 ||
                               i == B_Q_FULL || i == B_Q_FULL + 1 || i == B_SEEN ||
                               (i >= B_P_FULL && i < B_O_FULL);
            const bool free = (i >= B_K_FREE && i < B_V_FULL) || (i >= B_V_FREE && i < B_Q_FULL);
            mbar_init(bar + i, warps ? 4 : free ? 2 : 1);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    plan.build(a);                  // (its barriers cover the initialisation)
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const long long ctas = min((long long)gridDim.x, plan.total);
    if (a.cuts && tid == 0) a.cuts[blockIdx.x].pieces = 0;
    const Waits waits{&abort_flag, a.err, a.wait_limit};
    const long long beg = quot(plan.total * blockIdx.x, max(ctas, 1ll));
    const long long end = quot(plan.total * (blockIdx.x + 1), max(ctas, 1ll));

    if (blockIdx.x < ctas) {
        W w;
        if (tid < kConvert) {
            // ------------------------------------------------------------ softmax
            regs_more<kSoftmaxRegs>();
            const int m = tid >> 7, row = tid & 127;
            const uint32_t lanes = (uint32_t)(row & 96) << 16;       // the warp's TMEM lanes
            const uint32_t tS = tmem + L::TM_S + 128 * m + lanes, tO = tmem + L::TM_O + 128 * m + lanes;
            const uint32_t tile_q = base + L::OFF_Q + m * L::kOperand;
            uint32_t done = 0;           // this row tile's token tiles so far
            uint32_t all = 0;            // the CTA's token tiles so far
            w.start(a, plan, beg, end);
            do {
                const Seq sq = w.sq;
                const int h = w.h, rows = w.rows(a), count = w.count(), place0 = w.place0();
                const int mine = m * kRowTile + row, r = w.row0() + mine;
                bool there = mine < rows;
                const int j = there ? r / a.G : 0, hq = h * a.G + (there ? r - j * a.G : 0);
                if (there) there = a.row_ok((long long)sq.first + j, hq);
                const float gv = a.kv.head_scale ? __ldg(a.kv.head_scale + a.kv.H + h) : 1.f;
                int from = 0, to = sq.len;
                if (there) sq.sees(a, j, from, to);
                float sub = 0.f, sum = 0.f;
                bool started = false;       // whether `sub` is set
                uint32_t nan = 0;           // blocks of d in which the row sees a NaN
                const bool active = m * kRowTile < rows;
                if (active && count > 0) {
                    float mul;
                    {   // the row's queries, into the operand tile
                        const T *p = static_cast<const T *>(a.q) + (sq.first + j) * a.q_tok +
                                     (long long)hq * a.q_head;
                        auto piece = [&](int i) {
                            return there ? __ldg(reinterpret_cast<const uint4 *>(p) + i)
                                         : make_uint4(0, 0, 0, 0);
                        };
                        float most = 0.f;
#pragma unroll 4
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 x = piece(i);
                            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                most = fmaxf(most, fmaxf(fabsf(__uint_as_float(u[e] << 16)),
                                                         fabsf(__uint_as_float(u[e] & 0xffff0000u))));
                        }
                        float down;
                        const float up = row_up(most, down);
                        mul = down * a.scale_log2 *
                              (a.kv.head_scale ? __ldg(a.kv.head_scale + h) : 1.f);
                        // (so that -infinity stays what it is; scores are below 2^40)
                        if (mul == 0.f) mul = 0x1p-126f;
#pragma unroll 4
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 x = piece(i);
                            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = pack_f16(__uint_as_float(u[e] << 16) * up,
                                                __uint_as_float(u[e] & 0xffff0000u) * up);
                            st_shared16(chunk_at(tile_q, row, i), y[0], y[1], y[2], y[3]);
                        }
                    }
                    const uint32_t hidden = __float_as_uint(mul < 0.f ? INFINITY : -INFINITY);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + B_Q_FULL + m);

                    // NaN blocks of V of the piece's tile i, known when a product with it is done
                    auto see_nan = [&](int i) {
                        const uint32_t *any = nan_any[(all + i) & 3];
                        if ((any[0] | any[1] | any[2] | any[3]) == 0) return;
                        const uint8_t *of = nan_of[(all + i) & 3];
                        const int t0 = place0 + i * kTile;
                        for (int e = max(0, from - t0); e < min(kTile, to - t0); ++e) nan |= of[e];
                    };
                    for (int i = 0; i < count; ++i, ++done) {
                        const int t0 = place0 + i * kTile;
                        // (every lane of a warp takes part in what follows, whatever it sees)
                        const bool whole = __all_sync(0xffffffffu, t0 >= from && t0 + kTile <= to);
                        // Half a tile at a time, in columns of its own: while one half's numbers are
                        // formed, the tensor cores finish the other's and score the next tile's.
                        for (int half = 0; half < 2; ++half) {
                            const int h0 = t0 + half * kHalf;       // first place
                            const uint32_t tH = tS + half * kHalf;
                            const bool ok = waits.on(bar + B_S_FULL + 2 * m + half, done & 1);
                            tc_fence_after();
                            if (half == 0 && i > 0) see_nan(i - 1);
                            uint32_t pk[kHalf / 2];
                            float part = 0.f;
                            if (ok) {
                                if (!whole) {
                                    // what the row does not see becomes a score of -infinity
#pragma unroll 1
                                    for (int c = 0; c < kHalf; c += 32) {
                                        uint32_t x[32];
                                        tmem_ld32(tH + c, x);
                                        tmem_wait32(x);
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            if (h0 + c + e < from || h0 + c + e >= to) x[e] = hidden;
                                        tmem_st32(tH + c, x);
                                    }
                                    tmem_st_wait();
                                }
                                // A second pass where `sub` had to move: one copy of this code, as
                                // fetching instructions is what waits otherwise.
#pragma unroll 1
                                for (int pass = 0;; ++pass) {
                                    const uint64_t mul2 = pack64(mul, mul), sub2 = pack64(-sub, -sub);
                                    uint64_t p2[2] = {};
                                    uint32_t x[2][32];
                                    tmem_ld32(tH, x[0]);
                                    tmem_wait32(x[0]);
                                    tmem_ld32(tH + 32, x[1]);
#pragma unroll
                                    for (int c = 0; c < 2; ++c) {
                                        if (c == 1) tmem_wait32(x[1]);
#pragma unroll
                                        for (int e = 0; e < 32; e += 2) {
                                            float t[2];
                                            unpack64(fma_f32x2(pack64(x[c][e], x[c][e + 1]), mul2,
                                                               sub2), t[0], t[1]);
                                            t[0] = ex2(t[0]);
                                            t[1] = ex2(t[1]);
                                            p2[(e >> 1) & 1] =
                                                add_f32x2(p2[(e >> 1) & 1], pack64(t[0], t[1]));
                                            pk[16 * c + e / 2] = pack_f16(t[0], t[1]);
                                        }
                                    }
                                    float y[4];
                                    unpack64(p2[0], y[0], y[1]);
                                    unpack64(p2[1], y[2], y[3]);
                                    part = (y[0] + y[1]) + (y[2] + y[3]);
                                    const bool move = pass == 0 && (!started || part > kMostSum);
                                    if (!__any_sync(0xffffffffu, move)) break;

                                    // the row's maximum of these scores, and `sub` by it
                                    float top = -INFINITY;
#pragma unroll 1
                                    for (int c = 0; c < kHalf; c += 32) {
                                        uint32_t z[32];
                                        tmem_ld32(tH + c, z);
                                        tmem_wait32(z);
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            top = fmaxf(top, __uint_as_float(z[e]) * mul);
                                    }
                                    float f = 1.f;
                                    if (move && top > -INFINITY) {
                                        const float to_new = top - kLift;
                                        if (!started) {
                                            sub = to_new;
                                            started = true;
                                        } else if (to_new > sub) {
                                            f = ex2(sub - to_new);
                                            sub = to_new;
                                        }
                                    }
                                    sum *= f;
                                    if ((i > 0 || half > 0) && __any_sync(0xffffffffu, f != 1.f)) {
                                        // (the half before this one; of tile i - 1 before its first)
                                        waits.on(bar + B_O_FULL + 2 * m + (half ^ 1),
                                                 (done - (half ^ 1)) & 1);
                                        tc_fence_after();
#pragma unroll 1
                                        for (int c = 0; c < D; c += 32) {
                                            uint32_t z[32];
                                            tmem_ld32(tO + c, z);
                                            tmem_wait32(z);
#pragma unroll
                                            for (int e = 0; e < 32; ++e)
                                                z[e] = __float_as_uint(__uint_as_float(z[e]) * f);
                                            tmem_st32(tO + c, z);
                                        }
                                        tmem_st_wait();
                                    }
                                }
                                sum += part;
                                tmem_st32(tH, pk);
                                tmem_st_wait();
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar + B_P_FULL + 2 * m + half);
                        }
                    }
                    waits.on(bar + B_O_FULL + 2 * m + 1, (done - 1) & 1);
                    tc_fence_after();
                    see_nan(count - 1);
                    if (m == 1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar + B_SEEN);
                    }
                }
                all += count;

                // the piece's result
                const bool complete = w.complete();
                const long long slot = 2ll * blockIdx.x + (w.cur == beg ? 0 : 1);
                if (tid == 0 && w.tile0 == 0 && !complete) {
                    const int last = (int)quot((w.cur + w.n_tiles) * ctas - 1, plan.total);
                    a.cuts[blockIdx.x] =
                        Cut{last - (int)blockIdx.x + 1, (int)slot, sq.first, h, w.row0(), rows};
                }
                if (active) {
                    const float scale = complete ? (sum == 0.f ? 0.f : gv / sum) : 1.f;
                    const float lost = started ? sub : -INFINITY;
                    T *po = static_cast<T *>(a.o) + (sq.first + j) * a.o_tok + (long long)hq * a.o_head;
                    float *pp = a.part_o + (slot * kRows + mine) * D;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t x[32];
                        if (count > 0) {
                            tmem_ld32(tO + 32 * c, x);
                            tmem_wait32(x);
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float v[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                v[k] = count > 0 ? __uint_as_float(x[e + k]) * scale : 0.f;
                                if ((nan >> (2 * c + e / 16)) & 1) v[k] = NAN;
                            }
                            if (!there) continue;
                            if (complete) store8(po + 32 * c + e, v);
                            else if (a.part_ok(slot * kRows + mine, kRows))
                                store8(pp + 32 * c + e, v);
                        }
                    }
                    if (there) {
                        if (!complete) {
                            if (a.part_ok(slot * kRows + mine, kRows))
                                a.part_ml[slot * kRows + mine] = make_float2(lost, sum);
                        } else if (a.lse)
                            a.lse[(long long)(sq.first + j) * a.Hq + hq] = lse_of(lost, sum);
                    }
                }
            } while (w.next(a));
        } else if (tid < kIssuer) {
            // --------------------------------------------------------- conversion
            regs_less<kConvertRegs>();
            const int tok = tid - kConvert;
            uint32_t n = 0;               // the CTA's token tiles so far
            w.start(a, plan, beg, end);
            do {
                const int count = w.count(), place0 = w.place0(), len = w.sq.len, h = w.h;
                const int psz = a.kv.page_size();
                auto page_at = [&](int i) {
                    const int at = place0 + i * kTile + tok;
                    return i < count && at < len ? a.kv.page_raw(w.b, at) : Kv::kNoPage;
                };
                Token<D> k, v;
                auto load = [&](Token<D> &x, int i, int raw, bool key) {
                    const int page = a.kv.page_checked(raw, a.err);
                    if (page < 0) {
                        x.clear();
                        return;
                    }
                    const int row = (place0 + i * kTile + tok) & (psz - 1);
                    if (!a.kv.bytes_ok(page, h, v_scale_at(psz, D, row), D / 16)) {
                        x.clear();
                        return;
                    }
                    const uint8_t *blk = a.kv.pages + a.kv.block(page, h);
                    x.load(blk + (key ? k_code_at(psz, D, row) : v_code_at(psz, D, row)),
                           blk + (key ? k_scale_at(psz, D, row) : v_scale_at(psz, D, row)));
                };
                // brings a token of a tile to come into L2: its lines from DRAM would take
                // longer than the conversion of a tile
                auto prefetch = [&](int i, int raw) {
                    if ((unsigned)raw >= (unsigned)a.kv.n_pages) return;
                    const int row = (place0 + i * kTile + tok) & (psz - 1);
                    const uint8_t *blk = a.kv.pages + a.kv.block(raw, h);
                    prefetch_l2(blk + k_code_at(psz, D, row));
                    prefetch_l2(blk + v_code_at(psz, D, row));
                    if ((tok & 15) == 0) {      // (a page has 16 tokens at least)
                        prefetch_l2(blk + k_scale_at(psz, D, row));
                        prefetch_l2(blk + v_scale_at(psz, D, row));
                    }
                };
                int page = page_at(0), next_page = page_at(1), ahead[2] = {page_at(2), page_at(3)};
                prefetch(1, next_page);
                prefetch(2, ahead[0]);
                load(k, 0, page, true);
                load(v, 0, page, false);
                for (int i = 0; i < count; ++i, ++n) {
                    const int buf = n & 1;
                    const uint32_t reuse = ((n >> 1) + 1) & 1;
                    const bool k_ok = n < 2 || waits.on_lane(bar + B_K_FREE + buf, reuse);
                    if (k_ok) k.convert(base + L::OFF_K + buf * L::kOperand, tok);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + B_K_FULL + buf);
                    page = next_page;
                    next_page = ahead[0];
                    ahead[0] = ahead[1];
                    prefetch(i + 3, ahead[0]);
                    ahead[1] = page_at(i + 4);
                    load(k, i + 1, page, true);
                    const bool v_ok = n < 2 || waits.on_lane(bar + B_V_FREE + buf, reuse);
                    const uint32_t bad = v.take_nan();
                    nan_of[n & 3][tok] = (uint8_t)bad;
                    const uint32_t found = __ballot_sync(0xffffffffu, bad != 0);
                    if (lane == 0) nan_any[n & 3][warp & 3] = found;
                    if (v_ok) v.convert(base + L::OFF_V + buf * L::kOperand, tok);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + B_V_FULL + buf);
                    load(v, i + 1, page, false);
                }
            } while (w.next(a));
        } else {
            regs_less<kIssuerRegs>();
            if (warp < kIssuer / 32 + 2)
                issue<D>(a, plan, w, beg, end, base, tmem, bar, waits, warp - kIssuer / 32);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer / 32) tmem_dealloc(tmem, 512);
}

template <int D>
gdn_status launch(AttnArgs &a, cudaStream_t st) {
    auto kern = k_kv_attn_tc<D>;
    static std::atomic<int> memo[kMaxDeviceMemo];
    const int sms = per_device(memo, [&](int dev) {
        int n = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::SIZE) !=
                cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return -1;
        return n;
    }, 0);
    if (sms < 1) return GDN_ERR_CUDA;
    const long long rt = ((long long)a.max_new * a.G + kRows - 1) / kRows;
    long long most = rt * a.kv.H * (a.max_len / kTile + 2);     // of one sequence
    most = most > sms ? sms : most * a.kv.N;
    const int grid = (int)(most < sms ? (most < 1 ? 1 : most) : sms);
    void *scratch = nullptr;
    if (alloc_pieces<D, kRows>(a, grid, &scratch, st) != cudaSuccess) return GDN_ERR_CUDA;
    const int slot = timer_begin(st, "k_kv_attn_tc");
    kern<<<grid, kThreads, Lay<D>::SIZE, st>>>(a);
    timer_end(slot, st);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_join<__nv_bfloat16, D, kRows, 4, 1>(a, grid, st);
    const cudaError_t f = scratch_free(scratch, st);
    if (e == cudaSuccess) e = f;
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

gdn_status attn_many(AttnArgs &a, cudaStream_t st) {
    return a.kv.d == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace kv
}  // namespace gdn
