// gdn_kv_attn.cu -- attention over the 4-bit paged cache for few rows (single
// tokens, drafts, fp32 I/O).
//
// S = Q K^T and O = P V with one pass over the cache, the running maximum and
// sum of the softmax kept per row.  Reading the cache bounds it, and next to
// that the instructions that turn 4-bit numbers into fp16 operands: at 144 bytes
// a (token, head) of d = 128 and 6.8 TB/s an SM has 3 issue slots per element.
//
// - A warp takes 16 tokens at a time, by itself: cp.async into its own ring of
//   kStages groups (all four parts of a group lie contiguous in the page), no
//   barrier between warps until a piece of work ends.
// - Tokens are the M side of the products: S^T[16 x 8] = K[16 x d] Q^T[d x 8],
//   O^T[d x 8] += V^T[d x 16] P^T[16 x 8], so 8 query rows of a key/value head
//   cost one n = 8 tile and a single row no more.
// - The order of the contraction is free, so a lane's operand registers hold
//   the d / 4 neighbours that it reads with one wide load, and the lane's 16
//   d-neighbours of V for 4 tokens.  V's operand wants two TOKENS in a register:
//   nibbles of two tokens are merged before the conversion (4 instructions per
//   16 numbers).  e2m1 -> fp16 is the hardware conversion (64 a clock an SM);
//   times the block's e4m3 scale it is exact in fp16.
// - The running maximum of a row moves only when a score passes it by more than
//   kRaise (log2 units), so the output's registers are seldom rescaled.
//   Probabilities are carried times 2^kLift, which fills fp16's range: at most
//   2^15, and a weight keeps its bits down to 2^-28 of the row's largest (2^-17
//   as two numbers).  Smaller ones are multiplied up into that range and added
//   by a product of their own, so that they count where the largest weights
//   meet zeros.
// - A CTA's tiles are a contiguous share of all tiles (Plan, gdn_kv_attn.cuh);
//   pieces of a cut (sequence, head) go to scratch as fp32 sums and k_kv_join
//   adds them in a fixed order.
#include <cmath>
#include <type_traits>

#include "gdn_kv_attn.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace kv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;                    // tokens of a warp's step
constexpr int kTile = kWarps * kGroup;
constexpr float kRaise = 1.f;                 // log2: when the running maximum moves
constexpr float kLift = 14.f;                 // log2: probabilities at the maximum

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
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

// Place within its group of 16 of S^T's row g (rows g + 8: 8 more).  Rows 2 i and
// 2 i + 1 are places i and 4 + (i ^ 1): the four lanes that share a V operand
// register's tokens then read four neighbouring rows, and the two rows that a
// quarter warp reads of K differ in parity, which keeps its banks apart.
__device__ __forceinline__ int place_of(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1; }

// Probabilities p of S^T's rows g (p[0], p[1]: two columns) and g + 8 as the B
// operand of the second product; kSplit: what hi leaves of them in lo.
template <bool kSplit>
__device__ __forceinline__ void operand_of(const float (&p)[4], uint32_t (&hi)[2],
                                           uint32_t (&lo)[2]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t h = pack_f16(p[2 * e], p[2 * e + 1]);
        hi[e] = transpose8x8(h);
        if constexpr (kSplit) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            lo[e] = transpose8x8(pack_f16(p[2 * e] - x.x, p[2 * e + 1] - x.y));
        }
    }
}

// kSplit: queries and probabilities as two fp16 numbers each (fp32 I/O).
template <int D, int NT, bool kSplit, int kStages>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kGroupBytes = kGroup * D * 9 / 8;
    static constexpr int kRing = kWarps * kStages * kGroupBytes;
    static constexpr int kMerge = kWarps * kRows * D * 4;
    static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
};

// A lane's share of copying groups of one head into the ring: 16 tokens' key
// codes, value codes, key scales and value scales, each contiguous in the page,
// in this order.  Pieces of 16 bytes: kCode of key codes, as many of value
// codes, then D / 8 of scales.
template <int D>
struct Loader {
    static constexpr int kCode = D / 2, kScale = D / 16;
    const uint8_t *code, *scale;   // of page 0, row 0
    uint32_t page_bytes, v_code;
    bool scales;                   // whether this lane copies scales

    __device__ __forceinline__ void init(const Kv &kv, int h, int lane) {
        const int psz = kv.page_size();
        page_bytes = kv.H * block_bytes(psz, D);
        const uint8_t *blk = kv.pages + (long long)h * block_bytes(psz, D);
        code = blk + 16 * lane;
        v_code = psz * (D / 2);
        scales = lane < 2 * kScale;
        scale = blk + (lane < kScale ? k_scale_at(psz, D, 0) + 16 * lane
                                     : v_scale_at(psz, D, 0) + 16 * (lane - kScale));
    }
    __device__ __forceinline__ void copy(uint32_t dst, int page, int row, int lane) const {
        const uint8_t *c = code + (uint64_t)page * page_bytes + (uint32_t)(row * (D / 2));
        const uint8_t *v = c + v_code;
        const uint32_t d = dst + 16 * lane;
        if constexpr (D == 64) {
            cp_async16(d, c);
            cp_async16(d + 16 * kCode, v);
        } else {
#pragma unroll
            for (int i = 0; i < kCode / 32; ++i) {
                cp_async16(d + 512 * i, c + 512 * i);
                cp_async16(d + 16 * kCode + 512 * i, v + 512 * i);
            }
        }
        if (scales)
            cp_async16(d + 32 * kCode,
                       scale + (uint64_t)page * page_bytes + (uint32_t)(row * (D / 16)));
    }
};

template <typename T>
__device__ __forceinline__ void store4(T *p, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d) {
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
template <>
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(a, b), pack2(c, d));
}

template <typename T, int D, int NT, bool kSplit, int kStages, int kMinCtas>
__global__ void __launch_bounds__(kThreads, kMinCtas) k_kv_attn(const AttnArgs a) {
    using Sh = Shape<D, NT, kSplit, kStages>;
    using P = Plan<kTile, Sh::kRows, kThreads>;
    constexpr int kW = D / 32;      // 32-bit words of a lane's share of a K row
    constexpr int kV = D / 64;      // of a V row
    constexpr int kT = D / 16;      // m tiles of O^T = k steps of S^T
    constexpr int kParts = kSplit ? 2 : 1;
    // Least probability (lifted) whose fp16 parts keep all their bits, how far the
    // lifted maximum lies above it, and that range's middle and half in log2 units.
    constexpr float kLow = kSplit ? 0x1p-3f : 0x1p-14f, kBand = kSplit ? 0x1p18f : 0x1p29f;
    constexpr float kMid = kSplit ? 6.f : 0.5f, kHalf = kLift + kRaise - kMid;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ P plan;
    __shared__ float2 warp_ml[kWarps][Sh::kRows];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    plan.build(a);
    const long long ctas = min((long long)gridDim.x, plan.total);
    if (a.cuts && threadIdx.x == 0) a.cuts[blockIdx.x].pieces = 0;
    if (blockIdx.x >= ctas) return;
    const long long beg = plan.total * blockIdx.x / ctas, end = plan.total * (blockIdx.x + 1) / ctas;
    const uint32_t my_ring =
        static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * kStages * Sh::kGroupBytes;
    const uint8_t *my_buf = ring + warp * kStages * Sh::kGroupBytes;

    int b;
    long long seq_start;
    Seq sq;
    plan.find(a, beg, b, seq_start, sq);
    for (long long cur = beg; cur < end;) {
        int n_tiles = P::tiles(sq), n_rt = P::row_tiles(a, sq);
        while (cur >= seq_start + (long long)n_rt * a.kv.H * n_tiles) {
            seq_start += (long long)n_rt * a.kv.H * n_tiles;
            sq.get(a, ++b);
            n_tiles = P::tiles(sq);
            n_rt = P::row_tiles(a, sq);
        }
        const long long within = cur - seq_start;
        const int seg = (int)(within / n_tiles), tile0 = (int)(within - (long long)seg * n_tiles);
        const int tile1 = (int)min((long long)n_tiles, tile0 + (end - cur));
        const int h = seg / n_rt, row0 = (seg - h * n_rt) * Sh::kRows;
        const int rows = min(Sh::kRows, sq.n * a.G - row0);

        // groups of this piece, and this warp's among them
        const int n_groups = (sq.span + kGroup - 1) / kGroup;
        const int grp0 = tile0 * kWarps + warp, grp1 = min(tile1 * kWarps, n_groups);
        const int steps = grp1 > grp0 ? (grp1 - grp0 + kWarps - 1) / kWarps : 0;
        // page of the warp's step i: held by lane i % 32 of `pages`, the next 32 in `ahead`
        auto fetch = [&](int i) {
            const int grp = grp0 + (i + lane) * kWarps;
            return i + lane < steps ? a.kv.page_of(b, sq.lo + grp * kGroup, a.err) : -1;
        };
        int pages = fetch(0), ahead = steps > 32 ? fetch(32) : -1;
        Loader<D> loader;
        loader.init(a.kv, h, lane);
        uint32_t fill = my_ring;
        auto issue = [&](int i) {   // whole warp, i in order
            if (i < steps) {
                if ((i & 31) == 0 && i > 0) {
                    pages = ahead;
                    if (i + 32 < steps) ahead = fetch(i + 32);
                }
                const int page = __shfl_sync(0xffffffffu, pages, i & 31);
                const int at = sq.lo + (grp0 + i * kWarps) * kGroup;
                if (page >= 0) loader.copy(fill, page, at & (a.kv.page_size() - 1), lane);
                fill = fill == my_ring + (kStages - 1) * Sh::kGroupBytes ? my_ring
                                                                         : fill + Sh::kGroupBytes;
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(i);

        // queries: lane's part of row 8 nt + g, as the B operand, scaled by a power
        // of two that brings the row's largest number to [2^13, 2^14)
        const float gk = a.kv.head_scale ? __ldg(a.kv.head_scale + h) : 1.f;
        const float gv = a.kv.head_scale ? __ldg(a.kv.head_scale + a.kv.H + h) : 1.f;
        uint32_t qf[kParts][NT][kT][2];
        float mul[NT][2];
        int from[NT][2], to[NT][2];
        int all_from = 0, all_to = 0x7fffffff;     // places that every row sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + 8 * nt + g;
            const bool there = 8 * nt + g < rows;
            const int j = there ? r / a.G : 0;
            const T *p = static_cast<const T *>(a.q) + (sq.first + j) * a.q_tok +
                         (long long)(h * a.G + (there ? r - j * a.G : 0)) * a.q_head + t4 * (D / 4);
            float x[D / 4];
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                float v[8];
                if (there) load8(p + 8 * i, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[8 * i + e] = there ? v[e] : 0.f;
                    m = fmaxf(m, fabsf(x[8 * i + e]));
                }
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t ex = max(27u, __float_as_uint(m) >> 23);
            const float up = __uint_as_float((267u - ex) << 23);
            const float down = __uint_as_float((ex - 13u) << 23) * a.scale_log2 * gk;
#pragma unroll
            for (int s = 0; s < kT; ++s) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float u = x[4 * s + 2 * e] * up, w = x[4 * s + 2 * e + 1] * up;
                    qf[0][nt][s][e] = pack_f16(u, w);
                    if constexpr (kSplit) {
                        const float2 hi =
                            __half22float2(*reinterpret_cast<const __half2 *>(&qf[0][nt][s][e]));
                        qf[1][nt][s][e] = pack_f16(u - hi.x, w - hi.y);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mul[nt][e] = __shfl_sync(0xffffffffu, down, 4 * (2 * t4 + e));
                const int rr = 8 * nt + 2 * t4 + e;
                from[nt][e] = 0;
                to[nt][e] = sq.len;
                if (rr < rows) sq.sees(a, (row0 + rr) / a.G, from[nt][e], to[nt][e]);
                all_from = max(all_from, from[nt][e]);
                all_to = min(all_to, to[nt][e]);
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            all_from = max(all_from, __shfl_xor_sync(0xffffffffu, all_from, o));
            all_to = min(all_to, __shfl_xor_sync(0xffffffffu, all_to, o));
        }

        float o[NT][kT][4], sub[NT][2], sum[NT][2];   // sub: what scores lose before ex2
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < kT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sub[nt][e] = -INFINITY;
                sum[nt][e] = 0.f;
            }
        }

        const uint8_t *buf = my_buf + (kStages - 1) * Sh::kGroupBytes;
        int t0 = sq.lo + (grp0 - kWarps) * kGroup;
        for (int i = 0; i < steps; ++i) {
            cp_wait<kStages - 2>();
            __syncwarp();
            issue(i + kStages - 1);
            buf = buf == my_buf + (kStages - 1) * Sh::kGroupBytes ? my_buf : buf + Sh::kGroupBytes;
            t0 += kTile;
            const bool whole = t0 >= all_from && t0 + kGroup <= all_to;

            // S^T
            float s[NT][4];
            {
                uint32_t kw[2][kW];
                __half2 ks[2][kW / 2];      // scale of each block, twice
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = place_of(g) + 8 * r;
                    const uint8_t *p = buf + row * (D / 2) + t4 * (D / 8);
                    const uint8_t *sp = buf + 16 * D + row * (D / 16) + t4 * (D / 64);
                    if constexpr (D == 64) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(p);
                        kw[r][0] = w.x; kw[r][1] = w.y;
                        const uint32_t one = e4m3x2_f16(*sp);
                        ks[r][0] = __low2half2(*reinterpret_cast<const __half2 *>(&one));
                    } else {
#pragma unroll
                        for (int w4 = 0; w4 < kW / 4; ++w4) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(p + 16 * w4);
                            kw[r][4 * w4] = w.x; kw[r][4 * w4 + 1] = w.y;
                            kw[r][4 * w4 + 2] = w.z; kw[r][4 * w4 + 3] = w.w;
                            const uint32_t two = e4m3x2_f16(
                                *reinterpret_cast<const uint16_t *>(sp + 2 * w4));
                            ks[r][2 * w4] =
                                __low2half2(*reinterpret_cast<const __half2 *>(&two));
                            ks[r][2 * w4 + 1] =
                                __high2half2(*reinterpret_cast<const __half2 *>(&two));
                        }
                    }
                }
                float s2[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
                for (int w = 0; w < kW; ++w) {
                    uint32_t r0[4], r1[4];
                    e2m1x8_f16(kw[0][w], r0);
                    e2m1x8_f16(kw[1][w], r1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        r0[e] = mul2(r0[e], ks[0][w / 2]);
                        r1[e] = mul2(r1[e], ks[1][w / 2]);
                    }
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816(s[nt], r0[0], r1[0], r0[1], r1[1], qf[part][nt][2 * w][0],
                                     qf[part][nt][2 * w][1]);
                            mma16816(s2[nt], r0[2], r1[2], r0[3], r1[3], qf[part][nt][2 * w + 1][0],
                                     qf[part][nt][2 * w + 1][1]);
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];
            }

            // Scores in log2 units less the row's `sub`, so that the row's largest number
            // is about kLift.  One comparison finds those that call for more: above
            // kLift + kRaise the maximum moves; below kLow probabilities lose bits.
            float t[NT][4], rest[NT][4];
            bool more = false, low = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t[nt][e] = fmaf(s[nt][e], mul[nt][e & 1], -sub[nt][e & 1]);
                    if (!whole) {
                        const int at = t0 + place_of(g) + 8 * (e >> 1);
                        if (at < from[nt][e & 1] || at >= to[nt][e & 1]) t[nt][e] = -INFINITY;
                    }
                    more = more || fabsf(t[nt][e] - kMid) > kHalf;
                }
            }
            const bool extra = __any_sync(0xffffffffu, more);
            if (extra) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // (an infinite t: the row's first score; its own score decides then)
                        float y[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const bool out = t[nt][e + 2 * k] == -INFINITY;
                            y[k] = out ? -INFINITY : s[nt][e + 2 * k] * mul[nt][e];
                        }
                        float m = fmaxf(y[0], y[1]);
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m -= kLift;
                        if (m > sub[nt][e] + kRaise) {
                            const float f = ex2(sub[nt][e] - m);
                            sub[nt][e] = m;
                            sum[nt][e] *= f;
#pragma unroll
                            for (int k = 0; k < kT; ++k) {
                                o[nt][k][e] *= f;
                                o[nt][k][e + 2] *= f;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (t[nt][e + 2 * k] != -INFINITY)
                                t[nt][e + 2 * k] =
                                    fmaf(s[nt][e + 2 * k], mul[nt][e], -sub[nt][e]);
                    }
            }
            uint32_t pf[kParts][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(t[nt][e]);
                    sum[nt][e & 1] += p[e];
                }
                if (extra) {      // the small ones later, in a product of their own
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        rest[nt][e] = 0.f;
                        if (p[e] < kLow) {
                            rest[nt][e] = p[e];
                            p[e] = 0.f;
                        }
                        low = low || rest[nt][e] > 0.f;
                    }
                }
                operand_of<kSplit>(p, pf[0][nt], pf[kParts - 1][nt]);
            }

            // O^T
            uint32_t vw[4][kV], vs[4];       // lane's tokens t4, 4 + (t4 ^ 1), 8 more each
            constexpr int kBlocks = D == 256 ? 2 : 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 4 * j + ((j & 1) ? t4 ^ 1 : t4);
                const uint8_t *p = buf + 8 * D + row * (D / 2) + g * (D / 16);
                const uint8_t *sp = buf + 17 * D + row * (D / 16) + g * D / 128;
                if constexpr (D == 64) {
                    vw[j][0] = *reinterpret_cast<const uint32_t *>(p);
                    vs[j] = *sp;
                } else if constexpr (D == 128) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(p);
                    vw[j][0] = w.x; vw[j][1] = w.y;
                    vs[j] = *sp;
                } else {
                    const uint4 w = *reinterpret_cast<const uint4 *>(p);
                    vw[j][0] = w.x; vw[j][1] = w.y; vw[j][2] = w.z; vw[j][3] = w.w;
                    vs[j] = *reinterpret_cast<const uint16_t *>(sp);
                }
            }
            if (!whole) {
                // Places behind the sequence's end (or before what any row sees) may hold
                // anything: their scales become 0.  A NaN that some rows see and others do
                // not would reach all of them through 0 * NaN: it is taken out of the
                // product and put into the rows that see it.
                uint32_t nan[kBlocks] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int off = 4 * j + ((j & 1) ? t4 ^ 1 : t4);
                    if (t0 + off >= sq.len) vs[j] = 0;
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k)
                        if (((vs[j] >> (8 * k)) & 0x7f) == 0x7f) {
                            nan[k] |= 1u << off;
                            vs[j] &= ~(0xffu << (8 * k));
                        }
                }
                bool any = false;
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) any = any || nan[k];
                if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k) {
                        nan[k] |= __shfl_xor_sync(0xffffffffu, nan[k], 1);
                        nan[k] |= __shfl_xor_sync(0xffffffffu, nan[k], 2);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int lo = min(16, max(0, from[nt][e] - t0));
                                const int hi = min(16, max(0, to[nt][e] - t0));
                                const uint32_t seen = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
                                if (nan[k] & seen) {
#pragma unroll
                                    for (int m = 0; m < kT / kBlocks; ++m) {
                                        o[nt][k * (kT / kBlocks) + m][e] = NAN;
                                        o[nt][k * (kT / kBlocks) + m][e + 2] = NAN;
                                    }
                                }
                            }
                    }
                }
            }
            uint32_t sc[kBlocks][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t x = vs[2 * e], y = vs[2 * e + 1];
                sc[0][e] = e4m3x2_f16(__byte_perm(x, y, 0x0040));
                if constexpr (kBlocks == 2) sc[kBlocks - 1][e] = e4m3x2_f16(__byte_perm(x, y, 0x0051));
            }
            // O^T += V^T P^T, or O^T += factor * (V^T P^T)
            auto product = [&](auto plain, float factor) {
#pragma unroll
                for (int w = 0; w < kV; ++w) {
                    constexpr uint32_t kEven = 0x0f0f0f0fu;
                    uint32_t e1[4], d1[4], e2[4], d2[4];   // even and odd elements of the two pairs
                    e2m1x8_f16((vw[0][w] & kEven) | ((vw[1][w] << 4) & ~kEven), e1);
                    e2m1x8_f16(((vw[0][w] >> 4) & kEven) | (vw[1][w] & ~kEven), d1);
                    e2m1x8_f16((vw[2][w] & kEven) | ((vw[3][w] << 4) & ~kEven), e2);
                    e2m1x8_f16(((vw[2][w] >> 4) & kEven) | (vw[3][w] & ~kEven), d2);
                    const __half2 s1 = *reinterpret_cast<const __half2 *>(&sc[w / 2 % kBlocks][0]);
                    const __half2 s2 = *reinterpret_cast<const __half2 *>(&sc[w / 2 % kBlocks][1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t a0 = mul2(e1[k], s1), a1 = mul2(d1[k], s1);
                        const uint32_t a2 = mul2(e2[k], s2), a3 = mul2(d2[k], s2);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float (&acc)[4] = o[nt][4 * w + k];
                            if constexpr (plain.value) {
#pragma unroll
                                for (int part = 0; part < kParts; ++part)
                                    mma16816(acc, a0, a1, a2, a3, pf[part][nt][0], pf[part][nt][1]);
                            } else {
                                float x[4] = {};
#pragma unroll
                                for (int part = 0; part < kParts; ++part)
                                    mma16816(x, a0, a1, a2, a3, pf[part][nt][0], pf[part][nt][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[e], factor, acc[e]);
                            }
                        }
                    }
                }
            };
            product(std::true_type{}, 1.f);
            if (extra && __any_sync(0xffffffffu, low)) {
                // what lies a factor kBand below the last product's range, until nothing is left
                float factor = 1.f;
                do {
                    factor *= 1.f / kBand;
                    low = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            rest[nt][e] *= kBand;
                            p[e] = rest[nt][e] >= kLow ? rest[nt][e] : 0.f;
                            if (p[e] > 0.f) rest[nt][e] = 0.f;
                            low = low || rest[nt][e] > 0.f;
                        }
                        operand_of<kSplit>(p, pf[0][nt], pf[kParts - 1][nt]);
                    }
                    product(std::false_type{}, factor);
                } while (__any_sync(0xffffffffu, low));
            }
        }
        cp_wait<0>();

        // the warps' sums of this piece
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = sum[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                sum[nt][e] = x;
                if (g == 0) warp_ml[warp][8 * nt + 2 * t4 + e] = make_float2(sub[nt][e], x);
            }
        __syncthreads();      // every warp is done with its ring as well
        float *merge = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * t4 + e;
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_ml[w][r].x);
                const float f = m == -INFINITY ? 1.f : ex2(sub[nt][e] - m);
                float *p = merge + (warp * Sh::kRows + r) * D + g * (D / 8);
#pragma unroll
                for (int k = 0; k < kT; ++k)
                    *reinterpret_cast<float2 *>(p + 2 * k) =
                        make_float2(o[nt][k][e] * f, o[nt][k][e + 2] * f);
            }
        __syncthreads();
        const bool complete = tile0 == 0 && tile1 == n_tiles;
        const long long slot = 2ll * blockIdx.x + (cur == beg ? 0 : 1);
        if (threadIdx.x == 0 && tile0 == 0 && !complete) {
            const long long end_tile = cur + n_tiles;    // CTA of its last tile: below
            const int last = (int)((end_tile * ctas - 1) / plan.total);
            a.cuts[blockIdx.x] = Cut{last - (int)blockIdx.x + 1, (int)slot, sq.first, h, row0, rows};
        }
        for (int x = threadIdx.x; x < rows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = 4 * (x - r * (D / 4));
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_ml[w][r].x);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = warp_ml[w][r];
                l += ml.y * (m == -INFINITY ? 1.f : ex2(ml.x - m));
                const float4 y =
                    *reinterpret_cast<const float4 *>(merge + (w * Sh::kRows + r) * D + d);
                v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
            }
            if (complete) {
                const int rr = row0 + r, j = rr / a.G, hq = h * a.G + rr - j * a.G;
                const float inv = l == 0.f ? 0.f : gv / l;
                T *p = static_cast<T *>(a.o) + (sq.first + j) * a.o_tok + hq * a.o_head + d;
                store4(p, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                if (a.lse && d == 0)
                    a.lse[(long long)(sq.first + j) * a.Hq + hq] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            } else {
                store4(a.part_o + (slot * Sh::kRows + r) * D + d, v.x, v.y, v.z, v.w);
                if (d == 0) a.part_ml[slot * Sh::kRows + r] = make_float2(m, l);
            }
        }
        __syncthreads();
        cur += tile1 - tile0;
    }
}

// Adds the pieces of what was cut, in order: CTA (i, r) row r of the one whose
// first piece CTA i of k_kv_attn had.
constexpr int kJoinWarps = 4;
template <typename T, int D, int kRows>
__global__ void __launch_bounds__(kJoinWarps * 32) k_kv_join(const AttnArgs a) {
    constexpr int kVec = D / 32;
    __shared__ float sums[kJoinWarps][D];
    __shared__ float2 warp_ml[kJoinWarps];
    ptx::griddep_wait();
    const Cut c = a.cuts[blockIdx.x];
    const int r = blockIdx.y;
    if (r >= c.rows || c.pieces == 0) return;
    auto slot = [&](int k) {
        return (k == 0 ? (long long)c.slot0 : 2ll * (blockIdx.x + k)) * kRows + r;
    };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY;
    for (int k = threadIdx.x; k < c.pieces; k += kJoinWarps * 32) m = fmaxf(m, a.part_ml[slot(k)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) warp_ml[warp].x = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, warp_ml[w].x);
    float v[kVec] = {}, l = 0.f;
#pragma unroll 4
    for (int k = warp; k < c.pieces; k += kJoinWarps) {
        const float2 ml = a.part_ml[slot(k)];
        const float f = m == -INFINITY ? 1.f : ex2(ml.x - m);
        const float *p = a.part_o + slot(k) * D + lane * kVec;
        l += ml.y * f;
        if constexpr (kVec == 2) {
            const float2 x = *reinterpret_cast<const float2 *>(p);
            v[0] += x.x * f; v[1] += x.y * f;
        } else {
#pragma unroll
            for (int e = 0; e < kVec; e += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(p + e);
                v[e] += x.x * f; v[e + 1] += x.y * f; v[e + 2] += x.z * f; v[e + 3] += x.w * f;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sums[warp][lane * kVec + e] = v[e];
    if (lane == 0) warp_ml[warp].y = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += warp_ml[w].y;
    const int rr = c.row0 + r, j = rr / a.G, hq = c.h * a.G + rr - j * a.G;
    const float gv = a.kv.head_scale ? __ldg(a.kv.head_scale + a.kv.H + c.h) : 1.f;
    const float inv = l == 0.f ? 0.f : gv / l;
    T *p = static_cast<T *>(a.o) + (c.first + j) * a.o_tok + hq * a.o_head;
    for (int d = 4 * threadIdx.x; d < D; d += 4 * kJoinWarps * 32) {
        float x[4] = {};
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += sums[w][d + e];
        store4(p + d, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(long long)(c.first + j) * a.Hq + hq] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <typename T, int D, int NT, bool kSplit, int kStages, int kMinCtas>
gdn_status launch(AttnArgs &a, cudaStream_t st) {
    using Sh = Shape<D, NT, kSplit, kStages>;
    auto kern = k_kv_attn<T, D, NT, kSplit, kStages, kMinCtas>;
    static std::atomic<int> memo[kMaxDeviceMemo];
    // resident CTAs of the device, and the opt-in to the ring's shared memory
    const int resident = per_device(memo, [&](int dev) {
        int sms = 0, per = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) !=
                cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kThreads, Sh::kSmem) !=
                cudaSuccess)
            return -1;
        return sms * per;
    }, 0);
    if (resident < 1) return GDN_ERR_CUDA;
    const long long rt = ((long long)a.max_new * a.G + Sh::kRows - 1) / Sh::kRows;
    const long long tiles = a.max_len / kTile + 1;
    long long most = rt * a.kv.H * tiles;   // of one sequence; of all, without overflow:
    most = most > resident ? resident : most * a.kv.N;
    const int grid = (int)(most < resident ? (most < 1 ? 1 : most) : resident);
    const bool cut = a.max_len > kTile;     // else no piece of work has two tiles
    void *scratch = nullptr;
    const size_t po = (size_t)2 * grid * Sh::kRows * D * 4, pm = (size_t)2 * grid * Sh::kRows * 8;
    if (cut) {
        if (scratch_alloc(&scratch, po + pm + grid * sizeof(Cut), st) != cudaSuccess)
            return GDN_ERR_CUDA;
        a.part_o = static_cast<float *>(scratch);
        a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(scratch) + po);
        a.cuts = reinterpret_cast<Cut *>(static_cast<uint8_t *>(scratch) + po + pm);
    }
    const int slot = timer_begin(st, "k_kv_attn");
    kern<<<grid, kThreads, Sh::kSmem, st>>>(a);
    timer_end(slot, st);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (cut) {
        if (e == cudaSuccess && grid > 1 && a.max_new > 0) {
            // launched while k_kv_attn runs: it waits for that to end before it reads
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr.val.programmaticStreamSerializationAllowed = 1;
            cudaLaunchConfig_t cfg{};
            const long long rows = (long long)a.max_new * a.G;
            cfg.gridDim = dim3(grid, (unsigned)(rows < Sh::kRows ? rows : Sh::kRows));
            cfg.blockDim = dim3(kJoinWarps * 32);
            cfg.stream = st;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaLaunchKernelEx(&cfg, k_kv_join<T, D, Sh::kRows>, (const AttnArgs)a);
            count_launch();
        }
        const cudaError_t f = scratch_free(scratch, st);
        if (e == cudaSuccess) e = f;
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, bool kSplit>
gdn_status pick(AttnArgs &a, cudaStream_t st) {
    switch (a.kv.d) {
        case 64: return launch<T, 64, 1, kSplit, 4, kSplit ? 1 : 2>(a, st);
        case 128: return launch<T, 128, 1, kSplit, 4, kSplit ? 1 : 2>(a, st);
        default: return launch<T, 256, 1, kSplit, 3, 1>(a, st);
    }
}

}  // namespace
}  // namespace kv
}  // namespace gdn

extern "C" gdn_status gdn_kv_attn(const gdn_kv *kv, const gdn_rows *q, const gdn_rows *o,
                                  float *lse, int max_len, int max_new, float scale, int window,
                                  unsigned flags, gdn_dtype dt, void *stream) {
    using namespace gdn::kv;
    if (!kv || kv->N < 0 || kv->n_tokens < 0 || max_len < 0 || max_new < 0 || window < 0)
        return GDN_ERR_INVALID_ARG;
    if (flags & ~(unsigned)GDN_ATTN_CAUSAL) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (kv->n_tokens == 0) return GDN_OK;
    if (kv->N == 0) return GDN_ERR_INVALID_ARG;
    AttnArgs a{};
    gdn_status rc = check_kv(kv, &a.kv);
    if (rc != GDN_OK) return rc;
    if ((rc = check_rows(q, dt)) != GDN_OK || (rc = check_rows(o, dt)) != GDN_OK) return rc;
    if (q->heads != o->heads || q->heads % kv->heads) return GDN_ERR_INVALID_ARG;
    if (!aligned4(lse)) return GDN_ERR_ALIGNMENT;
    if ((long long)kv->n_tokens * q->heads > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    const long long cap = (long long)kv->max_pages * kv->page_size;
    a.q = q->data;
    a.o = o->data;
    a.lse = lse;
    a.q_head = q->stride_head;
    a.q_tok = q->stride_tok;
    a.o_head = o->stride_head;
    a.o_tok = o->stride_tok;
    a.Hq = q->heads;
    a.G = q->heads / kv->heads;
    a.max_len = (int)(max_len < cap ? max_len : cap);
    a.max_new = max_new < kv->n_tokens ? max_new : kv->n_tokens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.window = window;
    a.causal = (flags & GDN_ATTN_CAUSAL) != 0;
    a.err = gdn::device_error_word();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == GDN_BF16 ? pick<__nv_bfloat16, false>(a, st) : pick<float, true>(a, st);
}
