// gdn_kv_attn.cu -- attention over the paged cache, in 4 or 8 bits, for few rows (single
// tokens, drafts, fp32 I/O).
//
// S = Q K^T and O = P V with one pass over the cache, the running maximum and
// sum of the softmax kept per row.  Its floor is reading the cache, and next to
// that stand the instructions that turn 4-bit numbers into fp16 operands: at 144
// bytes a (token, head) of d = 128 and 6.8 TB/s an SM has 3 issue slots per element.
//
// - A tile (256 tokens; 128 at d = 256) is copied into a ring of shared memory by
//   bulk copies, one per page and part of it, each warp issuing every eighth
//   tile's; a warp takes its 16 or 32 tokens of every tile, and no barrier joins
//   the warps until a piece of work ends.  The next piece's first tile is copied
//   with the last tile of the piece before it, and its queries and the place of
//   the piece after it are found while that one's sums are merged (64 ragged
//   sequences below: 178 us without either, 165 without the second).
// - Tokens are the M side of the products: S^T[16 x 8] = K[16 x d] Q^T[d x 8],
//   O^T[d x 8] += V^T[d x 16] P^T[16 x 8], so 8 query rows of a key/value head
//   cost one n = 8 tile and a single row no more.
// - The order of the contraction is free, so a lane's operand registers hold
//   the d / 4 neighbours that it reads with one wide load, and the lane's 16
//   d-neighbours of V for 4 tokens.  V's operand wants two TOKENS in a register:
//   nibbles of two tokens are merged before the conversion (4 instructions per
//   16 numbers).  e2m1 -> fp16 is the hardware conversion (64 a clock an SM);
//   times the block's e4m3 scale it is exact in fp16.
// - Rows are scaled by a power of two and rounded to fp16 (fp32 rows to two fp16
//   numbers, 22 bits).  bf16 rows keep all their 8 bits.
// - The running maximum of a row moves only when a score passes it by more than
//   kRaise (log2 units), so the output's registers are seldom rescaled.
//   Probabilities are rounded to fp16, the products' type, times 2^kLift, which
//   fills that type's range: at most 2^15, and a weight keeps its bits down to
//   2^-28 of the row's largest (2^-17 as two numbers).  Smaller ones are
//   multiplied up into that range and added by a product of their own, so that
//   they count where the largest weights meet zeros.  Sums are fp32.
// - A CTA's tiles are a contiguous share of all tiles (Plan, gdn_kv_attn.cuh);
//   pieces of a cut (sequence, head) go to scratch as fp32 sums and k_kv_join
//   adds them in a fixed order.
//
// Measured, join included (bf16, d = 128, one token a sequence, pages read cold):
//   256 sequences of 8000 to 8192, 8 heads:    464 us, 5.1 TB/s (2.39 GB);
//   64 ragged ones of 128 to 16384, 8 heads:   163 us, 4.1 TB/s (665 MB);
//   one of 131072, 4 heads:                     33 us, 2.3 TB/s (75 MB).
// No unit is full in the first two: issue slots 66 and 63 % (about 340 instructions per
// 16 tokens and warp), DRAM 5.2 and 4.3 TB/s without the join, 77 and 63 % of a copy's.
// Registers and the ring allow 16 warps an SM, and of the 6 cycles between two
// instructions of a warp 1.4 go by for the fixed latency of the one before, 1.0 for other
// warps' turns and 0.65 for a pipe.  The last one's first copy starts 5 us in: the
// division of the work 2, its place in it 2, the page numbers 1; the join takes 5.
//
// In 8 bits (Fmt8) the same kernel reads e4m3 codes: a warp's 16 tokens are one block, so
// its keys' exponent is a factor of the scores, and its values' one of the converted numbers
// (exact in fp16).  Two tokens' bytes are put side by side before the conversion (one
// instruction per 2 numbers).  Above 8 rows a piece has two or three n = 8 tiles, which share
// the conversion (eights_of).  It reads twice the bytes with hardly more instructions, and
// DRAM bounds it:
//   256 sequences of 8000 to 8192, 8 heads:    646 us, 6.6 TB/s (4.25 GB);
//   64 ragged ones of 128 to 16384, 8 heads:   196 us, 6.0 TB/s (1.18 GB; 189 without the
//                                              join: 6.3 TB/s, issue slots 43 %);
//   one of 131072, 4 heads:                     40 us, 3.3 TB/s (134 MB).
#include "gdn_kv_attn.cuh"

namespace gdn {
namespace kv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;                    // tokens of a warp's step
// Rows of a key/value head above which the products go to tcgen05 (gdn_kv_attn_tc.cu),
// whose time hardly depends on them up to 128: 20 rows of 64 ragged sequences take 447 us
// there and 474 in three passes of 8 rows here, 16 sequences in a window of 4096 places 34
// and 42; up to 16 rows take 329 here.  (Some hundred places, which the rule does not look
// at: 16 sequences of 200 to 800 take 25 and 26 us, 64 of 128 to 512 take 82 there and 63
// here.)  In 8 bits, up to 24 rows at once, 32 rows of the 64 ragged ones take 532 us here
// and 517 there (at d = 64 295 and 395), of 64 of 128 to 512 places 74 and 103, in the window
// of 4096 places 52 both; 40 rows 699 and 518 (421 and 396), 88 and 105, 65 and 53.
constexpr int kMany4 = 16, kMany8 = 32;
constexpr int kQueryWarp = 4, kWalkWarp = 5;  // (the first tile is copied by warp 0)
// Which eight rows each warp brings the queries of, a hexadecimal digit a warp from the right: warps
// 4, 6 and 7 in turn.
constexpr uint32_t kQueryTurn = 0x21f0ffffu;
// 8 bits: what the end of a piece is counted as.  64 ragged sequences of 128 to 16384 take 198 us,
// uncounted 219 and as one tile 204, 128 of up to 8192 190 (212, 203), at d = 256 230 (291, 271);
// as six tiles they take 198, 193 and 230.
constexpr int kEndTiles = 3;
constexpr float kRaise = 1.f;                 // log2: when the running maximum moves
constexpr float kLift = 14.f;                 // log2: probabilities at the maximum

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Bits of a where `mask` is set, of b elsewhere.
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t mask) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(a), "r"(b), "r"(mask));
    return r;
}
// Place within its group of 16 of S^T's row g (rows g + 8: 8 more).  Rows 2 i and
// 2 i + 1 are places i and 4 + (i ^ 1): the four lanes that share a V operand
// register's tokens then read four neighbouring rows, and the two rows that a
// quarter warp reads of K differ in parity, which keeps its banks apart.
__device__ __forceinline__ int place_of(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1; }

// The row of K that S^T's row g is.
template <typename F>
__device__ __forceinline__ int row_of_place(int g) {
    return F::kBits == 4 ? place_of(g) : g;
}

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
// kU: groups of a warp in a tile.  Two groups and three stages leave room for two
// CTAs an SM (bf16, d <= 128); two stages took 522 us where three took 462.
// kN: rows of a piece, in eights (8 bits: up to three, which share a token's conversion).
template <typename F, int D, bool kSplit, int kN, int kU, int kStages>
struct Shape {
    static constexpr int kTile = kWarps * kU * kGroup;
    static constexpr int kRows = 8 * kN;
    static constexpr int kParts = kSplit ? 2 : 1;
    // a stage: key codes, value codes, key scales, value scales of a tile (8 bits: and the
    // exponents, 16 bytes a page or 128 places of it)
    static constexpr int kRowBytes = D * F::kBits / 8;
    static constexpr int kVCode = kTile * kRowBytes, kKScale = 2 * kVCode;
    static constexpr int kVScale = kKScale + (F::kBits == 4 ? kTile * D / 16 : 0);
    static constexpr int kStage = kKScale + (F::kBits == 4 ? kTile * D / 8 : kTile);
    static constexpr int kRing = kStages * kStage;
    static constexpr int kQueries = kN * kParts * (D / 16) * 32 * 8;
    // rows of every warp that are merged at a time, in one stage
    static constexpr int kMergeRows = kWarps * 8 * D * 4 <= kStage ? 8 : 4;
    static_assert(kWarps * kMergeRows * D * 4 <= kStage, "a stage holds a merge");
    // After the ring and the queries: which stages are full, which empty.  (bf16, d = 128:
    // 112688 bytes, next to 2960 static ones; above 115712 in all a second CTA does not fit,
    // and 256 sequences take 637 us instead of 464.  Hence no more alignment than copies want.)
    static constexpr int kBars = kRing + kQueries;
    static constexpr int kSmem = kBars + 2 * kStages * 8;
    static constexpr int kLead = kStages - 2;                  // tiles copied ahead
    static constexpr bool kEnds = F::kBits == 8;
};

// S^T of a warp's group (its first row at `codes` and `scales`): K, rows
// place_of(g) and 8 more, times Q^T.
template <int D, int kParts>
__device__ __forceinline__ void scores(Fmt4, const uint8_t *codes, const uint8_t *scales, int g,
                                       int t4, const uint4 *queries, float (&s1)[1][4]) {
    float (&s)[4] = s1[0];
    constexpr int kW = D / 32;      // 32-bit words of a lane's share of a row
    uint32_t kw[2][kW];
    __half2 ks[2][kW / 2];          // scale of each block, twice
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = place_of(g) + 8 * r;
        const uint8_t *p = codes + row * (D / 2) + t4 * (D / 8);
        const uint8_t *sp = scales + row * (D / 16) + t4 * (D / 64);
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
                const uint32_t two = e4m3x2_f16(*reinterpret_cast<const uint16_t *>(sp + 2 * w4));
                ks[r][2 * w4] = __low2half2(*reinterpret_cast<const __half2 *>(&two));
                ks[r][2 * w4 + 1] = __high2half2(*reinterpret_cast<const __half2 *>(&two));
            }
        }
    }
    float s2[4];                    // a second chain of products
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
        for (int part = 0; part < kParts; ++part) {
            const uint4 q = queries[(part * kW + w) * 32];
            if (w == 0 && part == 0) {
                mma16816_zero(s, r0[0], r1[0], r0[1], r1[1], q.x, q.y);
                mma16816_zero(s2, r0[2], r1[2], r0[3], r1[3], q.z, q.w);
            } else {
                mma16816(s, r0[0], r1[0], r0[1], r1[1], q.x, q.y);
                mma16816(s2, r0[2], r1[2], r0[3], r1[3], q.z, q.w);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += s2[e];
}

// The same of 8-bit numbers, rows g and g + 8: the group is one block, whose exponent
// (at `exponent`) the scores are multiplied by.
template <int D, int kParts, int kN>
__device__ __forceinline__ void scores(Fmt8, const uint8_t *codes, const uint8_t *exponent, int g,
                                       int t4, const uint4 *queries, float (&s)[kN][4]) {
    float s2[kN][4];                // a second chain of products
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {      // 16 numbers of a row at a time
        uint32_t k[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint4 x = *reinterpret_cast<const uint4 *>(codes + (g + 8 * r) * D + t4 * (D / 4) +
                                                             16 * w);
            k[r][0] = x.x; k[r][1] = x.y; k[r][2] = x.z; k[r][3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint32_t a0[2], a1[2], b0[2], b1[2];
            e4m3x4_f16(k[0][i], a0);
            e4m3x4_f16(k[1][i], a1);
            e4m3x4_f16(k[0][i + 1], b0);
            e4m3x4_f16(k[1][i + 1], b1);
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const uint4 q = queries[((n * kParts + part) * (D / 32) + 2 * w + i / 2) * 32];
                    if (w == 0 && i == 0 && part == 0) {
                        mma16816_zero(s[n], a0[0], a1[0], a0[1], a1[1], q.x, q.y);
                        mma16816_zero(s2[n], b0[0], b1[0], b0[1], b1[1], q.z, q.w);
                    } else {
                        mma16816(s[n], a0[0], a1[0], a0[1], a1[1], q.x, q.y);
                        mma16816(s2[n], b0[0], b1[0], b0[1], b1[1], q.z, q.w);
                    }
                }
        }
    }
    const float f = exponent_f32(*exponent);
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = (s[n][e] + s2[n][e]) * f;
}

// A lane's numbers of V of one group: D / 8 elements of the tokens t4, 4 + (t4 ^ 1)
// and those 8 further, with their scales.
template <typename F, int D>
struct VShare;
template <int D>
struct VShare<Fmt4, D> {
    static constexpr int kWords = D / 64, kBlocks = D == 256 ? 2 : 1;
    uint32_t w[4][kWords], sb[4];

    __device__ static __forceinline__ int place(int j, int t4) {
        return 4 * j + ((j & 1) ? t4 ^ 1 : t4);
    }
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, int g,
                                         int t4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = place(j, t4);
            const uint8_t *p = codes + row * (D / 2) + g * (D / 16);
            const uint8_t *sp = scales + row * (D / 16) + g * D / 128;
            if constexpr (D == 64) {
                w[j][0] = *reinterpret_cast<const uint32_t *>(p);
                sb[j] = *sp;
            } else if constexpr (D == 128) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[j][0] = x.x; w[j][1] = x.y;
                sb[j] = *sp;
            } else {
                const uint4 x = *reinterpret_cast<const uint4 *>(p);
                w[j][0] = x.x; w[j][1] = x.y; w[j][2] = x.z; w[j][3] = x.w;
                sb[j] = *reinterpret_cast<const uint16_t *>(sp);
            }
        }
    }
    // The scale of block k of the tokens 2 e and 2 e + 1 of the four.
    __device__ __forceinline__ __half2 scale(int k, int e) const {
        const uint32_t two =
            e4m3x2_f16(__byte_perm(sb[2 * e], sb[2 * e + 1], k == 0 ? 0x0040 : 0x0051));
        return *reinterpret_cast<const __half2 *>(&two);
    }
    // Takes token j out of the product.
    __device__ __forceinline__ void clear(int j) { sb[j] = 0; }
    // Whether token j has a NaN in block k; it is taken out if so.
    __device__ __forceinline__ bool take_nan(int j, int k) {
        if (((sb[j] >> (8 * k)) & 0x7f) != 0x7f) return false;
        sb[j] &= ~(0xffu << (8 * k));
        return true;
    }
};
// Of 8-bit numbers: of the tokens 2 t4, 2 t4 + 1 and those 8 further, which share one
// exponent.
template <int D>
struct VShare<Fmt8, D> {
    static constexpr int kWords = D / 32, kBlocks = D == 256 ? 2 : 1;
    uint32_t w[4][kWords], e;

    __device__ static __forceinline__ int place(int j, int t4) {
        return 2 * t4 + (j & 1) + 8 * (j >> 1);
    }
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *exponent, int g,
                                         int t4) {
        e = *exponent;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *p = codes + place(j, t4) * D + g * (D / 8);
            if constexpr (D == 64) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[j][0] = x.x; w[j][1] = x.y;
            } else {
#pragma unroll
                for (int i = 0; i < kWords; i += 4) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(p + 4 * i);
                    w[j][i] = x.x; w[j][i + 1] = x.y; w[j][i + 2] = x.z; w[j][i + 3] = x.w;
                }
            }
        }
    }
    __device__ __forceinline__ void clear(int j) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[j][i] = 0;
    }
    __device__ __forceinline__ bool take_nan(int j, int k) {
        uint32_t bad = 0;
#pragma unroll
        for (int i = k * (kWords / kBlocks); i < (k + 1) * (kWords / kBlocks); ++i)
            bad |= e4m3x4_nan(w[j][i]);
        if (bad == 0) return false;
#pragma unroll
        for (int i = k * (kWords / kBlocks); i < (k + 1) * (kWords / kBlocks); ++i) w[j][i] = 0;
        return true;
    }
};

// acc += A B, or with kScaled acc += factor * (A B), B in kParts parts.
template <int kParts, bool kScaled>
__device__ __forceinline__ void add_product(float (&acc)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, const uint32_t (&b)[kParts][2],
                                            float factor) {
    if constexpr (!kScaled) {
#pragma unroll
        for (int part = 0; part < kParts; ++part)
            mma16816(acc, a0, a1, a2, a3, b[part][0], b[part][1]);
    } else {
        float x[4] = {};
#pragma unroll
        for (int part = 0; part < kParts; ++part)
            mma16816(x, a0, a1, a2, a3, b[part][0], b[part][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[e], factor, acc[e]);
    }
}

// O^T += V^T P^T, or with kScaled O^T += factor * (V^T P^T).
template <int D, int kParts, bool kScaled>
__device__ __forceinline__ void product(const VShare<Fmt4, D> &v,
                                        const uint32_t (&pf)[1][kParts][2], float factor,
                                        float (&o)[1][D / 16][4]) {
    using V = VShare<Fmt4, D>;
    __half2 sc[V::kBlocks][2];
#pragma unroll
    for (int k = 0; k < V::kBlocks; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) sc[k][e] = v.scale(k, e);
#pragma unroll
    for (int w = 0; w < V::kWords; ++w) {
        constexpr uint32_t kEven = 0x0f0f0f0fu;
        uint32_t e1[4], d1[4], e2[4], d2[4];   // even and odd elements of the two token pairs
        e2m1x8_f16(select_bits(v.w[0][w], v.w[1][w] << 4, kEven), e1);
        e2m1x8_f16(select_bits(v.w[0][w] >> 4, v.w[1][w], kEven), d1);
        e2m1x8_f16(select_bits(v.w[2][w], v.w[3][w] << 4, kEven), e2);
        e2m1x8_f16(select_bits(v.w[2][w] >> 4, v.w[3][w], kEven), d2);
        const __half2 s1 = sc[w / 2 % V::kBlocks][0], s2 = sc[w / 2 % V::kBlocks][1];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            add_product<kParts, kScaled>(o[0][4 * w + k], mul2(e1[k], s1), mul2(d1[k], s1),
                                         mul2(e2[k], s2), mul2(d2[k], s2), pf[0], factor);
    }
}
template <int D, int kParts, bool kScaled, int kN>
__device__ __forceinline__ void product(const VShare<Fmt8, D> &v,
                                        const uint32_t (&pf)[kN][kParts][2], float factor,
                                        float (&o)[kN][D / 16][4]) {
    const __half2 f = exponent_f16x2(v.e);
#pragma unroll
    for (int w = 0; w < VShare<Fmt8, D>::kWords; ++w) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            // two elements of four tokens: bytes of two tokens side by side
            uint32_t x[2], y[2];
            e4m3x4_f16(__byte_perm(v.w[0][w], v.w[1][w], k == 0 ? 0x5140 : 0x7362), x);
            e4m3x4_f16(__byte_perm(v.w[2][w], v.w[3][w], k == 0 ? 0x5140 : 0x7362), y);
            const uint32_t a[4] = {mul2(x[0], f), mul2(x[1], f), mul2(y[0], f), mul2(y[1], f)};
#pragma unroll
            for (int n = 0; n < kN; ++n)
                add_product<kParts, kScaled>(o[n][2 * w + k], a[0], a[1], a[2], a[3], pf[n], factor);
        }
    }
}

template <typename F, typename T, int D, bool kSplit, int kN, int kU, int kStages, int kMinCtas>
__global__ void __launch_bounds__(kThreads, kMinCtas) k_kv_attn(const AttnArgs a) {
    using Sh = Shape<F, D, kSplit, kN, kU, kStages>;
    using V = VShare<F, D>;
    constexpr int kTile = Sh::kTile;
    using W = Walk<kTile, Sh::kRows, kThreads, Sh::kEnds>;
    constexpr int kT = D / 16;      // m tiles of O^T = k steps of S^T
    constexpr int kParts = Sh::kParts, kRows = Sh::kRows;
    // Least probability (lifted) whose fp16 parts keep all their bits, how far the
    // lifted maximum lies above it, and that range's middle and half in log2 units.
    constexpr float kLow = kSplit ? 0x1p-3f : 0x1p-14f, kBand = kSplit ? 0x1p18f : 0x1p29f;
    constexpr float kMid = kSplit ? 6.f : 0.5f, kHalf = kLift + kRaise - kMid;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ typename W::P plan;
    __shared__ uint32_t armed[kStages];     // tiles that were copied into each stage
    __shared__ int abort_flag;
    __shared__ float2 warp_ml[kWarps][kRows];
    __shared__ float row_mul[kRows];
    __shared__ W walk[3];           // the piece at work and the two after it, in a ring
    __shared__ bool walk_more[3];   // whether there is one behind each
    __shared__ int row_from[kRows], row_to[kRows], all_seen[kN][2];
    uint4 *queries = reinterpret_cast<uint4 *>(smem + Sh::kRing);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Sh::kBars), *empty = full + kStages;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, kWarps);
            armed[i] = 0;
        }
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    ptx::griddep_launch_dependents();   // (the join, which waits for this kernel's end)
    // 8 bits: calls that need no plan.  A token of each of 8 sequences of up to 100 places takes
    // 6.5 us (with a plan 7.6), of 64 13.1 (14.3), of one of 77 in fp32 7.1 (8.3).
    bool alike = false;
    if constexpr (Sh::kEnds) alike = !a.cuts && !a.kv.cu && a.kv.n_tokens / a.kv.N <= a.max_new;
    if (!alike) plan.build(a);
    const long long total = alike ? W::alike_total(a) : plan.total;
    const long long ctas = min((long long)gridDim.x, total);
    if (a.cuts && threadIdx.x == 0) a.cuts[blockIdx.x].pieces = 0;
    if (blockIdx.x >= ctas) return;
    const long long beg = quot(total * blockIdx.x, ctas);
    const long long end = quot(total * (blockIdx.x + 1), ctas);
    const Waits waits{&abort_flag, a.err, a.wait_limit};
    const uint32_t ring_at = ptx::smem_u32(smem);

    // Copies: lane (run, part) of the issuing warp copies one part of a run of tokens
    // that lie together, a page's or as many of it as make a tile.
    const int run_shift = min(a.kv.page_shift, 7), run = 1 << run_shift;
    const int lane_run = lane >> 2, lane_part = lane & 3;
    const int row_bytes = lane_part < 2 ? Sh::kRowBytes : D / 16;
    const uint32_t lane_dst = lane_part == 0   ? 0
                              : lane_part == 1 ? Sh::kVCode
                              : lane_part == 2 ? Sh::kKScale
                                               : Sh::kVScale;
    constexpr int kRuns = kTile / 16 / 8;         // of a lane, at the smallest pages
    // pages of the lane's runs (8 apart) of the tile at `place`, as the table has them
    auto fetch = [&](bool there, int b, int place, int len, int (&raw)[kRuns]) {
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            const int in_tile = (lane_run + 8 * k) * run, at = place + in_tile;
            raw[k] = there && in_tile < kTile && at < len ? a.kv.page_raw(b, at) : Kv::kNoPage;
        }
    };
    // Copies the CTA's tile n, whose first place is `place` (one warp).  Once a wait has given
    // up nothing more is copied, and a warp frees no stage that it has not waited for: a
    // stage is filled again only behind eight warps that had its tile.
    auto produce = [&](uint32_t n, int place, int h, const int (&raw)[kRuns]) {
        int page[kRuns];
#pragma unroll
        for (int k = 0; k < kRuns; ++k) page[k] = a.kv.page_checked(raw[k], a.err);
        const uint32_t stage = n % kStages;
        if (n >= kStages && !waits.on(empty + stage, ((n / kStages) + 1) & 1)) return;
        if (__any_sync(0xffffffffu, *waits.abort != 0)) return;
        uint32_t runs = 0;
#pragma unroll
        for (int k = 0; k < kRuns; ++k)
            runs += __popc(__ballot_sync(0xffffffffu, page[k] >= 0 && lane_part == 0));
        if (lane == 0) {
            armed[stage] = n / kStages + 1;
            ptx::mbar_arrive_expect_tx(full + stage, F::kBits == 4 ? runs * run * (D * 9 / 8)
                                                                   : runs * (run * (2 * D) + 16));
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            if (page[k] < 0) continue;
            const int psz = a.kv.page_size(), in_tile = (lane_run + 8 * k) * run;
            const int at = (place + in_tile) & (psz - 1);
            int from, bytes;
            uint32_t to = ring_at + stage * Sh::kStage + lane_dst;
            if constexpr (F::kBits == 4) {
                from = at * row_bytes + (lane_part == 0   ? 0
                                         : lane_part == 1 ? v_code_at(psz, D, 0)
                                         : lane_part == 2 ? k_scale_at(psz, D, 0)
                                                          : v_scale_at(psz, D, 0));
                bytes = run * row_bytes;
                to += in_tile * row_bytes;
            } else {
                if (lane_part == 3) continue;
                from = lane_part == 2 ? F::exponents_at(psz, D, at)
                                      : F::code_at(D, lane_part == 0 ? at : psz + at);
                bytes = lane_part == 2 ? 16 : run * D;
                to += lane_part == 2 ? 16 * (lane_run + 8 * k) : in_tile * D;
            }
            if (!a.kv.bytes_ok<F>(page[k], h, from, bytes)) continue;
            bulk_load(to, a.kv.pages + a.kv.block<F>(page[k], h) + from, bytes, full + stage);
        }
    };

    // Queries of a piece, eight rows a warp: the lane's part of row 8 n + g, loaded ...
    const int q_n = kN == 1 ? 0 : (int)(kQueryTurn >> 4 * warp) & 15;
    const bool q_warp = kN == 1 ? warp == kQueryWarp : q_n < kN;
    auto row_of = [&](const W &w, bool &there, int &j) {
        const int r = w.row0() + 8 * q_n + g;
        there = 8 * q_n + g < w.rows(a);
        j = there ? r / a.G : 0;
        const int i = there ? r - j * a.G : 0;
        if (there) there = a.row_ok((long long)w.sq.first + j, w.h * a.G + i);
        return i;
    };
    auto load_queries = [&](const W &w, Run<T> (&x)[D / 32]) {
        bool there;
        int j;
        const int i = row_of(w, there, j);
        const T *p = static_cast<const T *>(a.q) + (w.sq.first + j) * a.q_tok +
                     (long long)(w.h * a.G + i) * a.q_head + t4 * (D / 4);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            x[k] = Run<T>{};
            if (there) x[k].load(p + 8 * k);
        }
    };
    // ... and as the B operand, scaled by a power of two that brings the row's largest
    // number to [2^13, 2^14), with what the rows see.
    auto put_queries = [&](const W &w, const Run<T> (&x)[D / 32]) {
        bool there;
        int j;
        row_of(w, there, j);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            float v[8];
            x[k].get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
        }
        if (!there) m = 0.f;
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float down;
        const float up = row_up(m, down);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            float v[8];
            x[k].get(v);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float u = there ? v[2 * e] * up : 0.f, y = there ? v[2 * e + 1] * up : 0.f;
                hi[e] = pack_f16(u, y);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi[e]));
                lo[e] = pack_f16(u - f.x, y - f.y);
            }
            uint4 *q = queries + (q_n * kParts * (D / 32) + k) * 32 + lane;
            q[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (kSplit) q[(D / 32) * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        int from = 0, to = w.sq.len;
        if (there) w.sq.sees(a, j, from, to);
        if (t4 == 0) {
            const float gk = a.kv.head_scale ? __ldg(a.kv.head_scale + w.h) : 1.f;
            row_mul[8 * q_n + g] = down * a.scale_log2 * gk;
            row_from[8 * q_n + g] = from;
            row_to[8 * q_n + g] = to;
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            from = max(from, __shfl_xor_sync(0xffffffffu, from, o));
            to = min(to, __shfl_xor_sync(0xffffffffu, to, o));
        }
        if (lane == 0) {
            all_seen[q_n][0] = from;
            all_seen[q_n][1] = to;
        }
    };

    // the piece behind that of `at`, into `to` (one warp)
    auto walk_on = [&](int at, int to) {
        W x = walk[at];
        const bool more = x.next(a);
        __syncwarp();
        if (lane == 0) {
            walk[to] = x;
            walk_more[at] = more;
        }
    };
    {
        W w;
        if (alike) w.start_alike(a, beg, end);
        else w.start(a, plan, beg, end);
        if (threadIdx.x == 0) walk[0] = w;
    }
    __syncthreads();                // (covers the initialisation as well)
    Run<T> raw_q[D / 32];
    if (q_warp) {
        load_queries(walk[0], raw_q);
        put_queries(walk[0], raw_q);
    } else if (warp == kWalkWarp) {
        walk_on(0, 1);
    }
    // Tile n of the CTA (over all its pieces) is copied by warp n % kWarps; a piece's
    // first tile already while the last tile of the piece before it is worked on.
    uint32_t tiles_before = 0;      // of the earlier pieces
    uint32_t stage = 0, phase = 0;  // of the tile at work
    int made = 0;                   // tiles of this piece that are on their way already
    for (int piece = 0, after_piece = 1;;) {
        const int n_copy = walk[piece].count(), place0 = walk[piece].place0();
        const int len = walk[piece].sq.len;
        int next = (warp - (int)tiles_before) & (kWarps - 1);   // the warp's next tile to copy
        if (next < made) next += kWarps;
        int next_page[kRuns];
        auto fetch_next = [&]() {
            fetch(next < n_copy, walk[piece].b, place0 + next * kTile, len, next_page);
        };
        auto produce_next = [&]() {
            produce(tiles_before + next, place0 + next * kTile, walk[piece].h, next_page);
            next += kWarps;
            fetch_next();
        };
        fetch_next();
        if (next < min(Sh::kLead, n_copy)) produce_next();
        if (tiles_before == 0) __syncthreads();     // (later ones: with the merge's last)
        int all_from = all_seen[0][0], all_to = all_seen[0][1];   // places that every row sees
#pragma unroll
        for (int n = 1; n < kN; ++n) {
            all_from = max(all_from, all_seen[n][0]);
            all_to = min(all_to, all_seen[n][1]);
        }
        float mul[kN][2], o[kN][kT][4], sub[kN][2], sum[kN][2];   // sub: what scores lose before ex2
#pragma unroll
        for (int n = 0; n < kN; ++n) {
#pragma unroll
            for (int i = 0; i < kT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mul[n][e] = row_mul[8 * n + 2 * t4 + e];
                sub[n][e] = -INFINITY;
                sum[n][e] = 0.f;
            }
        }
        // The first tile of the piece after this one, copied by warp `after`: its pages are
        // looked up before this piece's last tile is worked on and copied behind it.
        const int after = (tiles_before + n_copy) & (kWarps - 1);
        auto look_after = [&]() {
            const W &x = walk[after_piece];
            next = walk_more[piece] && x.count() > 0 ? 0 : -1;
            fetch(next == 0, x.b, x.place0(), x.sq.len, next_page);
        };
        // the iteration at which this warp copies or looks pages up next
        auto due_at = [&]() {
            return next < n_copy ? next - Sh::kLead : warp == after ? n_copy - 1 : n_copy;
        };
        int due = due_at();
        for (int i = 0; i < n_copy; ++i) {
            if (i == due) {
                if (next < n_copy) produce_next();
                if (i + 1 == n_copy && warp == after) look_after();
                due = due_at();
            }
            const bool arrived = waits.on(full + stage, phase);
            const uint8_t *buf = smem + stage * Sh::kStage + warp * (kU * kGroup * Sh::kRowBytes);
            const uint8_t *sbuf =
                smem + stage * Sh::kStage + Sh::kKScale + warp * (kU * kGroup * D / 16);
            int t0 = place0 + i * kTile + warp * (kU * kGroup);
#pragma unroll 1
            for (int u = 0; u < kU;
                 ++u, t0 += kGroup, buf += kGroup * Sh::kRowBytes, sbuf += kGroup * D / 16) {
                if (!arrived || t0 >= len) break;
                const bool whole = t0 >= all_from && t0 + kGroup <= all_to;

                float s[kN][4];
                V v;
                if constexpr (F::kBits == 4) {
                    scores<D, kParts>(F(), buf, sbuf, g, t4, queries + lane, s);
                    v.load(buf + Sh::kVCode, sbuf + (Sh::kVScale - Sh::kKScale), g, t4);
                } else {
                    // the group's exponents, among the 16 bytes of its run of places
                    const int in_tile = (warp * kU + u) * kGroup;
                    const uint8_t *ex = smem + stage * Sh::kStage + Sh::kKScale +
                                        16 * (in_tile >> run_shift) +
                                        ((in_tile & (run - 1)) / F::kBlock);
                    scores<D, kParts>(F(), buf, ex, g, t4, queries + lane, s);
                    v.load(buf + Sh::kVCode, ex + 8, g, t4);
                }

                // Scores in log2 units less the row's `sub`, so that the row's largest number
                // is about kLift.  One comparison finds those that call for more: above
                // kLift + kRaise the maximum moves; below kLow probabilities lose bits.
                float t[kN][4];
                bool more = false;
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t[n][e] = fmaf(s[n][e], mul[n][e & 1], -sub[n][e & 1]);
                        if (!whole) {
                            const int at = t0 + row_of_place<F>(g) + 8 * (e >> 1);
                            const int r = 8 * n + 2 * t4 + (e & 1);
                            if (at < row_from[r] || at >= row_to[r]) t[n][e] = -INFINITY;
                        }
                        more |= fabsf(t[n][e] - kMid) > kHalf;
                    }
                const bool extra = __any_sync(0xffffffffu, more);
                if (extra) {
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // (+infinity in t is a row's first score: its own value decides)
                            float m = -INFINITY;
#pragma unroll
                            for (int k = e; k < 4; k += 2)
                                m = fmaxf(m, t[n][k] == -INFINITY ? -INFINITY : s[n][k] * mul[n][e]);
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            m -= kLift;
                            if (m > sub[n][e] + kRaise) {
                                const float f = ex2(sub[n][e] - m);
                                sub[n][e] = m;
                                sum[n][e] *= f;
#pragma unroll
                                for (int k = 0; k < kT; ++k) {
                                    o[n][k][e] *= f;
                                    o[n][k][e + 2] *= f;
                                }
                            }
#pragma unroll
                            for (int k = e; k < 4; k += 2)
                                if (t[n][k] != -INFINITY)
                                    t[n][k] = fmaf(s[n][k], mul[n][e], -sub[n][e]);
                        }
                }

                uint32_t pf[kN][kParts][2];
                float p[kN][4], rest[kN][4];
                bool low = false;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[n][e] = ex2(t[n][e]);
                        sum[n][e & 1] += p[n][e];
                    }
                    if (extra) {      // the small ones later, in a product of their own
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            rest[n][e] = 0.f;
                            if (p[n][e] < kLow) {
                                rest[n][e] = p[n][e];
                                p[n][e] = 0.f;
                            }
                            low |= rest[n][e] > 0.f;
                        }
                    }
                    operand_of<kSplit>(p[n], pf[n][0], pf[n][kParts - 1]);
                }
                if (!whole) {
                    // Places behind the sequence's end may hold anything: they become 0.  A NaN
                    // that some rows see and others do not would reach all of them through
                    // 0 * NaN: it is taken out of the product and put into the rows that see it.
                    constexpr int kBlocks = V::kBlocks;
                    uint32_t nan[kBlocks] = {};
                    bool any = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int off = v.place(j, t4);
                        if (t0 + off >= len) v.clear(j);
#pragma unroll
                        for (int k = 0; k < kBlocks; ++k)
                            if (v.take_nan(j, k)) {
                                nan[k] |= 1u << off;
                                any = true;
                            }
                    }
                    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                        for (int k = 0; k < kBlocks; ++k) {
                            nan[k] |= __shfl_xor_sync(0xffffffffu, nan[k], 1);
                            nan[k] |= __shfl_xor_sync(0xffffffffu, nan[k], 2);
#pragma unroll
                            for (int n = 0; n < kN; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int r = 8 * n + 2 * t4 + e;
                                    const int lo = min(16, max(0, row_from[r] - t0));
                                    const int hi = min(16, max(0, row_to[r] - t0));
                                    const uint32_t seen = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
                                    if (nan[k] & seen) {
#pragma unroll
                                        for (int m = 0; m < kT / kBlocks; ++m) {
                                            o[n][k * (kT / kBlocks) + m][e] = NAN;
                                            o[n][k * (kT / kBlocks) + m][e + 2] = NAN;
                                        }
                                    }
                                }
                        }
                    }
                }
                product<D, kParts, false>(v, pf, 1.f, o);
                if (extra && __any_sync(0xffffffffu, low)) {
                    // what lies a factor kBand below the last product's range, until nothing is
                    // left
                    float factor = 1.f;
                    do {
                        factor *= 1.f / kBand;
                        low = false;
#pragma unroll
                        for (int n = 0; n < kN; ++n) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                rest[n][e] *= kBand;
                                p[n][e] = rest[n][e] >= kLow ? rest[n][e] : 0.f;
                                if (p[n][e] > 0.f) rest[n][e] = 0.f;
                                low |= rest[n][e] > 0.f;
                            }
                            operand_of<kSplit>(p[n], pf[n][0], pf[n][kParts - 1]);
                        }
                        product<D, kParts, true>(v, pf, factor, o);
                    } while (__any_sync(0xffffffffu, low));
                }
            }
            if (!arrived) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty + stage);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (warp == after) {
            if (n_copy == 0) look_after();
            if (next == 0)
                produce(tiles_before + n_copy, walk[after_piece].place0(), walk[after_piece].h,
                        next_page);
        }
        tiles_before += n_copy;

        // the warps' sums of this piece
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = sum[n][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) warp_ml[warp][8 * n + 2 * t4 + e] = make_float2(sub[n][e], x);
            }
        __syncthreads();
        if (*waits.abort) break;        // (no wait is made between here and the next barrier)
        const W &w = walk[piece];
        const int h = w.h, row0 = w.row0(), rows = w.rows(a);
        const bool complete = w.complete();
        const long long slot = 2ll * blockIdx.x + (w.cur == beg ? 0 : 1);
        if (threadIdx.x == 0 && w.tile0 == 0 && !complete) {
            const long long end_tile = w.cur + w.n_tiles;
            const int last = (int)quot(end_tile * ctas - 1, total);   // CTA of its last tile
            a.cuts[blockIdx.x] = Cut{last - (int)blockIdx.x + 1, (int)slot, w.sq.first, h, row0, rows};
        }
        // The merge goes into the stage behind the one that the next piece's first tile may
        // be on its way to: every warp is done with it, and it is filled again only in the
        // next piece.
        float *merge =
            reinterpret_cast<float *>(smem + (tiles_before + 1) % kStages * Sh::kStage);
        constexpr int kMr = Sh::kMergeRows;
        const bool more = walk_more[piece];
        // what the next piece starts with, by warps that have less of the merge to do
        if (more && q_warp) load_queries(walk[after_piece], raw_q);
#pragma unroll
        for (int half = 0; half < kRows / kMr; ++half) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * t4 + e - half * kMr;
                    if (r < 0 || r >= kMr) continue;
                    float m = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) m = fmaxf(m, warp_ml[k][8 * n + 2 * t4 + e].x);
                    const float f = m == -INFINITY ? 1.f : ex2(sub[n][e] - m);
                    float *p = merge + (warp * kMr + r) * D + g * (D / 8);
#pragma unroll
                    for (int k = 0; k < kT; ++k)
                        *reinterpret_cast<float2 *>(p + 2 * k) =
                            make_float2(o[n][k][e] * f, o[n][k][e + 2] * f);
                }
            __syncthreads();
            if (half == 0 && more) {
                if (q_warp) put_queries(walk[after_piece], raw_q);
                else if (warp == kWalkWarp) walk_on(after_piece, 3 - piece - after_piece);
            }
            for (int x = threadIdx.x; x < min(kMr, rows - half * kMr) * (D / 4); x += kThreads) {
                const int rm = x / (D / 4), r = half * kMr + rm, d = 4 * (x - rm * (D / 4));
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) m = fmaxf(m, warp_ml[k][r].x);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 ml = warp_ml[k][r];
                    l += ml.y * (m == -INFINITY ? 1.f : ex2(ml.x - m));
                    const float4 y =
                        *reinterpret_cast<const float4 *>(merge + (k * kMr + rm) * D + d);
                    v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
                }
                if (complete) {
                    const int rr = row0 + r, j = rr / a.G, hq = h * a.G + rr - j * a.G;
                    const float gv = a.kv.head_scale ? __ldg(a.kv.head_scale + a.kv.H + h) : 1.f;
                    const float inv = l == 0.f ? 0.f : gv / l;
                    if (!a.row_ok((long long)w.sq.first + j, hq)) continue;
                    T *p = static_cast<T *>(a.o) + (w.sq.first + j) * a.o_tok + hq * a.o_head + d;
                    store4(p, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    if (a.lse && d == 0) a.lse[(long long)(w.sq.first + j) * a.Hq + hq] = lse_of(m, l);
                } else if (a.part_ok(slot * kRows + r, kRows)) {
                    store4(a.part_o + (slot * kRows + r) * D + d, v.x, v.y, v.z, v.w);
                    if (d == 0) a.part_ml[slot * kRows + r] = make_float2(m, l);
                }
            }
            ptx::fence_proxy_async_smem();     // before copies go into that stage again
            __syncthreads();
        }
        if (!more) break;
        made = walk[after_piece].count() > 0 ? 1 : 0;
        const int third = 3 - piece - after_piece;
        piece = after_piece;
        after_piece = third;
    }
    // a wait gave up: copies that no warp has waited for may still be on their way
    if (*waits.abort && warp == 0) drain_ring<kStages>(full, armed);
}

template <typename F, typename T, int D, bool kSplit, int kN, int kU, int kStages, int kMinCtas>
gdn_status launch(AttnArgs &a, cudaStream_t st) {
    using Sh = Shape<F, D, kSplit, kN, kU, kStages>;
    auto kern = k_kv_attn<F, T, D, kSplit, kN, kU, kStages, kMinCtas>;
    constexpr int kTile = Sh::kTile;
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
    const long long tiles = a.max_len / kTile + 2;
    long long most = rt * a.kv.H * tiles;   // of one sequence; of all, without overflow:
    most = most > resident ? resident : most * a.kv.N;
    const int grid = (int)(most < resident ? (most < 1 ? 1 : most) : resident);
    const bool cut = a.max_len > kTile;     // else no piece of work has two tiles
    a.end_tiles = cut && Sh::kEnds ? kEndTiles : 0;
    void *scratch = nullptr;
    if (cut && alloc_pieces<D, Sh::kRows>(a, grid, &scratch, st) != cudaSuccess) return GDN_ERR_CUDA;
    const int slot = timer_begin(st, F::kBits == 4 ? "k_kv_attn" : "k_kv8_attn");
    kern<<<grid, kThreads, Sh::kSmem, st>>>(a);
    timer_end(slot, st);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (cut) {
        if (e == cudaSuccess) e = launch_join<T, D, Sh::kRows, kWarps, kWarps>(a, grid, st);
        const cudaError_t f = scratch_free(scratch, st);
        if (e == cudaSuccess) e = f;
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Eights of rows that a piece has in 8 bits: as many as the registers hold sums for (d / 4 a lane
// each), in passes of the same number.  64 ragged sequences of 128 to 16384 places, 16 rows: two
// eights 276 us, one by one 384 (d = 256 340 and 468, fp32 rows 345 and 454); 24 rows three eights
// 372, two 517, one 564 (fp32 490, 635; d = 64 in fp32 338, 439).  512 rows over 12001 to 16384
// places, fp32: three eights 872 us, two 900, one 1238; at d = 256 two 1458, one 2121.  At d = 64
// two fit twice on an SM: 24 rows 285 us, as three once 270; 16 rows 163, once 200.  Up to 1024
// places the ends of the pieces count for more, and twice as many CTAs an SM (bf16, d = 128) take
// 47 us for 16 rows of 64 sequences of 512 where two eights take 52, 63 and 65 at 1024 places
// (at 2048 92 and 87).
int eights_of(const AttnArgs &a, bool split) {
    if (a.kv.d == 128 && !split && a.max_len <= 1024) return 1;
    const int most = a.kv.d == 256 || (a.kv.d == 64 && !split) ? 2 : 3;
    const long long rows = (long long)a.max_new * a.G, all = rows > 8 ? (rows + 7) / 8 : 1;
    const long long passes = (all + most - 1) / most;
    return (int)((all + passes - 1) / passes);
}

// By the head's width: registers hold d / 4 sums a lane and eight rows, and a stage has to
// hold the merge of the warps' sums.  8 bits: tiles of half the places, of as many bytes, but
// where one CTA an SM has the whole ring (64 ragged sequences with fp32 rows 226 us, in tiles
// of 128 places and three stages 272, six stages 237; at d = 64 158, 172 and 167).
template <typename F, typename T, bool kSplit>
gdn_status pick(AttnArgs &a, cudaStream_t st) {
    constexpr int kCtas = kSplit ? 1 : 2, kWide = kSplit ? 2 : 1;
    if constexpr (F::kBits == 4) {
        switch (a.kv.d) {
            case 64: return launch<F, T, 64, kSplit, 1, 2, 3, kCtas>(a, st);
            case 128: return launch<F, T, 128, kSplit, 1, 2, 3, kCtas>(a, st);
            default: return launch<F, T, 256, kSplit, 1, 1, 4, 1>(a, st);
        }
    } else {
        const int n = eights_of(a, kSplit);
        if (a.kv.d == 64) {
            if (n == 1) return launch<F, T, 64, kSplit, 1, 2 * kWide, 3, kCtas>(a, st);
            if constexpr (kSplit)
                if (n == 3) return launch<F, T, 64, kSplit, 3, 2 * kWide, 3, kCtas>(a, st);
            return launch<F, T, 64, kSplit, 2, 2 * kWide, 3, kCtas>(a, st);
        }
        if (a.kv.d == 128) {
            if (n == 1) return launch<F, T, 128, kSplit, 1, kWide, 3, kCtas>(a, st);
            return n == 2 ? launch<F, T, 128, kSplit, 2, 2, 3, 1>(a, st)
                          : launch<F, T, 128, kSplit, 3, 2, 3, 1>(a, st);
        }
        return n == 1 ? launch<F, T, 256, kSplit, 1, 1, 3, 1>(a, st)
                      : launch<F, T, 256, kSplit, 2, 1, 3, 1>(a, st);
    }
}

template <typename F>
gdn_status attention(const gdn_kv *kv, const gdn_rows *q, const gdn_rows *o, float *lse,
                     int max_len, int max_new, float scale, int window, unsigned flags,
                     gdn_dtype dt, void *stream) {
    if (!kv || kv->N < 0 || kv->n_tokens < 0 || max_len < 0 || max_new < 0 || window < 0)
        return GDN_ERR_INVALID_ARG;
    if (flags & ~(unsigned)GDN_ATTN_CAUSAL) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (kv->n_tokens == 0) return GDN_OK;
    if (kv->N == 0) return GDN_ERR_INVALID_ARG;
    AttnArgs a{};
    gdn_status rc = check_kv(kv, &a.kv);
    if (rc != GDN_OK) return rc;
    if ((rc = check_rows(q, dt, true)) != GDN_OK ||
        (rc = check_rows(o, dt, true)) != GDN_OK)
        return rc;
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
    a.err = device_error_word();
    const long long limit = option(GDN_OPT_WAIT_LIMIT);
    a.wait_limit = limit > 0 ? (uint32_t)(limit > 0x7fffffffLL ? 0x7fffffffLL : limit) : (1u << 22);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dt == GDN_F32) return pick<F, float, true>(a, st);
    constexpr int kMany = F::kBits == 4 ? kMany4 : kMany8;
    if (a.kv.d <= 128 && (long long)a.max_new * a.G > kMany) return attn_many<F>(a, st);
    return pick<F, __nv_bfloat16, false>(a, st);
}

}  // namespace
}  // namespace kv
}  // namespace gdn

extern "C" gdn_status gdn_kv_attn(const gdn_kv *kv, const gdn_rows *q, const gdn_rows *o,
                                  float *lse, int max_len, int max_new, float scale, int window,
                                  unsigned flags, gdn_dtype dt, void *stream) {
    return gdn::kv::attention<gdn::kv::Fmt4>(kv, q, o, lse, max_len, max_new, scale, window, flags,
                                             dt, stream);
}
extern "C" gdn_status gdn_kv8_attn(const gdn_kv *kv, const gdn_rows *q, const gdn_rows *o,
                                   float *lse, int max_len, int max_new, float scale, int window,
                                   unsigned flags, gdn_dtype dt, void *stream) {
    return gdn::kv::attention<gdn::kv::Fmt8>(kv, q, o, lse, max_len, max_new, scale, window, flags,
                                             dt, stream);
}
