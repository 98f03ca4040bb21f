// gdn_beam.cu -- beam search over a hybrid decoder (gdn_beam.h): selection over beams
// and vocabulary, and reordering of states and pages.
//
// Selection: score(w, v) = scores[w] + x[w][v] - log sum_u exp(x[w][u]), the n best of a
// group's W V.  Within a row the order is that of the logits, so a row's n best need no
// logarithm, and its logits are read once:
// - k_beam_rows: a CTA takes a run of a row, up to 32 vectors of 16 bytes a thread, in one pass
//   for the largest number and the sum of exponentials.  What a thread keeps of two vectors
//   is their largest number.  With k = n / 4 rounded up, the k-th largest thread's of every one
//   of 4 warps is reached by k numbers, so the least of the 4 is a bound that n numbers of
//   the run reach; pairs that reach it are few, and their numbers are read again from
//   the caches to be listed (64-bit keys: the number, then the lower index).
//   Runs are cut by index, not by address, and sums do not depend on where a row starts.
// - k_beam_pick, a CTA a group: a warp a row joins the runs' sums and finds the n best of
//   their lists; the beams' candidates that a like bound leaves are ranked by their scores,
//   sums of two fp32 numbers.
// Reading the logits bounds a large batch, latency of two launches a small one: 64 groups of 8
// beams over 128256 bf16 logits take 34 us (131 MB; the first kernel 30, in a copy's time 19),
// one group of 4 over 32000 in fp32 8 us.  One pass without the lists would take 23 us; the
// rest is the end of a run, which no loads run beside.  Warps that each listed the n best of
// their runs took 154 us for the first kernel; scores in fp64 3 us more for the second.  Rows that do
// not begin at a multiple of 16 bytes load nothing ahead (64 x 8 beams over 50257 take 25 us, over
// 50264 17), and of a run whose numbers are nearly all alike all are listed (the 64 groups over 128256,
// all tokens but 30 neighbours masked: 128 us with -infinity, 160 with a number, whose sums are
// formed again as well; with 1 % of the tokens left 35).
//
// Reordering: every CTA finds by itself which beams have to move (a few instructions a
// group, a warp each) and copies its share of 16 KB pieces.  Copying bounds it: 96 beams of six
// recurrent layers of 16 heads and two attention layers, 34 of which move, take 66 us (437
// MB read and written, as much as a plain copy of them would take).  Lists of what moves in
// shared memory instead of a look-up and two barriers a piece took 73 us, pieces of 32 KB 75.
#include <cmath>

#include "gdn_beam.h"
#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace beam {
namespace {

constexpr int kMaxBeams = 32, kMaxBest = 32;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ selection

// Numbers as integers of the same order (-0 as 0; NaN is looked after elsewhere).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((int)u < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float number_of(uint32_t o) {
    return __uint_as_float(o ^ ((int)o < 0 ? 0x80000000u : 0xffffffffu));
}
// A sum held as two fp32 numbers, the second at most half a step of the first: 48 bits, in
// instructions that take a tenth of fp64's time here.
struct Two {
    float hi, lo;
};
// a + b, exactly (where it does not overflow).
__device__ __forceinline__ Two sum_of(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Two{s, isinf(s) ? 0.f : __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two h = sum_of(a.hi, b.hi);
    return sum_of(h.hi, __fadd_rn(h.lo, __fadd_rn(a.lo, b.lo)));
}
// As integers of the same order, NaN above everything.  A second number that fp64 would not hold
// beside the first (next to a logit that masks with its type's lowest number) is left out.
__device__ __forceinline__ unsigned long long order_of(Two x) {
    if (isnan(x.hi)) return ~0ull;
    if (fabsf(x.lo) < fabsf(x.hi) * 0x1p-53f) x.lo = 0.f;
    return (unsigned long long)order_of(x.hi) << 32 | order_of(x.lo);
}
__device__ __forceinline__ float number_of(unsigned long long o) {
    return o == ~0ull ? NAN : number_of((uint32_t)(o >> 32));
}
// Keys: the number, then the lower index; 0 is none.
using Key = unsigned long long;
__device__ __forceinline__ Key key_of(uint32_t order, uint32_t index) {
    return (Key)order << 32 | (0xffffffffu - index);
}
__device__ __forceinline__ uint32_t index_of(Key k) { return 0xffffffffu - (uint32_t)k; }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Descending order over a warp of one key a lane.  (Called, so that it is fetched once.)
__device__ __noinline__ Key sorted32(Key x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const Key y = __shfl_xor_sync(kAll, x, j);
            const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
            x = larger ? (x > y ? x : y) : (x < y ? x : y);
        }
    return x;
}

// The n-th largest of a warp's numbers, one a lane.
__device__ __forceinline__ uint32_t nth32(uint32_t x, int n) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const uint32_t y = __shfl_xor_sync(kAll, x, j);
            x = ((lane & j) == 0) == ((lane & k) == 0) ? max(x, y) : min(x, y);
        }
    return __shfl_sync(kAll, x, n - 1);
}

// The n best of the keys that a warp has seen, in 64 places of shared memory.
struct Best {
    Key *buf;
    Key least;        // keys below it are not among the n best
    int count, n;

    // Sorts what there is and keeps n.
    __device__ __forceinline__ void cut() {
        const int lane = threadIdx.x & 31;
        __syncwarp();
        Key a = lane < count ? buf[lane] : 0;
        a = sorted32(a);
        if (count > 32) {
            // the upper half sorted too, turned around: the larger ones of each pair are the 32
            // largest, and are sorted once more
            const Key b = sorted32(lane + 32 < count ? buf[lane + 32] : 0);
            const Key c = __shfl_sync(kAll, b, 31 - lane);
            a = sorted32(a > c ? a : c);
        }
        __syncwarp();
        if (lane < n) buf[lane] = a;
        const Key last = __shfl_sync(kAll, a, n - 1);
        if (count >= n) {
            least = last;
            count = n;
        }
        __syncwarp();
    }
    // One key of each lane that has one (`take`), none below `least` and none seen before.
    __device__ __forceinline__ void add(Key k, bool take) {
        uint32_t mask = __ballot_sync(kAll, take);
        if (mask == 0) return;
        if (count + __popc(mask) > 64) {
            cut();
            take = take && k > least;
            mask = __ballot_sync(kAll, take);
        }
        const int lane = threadIdx.x & 31;
        if (take) buf[count + __popc(mask & ((1u << lane) - 1u))] = k;
        count += __popc(mask);
    }
};

constexpr int kRowWarps = 4, kRowThreads = kRowWarps * 32;

struct RowArgs {
    const void *logits;
    long long stride;          // elements
    const float *scores;
    const uint8_t *done;
    int rows, V, n, runs;      // runs of a row, `batches` batches each
    int batches;
    Key *keys;                 // [rows][runs][kRowWarps n]: the run's n best among them, then 0
    unsigned long long *sums;  // [rows][runs], of exp(x - top), in units of 1 / kOne; kNanSum
    float *tops;               // the run's largest number
};
// Sums over threads are integers, so that their order does not matter.
constexpr float kOne = 0x1p40f;
constexpr unsigned long long kNanSum = ~0ull;

// 16 bytes of logits as they lie in memory.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static constexpr uint32_t kHidden = 0xff80ff80u;     // -infinity
    __device__ static __forceinline__ float at(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    __device__ static __forceinline__ float get(const uint32_t (&w)[4], int i) {
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ static __forceinline__ uint32_t element(const __nv_bfloat16 *p) {
        return *reinterpret_cast<const uint16_t *>(p);
    }
    // the largest of a vector, two numbers of which one is it; of two of these; as a number
    using Top = __nv_bfloat162;
    __device__ static __forceinline__ Top top(const uint32_t (&w)[4]) {
        const Top *b = reinterpret_cast<const Top *>(w);
        return __hmax2(__hmax2(b[0], b[1]), __hmax2(b[2], b[3]));
    }
    __device__ static __forceinline__ Top larger(Top a, Top b) { return __hmax2(a, b); }
    __device__ static __forceinline__ float number(Top t) {
        return fmaxf(__low2float(t), __high2float(t));
    }
    // whether one of the two reaches `bound`, a bf16 number
    __device__ static __forceinline__ bool reaches(Top t, float bound) {
        uint32_t r;
        asm("{\n\t.reg .pred p, q;\n\tsetp.ge.bf16x2 p|q, %1, %2;\n\tor.pred p, p, q;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(r)
            : "r"(*reinterpret_cast<const uint32_t *>(&t)),
              "r"(__byte_perm(__float_as_uint(bound), 0, 0x3232)));
        return r != 0;
    }
};
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static constexpr uint32_t kHidden = 0xff800000u;
    __device__ static __forceinline__ float at(const float *p) { return *p; }
    __device__ static __forceinline__ float get(const uint32_t (&w)[4], int i) {
        return __uint_as_float(w[i]);
    }
    __device__ static __forceinline__ uint32_t element(const float *p) {
        return *reinterpret_cast<const uint32_t *>(p);
    }
    using Top = float;
    __device__ static __forceinline__ Top top(const uint32_t (&w)[4]) {
        return fmaxf(fmaxf(get(w, 0), get(w, 1)), fmaxf(get(w, 2), get(w, 3)));
    }
    __device__ static __forceinline__ Top larger(Top a, Top b) { return fmaxf(a, b); }
    __device__ static __forceinline__ float number(Top t) { return t; }
    __device__ static __forceinline__ bool reaches(Top t, float bound) { return t >= bound; }
};

// The 16 bytes that hold elements [i, i + kN) of a row, whose address is a multiple of 16;
// elements outside [0, V) become -infinity and are not read.
template <typename T>
__device__ __forceinline__ void load_whole(const T *row, int i, int V, uint32_t (&w)[4]) {
    uint4 x = make_uint4(Vec<T>::kHidden, Vec<T>::kHidden, Vec<T>::kHidden, Vec<T>::kHidden);
    if (i >= 0 && i + Vec<T>::kN <= V) x = __ldg(reinterpret_cast<const uint4 *>(row + i));
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
}
// The same where an end of the row lies among them: one by one, into what load_whole left.
template <typename T>
__device__ __noinline__ uint4 load_ends(const T *row, int i, int V) {
    using X = Vec<T>;
    uint32_t w[4] = {X::kHidden, X::kHidden, X::kHidden, X::kHidden};
#pragma unroll
    for (int e = 0; e < X::kN; ++e) {
        if (i + e < 0 || i + e >= V) continue;
        const uint32_t x = X::element(row + i + e);
        if constexpr (X::kN == 4) w[e] = x;
        else w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | x << 16 : (w[e / 2] & 0xffff0000u) | x;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void mend_ends(const T *row, int i, int V, uint32_t (&w)[4]) {
    constexpr int kN = Vec<T>::kN;
    if ((i < 0 && i + kN > 0) || (i < V && i + kN > V)) {
        const uint4 x = load_ends(row, i, V);
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    }
}

// Bytes [shift, shift + 16) of the 32 bytes a, b (shift below 16, the same in every lane).
__device__ __forceinline__ void shifted(const uint32_t (&a)[4], const uint32_t (&b)[4], int shift,
                                        uint32_t (&w)[4]) {
    uint32_t x[7];
    const bool two = shift & 8, one = shift & 4;
    uint32_t y[6];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = a[k];
#pragma unroll
    for (int k = 0; k < 3; ++k) x[4 + k] = b[k];
    // (words 0 .. 5 from word 0 or 2; word 7 is needed only for a shift of 12 and more)
#pragma unroll
    for (int k = 0; k < 6; ++k) y[k] = two ? (k + 2 < 7 ? x[k + 2] : b[3]) : x[k];
    uint32_t z[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) z[k] = one ? y[k + 1] : y[k];
    const int bits = 8 * (shift & 3);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(z[k], z[k + 1], bits);
}

__device__ __forceinline__ uint64_t pack64(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack64(uint64_t x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// sum2 += 2^(x kLog2e - base), two sums.  The product is not rounded before the difference, so
// terms that matter, whose exponents are near 0, have their 24 bits; what base is off from
// top kLog2e by is made up for at the end.
template <typename T>
__device__ __forceinline__ void add_exponentials(const uint32_t (&w)[4], float base,
                                                 uint64_t (&sum2)[2]) {
    using X = Vec<T>;
    const uint64_t less = pack64(-base, -base), log2e = pack64(kLog2e, kLog2e);
#pragma unroll
    for (int e = 0; e < X::kN; e += 2) {
        float t0, t1;
        unpack64(fma_f32x2(pack64(X::get(w, e), X::get(w, e + 1)), log2e, less), t0, t1);
        sum2[(e >> 1) & 1] = add_f32x2(sum2[(e >> 1) & 1], pack64(ex2(t0), ex2(t1)));
    }
}
// Where base = top kLog2e is rounded, every term is off by 2^r, r up to half a step of base.  Below
// kFar r is at most 2^-11, and 1 - r ln 2 makes up for it to 2^-24.  Further out (a vocabulary
// masked with -1e10, say) only a sum of exp(x - top), top taken off first, is right.
constexpr float kFar = 1e4f;
// So base stops here, where a thread's top is that far down: its terms become 0, not infinite.
constexpr float kLeastBase = -16384.f;
static_assert(kLeastBase < -kFar * kLog2e, "numbers that are not far have their own base");
// log2 of what a thread's sum is at least divided by where it does not count any more (of 2^8 terms,
// in units of 1 / kOne).
constexpr float kApart = 64.f;
// A thread's sum of exp(x - top) over its vectors i, i + step, ..., in the plainest form.
template <typename T>
__device__ __noinline__ float far_sum(const T *row, int i, int step, int end, float top) {
    float sum = 0.f;
    for (; i < end; i += step)
        for (int e = 0; e < Vec<T>::kN && i + e < end; ++e)
            sum += ex2((Vec<T>::at(row + i + e) - top) * kLog2e);
    return sum;
}

constexpr int kBatch = 4;                             // vectors of a thread in flight
constexpr int kMostBatches = 8;
constexpr int kMostV = 1 << 22;                      // (a row's sum stays below 2^63 / kOne)

// A batch of a row that begins `shift` bytes behind an address that is a multiple of 16, vectors
// at i, i + step, ...; -infinity behind its end.
template <typename T>
__device__ __forceinline__ void load_any(const T *row, int i, int step, int V, int shift,
                                         uint32_t (&w)[kBatch][4]) {
    constexpr int kN = Vec<T>::kN;
    i -= shift / (int)sizeof(T);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) load_whole(row, i + j * step, V, w[j]);
    if (shift == 0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mend_ends(row, i + j * step, V, w[j]);
        return;
    }
    uint32_t b[kBatch][4];                    // (a vector lies in two pieces of 16 bytes)
#pragma unroll
    for (int j = 0; j < kBatch; ++j) load_whole(row, i + j * step + kN, V, b[j]);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
        mend_ends(row, i + j * step, V, w[j]);
        mend_ends(row, i + j * step + kN, V, b[j]);
        shifted(w[j], b[j], shift, w[j]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 8) k_beam_rows(const RowArgs a) {
    using X = Vec<T>;
    using Top = typename X::Top;
    constexpr int kStep = kRowThreads * X::kN;        // elements from a thread's vector to its next
    constexpr int kMostKept = kMostBatches * kBatch / 2;
    __shared__ Key buffers[kRowWarps][64];
    // what a thread keeps: the largest numbers of two vectors each
    __shared__ Top kept[kMostKept][kRowThreads];
    __shared__ uint16_t pairs[kRowWarps][32 * kMostKept];
    __shared__ uint32_t warp_bound[kRowWarps], warp_top[kRowWarps];
    __shared__ unsigned long long warp_sum[kRowWarps];
    __shared__ int warp_count[kRowWarps];
    ptx::griddep_wait();          // (launched while the kernel before it in the stream ends)
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.x, run = blockIdx.y;
    // the run: from run0 on, `there` numbers
    const int run0 = run * a.batches * (kBatch * kStep);
    const int there = min(a.V - run0, a.batches * (kBatch * kStep));
    const T *row = static_cast<const T *>(a.logits) + (long long)r * a.stride;
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15);    // bytes
    // batches that hold anything, and the first ones of them that can be loaded as they are
    const int batches = (there + kBatch * kStep - 1) / (kBatch * kStep);
    const int plain = shift ? 0 : there / (kBatch * kStep);
    const long long job = (long long)r * a.runs + run;

    float top = -INFINITY, base = 0.f;
    uint64_t sum2[2] = {};
    // A batch: the same steps wherever it is loaded from, so that equal rows have equal sums.
    auto add = [&](const uint32_t (&w)[kBatch][4], int b) {
        Top t;
#pragma unroll
        for (int j = 0; j < kBatch; j += 2) {
            const Top two = X::larger(X::top(w[j]), X::top(w[j + 1]));
            kept[(b * kBatch + j) / 2][threadIdx.x] = two;
            t = j == 0 ? two : X::larger(t, two);
        }
        const float most = X::number(t);
        if (most > top) {
            // (what lies far off is put right below, but a NaN is never lost)
            const float to = fmaxf(most * kLog2e, kLeastBase), f = top == -INFINITY ? 1.f : ex2(base - to);
            sum2[0] = mul_f32x2(sum2[0], pack64(f, f));
            sum2[1] = mul_f32x2(sum2[1], pack64(f, f));
            top = most;
            base = to;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) add_exponentials<T>(w[j], base, sum2);
    };
    const T *from = row + run0 + threadIdx.x * X::kN;
    uint32_t next[kBatch][4];
    auto load = [&]() {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(from + j * kStep));
            next[j][0] = x.x; next[j][1] = x.y; next[j][2] = x.z; next[j][3] = x.w;
        }
        from += kBatch * kStep;
    };
    // (A dead or finished beam's first batch is loaded too: nothing reads its lists or sum, but
    // to wait for that look-up first took 64 x 8 beams of 128256 2 us of 47 more.)
    if (plain > 0) load();
    if ((a.done && a.done[r]) || a.scores[r] == -INFINITY) return;
    if (plain > 0) {
#pragma unroll 2
        for (int b = 0; b < plain; ++b) {
            uint32_t w[kBatch][4];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) w[j][q] = next[j][q];
            if (b + 1 < plain) load();
            add(w, b);
        }
    }
#pragma unroll 1
    for (int b = plain; b < batches; ++b) {
        uint32_t w[kBatch][4];
        load_any<T>(row, run0 + (int)threadIdx.x * X::kN + b * (kBatch * kStep), kStep, a.V, shift, w);
        add(w, b);
    }
    // A number that n of the run reach: the k-th largest thread's of every warp is reached by k.
    const uint32_t mine = order_of(top);
    uint32_t left = mine, bound = 0;
    for (int k = 0; k < a.n; k += kRowWarps) {
        bound = __reduce_max_sync(kAll, left);
        if (k == 0 && lane == 0) warp_top[warp] = bound;
        if (lane == __ffs(__ballot_sync(kAll, left == bound)) - 1) left = 0;
    }
    if (lane == 0) warp_bound[warp] = bound;
    __syncthreads();
    const uint32_t run_top = __reduce_max_sync(kAll, warp_top[lane & (kRowWarps - 1)]);
    bound = __reduce_min_sync(kAll, warp_bound[lane & (kRowWarps - 1)]);
    const float all = number_of(run_top);

    // A thread with numbers that are far down alone, next to others in the run: its sum does not
    // count.  (It is 0, or NaN; above 0 it may be infinite, and is always formed again.)  So 512
    // rows of 128256, 99 % of them masked, take what unmasked ones do; with every such thread's
    // numbers read again they took 41 us more.
    if (fabsf(top) > kFar && top != -INFINITY) {
        base = 0.f;
        if (top > 0.f || (all - top) * kLog2e < kApart) {
            sum2[0] = pack64(far_sum<T>(row, run0 + (int)threadIdx.x * X::kN, kStep, run0 + there, top), 0.f);
            sum2[1] = 0;
        }
    }

    // the pairs of vectors that reach the bound ...
    int count = 0;
    {
        const float least = number_of(bound);
        uint32_t reach = 0;
#pragma unroll
        for (int j = 0; j < kMostKept; ++j)
            if (j < batches * (kBatch / 2))
                reach |= X::reaches(kept[j][threadIdx.x], least) ? 1u << j : 0u;
        for (;;) {
            const uint32_t mask = __ballot_sync(kAll, reach != 0);
            if (mask == 0) break;
            if (reach) {
                const int j = __ffs(reach) - 1;
                pairs[warp][count + __popc(mask & ((1u << lane) - 1u))] = (uint16_t)(j * 32 + lane);
                reach &= reach - 1;
            }
            count += __popc(mask);
        }
        count *= 2 * X::kN;
    }
    __syncwarp();
    // ... and their numbers, kAhead loads of a lane together
    constexpr int kAhead = 4;
    int index[kAhead];
    float number[kAhead];
    bool in[kAhead];
    auto look = [&](int q0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int q = q0 + 32 * k + lane, v = q < count ? pairs[warp][q / (2 * X::kN)] : 0;
            const int vec = (v >> 5) * 2 + q / X::kN % 2;
            index[k] = run0 + vec * kStep + (warp * 32 + (v & 31)) * X::kN + q % X::kN;
            in[k] = q < count && index[k] < run0 + there;
            number[k] = in[k] ? X::at(row + index[k]) : 0.f;
        }
    };
    look(0);

    // (meanwhile) the sum, over exp(the run's largest number)
    {
        float s[4];
        unpack64(sum2[0], s[0], s[1]);
        unpack64(sum2[1], s[2], s[3]);
        float sum = (s[0] + s[1]) + (s[2] + s[3]);
        if (base != 0.f) sum = fmaf(sum, fmaf(-top, kLog2e, base) * 0.69314718f, sum);
        if (top != all) sum *= ex2((top - all) * kLog2e);
        const bool nan = __any_sync(kAll, isnan(sum));
        // (a thread's is below 2^9 kOne; summed in two parts that stay below 2^32)
        const unsigned long long x = __float2ull_rn(sum * kOne);
        const uint32_t lo = __reduce_add_sync(kAll, (uint32_t)x & 0xffffffu);
        const uint32_t hi = __reduce_add_sync(kAll, (uint32_t)(x >> 24));
        if (lane == 0) warp_sum[warp] = nan ? kNanSum : ((unsigned long long)hi << 24) + lo;
    }

    Best best{buffers[warp], (Key)bound << 32, 0, a.n};
    for (int q0 = 0;;) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const Key y = key_of(order_of(number[k]), (uint32_t)index[k]);
            best.add(y, in[k] && y >= best.least);
        }
        q0 += 32 * kAhead;
        if (q0 >= count) break;
        look(q0);
    }
    if (best.count > a.n) best.cut();
    if (lane == 0) warp_count[warp] = best.count;
    __syncthreads();
    const int c = lane < kRowWarps ? warp_count[lane] : 0;
    const int before = __reduce_add_sync(kAll, lane < warp ? c : 0), kept_all = __reduce_add_sync(kAll, c);
    Key *keys = a.keys + job * (kRowWarps * a.n);
    if (lane < best.count) keys[before + lane] = best.buf[lane];
    for (int i = kept_all + threadIdx.x; i < kRowWarps * a.n; i += kRowThreads) keys[i] = 0;
    if (warp == 0) {
        unsigned long long sum = lane < kRowWarps ? warp_sum[lane] : 0;
        const bool nan = __any_sync(kAll, sum == kNanSum);
#pragma unroll
        for (int o = kRowWarps / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            a.sums[job] = nan ? kNanSum : sum;
            a.tops[job] = number_of(run_top);
        }
    }
}

struct PickArgs {
    RowArgs rows;
    int W, eos;
    float *out_scores;
    int32_t *out_beam, *out_token;
};

// A CTA a group, a warp a beam (four at least), and one more for the logarithms of their sums
// (31 beams at most: a block has 32 warps).
__host__ __device__ constexpr bool has_log_warp(int W) { return W < kMaxBeams; }
__host__ __device__ constexpr int pick_warps(int W) {
    return (W < 4 ? 4 : W) + (has_log_warp(W) ? 1 : 0);
}
// Named barrier 1, on which the beams' warps only arrive.
__device__ __forceinline__ void sums_written(int warps) {
    asm volatile("bar.arrive 1, %0;" ::"r"(32 * warps) : "memory");
}
__device__ __forceinline__ void sums_awaited(int warps) {
    asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory");
}

__global__ void __launch_bounds__(kMaxBeams * 32) k_beam_pick(const PickArgs a) {
    constexpr int kMost = kMaxBeams * kMaxBest;
    // (keys are done with when candidates are written)
    __shared__ union {
        Key buffers[kMaxBeams][64];
        struct {
            unsigned long long order[kMost], id[kMost];     // of the scores; beam and token
        } all;
    } sh;
    __shared__ Two row_log[kMaxBeams];
    __shared__ unsigned long long row_sum[kMaxBeams], kth[kMaxBeams], nth[kMaxBeams];
    __shared__ int row_count[kMaxBeams];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, n = a.rows.n, V = a.rows.V;
    const int runs = a.rows.runs;
    const bool beam = w < a.W;
    const long long r = (long long)blockIdx.x * a.W + w;
    const float score = beam ? a.rows.scores[r] : -INFINITY;
    const bool dead = score == -INFINITY, done = beam && a.rows.done && a.rows.done[r];
    // Logarithms of the rows' sums, a row a lane of one warp: fp64 instructions are few here and
    // take long, so they run beside the other warps' search.
    const bool log_warp = has_log_warp(a.W) ? w == (int)(blockDim.x >> 5) - 1 : w == 0;
    auto logarithms = [&]() {
        if (lane >= a.W) return;
        const double x = log((double)row_sum[lane] * (1.0 / kOne));
        const float hi = (float)x;
        row_log[lane] = Two{hi, (float)(x - (double)hi)};
    };
    ptx::griddep_wait();

    // the row's n best, one a lane, and its sum
    uint32_t tok = kAll;             // none
    float x = -INFINITY, top = -INFINITY;
    bool nan = false;
    if (has_log_warp(a.W) && log_warp) {
        sums_awaited(a.W + 1);
        logarithms();
    }
    if (!beam) {
    } else if (dead || done) {
        if (lane == 0) row_sum[w] = (unsigned long long)kOne;
        __syncwarp();
        if (has_log_warp(a.W)) sums_written(a.W + 1);
    }
    if (!beam) {
    } else if (dead) {
        if (lane < n && lane < V) tok = lane;
    } else if (done) {
        // `eos` first, then the lowest tokens that it is not
        if (lane == 0) tok = a.eos;
        else if (lane < n && lane < V) tok = lane - 1 < a.eos ? lane - 1 : lane;
    } else {
        const long long job = r * runs;
        uint32_t most = 0;
        const float first_top = lane < runs ? a.rows.tops[job + lane] : -INFINITY;
        const unsigned long long first_sum = lane < runs ? a.rows.sums[job + lane] : 0;
        for (int i = lane; i < runs; i += 32)
            most = max(most, order_of(i < 32 ? first_top : a.rows.tops[job + i]));
        top = number_of(__reduce_max_sync(kAll, most));
        unsigned long long sum = 0;
        for (int i = lane; i < runs; i += 32) {
            const unsigned long long s = i < 32 ? first_sum : a.rows.sums[job + i];
            const float t = i < 32 ? first_top : a.rows.tops[job + i];
            nan |= s == kNanSum;
            sum += t == top ? s : (unsigned long long)((float)s * ex2((t - top) * kLog2e));
        }
        nan = __any_sync(kAll, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) row_sum[w] = sum;
        __syncwarp();
        if (has_log_warp(a.W)) sums_written(a.W + 1);
        if (nan) {
            if (lane < n && lane < V) tok = lane;
        } else {
            // keys of all runs, by a bound that n of them reach
            Best best{sh.buffers[w], 1, 0, n};             // (0 is no key)
            const Key *keys = a.rows.keys + job * (kRowWarps * n);
            const int total = runs * kRowWarps * n;
            constexpr int kHeld = 8;
            Key y[kHeld];                                  // (all of them, for a few runs)
            uint32_t lane_most = 0;
            auto get = [&](int k0) {
#pragma unroll
                for (int q = 0; q < kHeld; ++q) {
                    const int k = k0 + 32 * q + lane;
                    y[q] = k < total ? keys[k] : 0;
                }
            };
            for (int k0 = 0; k0 < total; k0 += 32 * kHeld) {
                get(k0);
#pragma unroll
                for (int q = 0; q < kHeld; ++q) lane_most = max(lane_most, (uint32_t)(y[q] >> 32));
            }
            best.least = max(1ull, (Key)nth32(lane_most, n) << 32);
            for (int k0 = 0; k0 < total; k0 += 32 * kHeld) {
                if (total > 32 * kHeld) get(k0);
#pragma unroll
                for (int q = 0; q < kHeld; ++q) best.add(y[q], y[q] >= best.least);
            }
            best.cut();
            if (lane < best.count && lane < n) {
                const Key y = best.buf[lane];
                tok = index_of(y);
                x = number_of((uint32_t)(y >> 32));
            }
        }
    }
    __syncthreads();
    if (!has_log_warp(a.W)) {
        if (log_warp) logarithms();
        __syncthreads();
    }
    Two val{-INFINITY, 0.f};
    if (done && !dead) {
        if (lane == 0) val.hi = score;
    } else if (nan) {
        val.hi = NAN;
    } else if (!dead && x != -INFINITY) {
        const Two l = row_log[w];
        val = add(add(sum_of(x, -top), Two{-l.hi, -l.lo}), Two{score, 0.f});
    }
    // (The lanes' logits fall, but their sums' roundings may turn two neighbours around: such a
    // sum counts as the one before it, so that a beam's k-th is the least of its first k.)
    unsigned long long mine = tok == kAll ? 0 : order_of(val);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) mine = min(mine, __shfl_up_sync(kAll, mine, o));

    // Candidates that can be among the n best: the k-th of every beam is reached by W k, and the
    // n-th of any by n.
    const int k = (n + a.W - 1) / a.W;
    if (beam && lane == k - 1) kth[w] = mine;
    if (beam && lane == n - 1) nth[w] = mine;
    __syncthreads();
    unsigned long long bound = ~0ull, high = 0;
    for (int i = 0; i < a.W; ++i) {
        bound = min(bound, kth[i]);
        high = max(high, nth[i]);
    }
    bound = max(bound, high);
    const bool in = tok != kAll && mine >= bound;
    const uint32_t mask = __ballot_sync(kAll, in);
    if (beam && lane == 0) row_count[w] = __popc(mask);
    __syncthreads();
    const int c = lane < a.W ? row_count[lane] : 0;
    const int total = __reduce_add_sync(kAll, c), before = __reduce_add_sync(kAll, lane < w ? c : 0);
    if (in) {
        const int at = before + __popc(mask & ((1u << lane) - 1u));
        sh.all.order[at] = mine;
        sh.all.id[at] = (unsigned long long)w << 32 | tok;
    }
    __syncthreads();
    // each one's rank, by eight threads
    const int each = blockDim.x / 8, part = threadIdx.x & 7;
    for (int c0 = 0; c0 < total; c0 += each) {
        const int i = c0 + threadIdx.x / 8;
        const unsigned long long o = i < total ? sh.all.order[i] : 0, id = i < total ? sh.all.id[i] : 0;
        int rank = 0;
        for (int q = part; q < total; q += 8) {
            const unsigned long long y = sh.all.order[q];
            rank += y > o || (y == o && sh.all.id[q] < id);
        }
        rank += __shfl_xor_sync(kAll, rank, 1);
        rank += __shfl_xor_sync(kAll, rank, 2);
        rank += __shfl_xor_sync(kAll, rank, 4);
        if (part == 0 && i < total && rank < n) {
            const long long at = (long long)blockIdx.x * n + rank;
            a.out_scores[at] = number_of(o);
            a.out_beam[at] = (int32_t)(id >> 32);
            a.out_token[at] = (int32_t)(uint32_t)id;
        }
    }
}

template <typename T>
gdn_status select(PickArgs a, int B, cudaStream_t st) {
    RowArgs &r = a.rows;
    // Batches of a run, by the time that they take, in batches: a CTA's, and two for its end, as
    // often as the CTAs that fit the GPU (8 an SM) are filled, and for a row's second kernel n / 14
    // for every run.  (8, 4, 2 and 1 of them, a call's GPU time in us: 512 rows of 128256 with
    // n = 16 41, 45, 56 and 79; 64 rows 12, 13, 14 and 20; 40 rows of 50257 with n = 5 12.6, 10.6,
    // 9.8 and 10.2; 4 rows of 32000 in fp32 with n = 4 8.4, 7.9, 7.8 and 7.4.)
    constexpr int kEach = kRowThreads * Vec<T>::kN * kBatch;
    const int all = (r.V + kEach - 1) / kEach;
    double least = 0.0;
    for (int b = kMostBatches; b >= 1; --b) {
        const int runs = (all + b - 1) / b;
        const double waves = ceil((double)r.rows * runs / (152 * 8));
        const double cost = waves * ((all + runs - 1) / runs + 2) + runs * r.n / 14.0;
        if (b == kMostBatches || cost < least) {
            least = cost;
            r.runs = runs;
        }
    }
    r.batches = (all + r.runs - 1) / r.runs;
    r.runs = (all + r.batches - 1) / r.batches;
    const long long jobs = (long long)r.rows * r.runs;
    if (r.runs > 65535 || jobs > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    void *scratch = nullptr;
    const size_t list = (size_t)kRowWarps * r.n;
    if (scratch_alloc(&scratch, jobs * (8 * list + 12), st) != cudaSuccess) return GDN_ERR_CUDA;
    r.keys = static_cast<Key *>(scratch);
    r.sums = r.keys + jobs * list;
    r.tops = reinterpret_cast<float *>(r.sums + jobs);
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(r.rows, r.runs);
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int slot = timer_begin(st, "k_beam_rows");
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_beam_rows<T>, r);
    timer_end(slot, st);
    count_launch();
    if (e == cudaSuccess) {
        cfg.gridDim = dim3(B);
        cfg.blockDim = dim3(32 * pick_warps(a.W));
        count_launch();
        e = cudaLaunchKernelEx(&cfg, k_beam_pick, a);
    }
    const cudaError_t f = scratch_free(scratch, st);
    return e == cudaSuccess && f == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// ------------------------------------------------------------------ reordering

constexpr int kMoveThreads = 256;
constexpr int kMostGroups = 2048;          // of a launch
constexpr int kMostPools = 64;
constexpr int kFly = 4;                    // 16-byte pieces of a thread in flight
constexpr int kPiece = kMoveThreads * 16 * kFly;

struct Pool {
    uint8_t *data;
    long long bytes;
    int count;
    int first;                 // piece of a moved beam that is this pool's first
};
struct MoveArgs {
    const int32_t *parent, *slots;
    int32_t *slots_out;        // nullptr: a launch that only copies
    int B, W, lanes;
    int n_pools, n_states;     // states first, then caches
    int pieces;                // of a moved beam
    gdn_beam_tables t;         // page_table nullptr: none
    int page_shift;
    int *err;
    Pool pools[kMostPools];
};

// What a warp knows of a group, a beam a lane (lanes from W on: nothing).
struct Group {
    int parent;                // the beam's parent
    uint32_t twins;            // beams whose parent goes on in an earlier one
    uint32_t childless;        // beams from which none goes on
    bool ok;

    __device__ static __forceinline__ int load(const MoveArgs &a, int b) {
        const int lane = threadIdx.x & 31;
        return lane < a.W && b < a.B ? __ldg(a.parent + (long long)b * a.W + lane) : lane;
    }
    __device__ __forceinline__ void get(const MoveArgs &a, int b) { set(a, load(a, b)); }
    __device__ __forceinline__ void set(const MoveArgs &a, int p) {
        const int lane = threadIdx.x & 31;
        const uint32_t beams = a.W == 32 ? kAll : (1u << a.W) - 1u;
        parent = p;
        const bool bad = lane < a.W && (unsigned)parent >= (unsigned)a.W;
        ok = __ballot_sync(kAll, bad) == 0;
        if (!ok) parent = lane;                    // (they stay where they are)
        const uint32_t same = __match_any_sync(kAll, parent);
        twins = __ballot_sync(kAll, lane < a.W && (same & ((1u << lane) - 1u)) != 0);
        childless = beams & ~__reduce_or_sync(kAll, lane < a.W ? 1u << parent : 0u);
    }
    // The beam whose lane the twin `w` takes: as many childless ones before it as twins.
    __device__ __forceinline__ int takes(int w) const {
        return __fns(childless, 0, __popc(twins & ((1u << w) - 1u)) + 1);
    }
};

__global__ void __launch_bounds__(kMoveThreads) k_beam_move(const __grid_constant__ MoveArgs a) {
    __shared__ int before[kMostGroups + 1];        // beams that move in the groups before
    __shared__ int warp_sum[kMoveThreads / 32];
    __shared__ long long copy[2];                  // of the piece at work: from, to (-1: nothing)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kMoveThreads / 32;

    constexpr int kAhead = 4;                      // groups whose parents are loaded together
    for (int b0 = warp; b0 < a.B; b0 += kWarps * kAhead) {
        int parent[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) parent[k] = Group::load(a, b0 + k * kWarps);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int b = b0 + k * kWarps;
            if (b >= a.B) break;
            Group g;
            g.set(a, parent[k]);
            if (lane == 0) {
                before[b + 1] = __popc(g.twins);
                if (!g.ok) atomicCAS(a.err, 0, kErrBadIndex);
            }
        }
    }
    if (threadIdx.x == 0) before[0] = 0;
    __syncthreads();
    // sums over the groups, a run of them a thread
    {
        const int share = (a.B + kMoveThreads - 1) / kMoveThreads;
        const int lo = min(a.B, (int)threadIdx.x * share), hi = min(a.B, lo + share);
        int own = 0;
        for (int b = lo; b < hi; ++b) own += before[b + 1];
        int x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sum[warp] = x;
        __syncthreads();
        int at = x - own;
        for (int i = 0; i < warp; ++i) at += warp_sum[i];
        for (int b = lo; b < hi; ++b) {
            at += before[b + 1];
            before[b + 1] = at;
        }
        __syncthreads();
    }

    // lanes and page tables, a warp a beam
    if (a.slots_out) {
        const long long beams = (long long)a.B * a.W;
        for (long long i = (long long)blockIdx.x * kWarps + warp; i < beams; i += (long long)gridDim.x * kWarps) {
            const int b = (int)(i / a.W), w = (int)(i - (long long)b * a.W);
            Group g;
            g.get(a, b);
            const bool twin = (g.twins >> w) & 1;
            const int p = __shfl_sync(kAll, g.parent, w);
            const int slot = __ldg(a.slots + (long long)b * a.W + (twin ? g.takes(w) : p));
            const bool in = (unsigned)slot < (unsigned)a.lanes;
            if (lane == 0) {
                a.slots_out[i] = slot;
                if (!in) atomicCAS(a.err, 0, kErrBadIndex);
            }
            if (!a.t.page_table) continue;
            const int32_t *from = a.t.page_table + ((long long)b * a.W + p) * a.t.table_stride;
            const int32_t *own = a.t.own_pages + (long long)(in ? slot : 0) * a.t.own_stride;
            int32_t *to = a.t.table_out + i * a.t.out_stride;
            const int len = __ldg(a.t.kv_len + (long long)b * a.W + p), len0 = __ldg(a.t.kv_len + i);
            if (lane == 0 && (len != len0 || len < 0 || len > (long long)a.t.max_pages << a.page_shift))
                atomicCAS(a.err, 0, kErrBadIndex);
            const int full = twin && in ? len >> a.page_shift : a.t.max_pages;
            for (int j = lane; j < a.t.max_pages; j += 32) to[j] = __ldg((j < full ? from : own) + j);
        }
    }

    // pieces of what moves
    const long long total = (long long)before[a.B] * a.pieces;
    for (long long item = blockIdx.x; item < total; item += gridDim.x) {
        const int move = (int)(item / a.pieces), piece = (int)(item - (long long)move * a.pieces);
        int p = 0;
        for (int q = a.n_pools; q - p > 1;) {
            const int m = (p + q) >> 1;
            if (a.pools[m].first <= piece) p = m;
            else q = m;
        }
        const Pool &pool = a.pools[p];
        if (warp == 0) {
            int b = 0;
            for (int q = a.B; q - b > 1;) {
                const int m = (b + q) >> 1;
                if (before[m] <= move) b = m;
                else q = m;
            }
            Group g;
            g.get(a, b);
            const int w = __fns(g.twins, 0, move - before[b] + 1);
            const int from_beam = __shfl_sync(kAll, g.parent, w);
            const long long at = (long long)b * a.W;
            int from = __ldg(a.slots + at + from_beam), to = __ldg(a.slots + at + g.takes(w));
            bool bad = (unsigned)from >= (unsigned)a.lanes || (unsigned)to >= (unsigned)a.lanes;
            bool none = false;
            if (p >= a.n_states && !bad) {
                const int len = __ldg(a.t.kv_len + at + from_beam), j = len >> a.page_shift;
                none = (len & ((1 << a.page_shift) - 1)) == 0;      // no page is partly filled
                if (len < 0 || j >= a.t.max_pages) {
                    bad = !none;
                    none = true;
                } else {
                    from = __ldg(a.t.page_table + (at + from_beam) * a.t.table_stride + j);
                    to = __ldg(a.t.own_pages + (long long)to * a.t.own_stride + j);
                }
            }
            if (!none) bad |= (unsigned)from >= (unsigned)pool.count || (unsigned)to >= (unsigned)pool.count;
            if (lane == 0) {
                if (bad) atomicCAS(a.err, 0, kErrBadIndex);
                copy[0] = bad || none || from == to ? -1 : from;
                copy[1] = to;
            }
        }
        __syncthreads();
        if (copy[0] >= 0) {
            const long long at = (long long)(piece - pool.first) * kPiece;
            const long long left = pool.bytes - at;
            const uint8_t *src = pool.data + copy[0] * pool.bytes + at;
            uint8_t *dst = pool.data + copy[1] * pool.bytes + at;
            uint4 x[kFly];
#pragma unroll
            for (int k = 0; k < kFly; ++k) {
                const int o = (k * kMoveThreads + threadIdx.x) * 16;
                if (o < left) x[k] = *reinterpret_cast<const uint4 *>(src + o);
            }
#pragma unroll
            for (int k = 0; k < kFly; ++k) {
                const int o = (k * kMoveThreads + threadIdx.x) * 16;
                if (o < left) *reinterpret_cast<uint4 *>(dst + o) = x[k];
            }
        }
        __syncthreads();
    }
}

gdn_status check_pool(const gdn_beam_pool &p) {
    if (p.bytes < 0 || p.count < 0 || (p.bytes > 0 && p.count > 0 && !p.data)) return GDN_ERR_INVALID_ARG;
    if (p.bytes % 16 || !kv::aligned16(p.data)) return GDN_ERR_ALIGNMENT;
    if (p.bytes / kPiece > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace
}  // namespace beam
}  // namespace gdn

using namespace gdn::beam;

extern "C" gdn_status gdn_beam_select(const void *logits, int64_t stride_row, const float *scores,
                                      const uint8_t *done, int eos, float *out_scores,
                                      int32_t *out_beam, int32_t *out_token, int B, int W, int V,
                                      int n, gdn_dtype dt, void *stream) {
    if (B < 0 || W < 1 || V < 1 || n < 1) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (W > kMaxBeams || n > kMaxBest || V > kMostV || (long long)B * W > (1 << 24))
        return GDN_ERR_UNSUPPORTED;
    if ((long long)W * V < n || (done && (eos < 0 || eos >= V))) return GDN_ERR_INVALID_ARG;
    if (B == 0) return GDN_OK;
    if (!logits || !scores || !out_scores || !out_beam || !out_token) return GDN_ERR_INVALID_ARG;
    const uintptr_t element = dt == GDN_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % element) return GDN_ERR_ALIGNMENT;
    const void *ptrs[] = {scores, out_scores, out_beam, out_token};
    for (const void *p : ptrs)
        if (!gdn::kv::aligned4(p)) return GDN_ERR_ALIGNMENT;
    PickArgs a{};
    a.rows.logits = logits;
    a.rows.stride = stride_row;
    a.rows.scores = scores;
    a.rows.done = done;
    a.rows.rows = B * W;
    a.rows.V = V;
    a.rows.n = n;
    a.W = W;
    a.eos = eos;
    a.out_scores = out_scores;
    a.out_beam = out_beam;
    a.out_token = out_token;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == GDN_BF16 ? select<__nv_bfloat16>(a, B, st) : select<float>(a, B, st);
}

extern "C" gdn_status gdn_beam_reorder(const int32_t *parent, const int32_t *slots,
                                       int32_t *slots_out, int B, int W, int lanes,
                                       const gdn_beam_pool *states, int n_states,
                                       const gdn_beam_tables *tables, const gdn_beam_pool *caches,
                                       int n_caches, void *stream) {
    if (B < 0 || W < 1 || lanes < 1 || n_states < 0 || n_caches < 0) return GDN_ERR_INVALID_ARG;
    if (W > kMaxBeams || B > (1 << 20) || n_states > 4096 || n_caches > 4096 - n_states)
        return GDN_ERR_UNSUPPORTED;
    if ((n_states > 0 && !states) || (n_caches > 0 && (!caches || !tables))) return GDN_ERR_INVALID_ARG;
    gdn_status rc;
    for (int i = 0; i < n_states; ++i) {
        if ((rc = check_pool(states[i])) != GDN_OK) return rc;
        if (states[i].count != lanes) return GDN_ERR_INVALID_ARG;
    }
    for (int i = 0; i < n_caches; ++i)
        if ((rc = check_pool(caches[i])) != GDN_OK) return rc;
    MoveArgs a{};
    if (tables) {
        a.t = *tables;
        if (a.t.max_pages < 1 || a.t.page_size < 1 || (a.t.page_size & (a.t.page_size - 1)))
            return GDN_ERR_INVALID_ARG;
        while ((1 << a.page_shift) < a.t.page_size) ++a.page_shift;
        if ((long long)a.t.max_pages << a.page_shift > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    }
    if (B == 0) return GDN_OK;
    if (!parent || !slots || !slots_out) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {parent, slots, slots_out, a.t.page_table, a.t.table_out, a.t.own_pages, a.t.kv_len};
    for (const void *p : ptrs)
        if (!gdn::kv::aligned4(p)) return GDN_ERR_ALIGNMENT;
    if (tables && (!a.t.page_table || !a.t.table_out || !a.t.own_pages || !a.t.kv_len))
        return GDN_ERR_INVALID_ARG;
    a.W = W;
    a.lanes = lanes;
    a.err = gdn::device_error_word();
    static std::atomic<int> memo[gdn::kMaxDeviceMemo];
    const int resident = gdn::per_device(memo, [&](int dev) {
        int sms = 0, per = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k_beam_move, kMoveThreads, 0) !=
                cudaSuccess)
            return -1;
        return sms * per;
    }, 0);
    if (resident < 1) return GDN_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int n_all = n_states + n_caches;
    for (int b0 = 0; b0 < B; b0 += kMostGroups) {
        const long long beam0 = (long long)b0 * W;
        a.B = B - b0 < kMostGroups ? B - b0 : kMostGroups;
        a.parent = parent + beam0;
        a.slots = slots + beam0;
        if (tables) {
            a.t.page_table = tables->page_table + beam0 * tables->table_stride;
            a.t.table_out = tables->table_out + beam0 * tables->out_stride;
            a.t.kv_len = tables->kv_len + beam0;
        }
        // (one launch at least: the lanes and tables)
        for (int i0 = 0; i0 == 0 || i0 < n_all; i0 += kMostPools) {
            a.slots_out = i0 == 0 ? slots_out + beam0 : nullptr;
            a.n_pools = n_all - i0 < kMostPools ? n_all - i0 : kMostPools;
            a.n_states = n_states - i0 < 0 ? 0 : n_states - i0 < a.n_pools ? n_states - i0 : a.n_pools;
            long long pieces = 0;
            for (int i = 0; i < a.n_pools; ++i) {
                const gdn_beam_pool &p = i0 + i < n_states ? states[i0 + i] : caches[i0 + i - n_states];
                a.pools[i] = Pool{static_cast<uint8_t *>(p.data), (long long)p.bytes, p.count, (int)pieces};
                pieces += (p.bytes + kPiece - 1) / kPiece;
            }
            if (pieces > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
            a.pieces = (int)pieces;
            const long long most = pieces * a.B * (W - 1), rows = ((long long)a.B * W + 7) / 8;
            long long grid = most > rows ? most : rows;
            grid = grid < resident ? (grid < 1 ? 1 : grid) : resident;
            const int slot = gdn::timer_begin(st, "k_beam_move");
            k_beam_move<<<(unsigned)grid, kMoveThreads, 0, st>>>(a);
            gdn::timer_end(slot, st);
            gdn::count_launch();
            if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
        }
    }
    return GDN_OK;
}
