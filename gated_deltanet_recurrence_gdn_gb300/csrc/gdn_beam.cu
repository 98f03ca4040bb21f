// gdn_beam.cu -- beam search over a hybrid decoder (gdn_beam.h): selection over beams
// and vocabulary, and reordering of states and pages.
//
// Selection: score(w, v) = scores[w] + x[w][v] - log sum_u exp(x[w][u]), the n best of a
// group's W V.  Within a row the order is that of the logits, so a row's n best need no
// logarithm, and its logits are read once:
// - k_beam_rows: a warp takes a run of a row, kVecs vectors of 16 bytes a lane, in one pass
//   for the largest number and the sum of exponentials.  What it keeps of a vector is its
//   largest number.  The n-th largest of the 32 lanes' largest numbers is a bound that
//   n numbers of the run reach at least; vectors that reach it are few, and are read again
//   from the caches to find the n best (64-bit keys: the number, then the lower index).
//   Runs are cut by index, not by address, and sums do not depend on where a row starts.
// - k_beam_pick, a CTA a group: a warp a row joins the runs' sums in fp64 and their lists
//   by the same bound, then the W n candidates are ranked by their fp64 scores.
// Reading the logits bounds a large batch, latency of two launches a small one.
//
// Reordering: every CTA finds by itself which beams have to move (a few instructions a
// group, a warp each) and copies its share of 16 KB pieces.  Copying bounds it.
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
// The same of fp64, NaN above everything.
__device__ __forceinline__ unsigned long long order_of(double x) {
    if (isnan(x)) return ~0ull;
    const long long u = __double_as_longlong(x + 0.0);
    return (unsigned long long)u ^ (u < 0 ? ~0ull : 0x8000000000000000ull);
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

// Descending order over a warp of one number a lane.
template <typename U>
__device__ __forceinline__ U sorted32(U x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const U y = __shfl_xor_sync(kAll, x, j);
            const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
            x = larger ? (x > y ? x : y) : (x < y ? x : y);
        }
    return x;
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

struct RowArgs {
    const void *logits;
    long long stride;          // elements
    const float *scores;
    const uint8_t *done;
    int rows, V, n, runs;      // runs of a row
    Key *keys;                 // [rows][runs][n]
    double *sums;              // [rows][runs]
    float *tops;
};

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
    // the largest of eight
    __device__ static __forceinline__ float top(const uint32_t (&w)[4]) {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(w);
        const __nv_bfloat162 m = __hmax2(__hmax2(b[0], b[1]), __hmax2(b[2], b[3]));
        return fmaxf(__low2float(m), __high2float(m));
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
    __device__ static __forceinline__ float top(const uint32_t (&w)[4]) {
        return fmaxf(fmaxf(get(w, 0), get(w, 1)), fmaxf(get(w, 2), get(w, 3)));
    }
};

// The 16 bytes that hold elements [i, i + kN) of a row, whose address is a multiple of 16;
// elements outside [0, V) become -infinity and are not read.
template <typename T>
__device__ __forceinline__ void load_whole(const T *row, long long i, int V, uint32_t (&w)[4]) {
    using X = Vec<T>;
    if (i >= 0 && i + X::kN <= V) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(row + i));
        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = X::kHidden;
#pragma unroll
    for (int e = 0; e < X::kN; ++e) {
        if (i + e < 0 || i + e >= V) continue;
        const uint32_t x = X::element(row + i + e);
        if constexpr (X::kN == 4) w[e] = x;
        else w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | x << 16 : (w[e / 2] & 0xffff0000u) | x;
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

constexpr int kRowWarps = 8;

template <typename T, int kVecs>
__global__ void __launch_bounds__(kRowWarps * 32) k_beam_rows(const RowArgs a) {
    using X = Vec<T>;
    constexpr int kBatch = kVecs < 4 ? kVecs : 4;
    __shared__ Key buffers[kRowWarps][64];
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long job = (long long)blockIdx.x * kRowWarps + warp;
    const int r = (int)(job / a.runs), run = (int)(job - (long long)r * a.runs);
    if (r >= a.rows) return;
    if ((a.done && a.done[r]) || a.scores[r] == -INFINITY) return;     // (nothing reads its lists)
    const T *row = static_cast<const T *>(a.logits) + (long long)r * a.stride;
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15);    // bytes
    const int ahead = shift / (int)sizeof(T);
    const long long i0 = (long long)run * (32 * X::kN * kVecs) + lane * X::kN;

    float top = -INFINITY, tops[kVecs];
    uint64_t sum2[2] = {};
#pragma unroll
    for (int j0 = 0; j0 < kVecs; j0 += kBatch) {
        uint32_t w[kBatch][4];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            load_whole(row, i0 + (j0 + j) * (32 * X::kN) - ahead, a.V, w[j]);
        if (shift) {
            // a vector lies in two pieces of 16 bytes, the second one the next lane's
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                uint32_t b[4], x[4];
                if (lane == 31)
                    load_whole(row, i0 + (j0 + j) * (32 * X::kN) + X::kN - ahead, a.V, x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    b[k] = __shfl_down_sync(kAll, w[j][k], 1);
                    if (lane == 31) b[k] = x[k];
                }
                shifted(w[j], b, shift, x);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[j][k] = x[k];
            }
        }
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            tops[j0 + j] = X::top(w[j]);
            most = fmaxf(most, tops[j0 + j]);
        }
        if (most > top) {
            const float f = ex2((top - most) * kLog2e);
            sum2[0] = mul_f32x2(sum2[0], pack64(f, f));
            sum2[1] = mul_f32x2(sum2[1], pack64(f, f));
            top = most;
        }
        // (x - top is exact where it matters, and right for numbers near fp32's end)
        const float less = top == -INFINITY ? 0.f : -top;
        const uint64_t less2 = pack64(less, less), log2e2 = pack64(kLog2e, kLog2e);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int e = 0; e < X::kN; e += 2) {
                float t0, t1;
                unpack64(mul_f32x2(add_f32x2(pack64(X::get(w[j], e), X::get(w[j], e + 1)), less2),
                                   log2e2), t0, t1);
                sum2[(e >> 1) & 1] = add_f32x2(sum2[(e >> 1) & 1], pack64(ex2(t0), ex2(t1)));
            }
    }

    // the run's largest number and its sum of exponentials
    const uint32_t mine = order_of(top);
    const float all_top = number_of(__reduce_max_sync(kAll, mine));
    {
        float s[4];
        unpack64(sum2[0], s[0], s[1]);
        unpack64(sum2[1], s[2], s[3]);
        const float f = top == all_top ? 1.f : ex2((top - all_top) * kLog2e);
        double sum = ((double)(s[0] + s[1]) + (double)(s[2] + s[3])) * (double)f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (lane == 0) {
            a.tops[job] = all_top;
            a.sums[job] = sum;
        }
    }

    // its n best
    Best best{buffers[warp], 0, 0, a.n};
    best.least = (Key)__shfl_sync(kAll, sorted32(mine), a.n - 1) << 32;
#pragma unroll 1
    for (int j = 0; j < kVecs; ++j) {
        float t = tops[0];
#pragma unroll
        for (int k = 1; k < kVecs; ++k) t = j == k ? tops[k] : t;
        const long long i = i0 + j * (32 * X::kN);
        const bool in = i < a.V && key_of(order_of(t), (uint32_t)i) >= best.least;
        if (!__any_sync(kAll, in)) continue;
        float x[X::kN];
#pragma unroll
        for (int e = 0; e < X::kN; ++e)
            x[e] = in && i + e < a.V ? X::at(row + i + e) : -INFINITY;
#pragma unroll 1
        for (int e = 0; e < X::kN; ++e) {
            float y = x[0];
#pragma unroll
            for (int k = 1; k < X::kN; ++k) y = e == k ? x[k] : y;
            const Key k = key_of(order_of(y), (uint32_t)(i + e));
            best.add(k, in && i + e < a.V && k >= best.least);
        }
    }
    best.cut();
    if (lane < a.n) a.keys[job * a.n + lane] = lane < best.count ? best.buf[lane] : 0;
}

struct PickArgs {
    RowArgs rows;
    int W, eos;
    float *out_scores;
    int32_t *out_beam, *out_token;
};

constexpr int kPickWarps = 16;

__global__ void __launch_bounds__(kPickWarps * 32) k_beam_pick(const PickArgs a) {
    __shared__ Key buffers[kPickWarps][64];
    __shared__ unsigned long long order[kMaxBeams * kMaxBest];   // of the candidates' scores
    __shared__ float value[kMaxBeams * kMaxBest];
    __shared__ uint32_t token[kMaxBeams * kMaxBest];             // kAll: no candidate
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = a.rows.n, V = a.rows.V;
    const int runs = a.rows.runs;
    ptx::griddep_wait();
    for (int w = warp; w < a.W; w += kPickWarps) {
        const long long r = (long long)blockIdx.x * a.W + w;
        const float score = a.rows.scores[r];
        const bool dead = score == -INFINITY, done = a.rows.done && a.rows.done[r];
        double val = -INFINITY;
        uint32_t tok = kAll;
        if (dead) {
            if (lane < n && lane < V) tok = lane;
        } else if (done) {
            // `eos` first, then the lowest tokens that it is not
            if (lane == 0) {
                tok = a.eos;
                val = score;
            } else if (lane < n && lane < V) {
                tok = lane - 1 < a.eos ? lane - 1 : lane;
            }
        } else {
            const float *tops = a.rows.tops + r * runs;
            const double *sums = a.rows.sums + r * runs;
            float top = -INFINITY;
            for (int i = lane; i < runs; i += 32) top = fmaxf(top, tops[i]);
            top = number_of(__reduce_max_sync(kAll, order_of(top)));
            double sum = 0.0;
            for (int i = lane; i < runs; i += 32) {
                const double s = sums[i];
                sum += tops[i] == top ? s : s * exp((double)tops[i] - (double)top);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            if (isnan(sum)) {
                if (lane < n && lane < V) {
                    tok = lane;
                    val = NAN;
                }
            } else {
                const Key *keys = a.rows.keys + r * runs * n;
                const int total = runs * n;
                Best best{buffers[warp], 0, 0, n};
                if (total > 32) {
                    Key most = 0;
                    for (int i = lane; i < total; i += 32) most = max(most, keys[i]);
                    best.least = __shfl_sync(kAll, sorted32(most), n - 1);
                }
                if (best.least == 0) best.least = 1;          // (0 is no key)
                for (int i = 0; i < total; i += 32) {
                    const Key k = i + lane < total ? keys[i + lane] : 0;
                    best.add(k, k >= best.least);
                }
                best.cut();
                if (lane < best.count) {
                    const Key k = best.buf[lane];
                    tok = index_of(k);
                    const float x = number_of((uint32_t)(k >> 32));
                    if (x != -INFINITY) val = (double)score + (((double)x - (double)top) - log(sum));
                }
                __syncwarp();
            }
        }
        if (lane < n) {
            order[w * n + lane] = order_of(val);
            value[w * n + lane] = (float)val;
            token[w * n + lane] = tok;
        }
    }
    __syncthreads();
    // each candidate's rank
    const int total = a.W * n;
    for (int c = threadIdx.x; c < total; c += kPickWarps * 32) {
        const unsigned long long mine = order[c];
        const uint32_t tok = token[c];
        const int w = c / n;
        if (tok == kAll) continue;
        int rank = 0;
        for (int i = 0; i < total; ++i) {
            const unsigned long long o = order[i];
            const uint32_t t = token[i];
            // (a row's candidates follow one another, so beams are in order)
            const bool before = o > mine || (o == mine && (i < w * n || (i < w * n + n && t < tok)));
            rank += t != kAll && before;
        }
        if (rank < n) {
            const long long at = (long long)blockIdx.x * n + rank;
            a.out_scores[at] = value[c];
            a.out_beam[at] = w;
            a.out_token[at] = (int32_t)tok;
        }
    }
}

template <typename T, int kVecs>
cudaError_t launch_rows(const RowArgs &a, cudaStream_t st) {
    const long long jobs = (long long)a.rows * a.runs;
    const int slot = timer_begin(st, "k_beam_rows");
    k_beam_rows<T, kVecs>
        <<<(unsigned)((jobs + kRowWarps - 1) / kRowWarps), kRowWarps * 32, 0, st>>>(a);
    timer_end(slot, st);
    count_launch();
    return cudaGetLastError();
}

template <typename T>
gdn_status select(PickArgs a, int B, cudaStream_t st) {
    RowArgs &r = a.rows;
    // Vectors of a lane: as many as leave some eight warps an SM.
    auto runs_of = [&](int vecs) {
        const long long each = 32ll * Vec<T>::kN * vecs;
        return (int)((r.V + each - 1) / each);
    };
    const int vecs = (long long)r.rows * runs_of(16) >= 152 * 8 ? 16 : 4;
    r.runs = runs_of(vecs);
    const long long jobs = (long long)r.rows * r.runs;
    if (jobs > (1ll << 33)) return GDN_ERR_UNSUPPORTED;
    void *scratch = nullptr;
    if (scratch_alloc(&scratch, (size_t)jobs * (8 * r.n + 12), st) != cudaSuccess) return GDN_ERR_CUDA;
    r.keys = static_cast<Key *>(scratch);
    r.sums = reinterpret_cast<double *>(r.keys + jobs * r.n);
    r.tops = reinterpret_cast<float *>(r.sums + jobs);
    cudaError_t e = vecs == 16 ? launch_rows<T, 16>(r, st) : launch_rows<T, 4>(r, st);
    if (e == cudaSuccess) {
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(B);
        cfg.blockDim = dim3(kPickWarps * 32);
        cfg.stream = st;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
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

    __device__ __forceinline__ void get(const MoveArgs &a, int b) {
        const int lane = threadIdx.x & 31;
        const uint32_t beams = a.W == 32 ? kAll : (1u << a.W) - 1u;
        parent = lane < a.W ? __ldg(a.parent + (long long)b * a.W + lane) : lane;
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

    for (int b = warp; b < a.B; b += kWarps) {
        Group g;
        g.get(a, b);
        if (lane == 0) {
            before[b + 1] = __popc(g.twins);
            if (!g.ok) atomicCAS(a.err, 0, kErrBadIndex);
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
    if (W > kMaxBeams || n > kMaxBest || (long long)B * W > (1 << 24)) return GDN_ERR_UNSUPPORTED;
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
