// gdn_kv8.cu -- the 8-bit paged key/value cache (gdn_attn.h): appending keys and
// values with the rotation applied on the way, and reading them back.
//
// An element is e4m3 * 2^(e - 15), one exponent e for the 16 places of a block of a
// head: the least under which the block's largest magnitude is at most 448.  Powers
// of two lose nothing against other scales (e4m3 is a floating type) and make a
// block's growth exact but for its smallest numbers: when a token does not fit under
// the exponent that its block has, the rows that are there are divided by the same
// power of two.
//
// Append, one launch of two kinds of CTAs:
// - keys and values: 16 units of 16 elements times 16 places, a thread each, so d
//   threads a block and 256 / d blocks a CTA.  They walk over the key heads (turn,
//   largest magnitude of the block, quantise) and the value heads: a warp's maximum is
//   one instruction (magnitudes compare as integers), the warps' maxima go through
//   shared memory.  The threads of places that were there before
//   move their codes when the block's exponent grows; in the middle of a prompt there
//   are none, for a single token they are the other 15 sixteenths.
// - queries: a thread holds a unit of one token with its cosines and sines and walks
//   over the heads.
// Every row is read once: HBM bounds a prompt, the launch a single token.  12 prompts of 700
// to 8192 tokens (59 k tokens, 32 + 8 + 8 heads, d = 128 bf16, 1.32 GB) take 225 us (5.9
// TB/s, 86 % of a copy's rate; keys and values alone 97: their instructions, which in CTAs
// of their own in front of the queries' took 239 in all), reading back 64 us (0.36 GB, of which
// DRAM carries 0.30: half of the codes are still in L2), a token of each of 64 sequences 4.6 us
// and 2.4.
#include "gdn_kv.cuh"

namespace gdn {
namespace kv {
namespace {

using F = Fmt8;
constexpr int kThreads = 256;

// The least exponent byte under which magnitude m is at most 448 = 1.75 * 2^8.
__device__ __forceinline__ int exponent_for(float m) {
    const int e = (int)((__float_as_uint(m) + 0x1fffffu) >> 23) - 120;
    return min(max(e, 0), F::kMostExponent);
}
// 2^(15 - e)
__device__ __forceinline__ float power_of(int e) { return __uint_as_float((142 - e) << 23); }

// Eight numbers times f as codes; all NaN if `nan`.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float f, bool nan) {
    if (nan) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    return make_uint2(
        e4m3x4_of(__fmul_rn(x[0], f), __fmul_rn(x[1], f), __fmul_rn(x[2], f), __fmul_rn(x[3], f)),
        e4m3x4_of(__fmul_rn(x[4], f), __fmul_rn(x[5], f), __fmul_rn(x[6], f), __fmul_rn(x[7], f)));
}

// 2^-by as fp16x2, 0 < by <= 22 (a subnormal number below 2^-14).
__device__ __forceinline__ __half2 down_f16x2(int by) {
    return __half2half2(__ushort_as_half((unsigned short)(by <= 14 ? (15 - by) << 10 : 0x400 >> (by - 14))));
}
// Four codes times 2^-by, rounded once as far as an e4m3 number can tell: a product is exact in
// fp16, or below 2^-20 and becomes 0 either way.
__device__ __forceinline__ uint32_t moved(uint32_t w, __half2 f) {
    uint32_t r[2];
    e4m3x4_f16(w, r);
    const __half2 a = __hmul2(*reinterpret_cast<const __half2 *>(&r[0]), f);
    const __half2 b = __hmul2(*reinterpret_cast<const __half2 *>(&r[1]), f);
    return e4m3x4_of_f16(*reinterpret_cast<const uint32_t *>(&a),
                         *reinterpret_cast<const uint32_t *>(&b));
}

// Blocks of 16 places that the new tokens of a sequence may touch, n > 0 of them.
__host__ __device__ inline int blocks_touched(int n) { return (n + 14) / F::kBlock + 1; }

struct Append {
    int Hq, q_ctas_x, q_heads_per;    // CTAs of queries: tokens, then heads
    long long kv_tasks;               // blocks of keys and values, kv_ctas_x CTAs of them
    int kv_ctas_x, kv_items_per;      // items: key heads, then value heads
    // The two kinds of CTAs in turn, so that the instructions of one run beside the other's
    // waits for memory: one of the `few` in every `stride`, from the grid's first on.
    int few, stride;
    bool few_are_kv;
    bool rotate;

    // This CTA's number among those of its kind.
    __device__ __forceinline__ int number(bool &kv) const {
        const int turn = blockIdx.x / stride, at = blockIdx.x - turn * stride;
        const bool one = at == 0 && turn < few;
        kv = one == few_are_kv;
        return one ? turn : (int)blockIdx.x - min(few, turn + 1);
    }
};

// The block of a task: sequence and how many blocks behind its first.  With offsets the
// tasks of sequence b begin at cu[b] / 16 + 2 b, which leaves room for every block that
// its tokens touch; without, every sequence has the same number.
__device__ __forceinline__ void task_block(const Kv &kv, long long task, int &b, int &behind) {
    if (!kv.cu) {
        const int each = blocks_touched(kv.n_tokens / kv.N);
        b = (int)(task / each);
        behind = (int)(task - (long long)b * each);
        return;
    }
    auto first = [&](int i) { return (long long)(__ldg(kv.cu + i) / F::kBlock) + 2ll * i; };
    int lo = 0, hi = kv.N;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (first(m) <= task) lo = m;
        else hi = m;
    }
    b = lo;
    const long long x = task - first(lo);
    behind = x < 0 ? -1 : (int)min(x, 0x7fffffffll);
}

template <typename T>
__device__ __forceinline__ void append_queries(const Kv &kv, const Append &ap, Rows<const T> q,
                                               Rows<T> qo, const Rotary &rot, int cta, int *err) {
    const int units = kv.d / 16, u = threadIdx.x & (units - 1);
    const int bx = cta % ap.q_ctas_x, by = cta / ap.q_ctas_x;
    const int t = bx * (kThreads / units) + threadIdx.x / units;
    if (t >= kv.n_tokens) return;
    const Unit un = unit_of(rot, u);
    const int h0 = by * ap.q_heads_per, h1 = min(h0 + ap.q_heads_per, ap.Hq);
    Run<T> x, y;
    auto load = [&](int h) {
        if (h >= h1) return;
        const T *p = q.at(0, h, t);
        x.load(p + un.lo);
        y.load(p + un.hi);
    };
    load(h0);
    const bool turned = ap.rotate && un.turned;
    float c[8], s[8];
    if (turned) unit_angles(rot, u, 0, t, c, s, err);
    for (int h = h0; h < h1; ++h) {
        float v[8], w[8];
        x.get(v);
        y.get(w);
        load(h + 1);
        if (turned) turn(rot.adjacent, c, s, v, w);
        T *p = qo.at(0, h, t);
        store8(p + un.lo, v);
        store8(p + un.hi, w);
    }
}

template <typename T, int kMinCtas>
__global__ void __launch_bounds__(kThreads, kMinCtas)
k_kv8_append(const Kv kv, Rows<const T> k, Rows<const T> v, Rows<const T> q, Rows<T> qo,
             const Append ap, const __grid_constant__ Rotary rot, int *err) {
    __shared__ uint32_t warp_most[2][kThreads / 32];
    bool is_kv;
    const int cta = ap.number(is_kv);
    if (!is_kv) {
        append_queries<T>(kv, ap, q, qo, rot, cta, err);
        return;
    }
    const int units = kv.d / 16, psz = kv.page_size();
    const int u = threadIdx.x & (units - 1), place_in = threadIdx.x / units % F::kBlock;
    const int bx = cta % ap.kv_ctas_x, by = cta / ap.kv_ctas_x;
    const int i0 = by * ap.kv_items_per, i1 = min(i0 + ap.kv_items_per, 2 * kv.H);
    const Unit un = unit_of(rot, u);
    const Unit whole{16 * u, 16 * u + 8, false};
    const bool split = un.turned && !rot.adjacent;

    // this thread's place: a new token, or a row that is there already, or neither
    const long long task = (long long)bx * (kThreads / kv.d) + threadIdx.x / kv.d;
    int t = 0, page = -1, row = 0;
    bool fresh = false, old = false, had = false;
    if (task < ap.kv_tasks) {
        int b, behind, first, n, len;
        task_block(kv, task, b, behind);
        kv.tokens(b, first, n, len, err);
        const int start = max(0, len - n), block = start / F::kBlock + behind;
        const int p = block * F::kBlock + place_in;
        // (tokens at places below 0 are not written)
        if (behind >= 0 && n > 0 && block <= (len - 1) / F::kBlock && len > 0) {
            had = block * F::kBlock < start;
            page = kv.page_of(b, block * F::kBlock, err);
            if (!kv.bytes_ok<F>(max(page, 0), 0, F::exponents_at(psz, kv.d, p & (psz - 1)), 16))
                page = -1;
            fresh = page >= 0 && p >= start && p < len;
            old = page >= 0 && p < start;
            t = fresh ? first + (p - (len - n)) : 0;
            row = p & (psz - 1);
        }
    }
    Run<T> x{}, y{};
    auto load = [&](int i) {
        if (!fresh || i >= i1) return;
        const bool key = i < kv.H;
        const T *p = key ? k.at(0, i, t) : v.at(0, i - kv.H, t);
        const Unit &w = key ? un : whole;
        x.load(p + w.lo);
        y.load(p + w.hi);
    };
    load(i0);
    float c[8], s[8];
    const bool turned = ap.rotate && un.turned;
    if (turned && fresh) unit_angles(rot, u, 0, t, c, s, err);
    const int step = F::block_bytes(psz, kv.d);
    uint8_t *base = kv.pages + kv.block<F>(max(page, 0), 0);
    const int code_at = F::code_at(kv.d, row);
    const int exp_at = F::exponents_at(psz, kv.d, row) + F::exponent_of(row);
    const int warp = threadIdx.x / 32, warp0 = threadIdx.x / kv.d * (kv.d / 32);

    for (int i = i0, turn_no = 0; i < i1; ++i, turn_no ^= 1) {
        const bool key = i < kv.H;
        const int h = key ? i : i - kv.H;
        uint8_t *blk = base + (long long)h * step;
        uint8_t *codes = blk + code_at + (key ? 0 : F::code_at(kv.d, psz));
        uint8_t *exponent = blk + exp_at + (key ? 0 : 8);
        float a[8], e[8];
        x.get(a);
        y.get(e);
        load(i + 1);
        // (read before the barrier that the new one is written behind)
        const int was = had && page >= 0 ? *(volatile uint8_t *)exponent : 0;
        if (key && turned && fresh) turn(rot.adjacent, c, s, a, e);
        if (kv.head_scale) {
            const float inv = __frcp_rn(__ldg(kv.head_scale + (key ? 0 : kv.H) + h));
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                a[m] = __fmul_rn(a[m], inv);
                e[m] = __fmul_rn(e[m], inv);
            }
        }
        const float ma = amax8(a), me = amax8(e);
        // a NaN takes its 16 neighbours: of two lanes where the runs are halves of two
        const bool halves = key && split;
        const float oa = __shfl_xor_sync(0xffffffffu, ma, 1);
        const float oe = __shfl_xor_sync(0xffffffffu, me, 1);
        const bool nan_a = isnan(ma) || isnan(halves ? oa : me);
        const bool nan_e = isnan(me) || isnan(halves ? oe : ma);
        uint32_t most = 0;
        if (fresh) {
            if (!nan_a) most = __float_as_uint(ma);
            if (!nan_e) most = max(most, __float_as_uint(me));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if ((threadIdx.x & 31) == 0) warp_most[turn_no][warp] = most;
        __syncthreads();
        if (page < 0) continue;
        for (int w = 0; w < kv.d / 32; ++w) most = max(most, warp_most[turn_no][warp0 + w]);
        const int need = exponent_for(__uint_as_float(most)), now = had ? max(need, was) : need;
        if (place_in == 0 && u == 0) *exponent = (uint8_t)now;
        if (fresh) {
            const float p = power_of(now);
            const uint2 ca = codes_of(a, p, nan_a), ce = codes_of(e, p, nan_e);
            if (halves) {
                *reinterpret_cast<uint2 *>(codes + un.lo) = ca;
                *reinterpret_cast<uint2 *>(codes + un.hi) = ce;
            } else {
                *reinterpret_cast<uint4 *>(codes + whole.lo) = make_uint4(ca.x, ca.y, ce.x, ce.y);
            }
        } else if (old && now > was) {
            uint4 *at = reinterpret_cast<uint4 *>(codes + whole.lo);
            const uint4 w = *at;
            const __half2 p = down_f16x2(now - was);
            *at = make_uint4(moved(w.x, p), moved(w.y, p), moved(w.z, p), moved(w.w, p));
        }
    }
}

// One thread per 16 neighbours of a token's head: 16 bytes and an exponent in, 16 values out.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_kv8_read(const Kv kv, Rows<T> k, Rows<T> v, int heads_per, int *err) {
    const int units = kv.d / 16;
    const int u = threadIdx.x & (units - 1);
    const int t = blockIdx.x * (kThreads / units) + threadIdx.x / units;
    if (t >= kv.n_tokens) return;
    const int b = kv.seq_of(t);
    int first, n, len;
    kv.tokens(b, first, n, len, err);
    const int place = len - n + (t - first);
    int page = -1;
    if (place >= 0 && t >= first && t < first + n) page = kv.page_of(b, place, err);
    const int row = place & (kv.page_size() - 1), psz = kv.page_size();
    const uint8_t *base = kv.pages + kv.block<F>(page >= 0 ? page : 0, 0);
    const int step = F::block_bytes(psz, kv.d);
    const int exp_at = F::exponents_at(psz, kv.d, row) + F::exponent_of(row);
    const int i0 = blockIdx.y * heads_per, i1 = min(i0 + heads_per, 2 * kv.H);
    for (int i = i0; i < i1; ++i) {
        const bool key = i < kv.H;
        const int h = key ? i : i - kv.H;
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
        if (page >= 0) {
            const uint8_t *blk = base + (long long)h * step;
            const uint4 w = *reinterpret_cast<const uint4 *>(
                blk + F::code_at(kv.d, key ? row : psz + row) + 16 * u);
            const float s = exponent_f32(blk[exp_at + (key ? 0 : 8)]);
            const float g = kv.head_scale ? __ldg(kv.head_scale + (key ? 0 : kv.H) + h) : 1.f;
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t r[2];
                e4m3x4_f16(ws[e], r);
                const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&r[0]));
                const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&r[1]));
                float (&z)[8] = e < 2 ? x : y;
                const int at = 4 * (e & 1);
                z[at] = p.x * s * g;
                z[at + 1] = p.y * s * g;
                z[at + 2] = q.x * s * g;
                z[at + 3] = q.y * s * g;
            }
        }
        T *o = key ? k.at(0, h, t) : v.at(0, h, t);
        store8(o + 16 * u, x);
        store8(o + 16 * u + 8, y);
    }
}

// Items that a CTA walks over, so that few columns of CTAs still make `per_sm` CTAs an SM.
// Appending wants 3 (4096 tokens 17.5 us; at 1 an SM 21.7, at 6 19.5, at 16 26.0; 1024 tokens 8.4,
// 8.5, 8.6 and 10.5), reading back 10 (16384 tokens 18.5 us, at 3 20.7, at 24 19.9).
int items_per_cta(long long columns, int items, int per_sm, int least_split) {
    long long want = (152 * per_sm + columns - 1) / columns;
    if (want < least_split) want = least_split;
    const int split = (int)(want < items ? want : items);
    return (items + split - 1) / split;
}

template <typename T, int kMinCtas>
gdn_status launch_append(const Kv &kv, const gdn_rows *k, const gdn_rows *v, const gdn_rows *q,
                         const gdn_rows *qo, bool rotate, const Rotary &rot, cudaStream_t st) {
    Append ap{};
    ap.rotate = rotate;
    ap.kv_tasks = kv.cu ? (long long)kv.n_tokens / F::kBlock + 2ll * kv.N
                        : (long long)blocks_touched(kv.n_tokens / kv.N) * kv.N;
    const int tasks_per = kThreads / kv.d;
    const long long kx = (ap.kv_tasks + tasks_per - 1) / tasks_per;
    ap.kv_items_per = items_per_cta(kx, 2 * kv.H, 3, 1);
    const long long ky = (2 * kv.H + ap.kv_items_per - 1) / ap.kv_items_per;
    long long q_ctas = 0;
    if (q) {
        const int per = kThreads / (kv.d / 16);
        ap.Hq = q->heads;
        ap.q_ctas_x = (kv.n_tokens + per - 1) / per;
        ap.q_heads_per = items_per_cta(ap.q_ctas_x, ap.Hq, 3, 2);
        q_ctas = (long long)ap.q_ctas_x * ((ap.Hq + ap.q_heads_per - 1) / ap.q_heads_per);
    }
    if (kx * ky + q_ctas > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
    ap.kv_ctas_x = (int)kx;
    ap.few_are_kv = kx * ky <= q_ctas;
    ap.few = (int)(ap.few_are_kv ? kx * ky : q_ctas);
    ap.stride = ap.few > 0 ? (int)((kx * ky + q_ctas) / ap.few) : 1;
    const int slot = timer_begin(st, "k_kv8_append");
    k_kv8_append<T, kMinCtas><<<(unsigned)(kx * ky + q_ctas), kThreads, 0, st>>>(
        kv, rows_of<const T>(k), rows_of<const T>(v), rows_of<const T>(q), rows_of<T>(qo), ap, rot,
        device_error_word());
    timer_end(slot, st);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T>
gdn_status launch_read(const Kv &kv, const gdn_rows *k, const gdn_rows *v, cudaStream_t st) {
    const int per = kThreads / (kv.d / 16), items = 2 * kv.H;
    const int gx = (kv.n_tokens + per - 1) / per, heads_per = items_per_cta(gx, items, 10, 2);
    const dim3 grid(gx, (items + heads_per - 1) / heads_per);
    const int slot = timer_begin(st, "k_kv8_read");
    k_kv8_read<T><<<grid, kThreads, 0, st>>>(kv, rows_of<T>(k), rows_of<T>(v), heads_per,
                                             device_error_word());
    timer_end(slot, st);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace kv
}  // namespace gdn

using namespace gdn::kv;

extern "C" {

int64_t gdn_kv8_page_bytes(int page_size, int d) {
    if (gdn_kv_page_bytes(page_size, d) == 0) return 0;      // the same sizes
    return Fmt8::block_bytes(page_size, d);
}

gdn_status gdn_kv8_append(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v,
                          const gdn_rows *q, const gdn_rows *q_out, const gdn_rotary *rot,
                          gdn_dtype dt, void *stream) {
    if (!kv || kv->N < 0 || kv->n_tokens < 0 || (q != nullptr) != (q_out != nullptr))
        return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (kv->n_tokens == 0) return GDN_OK;
    if (kv->N == 0) return GDN_ERR_INVALID_ARG;
    Kv dev;
    gdn_status rc = check_kv(kv, &dev);
    if (rc != GDN_OK) return rc;
    if ((rc = check_rows(k, dt, true)) != GDN_OK || (rc = check_rows(v, dt, true)) != GDN_OK)
        return rc;
    if (k->heads != kv->heads || v->heads != kv->heads) return GDN_ERR_INVALID_ARG;
    if (q) {
        if ((rc = check_rows(q, dt, true)) != GDN_OK ||
            (rc = check_rows(q_out, dt, true)) != GDN_OK)
            return rc;
        if (q->heads != q_out->heads) return GDN_ERR_INVALID_ARG;
    }
    Rotary r{};
    if (rot && (rc = check_rotary(rot, kv->d, true, &r)) != GDN_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // (CTAs an SM: fp32 rows spill at four; bf16 rows took 268 us for the prompts above at three)
    return dt == GDN_BF16
               ? launch_append<__nv_bfloat16, 4>(dev, k, v, q, q_out, rot != nullptr, r, st)
               : launch_append<float, 3>(dev, k, v, q, q_out, rot != nullptr, r, st);
}

gdn_status gdn_kv8_read(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v, gdn_dtype dt,
                        void *stream) {
    if (!kv || kv->N < 0 || kv->n_tokens < 0) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (kv->n_tokens == 0) return GDN_OK;
    if (kv->N == 0) return GDN_ERR_INVALID_ARG;
    Kv dev;
    gdn_status rc = check_kv(kv, &dev);
    if (rc != GDN_OK) return rc;
    if ((rc = check_rows(k, dt, true)) != GDN_OK || (rc = check_rows(v, dt, true)) != GDN_OK)
        return rc;
    if (k->heads != kv->heads || v->heads != kv->heads) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dt == GDN_BF16 ? launch_read<__nv_bfloat16>(dev, k, v, st)
                          : launch_read<float>(dev, k, v, st);
}

}  // extern "C"
