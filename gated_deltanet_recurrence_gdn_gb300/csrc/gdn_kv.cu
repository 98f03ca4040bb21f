// gdn_kv.cu -- the 4-bit paged key/value cache (gdn_attn.h): appending keys and
// values with the rotation applied on the way, and reading them back.
//
// Append: a thread holds one unit of 8 pairs or 16 neighbours (gdn_kv.cuh) of
// one token, with its cosines and sines in registers, and walks over the query
// heads (turn, round, store), the key heads (turn, quantise, store) and the
// value heads (quantise, store).  Where pairs are (i, i + d_rot / 2), a block of
// 16 neighbours that share a scale lies half in the unit of this thread and half
// in that of the neighbouring lane (units 2 m and 2 m + 1), so its largest
// magnitude is taken over two lanes.  Every key and value is read once and
// 9/16 of a byte per element is written: HBM bounds a prompt, the launch a
// single token.
//
// A thread has two heads' rows in flight and an SM four CTAs: 230 us for 12
// prompts of 700 to 8192 tokens (60 k tokens, 32 + 8 + 8 heads, d = 128 bf16,
// 1.29 GB: 5.6 TB/s, 82 % of a copy's rate); one row in flight took 251 us, three
// CTAs 234 (fp32 rows: one, 4.2 us for few tokens where two took 4.8).  Reading
// back takes 61 us (0.31 GB).  A token of each of 64 sequences: 3.9 us and 3.2.
#include "gdn_kv.cuh"

namespace gdn {
namespace kv {
namespace {

constexpr int kThreads = 256;

// Quantises a unit held as runs x, y and stores its codes and scale bytes.
// `split`: the runs are halves of two blocks whose other halves are in lane ^ 1.
__device__ __forceinline__ void put_unit(uint8_t *code_row, uint8_t *scale_row, const Unit &un,
                                         bool split, bool live, float inv, float (&x)[8],
                                         float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = __fmul_rn(x[i], inv);
        y[i] = __fmul_rn(y[i], inv);
    }
    const float mx = amax8(x), my = amax8(y);
    const float ox = __shfl_xor_sync(0xffffffffu, mx, 1), oy = __shfl_xor_sync(0xffffffffu, my, 1);
    float fx, fy;
    const uint32_t sx = scale_of(max_nan(mx, split ? ox : my), fx);
    const uint32_t sy = scale_of(max_nan(my, split ? oy : mx), fy);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = __fmul_rn(x[i], fx);
        y[i] = __fmul_rn(y[i], fy);
    }
    const uint32_t cx = e2m1x8_of(x), cy = e2m1x8_of(y);
    if (!live) return;
    if (split) {
        *reinterpret_cast<uint32_t *>(code_row + (un.lo >> 1)) = cx;
        *reinterpret_cast<uint32_t *>(code_row + (un.hi >> 1)) = cy;
        // the even unit of the two stores the first runs' scale, the odd the second's
        if ((un.lo & 8) == 0) scale_row[un.lo >> 4] = (uint8_t)sx;
        else scale_row[un.hi >> 4] = (uint8_t)sy;
    } else {
        *reinterpret_cast<uint2 *>(code_row + (un.lo >> 1)) = make_uint2(cx, cy);
        scale_row[un.lo >> 4] = (uint8_t)sx;
    }
}

// blockIdx.y takes heads_per of the Hq + 2 H items (query, key, value heads).
// Every lane of a warp runs the same items (the scale is taken across lanes);
// lanes past the last token only take part in that.
template <typename T, int kFly>
__global__ void __launch_bounds__(kThreads, 4)
k_kv_append(const Kv kv, Rows<const T> k, Rows<const T> v, Rows<const T> q, Rows<T> qo, int Hq,
            int heads_per, bool rotate, const __grid_constant__ Rotary rot, int *err) {
    const int units = kv.d / 16;                     // 4, 8 or 16: divides a warp
    const int u = threadIdx.x & (units - 1);
    const int t0 = blockIdx.x * (kThreads / units) + threadIdx.x / units;
    const bool there = t0 < kv.n_tokens;
    const int t = there ? t0 : kv.n_tokens - 1;
    const Unit un = unit_of(rot, u);
    const Unit whole{16 * u, 16 * u + 8, false};
    const int i0 = blockIdx.y * heads_per, i1 = min(i0 + heads_per, Hq + 2 * kv.H);
    Run<T> x[kFly], y[kFly];
    auto load = [&](int i) {
#pragma unroll
        for (int f = 0; f < kFly; ++f)
            if (i + f < i1) {
                const int h = i + f;
                const T *p = h < Hq          ? q.at(0, h, t)
                             : h < Hq + kv.H ? k.at(0, h - Hq, t)
                                             : v.at(0, h - Hq - kv.H, t);
                const Unit &w = h < Hq + kv.H ? un : whole;
                x[f].load(p + w.lo);
                y[f].load(p + w.hi);
            }
    };
    load(i0);
    float c[8], s[8];
    if (rotate && un.turned) unit_angles(rot, u, 0, t, c, s, err);
    const int b = kv.seq_of(t);
    int first, n, len;
    kv.tokens(b, first, n, len, err);
    const int place = len - n + (t - first);
    int page = -1;
    if (there && place >= 0 && t >= first && t < first + n) page = kv.page_of(b, place, err);
    const bool live = page >= 0;
    const int row = place & (kv.page_size() - 1), psz = kv.page_size();
    uint8_t *base = kv.pages + kv.block(live ? page : 0, 0);
    const int step = block_bytes(psz, kv.d);
    for (int i = i0; i < i1;) {
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            if (i + f >= i1) break;
            float a[8], e[8];
            x[f].get(a);
            y[f].get(e);
            if (i + f < Hq + kv.H && rotate && un.turned) turn(rot.adjacent, c, s, a, e);
            if (i + f < Hq) {
                if (there) {
                    T *o = qo.at(0, i + f, t);
                    store8(o + un.lo, a);
                    store8(o + un.hi, e);
                }
            } else {
                const bool key = i + f < Hq + kv.H;
                const int h = key ? i + f - Hq : i + f - Hq - kv.H;
                const float inv =
                    kv.head_scale ? __frcp_rn(__ldg(kv.head_scale + (key ? 0 : kv.H) + h)) : 1.f;
                uint8_t *blk = base + (long long)h * step;
                put_unit(blk + (key ? k_code_at(psz, kv.d, row) : v_code_at(psz, kv.d, row)),
                         blk + (key ? k_scale_at(psz, kv.d, row) : v_scale_at(psz, kv.d, row)),
                         key ? un : whole, key && un.turned && !rot.adjacent, live, inv, a, e);
            }
        }
        i += kFly;
        load(i);
    }
}

// One thread per 16 neighbours of a token's head: 9 bytes in, 16 values out.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_kv_read(const Kv kv, Rows<T> k, Rows<T> v, int heads_per, int *err) {
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
    const uint8_t *base = kv.pages + kv.block(page >= 0 ? page : 0, 0);
    const int step = block_bytes(psz, kv.d);
    const int i0 = blockIdx.y * heads_per, i1 = min(i0 + heads_per, 2 * kv.H);
    for (int i = i0; i < i1; ++i) {
        const bool key = i < kv.H;
        const int h = key ? i : i - kv.H;
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
        if (page >= 0) {
            const uint8_t *blk = base + (long long)h * step;
            const int at = key ? k_code_at(psz, kv.d, row) : v_code_at(psz, kv.d, row);
            const int as = key ? k_scale_at(psz, kv.d, row) : v_scale_at(psz, kv.d, row);
            const uint2 w = *reinterpret_cast<const uint2 *>(blk + at + 8 * u);
            const float s = e4m3_f32(blk[as + u]);
            const float g = kv.head_scale ? __ldg(kv.head_scale + (key ? 0 : kv.H) + h) : 1.f;
            uint32_t a[4], c[4];
            e2m1x8_f16(w.x, a);
            e2m1x8_f16(w.y, c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&a[e]));
                const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&c[e]));
                x[2 * e] = p.x * s * g;
                x[2 * e + 1] = p.y * s * g;
                y[2 * e] = r.x * s * g;
                y[2 * e + 1] = r.y * s * g;
            }
        }
        T *o = key ? k.at(0, h, t) : v.at(0, h, t);
        store8(o + 16 * u, x);
        store8(o + 16 * u + 8, y);
    }
}

// Heads a CTA walks over: few tokens are spread over the heads until there are
// `per_sm` CTAs an SM, many still in two.  Appending wants 3 (1024 tokens of 32 + 8 +
// 8 heads 8.5 us, at 16 an SM 10.9, 4096 tokens 22.0 and 24.1), reading back 10 (16384
// tokens 17.7 us, at 3 an SM 20.8; 1024 tokens 3.8 either way); in one part 60 k
// tokens took 237 us to append, 230 in two.
int heads_per_cta(long long gx, int items, int per_sm) {
    long long want = (152 * per_sm + gx - 1) / gx;
    want = want < 2 ? 2 : want;
    const int split = (int)(want < items ? want : items);
    return (items + split - 1) / split;
}

template <typename T, int kFly>
cudaError_t launch_append(const Kv &kv, const gdn_rows *k, const gdn_rows *v, const gdn_rows *q,
                          const gdn_rows *qo, bool rotate, const Rotary &rot, cudaStream_t st) {
    const int per = kThreads / (kv.d / 16), Hq = q ? q->heads : 0, items = Hq + 2 * kv.H;
    const int gx = (kv.n_tokens + per - 1) / per, heads_per = heads_per_cta(gx, items, 3);
    const dim3 grid(gx, (items + heads_per - 1) / heads_per);
    const int slot = timer_begin(st, "k_kv_append");
    k_kv_append<T, kFly><<<grid, kThreads, 0, st>>>(kv, rows_of<const T>(k), rows_of<const T>(v),
                                              rows_of<const T>(q), rows_of<T>(qo), Hq, heads_per,
                                              rotate, rot, device_error_word());
    timer_end(slot, st);
    count_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_read(const Kv &kv, const gdn_rows *k, const gdn_rows *v, cudaStream_t st) {
    const int per = kThreads / (kv.d / 16), items = 2 * kv.H;
    const int gx = (kv.n_tokens + per - 1) / per, heads_per = heads_per_cta(gx, items, 10);
    const dim3 grid(gx, (items + heads_per - 1) / heads_per);
    const int slot = timer_begin(st, "k_kv_read");
    k_kv_read<T><<<grid, kThreads, 0, st>>>(kv, rows_of<T>(k), rows_of<T>(v), heads_per,
                                            device_error_word());
    timer_end(slot, st);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

gdn_status check_kv(const gdn_kv *kv, Kv *out) {
    if (!kv->pages || !kv->page_table || !kv->kv_len || kv->n_pages < 1 || kv->max_pages < 1 ||
        kv->heads < 1)
        return GDN_ERR_INVALID_ARG;
    if (gdn_kv_page_bytes(kv->page_size, kv->d) == 0 || kv->heads > 65535 || kv->N > (1 << 24) ||
        kv->n_tokens > kMaxTokens)
        return GDN_ERR_UNSUPPORTED;
    if (!kv->cu_seqlens && kv->n_tokens % kv->N) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {kv->head_scale, kv->page_table, kv->kv_len, kv->cu_seqlens};
    for (const void *p : ptrs)
        if (!aligned4(p)) return GDN_ERR_ALIGNMENT;
    if (!aligned16(kv->pages)) return GDN_ERR_ALIGNMENT;
    int shift = 4;
    while ((1 << shift) < kv->page_size) ++shift;
    if ((long long)kv->max_pages << shift > kMaxTokens) return GDN_ERR_UNSUPPORTED;
    *out = Kv{static_cast<uint8_t *>(kv->pages), kv->head_scale, kv->page_table, kv->kv_len,
              kv->cu_seqlens, kv->n_pages, shift, kv->heads, kv->d, kv->N, kv->max_pages,
              kv->n_tokens, (long long)kv->table_stride};
    return GDN_OK;
}

}  // namespace kv
}  // namespace gdn

using namespace gdn::kv;

extern "C" {

int64_t gdn_kv_page_bytes(int page_size, int d) {
    if (d != 64 && d != 128 && d != 256) return 0;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return 0;
    return (int64_t)page_size * d * 9 / 8;
}

gdn_status gdn_kv_append(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v, const gdn_rows *q,
                         const gdn_rows *q_out, const gdn_rotary *rot, gdn_dtype dt,
                         void *stream) {
    if (!kv || kv->N < 0 || kv->n_tokens < 0 || (q != nullptr) != (q_out != nullptr))
        return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (kv->n_tokens == 0) return GDN_OK;
    if (kv->N == 0) return GDN_ERR_INVALID_ARG;
    Kv dev;
    gdn_status rc = check_kv(kv, &dev);
    if (rc != GDN_OK) return rc;
    if ((rc = check_rows(k, dt, true)) != GDN_OK ||
        (rc = check_rows(v, dt, true)) != GDN_OK)
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
    const cudaError_t e =
        dt == GDN_BF16 ? launch_append<__nv_bfloat16, 2>(dev, k, v, q, q_out, rot != nullptr, r, st)
                       : launch_append<float, 1>(dev, k, v, q, q_out, rot != nullptr, r, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_kv_read(const gdn_kv *kv, const gdn_rows *k, const gdn_rows *v, gdn_dtype dt,
                       void *stream) {
    if (!kv || kv->N < 0 || kv->n_tokens < 0) return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (kv->n_tokens == 0) return GDN_OK;
    if (kv->N == 0) return GDN_ERR_INVALID_ARG;
    Kv dev;
    gdn_status rc = check_kv(kv, &dev);
    if (rc != GDN_OK) return rc;
    if ((rc = check_rows(k, dt, true)) != GDN_OK ||
        (rc = check_rows(v, dt, true)) != GDN_OK)
        return rc;
    if (k->heads != kv->heads || v->heads != kv->heads) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dt == GDN_BF16 ? launch_read<__nv_bfloat16>(dev, k, v, st)
                                         : launch_read<float>(dev, k, v, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
