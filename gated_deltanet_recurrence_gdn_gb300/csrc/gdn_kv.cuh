// gdn_kv.cuh -- what the attention-layer kernels (gdn_rope.cu, gdn_kv.cu,
// gdn_kv_attn.cu) share: rows and their strides, the rotation of a unit of
// pairs, the 4-bit page format, and where a sequence's tokens lie.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_attn.h"
#include "gdn_check.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace kv {

constexpr int kMaxAxes = 4;
constexpr int kMaxPairs = 128;   // d_rot / 2 at d = 256
constexpr long long kMaxTokens = 0x7fffff00;   // so that a grid's last tokens fit an int

// ------------------------------------------------------------------- rows

template <typename T>
struct Rows {
    T *p;
    long long seq, head, tok;
    __device__ __forceinline__ T *at(int b, int h, int t) const {
        return p + b * seq + h * head + t * tok;
    }
};

template <typename T>
inline Rows<T> rows_of(const gdn_rows *r) {
    if (!r) return Rows<T>{nullptr, 0, 0, 0};
    return Rows<T>{static_cast<T *>(r->data), (long long)r->stride_seq, (long long)r->stride_head,
                   (long long)r->stride_tok};
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// 8 neighbouring elements as fp32, one 16-byte access for bf16, two for fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// The same as loaded, for loads that are in flight together.
template <typename T>
struct Run;
template <>
struct Run<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        w = *reinterpret_cast<const uint4 *>(p);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};
template <>
struct Run<float> {
    float x_[8];
    __device__ __forceinline__ void load(const float *p) { load8(p, x_); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x_[i];
    }
};
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// --------------------------------------------------------------- rotation

// Kernel-side form of gdn_rotary: the axis of each pair by value.
struct Rotary {
    const float *cos, *sin;
    const int32_t *pos;
    long long stride_axis, stride_seq;
    int table_len, half, n_axes;   // half = d_rot / 2
    bool adjacent, inverse;
    uint8_t axes[kMaxPairs];
};

// A row is cut into units of 16 elements: unit u < half / 8 holds the pairs
// 8 u .. 8 u + 7, as two runs of 8 elements (first and second of each pair, or
// 16 neighbours where pairs are adjacent); the units after them hold 16
// neighbours each that are not turned.
struct Unit {
    int lo, hi;      // element offsets of the two runs
    bool turned;
};
__device__ __forceinline__ Unit unit_of(const Rotary &r, int u) {
    Unit x;
    x.turned = u < (r.half >> 3);
    const bool split = x.turned && !r.adjacent;
    x.lo = split ? 8 * u : 16 * u;
    x.hi = split ? 8 * u + r.half : 16 * u + 8;
    return x;
}

// Cosines and sines of the 8 pairs of a turned unit of one token (the sines
// negated for the inverse); false, with the device error recorded, if a
// position lies outside the table.
__device__ __forceinline__ bool unit_angles(const Rotary &r, int u, int b, int t, float (&c)[8],
                                            float (&s)[8], int *err) {
    const int32_t *pos = r.pos + (long long)b * r.stride_seq + t;
    bool ok = true;
    if (r.n_axes == 1) {
        int p = __ldg(pos);
        if ((unsigned)p >= (unsigned)r.table_len) {
            ok = false;
            p = 0;
        }
        const long long at = (long long)p * r.half + 8 * u;
        load8(r.cos + at, c);
        load8(r.sin + at, s);
    } else {
        int p[kMaxAxes];
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a) {
            p[a] = a < r.n_axes ? __ldg(pos + a * r.stride_axis) : 0;
            if ((unsigned)p[a] >= (unsigned)r.table_len) {
                ok = false;
                p[a] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int a = r.axes[8 * u + i];
            const int q = a == 0 ? p[0] : a == 1 ? p[1] : a == 2 ? p[2] : p[3];
            const long long at = (long long)q * r.half + 8 * u + i;
            c[i] = __ldg(r.cos + at);
            s[i] = __ldg(r.sin + at);
        }
    }
    if (!ok) atomicCAS(err, 0, kErrBadIndex);
    if (r.inverse) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
    return ok;
}

// Turns a unit held as its two runs x[0..7], y[0..7].  The products are rounded
// before the sum (no fma), so that the result does not depend on which of the
// two products a fused form would keep exact.
__device__ __forceinline__ void turn(bool adjacent, const float (&c)[8], const float (&s)[8],
                                     float (&x)[8], float (&y)[8]) {
    if (adjacent) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
            const float e = y[2 * i], f = y[2 * i + 1];
            y[2 * i] = __fsub_rn(__fmul_rn(e, c[4 + i]), __fmul_rn(f, s[4 + i]));
            y[2 * i + 1] = __fadd_rn(__fmul_rn(f, c[4 + i]), __fmul_rn(e, s[4 + i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x[i], b = y[i];
            x[i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
            y[i] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
    }
}

// -------------------------------------------------------------- page format

// Byte offsets inside the block of one (page, head).
__host__ __device__ __forceinline__ int block_bytes(int page, int d) { return page * d * 9 / 8; }
__host__ __device__ __forceinline__ int k_code_at(int, int d, int row) { return row * (d / 2); }
__host__ __device__ __forceinline__ int v_code_at(int page, int d, int row) {
    return (page + row) * (d / 2);
}
__host__ __device__ __forceinline__ int k_scale_at(int page, int d, int row) {
    return page * d + row * (d / 16);
}
__host__ __device__ __forceinline__ int v_scale_at(int page, int d, int row) {
    return page * d + (page + row) * (d / 16);
}

// Kernel-side form of gdn_kv.
struct Kv {
    uint8_t *pages;
    const float *head_scale;
    const int32_t *page_table, *kv_len, *cu;
    int n_pages, page_shift, H, d, N, max_pages, n_tokens;
    long long table_stride;

    __device__ __forceinline__ int page_size() const { return 1 << page_shift; }
    __device__ __forceinline__ long long block(int page, int h) const {
        return ((long long)page * H + h) * block_bytes(1 << page_shift, d);
    }
    // (the bounds-check build: `bytes` bytes from `at` in a page's block lie in the pool)
    __device__ __forceinline__ bool bytes_ok(int page, int h, int at, int bytes) const {
        return GDN_IDX_OK(h, 1, H) && GDN_IDX_OK(at, bytes, block_bytes(1 << page_shift, d)) &&
               GDN_IDX_OK(page, 1, n_pages);
    }
    // Page of place p of sequence b as the table has it, and the same checked: -1 with
    // the error recorded if it is outside the pool.  (Apart, so that a look-up made
    // ahead is not waited for where it is made; kNoPage passes through as -1.)
    static constexpr int kNoPage = -0x7fffffff;
    __device__ __forceinline__ int page_raw(int b, int p) const {
        if (!GDN_IDX_OK(b, 1, N) || !GDN_IDX_OK(p >> page_shift, 1, max_pages)) return kNoPage;
        return __ldg(page_table + b * table_stride + (p >> page_shift));
    }
    __device__ __forceinline__ int page_checked(int g, int *err) const {
        if ((unsigned)g < (unsigned)n_pages) return g;
        if (g != kNoPage) atomicCAS(err, 0, kErrBadIndex);
        return -1;
    }
    __device__ __forceinline__ int page_of(int b, int p, int *err) const {
        return page_checked(page_raw(b, p), err);
    }
    // Tokens [first, first + n) and length of sequence b.  Offsets or lengths
    // out of range are recorded, and the sequence then counts as having none; so are
    // offsets that do not begin at 0 or end at n_tokens (tokens of no sequence).
    __device__ __forceinline__ void tokens(int b, int &first, int &n, int &len, int *err) const {
        first = n = len = 0;
        if (!GDN_IDX_OK(b, 1, N)) return;
        if (cu) {
            first = __ldg(cu + b);
            n = __ldg(cu + b + 1) - first;
        } else {
            n = n_tokens / N;
            first = b * n;
        }
        len = __ldg(kv_len + b);
        const bool bad_n = first < 0 || n < 0 || n > n_tokens - first;
        const bool bad_len = len < 0 || len > (long long)max_pages << page_shift;
        if (bad_n || bad_len) {
            atomicCAS(err, 0, kErrBadIndex);
            if (bad_n) n = first = 0;
            if (bad_len) len = 0;
        } else if ((b == 0 && first != 0) || (b == N - 1 && first + n != n_tokens)) {
            atomicCAS(err, 0, kErrBadIndex);
        }
    }
    // Sequence of packed token t: the last b with cu[b] <= t (empty sequences
    // before it share its offset).
    __device__ __forceinline__ int seq_of(int t) const {
        if (!cu) return t / (n_tokens / N);
        int lo = 0, hi = N;   // cu[lo] <= t < cu[hi] for valid offsets
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (__ldg(cu + m) <= t) lo = m;
            else hi = m;
        }
        return lo;
    }
};

// Host side: checks a gdn_kv (n_tokens > 0 and N > 0 known), fills the kernel's form.
gdn_status check_kv(const gdn_kv *kv, Kv *out);
// Checks rows of elements of `dt`; packed: of packed tokens, which have no stride_seq.
gdn_status check_rows(const gdn_rows *r, gdn_dtype dt, bool packed);
// Checks a rotation over rows of d elements; unit = required divisor of d_rot.
gdn_status check_rotary(const gdn_rotary *r, int d, bool append, Rotary *out);

// ------------------------------------------------------------ 4-bit numbers

// e4m3 byte of x >= 0 (or NaN), to nearest even, at most 448.
__device__ __forceinline__ uint32_t e4m3_of(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}
// Two e4m3 bytes (low half of w) as fp16x2.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(w));
    return r;
}
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    const uint32_t h = e4m3x2_f16(byte);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
// Eight e2m1 codes of x[0..7], element 0 in the lowest 4 bits; |x| > 6 becomes 6.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
// The four bytes of w, two e2m1 codes each, as fp16x2 (low code in the low half).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float m = max_nan(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
    for (int i = 2; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
    return m;
}
// e4m3 scale byte of 16 neighbours whose largest magnitude is m, and the factor
// that their elements are multiplied by before they become e2m1 (0 where the
// scale is: everything then reads back as zero).
__device__ __forceinline__ uint32_t scale_of(float m, float &factor) {
    const float t = __fmul_rn(m, 1.0f / 6.0f);
    const uint32_t byte = e4m3_of(t > 448.f ? 448.f : t);
    const float s = e4m3_f32(byte);
    factor = s == 0.f ? 0.f : __frcp_rn(s);
    return byte;
}

}  // namespace kv
}  // namespace gdn
