// gdn_rope.cu -- rotary positions with one or several axes: turns the pairs of
// query and key rows (gdn_attn.h), or turns their gradients back.
//
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for every pair (a, b): each row is
// read once and written once, so HBM bounds it.  A thread holds one unit of 8
// pairs (gdn_kv.cuh) of one token, keeps that unit's cosines and sines in
// registers and walks over the heads, so the table is read once a token, not
// once a row.  The next head's loads are issued before this one's stores; what
// hides their latency is occupancy: four CTAs an SM with one head in flight take
// 29.9 us at B4 T4096, 16 + 4 heads, d = 128 bf16 (170 MB, 84 % of a copy's rate)
// and 64.9 us at 371 MB (84 %); two CTAs with four heads in flight took 44 and
// 97 us, five CTAs 35 and 72.  A few tokens take 2.7 us: the launch.
#include "gdn_kv.cuh"

namespace gdn {
namespace kv {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
k_rope(Rows<const T> q, Rows<T> qo, int Hq, Rows<const T> k, Rows<T> ko, int Hk, int Tn, int n,
       int units, int heads_per, const __grid_constant__ Rotary rot, int *err) {
    const int per = kThreads / units;
    const int local = threadIdx.x / units, u = threadIdx.x - local * units;
    const int bt = blockIdx.x * per + local;
    if (local >= per || bt >= n) return;
    const int b = bt / Tn, t = bt - b * Tn;
    const Unit un = unit_of(rot, u);
    const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, Hq + Hk);
    Run<T> x, y;
    auto load = [&](int h) {
        if (h >= h1) return;
        const T *p = h < Hq ? q.at(b, h, t) : k.at(b, h - Hq, t);
        x.load(p + un.lo);
        y.load(p + un.hi);
    };
    load(h0);
    float c[8], s[8];
    if (un.turned) unit_angles(rot, u, b, t, c, s, err);
    for (int h = h0; h < h1; ++h) {
        float v[8], w[8];
        x.get(v);
        y.get(w);
        load(h + 1);
        if (un.turned) turn(rot.adjacent, c, s, v, w);
        T *p = h < Hq ? qo.at(b, h, t) : ko.at(b, h - Hq, t);
        store8(p + un.lo, v);
        store8(p + un.hi, w);
    }
}

template <typename T>
cudaError_t launch(const gdn_rows *q, const gdn_rows *qo, const gdn_rows *k, const gdn_rows *ko,
                   int B, int Tn, int d, const Rotary &rot, cudaStream_t st) {
    const int units = d / 16, per = kThreads / units;
    const int Hq = q->heads, Hk = k ? k->heads : 0;
    const int n = B * Tn;
    const long long gx = ((long long)n + per - 1) / per;
    // Few tokens: the heads are spread over CTAs until there are 3 an SM (4096 tokens of 64
    // + 16 heads 30.2 us; at 4 an SM, a full wave before the tail, 36.5, at 2 32.5).
    const long long want = (152 * 3 + gx - 1) / gx;
    const int split = (int)(want < Hq + Hk ? want : Hq + Hk);
    const int heads_per = (Hq + Hk + split - 1) / split;
    const int gy = (Hq + Hk + heads_per - 1) / heads_per;
    const int slot = timer_begin(st, "k_rope");
    k_rope<T><<<dim3((unsigned)gx, gy), kThreads, 0, st>>>(
        rows_of<const T>(q), rows_of<T>(qo), Hq, rows_of<const T>(k), rows_of<T>(ko), Hk, Tn, n,
        units, heads_per, rot, device_error_word());
    timer_end(slot, st);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

gdn_status check_rows(const gdn_rows *r, gdn_dtype dt, bool packed) {
    if (!r || !r->data || r->heads < 1) return GDN_ERR_INVALID_ARG;
    if (r->heads > 65535) return GDN_ERR_UNSUPPORTED;
    const int e = dt == GDN_BF16 ? 8 : 4;   // elements in 16 bytes
    if (!aligned16(r->data) || (!packed && r->stride_seq % e) || r->stride_head % e ||
        r->stride_tok % e)
        return GDN_ERR_ALIGNMENT;
    return GDN_OK;
}

gdn_status check_rotary(const gdn_rotary *r, int d, bool append, Rotary *out) {
    if (r->d_rot != 0 && (!r->cos || !r->sin || !r->pos || r->table_len < 1))
        return GDN_ERR_INVALID_ARG;
    if (r->d_rot < 0 || r->d_rot > d || r->n_axes < 1) return GDN_ERR_INVALID_ARG;
    const unsigned known = GDN_ROPE_ADJACENT | (append ? 0u : (unsigned)GDN_ROPE_INVERSE);
    if (r->flags & ~known) return GDN_ERR_INVALID_ARG;
    if (r->n_axes > kMaxAxes) return GDN_ERR_UNSUPPORTED;
    const bool adjacent = (r->flags & GDN_ROPE_ADJACENT) != 0;
    if (r->d_rot % (append && !adjacent ? 32 : 16)) return GDN_ERR_UNSUPPORTED;
    if (!aligned16(r->cos) || !aligned16(r->sin) || !aligned4(r->pos)) return GDN_ERR_ALIGNMENT;
    out->cos = r->cos;
    out->sin = r->sin;
    out->pos = r->pos;
    out->stride_axis = r->stride_axis;
    out->stride_seq = r->stride_seq;
    out->table_len = r->table_len;
    out->half = r->d_rot / 2;
    out->adjacent = adjacent;
    out->inverse = (r->flags & GDN_ROPE_INVERSE) != 0;
    bool one = true;
    for (int i = 0; i < out->half; ++i) {
        out->axes[i] = r->axes ? r->axes[i] : 0;
        if (out->axes[i] >= r->n_axes) return GDN_ERR_INVALID_ARG;
        one = one && out->axes[i] == 0;
    }
    out->n_axes = one ? 1 : r->n_axes;
    return GDN_OK;
}

}  // namespace kv
}  // namespace gdn

extern "C" gdn_status gdn_rope(const gdn_rows *q, const gdn_rows *q_out, const gdn_rows *k,
                               const gdn_rows *k_out, int B, int T, int d, const gdn_rotary *rot,
                               gdn_dtype dt, void *stream) {
    using namespace gdn::kv;
    if (B < 0 || T < 0 || !rot || !q || !q_out || (k != nullptr) != (k_out != nullptr))
        return GDN_ERR_INVALID_ARG;
    if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
    if (d < 16 || d % 16 || d > 256) return GDN_ERR_UNSUPPORTED;
    if ((long long)B * T > kMaxTokens) return GDN_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return GDN_OK;
    gdn_status rc;
    const gdn_rows *rows[] = {q, q_out, k, k_out};
    for (const gdn_rows *r : rows)
        if (r && (rc = check_rows(r, dt, false)) != GDN_OK) return rc;
    if (q->heads != q_out->heads || (k && k->heads != k_out->heads)) return GDN_ERR_INVALID_ARG;
    Rotary r{};
    if ((rc = check_rotary(rot, d, false, &r)) != GDN_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dt == GDN_BF16
                              ? launch<__nv_bfloat16>(q, q_out, k, k_out, B, T, d, r, st)
                              : launch<float>(q, q_out, k, k_out, B, T, d, r, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
