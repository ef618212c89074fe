// ops_api.cpp -- the C ABI declared in include/lstm_ops.h: argument checks,
// workspace carve-up and the kernel launches.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/lstm_ops.h"
#include "host.h"
#include "ops.h"

using namespace lstm_amd;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxDim = 256;
constexpr int kMaxWidth = 1 << 28;         // of a normalised row
constexpr long long kMaxRows = 1 << 20;  // (batch row, head) pairs
// Tokens: the kernels count in int, up to the end of the last segment (of at
// most 512, each of whole chunks of 32: less than 2^14 past T) and the two
// chunks loaded ahead.
constexpr int kMaxTokens = INT_MAX - (1 << 15);

size_t elem(int dtype) { return dtype == LSTM_BF16 ? 2 : 4; }

// acc += a * b * c * d bytes, 256-byte aligned; false on overflow.
bool add_bytes(size_t *acc, size_t a, size_t b, size_t c, size_t d) {
    size_t n;
    if (__builtin_mul_overflow(a, b, &n) || __builtin_mul_overflow(n, c, &n) || __builtin_mul_overflow(n, d, &n))
        return false;
    if (n > SIZE_MAX / 4 - *acc) return false;
    *acc += (n + kAlign - 1) / kAlign * kAlign;
    return true;
}

lstm_status current_device(int *dev) {
    if (hipGetDevice(dev) == hipSuccess) return LSTM_OK;
    (void)hipGetLastError();
    return LSTM_ERR_DEVICE;
}

lstm_status launched(hipError_t e) {
    if (e == hipSuccess) return LSTM_OK;
    (void)hipGetLastError();
    return LSTM_ERR_LAUNCH;
}

lstm_status check_shape(const lstm_linear_attention_shape *s) {
    if (!s) return LSTM_ERR_ARG;
    if (s->dtype != LSTM_F32 && s->dtype != LSTM_BF16) return LSTM_ERR_DTYPE;
    if (s->heads < 1 || s->kv_heads < 1 || s->heads % s->kv_heads != 0) return LSTM_ERR_ARG;
    if (s->key_dim < 1 || s->value_dim < 1 || s->key_dim > kMaxDim || s->value_dim > kMaxDim) return LSTM_ERR_ARG;
    if (!std::isfinite(s->scale) || s->scale == 0.0f) return LSTM_ERR_ARG;
    if (s->T < 1 || s->T > kMaxTokens || s->B < 1) return LSTM_ERR_SHAPE;
    // a grid of 2^32 threads holds every workgroup of three passes
    if ((long long)s->B * s->heads > kMaxRows) return LSTM_ERR_SHAPE;
    return LSTM_OK;
}

bool view_ok(const lstm_view *v) { return v && v->data; }

// Token to token the kernels step by 32-bit byte counts.
bool steps_ok(const lstm_linear_attention_shape *s, const lstm_view *v) {
    const long long most = INT_MAX / (long long)elem(s->dtype);
    return v->time >= -most && v->time <= most;
}

// Every pointer of the list that is given lies on the device.
bool all_on_device(const void *const *p, int n, int dev) {
    for (int i = 0; i < n; ++i)
        if (p[i] && !is_device_ptr(p[i], dev)) return false;
    return true;
}

LaTensor tensor(const lstm_view *v, int hdiv) {
    return LaTensor{static_cast<const char *>(v->data), v->time, v->batch, v->head, hdiv};
}
LaOut output(const lstm_view *v) { return LaOut{static_cast<char *>(v->data), v->time, v->batch, v->head, 0}; }

// Workspace: segment states of each pass; backward with shared heads: fp32
// partial sums of dk and dv, [B][T][heads][dim] each.
struct LaLayout {
    size_t seg[3], part_k, part_v, total;
    int nseg, seg_tokens;
};

bool la_layout(const lstm_linear_attention_shape *s, bool backward, LaLayout *o) {
    const size_t rows = (size_t)s->B * s->heads;
    const int npass = backward ? 3 : 1;
    size_t floats = 0;
    la_segments(s->T, (long long)rows, npass, s->key_dim, s->value_dim, s->dtype, &o->nseg, &o->seg_tokens, &floats);
    size_t off = 0;
    for (int i = 0; i < npass; ++i) {
        o->seg[i] = off;
        if (o->nseg > 1 && !add_bytes(&off, (size_t)o->nseg, rows, floats, sizeof(float))) return false;
    }
    o->part_k = o->part_v = off;
    if (backward && s->heads != s->kv_heads) {
        const size_t n = (size_t)s->T * rows;
        if (!add_bytes(&off, n, (size_t)s->key_dim, sizeof(float), 1)) return false;
        o->part_v = off;
        if (!add_bytes(&off, n, (size_t)s->value_dim, sizeof(float), 1)) return false;
    }
    o->total = off;
    return true;
}

lstm_status la_size(const lstm_linear_attention_shape *s, bool backward, size_t *bytes) {
    const lstm_status rc = check_shape(s);
    if (rc != LSTM_OK) return rc;
    if (!bytes) return LSTM_ERR_ARG;
    LaLayout lay;
    if (!la_layout(s, backward, &lay)) return LSTM_ERR_SHAPE;
    *bytes = lay.total;
    return LSTM_OK;
}

}  // namespace

extern "C" {

lstm_status lstm_linear_attention_workspace_size(const lstm_linear_attention_shape *s, size_t *bytes) {
    return la_size(s, false, bytes);
}

lstm_status lstm_linear_attention_backward_workspace_size(const lstm_linear_attention_shape *s, size_t *bytes) {
    return la_size(s, true, bytes);
}

lstm_status lstm_linear_attention_forward(const lstm_linear_attention_shape *s, const lstm_view *q,
                                          const lstm_view *k, const lstm_view *v, const float *log_decay,
                                          const int *lengths, const float *state, const lstm_view *o,
                                          float *state_out, void *workspace, size_t workspace_bytes, void *stream) {
    lstm_status rc = check_shape(s);
    if (rc != LSTM_OK) return rc;
    if (!view_ok(q) || !view_ok(k) || !view_ok(v) || !view_ok(o) || !log_decay) return LSTM_ERR_ARG;
    if (!steps_ok(s, q) || !steps_ok(s, k) || !steps_ok(s, v)) return LSTM_ERR_SHAPE;
    LaLayout lay;
    if (!la_layout(s, false, &lay)) return LSTM_ERR_SHAPE;
    if (lay.total && (!workspace || workspace_bytes < lay.total)) return LSTM_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {q->data, k->data, v->data, o->data, log_decay, lengths, state, state_out,
                          lay.total ? workspace : nullptr};
    if (!all_on_device(ptrs, 9, dev)) return LSTM_ERR_DEVICE;
    const int group = s->heads / s->kv_heads;
    LaCall c{};
    c.npass = 1;
    c.pass[0] = LaPass{tensor(q, 1), tensor(k, group), tensor(v, group), output(o), s->key_dim, s->value_dim, state,
                       state_out, s->value_dim, 1, s->scale, 1.0f, 0,
                       lay.nseg > 1 ? reinterpret_cast<float *>(static_cast<char *>(workspace) + lay.seg[0])
                                    : nullptr};
    c.log_decay = log_decay;
    c.lengths = lengths;
    c.T = s->T;
    c.B = s->B;
    c.H = s->heads;
    c.dtype = s->dtype;
    c.nseg = lay.nseg;
    c.seg_tokens = lay.seg_tokens;
    return launched(launch_la(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_linear_attention_backward(const lstm_linear_attention_shape *s, const lstm_view *q,
                                           const lstm_view *k, const lstm_view *v, const float *log_decay,
                                           const int *lengths, const float *state, const lstm_view *do_,
                                           const float *dstate_out, const lstm_view *dq, const lstm_view *dk,
                                           const lstm_view *dv, float *dstate, void *workspace,
                                           size_t workspace_bytes, void *stream) {
    lstm_status rc = check_shape(s);
    if (rc != LSTM_OK) return rc;
    if (!view_ok(q) || !view_ok(k) || !view_ok(v) || !view_ok(do_) || !view_ok(dq) || !view_ok(dk) || !view_ok(dv) ||
        !log_decay)
        return LSTM_ERR_ARG;
    if (!steps_ok(s, q) || !steps_ok(s, k) || !steps_ok(s, v) || !steps_ok(s, do_)) return LSTM_ERR_SHAPE;
    LaLayout lay;
    if (!la_layout(s, true, &lay)) return LSTM_ERR_SHAPE;
    if (lay.total && (!workspace || workspace_bytes < lay.total)) return LSTM_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {q->data, k->data, v->data, do_->data, dq->data, dk->data, dv->data, log_decay, lengths,
                          state, dstate_out, dstate, lay.total ? workspace : nullptr};
    if (!all_on_device(ptrs, 13, dev)) return LSTM_ERR_DEVICE;
    const int group = s->heads / s->kv_heads, Dk = s->key_dim, Dv = s->value_dim, H = s->heads;
    char *ws = static_cast<char *>(workspace);
    float *seg[3];
    for (int i = 0; i < 3; ++i) seg[i] = lay.nseg > 1 ? reinterpret_cast<float *>(ws + lay.seg[i]) : nullptr;
    // a shared head's gradient is summed over its query heads afterwards
    LaOut ok = output(dk), ov = output(dv);
    float *pk = reinterpret_cast<float *>(ws + lay.part_k), *pv = reinterpret_cast<float *>(ws + lay.part_v);
    if (group > 1) {
        const long long T = s->T;
        ok = LaOut{reinterpret_cast<char *>(pk), (long long)H * Dk, T * H * Dk, Dk, 1};
        ov = LaOut{reinterpret_cast<char *>(pv), (long long)H * Dv, T * H * Dv, Dv, 1};
    }
    const LaTensor tq = tensor(q, 1), tk = tensor(k, group), tv = tensor(v, group), td = tensor(do_, 1);
    const float sc = s->scale;
    LaCall c{};
    c.npass = 3;
    c.pass[0] = LaPass{td, tv, tk, output(dq), Dv, Dk, state, nullptr, 1, Dv, sc, 1.0f, 0, seg[0]};
    c.pass[1] = LaPass{tv, td, tq, ok, Dv, Dk, dstate_out, nullptr, 1, Dv, 1.0f, sc, 1, seg[1]};
    c.pass[2] = LaPass{tk, tq, td, ov, Dk, Dv, dstate_out, dstate, Dv, 1, 1.0f, sc, 1, seg[2]};
    c.log_decay = log_decay;
    c.lengths = lengths;
    c.T = s->T;
    c.B = s->B;
    c.H = H;
    c.dtype = s->dtype;
    c.nseg = lay.nseg;
    c.seg_tokens = lay.seg_tokens;
    hipStream_t st = static_cast<hipStream_t>(stream);
    rc = launched(launch_la(c, st));
    if (rc != LSTM_OK || group == 1) return rc;
    return launched(launch_la_share(LaShare{pk, output(dk), Dk}, LaShare{pv, output(dv), Dv}, s->T, s->B, H,
                                    s->kv_heads, s->dtype, st));
}

lstm_status lstm_linear_attention_step(const lstm_linear_attention_shape *s, const lstm_view *q, const lstm_view *k,
                                       const lstm_view *v, const float *log_decay, const int *slots, int n_slots,
                                       float *pool, const lstm_view *o, void *stream) {
    lstm_status rc = check_shape(s);
    if (rc != LSTM_OK) return rc;
    if (!view_ok(q) || !view_ok(k) || !view_ok(v) || !view_ok(o) || !log_decay || !pool) return LSTM_ERR_ARG;
    if (s->T != 1 || n_slots < 1 || (!slots && n_slots < s->B)) return LSTM_ERR_SHAPE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {q->data, k->data, v->data, o->data, log_decay, slots, pool};
    if (!all_on_device(ptrs, 7, dev)) return LSTM_ERR_DEVICE;
    const int group = s->heads / s->kv_heads;
    const LaStep c{tensor(q, 1), tensor(k, group), tensor(v, group), output(o), log_decay, slots, pool, n_slots, s->B,
                   s->heads, s->key_dim, s->value_dim, s->dtype, s->scale};
    return launched(launch_la_step(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_layer_norm_forward(int dtype, const void *x, long long x_stride, const void *residual,
                                    long long residual_stride, const void *weight, const void *bias, long long rows,
                                    int width, float eps, void *y, void *sum, float *mean, float *rstd,
                                    void *stream) {
    if (dtype != LSTM_F32 && dtype != LSTM_BF16) return LSTM_ERR_DTYPE;
    if (rows < 0 || width < 1 || width > kMaxWidth || x_stride < width || (residual && residual_stride < width))
        return LSTM_ERR_SHAPE;
    if (!(eps >= 0.0f) || !std::isfinite(eps) || (!residual && sum)) return LSTM_ERR_ARG;
    if (rows == 0) return LSTM_OK;
    if (!x || !y) return LSTM_ERR_ARG;
    int dev = 0;
    const lstm_status rc = current_device(&dev);
    if (rc != LSTM_OK) return rc;
    const void *ptrs[] = {x, residual, weight, bias, y, sum, mean, rstd};
    if (!all_on_device(ptrs, 8, dev)) return LSTM_ERR_DEVICE;
    const LnForward c{static_cast<const char *>(x), static_cast<const char *>(residual),
                      static_cast<const char *>(weight), static_cast<const char *>(bias), static_cast<char *>(y),
                      static_cast<char *>(sum), mean, rstd, x_stride, residual_stride, rows, width, dtype, eps};
    return launched(launch_ln_forward(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_layer_norm_backward_workspace_size(long long rows, int width, size_t *bytes) {
    if (!bytes) return LSTM_ERR_ARG;
    if (rows < 0 || width < 1 || width > kMaxWidth) return LSTM_ERR_SHAPE;
    *bytes = (size_t)ln_parts(rows, width) * 2 * (size_t)width * sizeof(float);
    return LSTM_OK;
}

lstm_status lstm_layer_norm_backward(int dtype, const void *dy, long long dy_stride, const void *z,
                                     long long z_stride, const float *mean, const float *rstd, const void *weight,
                                     const void *dsum, long long rows, int width, void *dx, void *dweight,
                                     void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    if (dtype != LSTM_F32 && dtype != LSTM_BF16) return LSTM_ERR_DTYPE;
    if (rows < 0 || width < 1 || width > kMaxWidth || dy_stride < width || z_stride < width) return LSTM_ERR_SHAPE;
    if (rows > 0 && (!dy || !z || !mean || !rstd || !dx)) return LSTM_ERR_ARG;
    size_t need = 0;
    lstm_status rc = lstm_layer_norm_backward_workspace_size(rows, width, &need);
    if (rc != LSTM_OK) return rc;
    const bool sums = dweight || dbias;
    if (sums && need && (!workspace || workspace_bytes < need)) return LSTM_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {rows ? dy : nullptr, rows ? z : nullptr, rows ? mean : nullptr, rows ? rstd : nullptr,
                          weight, rows ? dsum : nullptr, rows ? dx : nullptr, dweight, dbias,
                          sums && need ? workspace : nullptr};
    if (!all_on_device(ptrs, 10, dev)) return LSTM_ERR_DEVICE;
    const LnBackward c{static_cast<const char *>(dy), static_cast<const char *>(z), static_cast<const char *>(weight),
                       static_cast<const char *>(dsum), mean, rstd, static_cast<char *>(dx),
                       static_cast<char *>(dweight), static_cast<char *>(dbias),
                       sums ? static_cast<float *>(workspace) : nullptr, dy_stride, z_stride, rows, width, dtype};
    return launched(launch_ln_backward(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_adamw_step(int dtype, int state_bits, const lstm_adamw_tensor *tensors, int count, double beta1,
                            double beta2, double eps, long long step, const float *grad_scale, unsigned seed,
                            void *stream) {
    if (dtype != LSTM_F32 && dtype != LSTM_BF16) return LSTM_ERR_DTYPE;
    if (state_bits != 8 && state_bits != 32) return LSTM_ERR_UNSUPPORTED;
    if (count < 0 || (count > 0 && !tensors)) return LSTM_ERR_ARG;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
        step < 1)
        return LSTM_ERR_ARG;
    for (int i = 0; i < count; ++i) {
        const lstm_adamw_tensor &t = tensors[i];
        if (t.n < 0) return LSTM_ERR_SHAPE;
        if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay)) return LSTM_ERR_ARG;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale)))
            return LSTM_ERR_ARG;
        if (t.master && dtype != LSTM_BF16) return LSTM_ERR_ARG;
    }
    int dev = 0;
    const lstm_status rc = current_device(&dev);
    if (rc != LSTM_OK) return rc;
    if (grad_scale && !is_device_ptr(grad_scale, dev)) return LSTM_ERR_DEVICE;
    for (int i = 0; i < count; ++i) {
        const lstm_adamw_tensor &t = tensors[i];
        if (t.n == 0) continue;
        const void *ptrs[] = {t.param, t.grad, t.m, t.v, state_bits == 8 ? t.m_scale : nullptr,
                              state_bits == 8 ? t.v_scale : nullptr, t.master};
        if (!all_on_device(ptrs, 7, dev)) return LSTM_ERR_DEVICE;
    }
    AdamwHyper h{};
    h.beta1 = (float)beta1;
    h.beta2 = (float)beta2;
    h.one_beta1 = (float)(1.0 - beta1);
    h.one_beta2 = (float)(1.0 - beta2);
    // The kernels multiply by a reciprocal, which is infinite for eps alone
    // (v = 0) below the normal range, and 0 times it not a number: there both
    // parts of the quotient are taken 2^30 times as large.
    const double up = eps > 0.0 && eps < 0x1p-100 ? 0x1p30 : 1.0;
    h.eps = eps > 0.0 ? (float)std::fmax(eps * up, 0x1p-126) : 0.0f;
    h.inv_bc1 = (float)(up / (1.0 - std::pow(beta1, (double)step)));
    h.inv_sqrt_bc2 = (float)(up / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    h.grad_scale = grad_scale;
    h.seed = seed;
    return launched(launch_adamw(dtype, state_bits, tensors, count, h, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
