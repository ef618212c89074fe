// linear_attention.hip -- linear attention with a decay for each head.
#include "device.h"
#include "ops.h"
#include "ops_dev.h"

namespace lstm_amd {

void la_segments(int T, long long rows, int da, int dc, int dtype, int *nseg, int *seg_tokens) {
    (void)rows, (void)da, (void)dc, (void)dtype;
    *nseg = 1;
    *seg_tokens = T;
}

namespace {

template <class DT>
__device__ inline float la_get(const LaTensor &x, int t, int b, int h, int d) {
    const size_t at = (size_t)((long long)t * x.t + (long long)b * x.b + (long long)(h / x.hdiv) * x.h + d);
    return DT::to_f(reinterpret_cast<const typename DT::S *>(x.p)[at]);
}

template <class DT>
__device__ inline void la_put(const LaOut &o, int t, int b, int h, int d, float v) {
    const size_t at = (size_t)((long long)t * o.t + (long long)b * o.b + (long long)h * o.h + d);
    if (o.f32)
        reinterpret_cast<float *>(o.p)[at] = v;
    else
        reinterpret_cast<typename DT::S *>(o.p)[at] = round_to<DT>(v);
}

// gamma^n for n >= 0; n = 0 is 1 also for gamma = 0 (log decay -infinity).
__device__ inline float la_pow(float g2, int n) { return n == 0 ? 1.0f : __builtin_amdgcn_exp2f((float)n * g2); }

// One wave per 64 columns of one (batch row, head): the recurrence itself,
// token by token, the carried matrix in LDS.
template <class DT>
__global__ __launch_bounds__(64) void k_la_tokens(LaPass p, const float *log_decay, const int *lengths, int T, int H) {
    extern __shared__ float S[];  // [da][64]
    const int lane = threadIdx.x, col = blockIdx.x * 64 + lane;
    const int h = blockIdx.y % H, b = blockIdx.y / H;
    const bool on = col < p.dc;
    int len = lengths ? lengths[b] : T;
    len = len < 0 ? 0 : len > T ? T : len;
    const float gamma = la_pow(log_decay[h] * 1.4426950408889634f, 1);
    const size_t sbase = ((size_t)b * H + h) * p.da * p.dc;
    for (int d = 0; d < p.da; ++d)
        S[d * 64 + lane] = p.s0 && on ? p.s0[sbase + (size_t)d * p.srow + (size_t)col * p.scol] * p.in_scale : 0.0f;
    for (int i = 0; i < len; ++i) {
        const int t = p.reverse ? len - 1 - i : i;
        const float cv = on ? la_get<DT>(p.c, t, b, h, col) : 0.0f;
        float sum = 0.0f;
        for (int d = 0; d < p.da; ++d) {
            float s = S[d * 64 + lane];
            if (!p.reverse) s *= gamma;
            s += la_get<DT>(p.b, t, b, h, d) * cv;
            sum += la_get<DT>(p.a, t, b, h, d) * s;
            if (p.reverse) s *= gamma;
            S[d * 64 + lane] = s;
        }
        if (on) la_put<DT>(p.o, t, b, h, col, sum * p.out_scale);
    }
    if (on)
        for (int t = len; t < T; ++t) la_put<DT>(p.o, t, b, h, col, 0.0f);
    if (p.s1 && on)
        for (int d = 0; d < p.da; ++d)
            p.s1[sbase + (size_t)d * p.srow + (size_t)col * p.scol] = S[d * 64 + lane] * p.s1_scale;
}

template <class DT>
__global__ __launch_bounds__(256) void k_la_share(const float *part, LaOut o, int T, int B, int H, int G, int D) {
    const size_t n = (size_t)T * B * G * D;
    const int per = H / G;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        const int d = (int)(i % D), g = (int)(i / D % G);
        const size_t row = i / ((size_t)D * G);  // b * T + t
        const float *p = part + (row * H + (size_t)g * per) * D + d;
        float sum = 0.0f;
        for (int j = 0; j < per; ++j) sum += p[(size_t)j * D];
        la_put<DT>(o, (int)(row % T), (int)(row / T), g, d, sum);
    }
}

// One wave per 64 value columns of one (request, head).
template <class DT>
__global__ __launch_bounds__(64) void k_la_step(LaStep c) {
    const int col = blockIdx.x * 64 + threadIdx.x, h = blockIdx.y % c.H, b = blockIdx.y / c.H;
    if (col >= c.Dv) return;
    const int slot = c.slots ? c.slots[b] : b;
    float sum = 0.0f;
    if (slot >= 0 && slot < c.n_slots) {
        const float gamma = la_pow(c.log_decay[h] * 1.4426950408889634f, 1);
        const float v = la_get<DT>(c.v, 0, b, h, col);
        float *s = c.pool + ((size_t)slot * c.H + h) * c.Dk * c.Dv + col;
        for (int d = 0; d < c.Dk; ++d) {
            const float x = s[(size_t)d * c.Dv] * gamma + la_get<DT>(c.k, 0, b, h, d) * v;
            s[(size_t)d * c.Dv] = x;
            sum += la_get<DT>(c.q, 0, b, h, d) * x;
        }
    }
    la_put<DT>(c.o, 0, b, h, col, sum * c.scale);
}

}  // namespace

hipError_t launch_la(const LaCall &c, hipStream_t s) {
    for (int i = 0; i < c.npass; ++i) {
        const LaPass &p = c.pass[i];
        const dim3 grid((p.dc + 63) / 64, c.B * c.H);
        const size_t lds = (size_t)p.da * 64 * sizeof(float);
        if (c.dtype == LSTM_BF16)
            hipLaunchKernelGGL(k_la_tokens<BF16>, grid, dim3(64), lds, s, p, c.log_decay, c.lengths, c.T, c.H);
        else
            hipLaunchKernelGGL(k_la_tokens<F32>, grid, dim3(64), lds, s, p, c.log_decay, c.lengths, c.T, c.H);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_la_share(const float *part, LaOut out, int T, int B, int H, int G, int D, int dtype, hipStream_t s) {
    const size_t n = (size_t)T * B * G * D, blocks = (n + 255) / 256;
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
    if (dtype == LSTM_BF16)
        hipLaunchKernelGGL(k_la_share<BF16>, grid, dim3(256), 0, s, part, out, T, B, H, G, D);
    else
        hipLaunchKernelGGL(k_la_share<F32>, grid, dim3(256), 0, s, part, out, T, B, H, G, D);
    return hipGetLastError();
}

hipError_t launch_la_step(const LaStep &c, hipStream_t s) {
    const dim3 grid((c.Dv + 63) / 64, c.B * c.H);
    if (c.dtype == LSTM_BF16)
        hipLaunchKernelGGL(k_la_step<BF16>, grid, dim3(64), 0, s, c);
    else
        hipLaunchKernelGGL(k_la_step<F32>, grid, dim3(64), 0, s, c);
    return hipGetLastError();
}

}  // namespace lstm_amd
