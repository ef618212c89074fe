// gated_recurrence.hip -- the gated linear recurrence, whole sequences forward
// and backward, and single tokens.
//     z = s(-f) (= 1 - a),  w = s(i) or z,  h_t = h_{t-1} - z h_{t-1} + w x_t
//     D_t = dy_t + E_{t+1},  E_t = D_t - z D_t  (E: what reaches h_{t-1})
//     dx = w D,  df = D (h_{t-1} - [w = z] x) z (1 - z),  di = D x w (1 - w)
// A thread walks the tokens of V neighbouring channels of a batch row, 16 bytes
// of each tensor at a time.  Where the channels do not fill the card the
// sequence is cut into segments: one launch takes each segment's own map
// (carry -> A carry + B, A the product of its 1 - z), one joins them, and one
// walks the segments from the states that they begin with.
#include <type_traits>

#include "blocks.h"
#include "device.h"
#include "ops_dev.h"

namespace lstm_amd {
namespace {

constexpr int U = 8;  // tokens on their way at a time

template <class DT, int V>
__device__ inline void gr_load(const char *p, float *v) {
    typename DT::S s[V];
    __builtin_memcpy(s, p, sizeof(s));
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = DT::to_f(s[e]);
}
// Values `own`.. of the piece: those before it are another thread's.
template <class DT, int V>
__device__ inline void gr_store(char *p, const float *v, int own = 0) {
    typename DT::S s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = round_to<DT>(v[e]);
    if (own == 0) {
        __builtin_memcpy(p, s, sizeof(s));
    } else {
#pragma unroll
        for (int e = 1; e < V; ++e)
            if (e >= own) __builtin_memcpy(p + e * sizeof(s[0]), &s[e], sizeof(s[0]));
    }
}

template <class DT, int V>
struct Raw {
    typename DT::S s[V];
    __device__ void load(const char *p) { __builtin_memcpy(s, p, sizeof(s)); }
    __device__ float at(int e) const { return DT::to_f(s[e]); }
};

// The thread's batch row and first channel.  Where the width is no multiple of
// V the last piece ends with the row, and its first `own` values are read but
// are the thread before's to write (state and state_out may be one memory).
template <int V>
__device__ inline bool gr_place(const GrCall &c, int *b, int *ch, int *own) {
    const int per = (c.width + V - 1) / V;
    const long long t = blockIdx.x * 256ll + threadIdx.x;
    if (t >= (long long)c.B * per) return false;
    *b = (int)(t / per);
    const int from = (int)(t % per) * V;
    *ch = min(from, c.width - V);
    *own = from - *ch;
    return true;
}

template <class DT>
__device__ inline const char *gr_at(const GrView &v, int b, int ch, int t) {
    return v.p + (v.t * t + v.b * b + ch) * (long long)sizeof(typename DT::S);
}

__device__ inline int gr_length(const GrCall &c, int b) {
    return c.lengths ? min(max(c.lengths[b], 0), c.T) : c.T;
}

// APPLY: the outputs; else the segment's map, to the workspace.
template <class DT, int V, bool INPUT, bool APPLY>
__global__ __launch_bounds__(256) void k_gr_forward(GrCall c) {
    int b, ch, own;
    if (!gr_place<V>(c, &b, &ch, &own)) return;
    const int sg = blockIdx.y, n = gr_length(c, b), t0 = sg * c.seg_tokens, t1 = min(t0 + c.seg_tokens, c.T);
    const int end = min(t1, n);  // of the tokens that count
    const size_t slab = (size_t)c.B * c.width, at = (size_t)b * c.width + ch;
    float h[V], A[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = 0.0f, A[e] = 1.0f;
    if (APPLY) {
        const float *s = c.nseg > 1 ? c.seg + sg * slab : c.s0;
        if (s) __builtin_memcpy(h, s + at, sizeof(h));
    }
    const long long sx = c.x.t * (long long)sizeof(typename DT::S), sf = c.f.t * (long long)sizeof(typename DT::S);
    const long long si = c.i.t * (long long)sizeof(typename DT::S), sy = c.y.t * (long long)sizeof(typename DT::S);
    const char *px = gr_at<DT>(c.x, b, ch, t0), *pf = gr_at<DT>(c.f, b, ch, t0);
    const char *pi = INPUT ? gr_at<DT>(c.i, b, ch, t0) : nullptr;
    char *py = APPLY ? const_cast<char *>(gr_at<DT>(c.y, b, ch, t0)) : nullptr;
    Raw<DT, V> x[U], f[U], g[U];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(t + u, end - 1) - t0;  // past the end: the last token again
            x[u].load(px + k * sx);
            f[u].load(pf + k * sf);
            if (INPUT) g[u].load(pi + k * si);
        }
    };
    for (int t = t0; t < end; t += U) {
        fetch(t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= end) break;
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float z = sigmoid_f(-f[u].at(e)), w = INPUT ? sigmoid_f(g[u].at(e)) : z;
                h[e] = fmaf(w, x[u].at(e), fmaf(-z, h[e], h[e]));
                if (!APPLY) A[e] = fmaf(-z, A[e], A[e]);
                y[e] = h[e];
            }
            if (APPLY) gr_store<DT, V>(py + (t + u - t0) * sy, y, own);
        }
    }
    if (!APPLY) {
        float *s = c.seg + sg * slab + at;
        gr_store<F32, V>(reinterpret_cast<char *>(s), h, own);
        gr_store<F32, V>(reinterpret_cast<char *>(s + c.nseg * slab), A, own);
        return;
    }
    const float zero[V] = {};
    for (int t = max(end, t0); t < t1; ++t) gr_store<DT, V>(py + (t - t0) * sy, zero, own);
    if (sg == c.nseg - 1 && c.s1) gr_store<F32, V>(reinterpret_cast<char *>(c.s1 + at), h, own);
}

template <class DT, int V, bool INPUT, bool APPLY>
__global__ __launch_bounds__(256) void k_gr_backward(GrCall c) {
    int b, ch, own;
    if (!gr_place<V>(c, &b, &ch, &own)) return;
    const int sg = blockIdx.y, n = gr_length(c, b), t0 = sg * c.seg_tokens, t1 = min(t0 + c.seg_tokens, c.T);
    const int end = min(t1, n);
    const size_t slab = (size_t)c.B * c.width, at = (size_t)b * c.width + ch;
    float E[V], A[V];
#pragma unroll
    for (int e = 0; e < V; ++e) E[e] = 0.0f, A[e] = 1.0f;
    if (APPLY) {
        const float *s = c.nseg > 1 ? c.seg + sg * slab : c.ds1;
        if (s) __builtin_memcpy(E, s + at, sizeof(E));
    }
    Raw<DT, V> x[U], f[U], g[U], d[U], h[U];
    if (APPLY) {
        const float zero[V] = {};
        for (int t = max(end, t0); t < t1; ++t) {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), zero, own);
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), zero, own);
            if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), zero, own);
        }
    }
    for (int t = end - 1; t >= t0; t -= U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = max(t - u, t0);
            f[u].load(gr_at<DT>(c.f, b, ch, k));
            d[u].load(gr_at<DT>(c.dy, b, ch, k));
            if (APPLY) {
                x[u].load(gr_at<DT>(c.x, b, ch, k));
                if (INPUT) g[u].load(gr_at<DT>(c.i, b, ch, k));
                h[u].load(gr_at<DT>(c.y, b, ch, max(k - 1, 0)));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = t - u;
            if (k < t0) break;
            float dx[V], df[V], di[V];
            float before[V];
            if (APPLY) {
#pragma unroll
                for (int e = 0; e < V; ++e) before[e] = h[u].at(e);
                if (k == 0) {
#pragma unroll
                    for (int e = 0; e < V; ++e) before[e] = 0.0f;
                    if (c.s0) __builtin_memcpy(before, c.s0 + at, sizeof(before));
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float z = sigmoid_f(-f[u].at(e)), D = d[u].at(e) + E[e];
                if (APPLY) {
                    const float a = sigmoid_f(f[u].at(e)), xv = x[u].at(e);
                    if (INPUT) {
                        const float w = sigmoid_f(g[u].at(e)), v = sigmoid_f(-g[u].at(e));
                        dx[e] = w * D;
                        df[e] = D * before[e] * (z * a);
                        di[e] = D * xv * (w * v);
                    } else {
                        dx[e] = z * D;
                        df[e] = D * (before[e] - xv) * (z * a);
                    }
                } else {
                    A[e] = fmaf(-z, A[e], A[e]);
                }
                E[e] = fmaf(-z, D, D);
            }
            if (APPLY) {
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, k)), dx, own);
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, k)), df, own);
                if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, k)), di, own);
            }
        }
    }
    if (!APPLY) {
        float *s = c.seg + sg * slab + at;
        gr_store<F32, V>(reinterpret_cast<char *>(s), E, own);
        gr_store<F32, V>(reinterpret_cast<char *>(s + c.nseg * slab), A, own);
    } else if (sg == 0 && c.ds0) {
        gr_store<F32, V>(reinterpret_cast<char *>(c.ds0 + at), E, own);
    }
}

// Each segment's B becomes the carry that it begins with.
template <bool BACK>
__global__ __launch_bounds__(256) void k_gr_join(GrCall c) {
    const size_t slab = (size_t)c.B * c.width, at = blockIdx.x * 256ull + threadIdx.x;
    if (at >= slab) return;
    const float *first = BACK ? c.ds1 : c.s0;
    float carry = first ? first[at] : 0.0f;
#pragma unroll 8
    for (int i = 0; i < c.nseg; ++i) {
        float *s = c.seg + (BACK ? c.nseg - 1 - i : i) * slab + at;
        const float b = *s, a = s[c.nseg * slab];
        *s = carry;
        carry = fmaf(a, carry, b);
    }
}

template <class DT, int V, bool INPUT>
__global__ __launch_bounds__(64) void k_gr_step(GrStep c) {
    const int per = c.width / V;  // whole pieces, or V = 1
    const long long t = blockIdx.x * 64ll + threadIdx.x;
    if (t >= (long long)c.B * per) return;
    const int b = (int)(t / per), ch = (int)(t % per) * V;
    const int slot = c.slots ? c.slots[b] : b;
    float x[V], f[V], g[V], h[V];
    gr_load<DT, V>(gr_at<DT>(c.x, b, ch, 0), x);
    gr_load<DT, V>(gr_at<DT>(c.f, b, ch, 0), f);
    if (INPUT) gr_load<DT, V>(gr_at<DT>(c.i, b, ch, 0), g);
    char *y = const_cast<char *>(gr_at<DT>(c.y, b, ch, 0));
    if (slot < 0 || slot >= c.n_slots) {
        const float zero[V] = {};
        gr_store<DT, V>(y, zero);
        return;
    }
    float *s = c.pool + (size_t)slot * c.width + ch;
    __builtin_memcpy(h, s, sizeof(h));
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float z = sigmoid_f(-f[e]), w = INPUT ? sigmoid_f(g[e]) : z;
        h[e] = fmaf(w, x[e], fmaf(-z, h[e], h[e]));
    }
    __builtin_memcpy(s, h, sizeof(h));
    gr_store<DT, V>(y, h);
}

// f(integral_constant V) for the widest piece that a row holds.
template <class DT, class F>
void with_piece(int width, F f) {
    if (width >= DT::PER16)
        f(std::integral_constant<int, DT::PER16>{});
    else
        f(std::integral_constant<int, 1>{});
}

template <class DT, bool INPUT, bool BACK>
hipError_t run(const GrCall &c, hipStream_t s) {
    with_piece<DT>(c.width, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const long long threads = (long long)c.B * ((c.width + V - 1) / V);
        const dim3 grid((unsigned)((threads + 255) / 256), c.nseg);
        if (c.nseg > 1) {
            if (BACK)
                hipLaunchKernelGGL((k_gr_backward<DT, V, INPUT, false>), grid, dim3(256), 0, s, c);
            else
                hipLaunchKernelGGL((k_gr_forward<DT, V, INPUT, false>), grid, dim3(256), 0, s, c);
            hipLaunchKernelGGL(k_gr_join<BACK>, dim3((unsigned)(((long long)c.B * c.width + 255) / 256)), dim3(256), 0,
                               s, c);
        }
        if (BACK)
            hipLaunchKernelGGL((k_gr_backward<DT, V, INPUT, true>), grid, dim3(256), 0, s, c);
        else
            hipLaunchKernelGGL((k_gr_forward<DT, V, INPUT, true>), grid, dim3(256), 0, s, c);
    });
    return hipGetLastError();
}

template <bool BACK>
hipError_t launch(const GrCall &c, hipStream_t s) {
    if (c.dtype == LSTM_BF16) return c.i.p ? run<BF16, true, BACK>(c, s) : run<BF16, false, BACK>(c, s);
    return c.i.p ? run<F32, true, BACK>(c, s) : run<F32, false, BACK>(c, s);
}

template <class DT, bool INPUT>
hipError_t run_step(const GrStep &c, hipStream_t s) {
    // (no overlapping pieces here: the pool is read and written)
    auto go = [&](auto v) {
        constexpr int V = decltype(v)::value;
        const long long n = (long long)c.B * (c.width / V);
        hipLaunchKernelGGL((k_gr_step<DT, V, INPUT>), dim3((unsigned)((n + 63) / 64)), dim3(64), 0, s, c);
    };
    if (c.width % 4 == 0)
        go(std::integral_constant<int, 4>{});
    else
        go(std::integral_constant<int, 1>{});
    return hipGetLastError();
}

}  // namespace

void gr_segments(int T, int B, int width, int dtype, bool backward, int *nseg, int *seg_tokens) {
    const int V = dtype == LSTM_BF16 ? 8 : 4;
    const long long rows = (long long)B * ((width + V - 1) / V);  // threads of one segment
    // Two waves a SIMD, in segments of 32 tokens at least.
    long long n = (1 << 17) / rows;
    const long long most = (T + 31) / 32;
    if (n > most) n = most;
    if (n > 512) n = 512;
    if (n < 2) n = 1;
    const int per = (int)((T + n - 1) / n);
    *seg_tokens = per;
    *nseg = (T + per - 1) / per;
}

hipError_t launch_gr_forward(const GrCall &c, hipStream_t s) { return launch<false>(c, s); }
hipError_t launch_gr_backward(const GrCall &c, hipStream_t s) { return launch<true>(c, s); }

hipError_t launch_gr_step(const GrStep &c, hipStream_t s) {
    if (c.dtype == LSTM_BF16) return c.i.p ? run_step<BF16, true>(c, s) : run_step<BF16, false>(c, s);
    return c.i.p ? run_step<F32, true>(c, s) : run_step<F32, false>(c, s);
}

}  // namespace lstm_amd
