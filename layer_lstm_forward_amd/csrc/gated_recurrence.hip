// gated_recurrence.hip -- the gated linear recurrence, whole sequences forward
// and backward, and single tokens.
//     z = s(-f) (= 1 - a),  w = s(i) or z,  h_t = h_{t-1} - z h_{t-1} + w x_t
//     D_t = dy_t + E_{t+1},  E_t = D_t - z D_t  (E: what reaches h_{t-1})
//     dx = w D,  df = D (h_{t-1} - [w = z] x) z a,  di = D x w (1 - w)
// Two ways, chosen by an estimate of their times (gr_plan):
// k_gr_lanes: a thread walks the tokens of V neighbouring channels of a batch
// row, the next tokens' values under way meanwhile.  Where the channels do not
// fill the card the sequence is cut into segments: one launch takes each
// segment's own map (carry -> A carry + B, A the product of its 1 - z), one
// joins them, and one walks the segments from the carries that they begin with.
// Bound by memory: 512 x 256 x 2048 bf16 304 us forward, 597 backward (5.3 and
// 5.4 TB/s, as a copy).  In segments the inputs are read twice: 16384 tokens of
// 2048 channels 23 + 6 + 35 us, where one read would take 38.
// k_gr_tile, for little work: a workgroup spreads the tokens of 32 channels over
// its threads and scans their maps: one launch, and memory is read once, but the
// scan's steps wait for each other (333 x 5 x 1001 fp32 with an input gate:
// 12 + 17 us, against 33 + 53 in segments; 512 x 256 x 2048 bf16 570 + 946).
#include <type_traits>

#include "blocks.h"
#include "device.h"
#include "ops_dev.h"

namespace lstm_amd {
namespace {

constexpr int LN = 8;  // lanes of a token's channels in a tile: 32 channels

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

template <class DT>
__device__ inline const char *gr_at(const GrView &v, int b, int ch, int t) {
    return v.p + (v.t * t + v.b * b + ch) * (long long)sizeof(typename DT::S);
}

__device__ inline int gr_length(const GrCall &c, int b) {
    return c.lengths ? min(max(c.lengths[b], 0), c.T) : c.T;
}

// s(-f) and s(f), each with all its digits.
__device__ inline void gates(float f, float &z, float &a) {
    const float e = __builtin_amdgcn_exp2f(fabsf(f) * -1.4426950408889634f), big = __builtin_amdgcn_rcpf(1.0f + e);
    const float small = e * big;
    z = f < 0.0f ? big : small;
    a = f < 0.0f ? small : big;
}

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

// SUM: the segment's map, to the workspace; else the outputs.  Backward the
// tokens count from the segment's end.
template <class DT, int V, bool INPUT, bool BACK, bool SUM>
__global__ __launch_bounds__(256) void k_gr_lanes(GrCall c) {
    // tokens loaded at a time, and as many under way: with more tensors fewer
    constexpr int U = BACK && !SUM ? 4 : 8;
    int b, ch, own;
    if (!gr_place<V>(c, &b, &ch, &own)) return;
    const int sg = blockIdx.y, n = gr_length(c, b), t0 = sg * c.seg_tokens, t1 = min(t0 + c.seg_tokens, c.T);
    const int end = min(t1, n), count = end - t0;  // of the tokens that count
    const size_t slab = (size_t)c.B * c.width, at = (size_t)b * c.width + ch;
    float h[V], A[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = 0.0f, A[e] = 1.0f;
    if (!SUM) {
        const float *s = c.nseg > 1 ? c.seg + sg * slab : BACK ? c.ds1 : c.s0;
        if (s) __builtin_memcpy(h, s + at, sizeof(h));
    }
    struct Tokens {
        Raw<DT, V> x[U], f[U], g[U], d[U], p[U];
    } q[2];
    auto token = [&](int o) { return BACK ? end - 1 - o : t0 + o; };
    auto fetch = [&](Tokens &k, int o) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = token(min(o + u, count - 1));  // past the end: the last token again
            k.f[u].load(gr_at<DT>(c.f, b, ch, t));
            if (BACK) k.d[u].load(gr_at<DT>(c.dy, b, ch, t));
            if (!BACK || !SUM) {
                k.x[u].load(gr_at<DT>(c.x, b, ch, t));
                if (INPUT) k.g[u].load(gr_at<DT>(c.i, b, ch, t));
            }
            if (BACK && !SUM) k.p[u].load(gr_at<DT>(c.y, b, ch, max(t - 1, 0)));
        }
    };
    auto walk = [&](Tokens &k, int o) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (o + u >= count) break;
            const int t = token(o + u);
            float r[3][V], was[V];
            if (BACK && !SUM) {
#pragma unroll
                for (int e = 0; e < V; ++e) was[e] = k.p[u].at(e);
                if (t == 0) {
#pragma unroll
                    for (int e = 0; e < V; ++e) was[e] = 0.0f;
                    if (c.s0) __builtin_memcpy(was, c.s0 + at, sizeof(was));
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float z, a;
                if (BACK && !SUM)
                    gates(k.f[u].at(e), z, a);
                else
                    z = sigmoid_f(-k.f[u].at(e));
                if (!BACK) {
                    const float w = INPUT ? sigmoid_f(k.g[u].at(e)) : z;
                    h[e] = fmaf(w, k.x[u].at(e), fmaf(-z, h[e], h[e]));
                    r[0][e] = h[e];
                } else {
                    const float D = k.d[u].at(e) + h[e];
                    if (!SUM) {
                        const float x = k.x[u].at(e);
                        if (INPUT) {
                            float v, w;
                            gates(k.g[u].at(e), v, w);
                            r[0][e] = w * D;
                            r[1][e] = D * was[e] * (z * a);
                            r[2][e] = D * x * (w * v);
                        } else {
                            r[0][e] = z * D;
                            r[1][e] = D * (was[e] - x) * (z * a);
                        }
                    }
                    h[e] = fmaf(-z, D, D);
                }
                if (SUM) A[e] = fmaf(-z, A[e], A[e]);
            }
            if (!SUM && !BACK) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), r[0], own);
            if (!SUM && BACK) {
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), r[0], own);
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), r[1], own);
                if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), r[2], own);
            }
        }
    };
    if (count > 0) fetch(q[0], 0);
    for (int o = 0; o < count; o += 2 * U) {
        if (o + U < count) fetch(q[1], o + U);
        walk(q[0], o);
        if (o + 2 * U < count) fetch(q[0], o + 2 * U);
        walk(q[1], o + U);
    }
    if (SUM) {
        float *s = c.seg + sg * slab + at;
        gr_store<F32, V>(reinterpret_cast<char *>(s), h, own);
        gr_store<F32, V>(reinterpret_cast<char *>(s + c.nseg * slab), A, own);
        return;
    }
    const float zero[V] = {};
    for (int t = max(end, t0); t < t1; ++t) {
        if (!BACK) {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), zero, own);
        } else {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), zero, own);
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), zero, own);
            if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), zero, own);
        }
    }
    // the state is what the row's last token leaves (or a row of none has)
    float *const last = BACK ? (sg == 0 ? c.ds0 : nullptr) : (n > t0 || sg == 0) && n <= t1 ? c.s1 : nullptr;
    if (last) gr_store<F32, V>(reinterpret_cast<char *>(last + at), h, own);
}

// Each segment's B becomes the carry that it begins with: 16 threads a channel
// compose a sixteenth of the segments' maps each, then walk them from the
// carries that these give.
template <bool BACK>
__global__ __launch_bounds__(256) void k_gr_join(GrCall c) {
    __shared__ float maps[2][16][16];
    const size_t slab = (size_t)c.B * c.width;
    const int x = threadIdx.x % 16, y = threadIdx.x / 16;
    const size_t at = blockIdx.x * 16ull + x;
    const int per = (c.nseg + 15) / 16, k0 = min(y * per, c.nseg), k1 = min(k0 + per, c.nseg);
    auto segment = [&](int k) { return c.seg + (BACK ? c.nseg - 1 - k : k) * slab + at; };
    float A = 1.0f, B = 0.0f;
    if (at < slab)
#pragma unroll 8
        for (int k = k0; k < k1; ++k) {
            const float *s = segment(k);
            const float b = *s, a = s[c.nseg * slab];
            B = fmaf(a, B, b);
            A *= a;
        }
    maps[0][y][x] = A;
    maps[1][y][x] = B;
    __syncthreads();
    if (at >= slab) return;
    const float *first = BACK ? c.ds1 : c.s0;
    float carry = first ? first[at] : 0.0f;
    for (int i = 0; i < y; ++i) carry = fmaf(maps[0][i][x], carry, maps[1][i][x]);
#pragma unroll 8
    for (int k = k0; k < k1; ++k) {
        float *s = segment(k);
        const float b = *s, a = s[c.nseg * slab];
        *s = carry;
        carry = fmaf(a, carry, b);
    }
}

// A tile's threads: LN lanes x TC runs of U tokens.
template <int TC_, int U_>
struct GrTile {
    static constexpr int TC = TC_, U = U_, THREADS = LN * TC, WAVES = THREADS / 64;
};

// Each thread composes the maps of its U tokens, the workgroup scans the
// threads' maps, and each thread walks its tokens again from the carry that it
// begins with.  Backward the tokens count from the row's end.
template <class DT, int V, bool INPUT, bool BACK, class TL>
__global__ __launch_bounds__(TL::THREADS) void k_gr_tile(GrCall c) {
    constexpr int U = TL::U, TC = TL::TC, WAVES = TL::WAVES;
    __shared__ float maps[2][WAVES][LN][2 * V];  // the waves' maps of a tile, in turn
    const int l = threadIdx.x % LN, run = threadIdx.x / LN, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int slabs = (c.width + LN * V - 1) / (LN * V), b = blockIdx.x / slabs;
    const int from = (blockIdx.x % slabs * LN + l) * V, ch = min(from, c.width - V), own = from - ch;
    const int count = gr_length(c, b);  // tokens that count
    const size_t at = (size_t)b * c.width + ch;
    const float *first = BACK ? c.ds1 : c.s0;
    float *const last = BACK ? c.ds0 : c.s1;
    float carry[V];
#pragma unroll
    for (int e = 0; e < V; ++e) carry[e] = 0.0f;
    if (first) __builtin_memcpy(carry, first + at, sizeof(carry));
    auto tokens = [&](int o) { return BACK ? count - 1 - o : o; };
    struct Tokens {
        Raw<DT, V> x[U], f[U], g[U], d[U], h[U];
    };
    auto fetch = [&](Tokens &q, int o0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = tokens(min(o0 + u, count - 1));  // past the end: the last token again
            q.f[u].load(gr_at<DT>(c.f, b, ch, t));
            if (BACK) q.d[u].load(gr_at<DT>(c.dy, b, ch, t));
            q.x[u].load(gr_at<DT>(c.x, b, ch, t));
            if (INPUT) q.g[u].load(gr_at<DT>(c.i, b, ch, t));
            if (BACK) q.h[u].load(gr_at<DT>(c.y, b, ch, max(t - 1, 0)));
        }
    };
    int turn = 0;
    for (int o0 = 0; o0 < count; o0 += TC * U, turn ^= 1) {
        const int mine = o0 + run * U;
        Tokens q;
        fetch(q, mine);
        // the thread's own map
        float A[V], B[V], z[U][V], w[INPUT && !BACK ? U : 1][V];
        auto in = [&](int u, int e) {  // x or dy, 0 past the end
            return mine + u < count ? BACK ? q.d[u].at(e) : q.x[u].at(e) : 0.0f;
        };
        auto gate = [&](int u, int e) { return INPUT ? w[INPUT && !BACK ? u : 0][e] : z[u][e]; };
#pragma unroll
        for (int e = 0; e < V; ++e) A[e] = 1.0f, B[e] = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool on = mine + u < count;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                z[u][e] = on ? sigmoid_f(-q.f[u].at(e)) : 0.0f;
                if (BACK) {
                    const float D = in(u, e) + B[e];
                    B[e] = fmaf(-z[u][e], D, D);
                } else {
                    if (INPUT) w[INPUT && !BACK ? u : 0][e] = on ? sigmoid_f(q.g[u].at(e)) : 0.0f;
                    B[e] = fmaf(gate(u, e), in(u, e), fmaf(-z[u][e], B[e], B[e]));
                }
                A[e] = fmaf(-z[u][e], A[e], A[e]);
            }
        }
        // Scan: the threads of a wave with the same channels (LN lanes apart),
        // then the waves.  (A, B) after (A', B') is (A A', A B' + B).
#pragma unroll
        for (int s = LN; s < 64; s *= 2) {
            const bool on = lane >= s;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float a = __shfl_up(A[e], s), p = __shfl_up(B[e], s);
                B[e] = on ? fmaf(A[e], p, B[e]) : B[e];
                A[e] = on ? A[e] * a : A[e];
            }
        }
        if (lane >= 64 - LN)
#pragma unroll
            for (int e = 0; e < V; ++e) maps[turn][wave][l][e] = A[e], maps[turn][wave][l][V + e] = B[e];
        // what a thread begins with: the thread's before it in the wave
#pragma unroll
        for (int e = 0; e < V; ++e) {
            A[e] = __shfl_up(A[e], LN);
            B[e] = __shfl_up(B[e], LN);
            if (lane < LN) A[e] = 1.0f, B[e] = 0.0f;
        }
        __syncthreads();  // (the other buffer's readers are past this barrier's predecessor)
        float h[V];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (w == wave) h[e] = carry[e];
                const float a = maps[turn][w][l][e];
                carry[e] = fmaf(a, carry[e], maps[turn][w][l][V + e]);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = fmaf(A[e], h[e], B[e]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (mine + u >= count) break;
            const int t = tokens(mine + u);
            if (!BACK) {
#pragma unroll
                for (int e = 0; e < V; ++e) h[e] = fmaf(gate(u, e), in(u, e), fmaf(-z[u][e], h[e], h[e]));
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), h, own);
            } else {
                float was[V], dx[V], df[V], di[V];
#pragma unroll
                for (int e = 0; e < V; ++e) was[e] = q.h[u].at(e);
                if (t == 0) {
#pragma unroll
                    for (int e = 0; e < V; ++e) was[e] = 0.0f;
                    if (c.s0) __builtin_memcpy(was, c.s0 + at, sizeof(was));
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float D = in(u, e) + h[e], x = q.x[u].at(e);
                    float zz, a;
                    gates(q.f[u].at(e), zz, a);
                    if (INPUT) {
                        float v, w;
                        gates(q.g[u].at(e), v, w);
                        dx[e] = w * D;
                        df[e] = D * was[e] * (zz * a);
                        di[e] = D * x * (w * v);
                    } else {
                        dx[e] = zz * D;
                        df[e] = D * (was[e] - x) * (zz * a);
                    }
                    h[e] = fmaf(-z[u][e], D, D);
                }
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), dx, own);
                gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), df, own);
                if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), di, own);
            }
        }
        // the state after the last token
        if (last && mine < count && mine + U >= count) gr_store<F32, V>(reinterpret_cast<char *>(last + at), h, own);
    }
    const float zero[V] = {};
    for (int t = count + run; t < c.T; t += TC) {
        if (!BACK) {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), zero, own);
        } else {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), zero, own);
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), zero, own);
            if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), zero, own);
        }
    }
    if (last && count == 0 && run == 0) gr_store<F32, V>(reinterpret_cast<char *>(last + at), carry, own);
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

// Channels of a thread: four, or one where the row is shorter.  (Of bf16 eight,
// 16 bytes, give half as many waves: 512 x 256 x 2048 backward 745 us against 598.)
int piece(int width) { return width >= 4 ? 4 : 1; }

constexpr int kU = 4;  // tokens of a tile's thread

template <class DT, int V, bool INPUT, bool BACK>
void run_piece(const GrCall &c, hipStream_t s) {
    if (c.nseg == 0) {
        const dim3 grid((unsigned)(c.B * (long long)((c.width + LN * V - 1) / (LN * V))));
        auto go = [&](auto tile) {
            using TL = decltype(tile);
            hipLaunchKernelGGL((k_gr_tile<DT, V, INPUT, BACK, TL>), grid, dim3(TL::THREADS), 0, s, c);
        };
        if (c.T <= 8 * kU)
            go(GrTile<8, kU>{});
        else if (c.T <= 32 * kU)
            go(GrTile<32, kU>{});
        else
            go(GrTile<64, kU>{});
        return;
    }
    const long long threads = (long long)c.B * ((c.width + V - 1) / V);
    const dim3 grid((unsigned)((threads + 255) / 256), c.nseg);
    if (c.nseg > 1) {
        hipLaunchKernelGGL((k_gr_lanes<DT, V, INPUT, BACK, true>), grid, dim3(256), 0, s, c);
        hipLaunchKernelGGL(k_gr_join<BACK>, dim3((unsigned)(((long long)c.B * c.width + 15) / 16)), dim3(256), 0, s, c);
    }
    hipLaunchKernelGGL((k_gr_lanes<DT, V, INPUT, BACK, false>), grid, dim3(256), 0, s, c);
}

template <class DT, bool INPUT, bool BACK>
hipError_t run(const GrCall &c, hipStream_t s) {
    if (piece(c.width) == 4)
        run_piece<DT, 4, INPUT, BACK>(c, s);
    else
        run_piece<DT, 1, INPUT, BACK>(c, s);
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

// The way with the least estimated time.  nseg 0: tiles.
void gr_plan(int T, int B, int width, int dtype, bool backward, int *nseg, int *seg_tokens) {
    const int V = piece(width);
    const double lanes = (double)B * ((width + V - 1) / V);
    const double groups = (double)B * ((width + LN * V - 1) / (LN * V));
    const double bytes = (double)T * B * width * (dtype == LSTM_BF16 ? 2 : 4) * (backward ? 6 : 3);
    // Tiles of 256 tokens take 4 us alone and 9 where a CU has always one (6 and 15 backward).
    const double tiles = (T + 255) / 256;
    const double turns = groups * tiles / 256;
    double least = 3.0 + (backward ? 6.0 : 4.0) * tiles;
    if (turns > 1 && 3.0 + (backward ? 15.0 : 9.0) * turns > least) least = 3.0 + (backward ? 15.0 : 9.0) * turns;
    *nseg = 0;
    *seg_tokens = T;
    // Lanes: 2.5 us for eight tokens that a thread waits for, 5 TB/s, and with
    // segments two launches more and two thirds of the reads again.
    for (int n = 1; n <= 512 && (n == 1 || T / n >= 16); n *= 2) {
        const int per = (T + n - 1) / n;
        double wait = (per + 7) / 8 * (backward ? 4.0 : 2.5), stream = bytes / 5e6;
        if (lanes * n < 32768) stream *= 32768 / (lanes * n);
        double us = 3.0 + (wait > stream ? wait : stream);
        if (n > 1) us += 10.0 + ((per + 7) / 8 * 2.5 > stream * 0.6 ? (per + 7) / 8 * 2.5 : stream * 0.6);
        if (us < least) {
            least = us;
            *seg_tokens = per;
            *nseg = (T + per - 1) / per;
        }
    }
}

hipError_t launch_gr_forward(const GrCall &c, hipStream_t s) { return launch<false>(c, s); }
hipError_t launch_gr_backward(const GrCall &c, hipStream_t s) { return launch<true>(c, s); }

hipError_t launch_gr_step(const GrStep &c, hipStream_t s) {
    if (c.dtype == LSTM_BF16) return c.i.p ? run_step<BF16, true>(c, s) : run_step<BF16, false>(c, s);
    return c.i.p ? run_step<F32, true>(c, s) : run_step<F32, false>(c, s);
}

}  // namespace lstm_amd
