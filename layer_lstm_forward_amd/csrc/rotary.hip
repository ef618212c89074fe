// rotary.hip -- the norm of each head and the rotation by its token's position,
// forward and backward.
//     r = 1 / sqrt(mean x^2 + eps), u = x r w, each pair (u_a, u_b) turned by p f_j
//     g = the output's gradient turned back, dx = r (g w - x r mean(g w x r)), dw = sum of g x r
// Bound by memory: 131072 tokens of 24 heads of 128 bf16 313 us forward, 501
// backward, 6 to join the weights' sums (5.2 and 4.8 TB/s).  A head's row lies over L lanes of a wave, each with two
// pieces of P values: the two halves of P pairs, so that a rotation needs no
// other lane's values.  A lane keeps its pairs' sines and cosines for all heads
// of a token that it takes.
#include "blocks.h"
#include "device.h"
#include "ops_dev.h"

namespace lstm_amd {
namespace {

constexpr int AHEAD = 4;  // heads loaded at a time

// What lane `j` of a row holds: values lo..lo+P-1 and hi..hi+P-1, turned pair
// by pair (half layout: lo[e] with hi[e]; neighbours: the 2P values from lo on).
template <int P>
struct Block {
    int lo, hi, pair;  // first pair's number, or -1: not turned
    bool on, odd;      // odd: only lo's one value exists (P = 1)
    __device__ void place(const RotCall &c, int j) {
        const int turned = c.rot / 2 / P;  // whole blocks: P divides rot / 2
        on = j * 2 * P < c.dim;
        odd = false;
        if (j < turned) {
            pair = j * P;
            lo = c.pairs ? 2 * j * P : j * P;
            hi = c.pairs ? lo + P : lo + c.rot / 2;
        } else {
            pair = -1;
            lo = 2 * j * P;
            hi = lo + P;
            odd = hi >= c.dim;
        }
    }
};

// The block's values of a row as they are in memory.
template <class DT, int P>
struct Row {
    typename DT::S s[2 * P];
    __device__ void load(const char *row, const Block<P> &b) {
        const typename DT::S *q = reinterpret_cast<const typename DT::S *>(row);
        __builtin_memcpy(s, q + b.lo, sizeof(s) / 2);
        if (!(P == 1 && b.odd))
            __builtin_memcpy(s + P, q + b.hi, sizeof(s) / 2);
        else
            s[P] = (typename DT::S)0;
    }
    __device__ void values(bool on, float *v) const {
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) v[e] = on ? DT::to_f(s[e]) : 0.0f;
    }
};

template <class DT, int P>
__device__ inline void rot_store(char *row, const Block<P> &b, const float *v) {
    using S = typename DT::S;
    S *q = reinterpret_cast<S *>(row), s[2 * P];
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) s[e] = round_to<DT>(v[e]);
    __builtin_memcpy(q + b.lo, s, sizeof(s) / 2);
    if (!(P == 1 && b.odd)) __builtin_memcpy(q + b.hi, s + P, sizeof(s) / 2);
}

// Pairs of the block turned by their angles (BACK: back).  A pair is (v[e],
// v[P + e]) in the half layout and (v[2e], v[2e + 1]) for neighbours; P = 1 is both.
template <int P, bool PAIRS, bool BACK>
__device__ inline void turn(float *v, const float *co, const float *si) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
        float &a = v[PAIRS ? 2 * e : e], &b = v[PAIRS ? 2 * e + 1 : P + e];
        const float s = BACK ? -si[e] : si[e], x = a, y = b;
        a = x * co[e] - y * s;
        b = y * co[e] + x * s;
    }
}

// Angles p f_j in 64 bits, as parts of a turn.  bf16 takes the hardware's sine and
// cosine of parts of a turn, whose error (below 2^-18) is lost in the results'
// rounding; fp32 the library's.
template <class DT, int P>
__device__ inline void angles(const RotCall &c, const Block<P> &b, int p, float *co, float *si) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
        co[e] = 1.0f;
        si[e] = 0.0f;
        if (b.pair >= 0) {
            const double turns = (double)p * c.freq[b.pair + e] * 0.15915494309189535;
            const float part = (float)(turns - __builtin_rint(turns));
            if (sizeof(typename DT::S) == 2) {
                si[e] = __builtin_amdgcn_sinf(part);
                co[e] = __builtin_amdgcn_cosf(part);
            } else {
                sincospif(2.0f * part, &si[e], &co[e]);
            }
            si[e] *= c.scale;
            co[e] *= c.scale;
        }
    }
}

template <int L>
__device__ inline float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Workgroup (x, y): tokens from x on, the y-th run of c.run heads (queries
// first).  NB blocks a lane.
template <class DT, int P, int L, int NB, bool PAIRS, bool BACK>
__global__ __launch_bounds__(256) void k_rot(RotCall c) {
    constexpr int GROUPS = 256 / L;
    __shared__ float sums[BACK ? GROUPS * L * NB * 2 * P : 1];
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const int cq = (c.side[0].heads + c.run - 1) / c.run;
    const int which = (int)blockIdx.y >= cq;
    const RotSide &s = c.side[which];
    const int h0 = (blockIdx.y - (which ? cq : 0)) * c.run, h1 = min(h0 + c.run, s.heads);
    constexpr long long ES = sizeof(typename DT::S);
    const float inv = 1.0f / (float)c.dim;
    Block<P> b[NB];
    float w[NB][2 * P], dw[NB][2 * P];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
        b[k].place(c, lane + k * L);
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) w[k][e] = 1.0f, dw[k][e] = 0.0f;
        if (s.w && b[k].on) {
            Row<DT, P> row;
            row.load(s.w, b[k]);
            row.values(true, w[k]);
        }
    }
    const int tokens = c.T * c.B;
    for (long long tok = (long long)blockIdx.x * GROUPS + group; tok < tokens; tok += (long long)gridDim.x * GROUPS) {
        const int t = (int)(tok / c.B), bt = (int)(tok % c.B);
        const int p = c.pos ? c.pos[c.pos_t * t + c.pos_b * bt] : t;
        const char *x = s.x.p + (s.x.t * t + s.x.b * bt) * ES;
        const char *yi = s.y.p + (s.y.t * t + s.y.b * bt) * ES;
        char *out = BACK ? s.dx.p + (s.dx.t * t + s.dx.b * bt) * ES : const_cast<char *>(yi);
        const long long oh = (BACK ? s.dx.h : s.y.h) * ES;
        Row<DT, P> rx[AHEAD][NB], ry[BACK ? AHEAD : 1][NB];
        auto fetch = [&](int h) {
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const long long q = min(h + a, h1 - 1);  // past the last head: it again
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    if (!b[k].on) continue;
                    if (!BACK || c.norm) rx[a][k].load(x + q * s.x.h * ES, b[k]);
                    if (BACK) ry[BACK ? a : 0][k].load(yi + q * s.y.h * ES, b[k]);
                }
            }
        };
        fetch(h0);
        float co[NB][P], si[NB][P];
#pragma unroll
        for (int k = 0; k < NB; ++k) angles<DT, P>(c, b[k], p, co[k], si[k]);
#pragma unroll 1
        for (int h = h0; h < h1; h += AHEAD) {
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                if (h + a >= h1) break;
                __builtin_amdgcn_sched_barrier(0);  // one head after the other, or all are widened at once
                float v[NB][2 * P], r = 1.0f;
#pragma unroll
                for (int k = 0; k < NB; ++k) rx[a][k].values(b[k].on && (!BACK || c.norm), v[k]);
                if (c.norm) {
                    float ss = 0.0f;
#pragma unroll
                    for (int k = 0; k < NB; ++k)
#pragma unroll
                        for (int e = 0; e < 2 * P; ++e) ss += v[k][e] * v[k][e];
                    r = 1.0f / sqrtf(lanes_sum<L>(ss) * inv + c.eps);
                }
                if (!BACK) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        if (c.norm)
#pragma unroll
                            for (int e = 0; e < 2 * P; ++e) v[k][e] *= r * w[k][e];
                        if (b[k].pair >= 0) turn<P, PAIRS, false>(v[k], co[k], si[k]);
                        if (b[k].on) rot_store<DT, P>(out + (h + a) * oh, b[k], v[k]);
                    }
                } else {
                    float g[NB][2 * P], dot = 0.0f;
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        ry[BACK ? a : 0][k].values(b[k].on, g[k]);
                        if (b[k].pair >= 0) turn<P, PAIRS, true>(g[k], co[k], si[k]);
                        if (c.norm)
#pragma unroll
                            for (int e = 0; e < 2 * P; ++e) {
                                v[k][e] *= r;
                                dw[k][e] += g[k][e] * v[k][e];
                                g[k][e] *= w[k][e];
                                dot += g[k][e] * v[k][e];
                            }
                    }
                    if (c.norm) dot = lanes_sum<L>(dot) * inv;
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        if (c.norm)
#pragma unroll
                            for (int e = 0; e < 2 * P; ++e) g[k][e] = r * (g[k][e] - v[k][e] * dot);
                        if (b[k].on) rot_store<DT, P>(out + (h + a) * oh, b[k], g[k]);
                    }
                }
            }
            if (h + AHEAD < h1) fetch(h + AHEAD);
        }
    }
    if (!BACK || !c.part) return;
    // the workgroup's sums, group by group
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) sums[(group * NB * 2 * P + k * 2 * P + e) * L + lane] = dw[k][e];
    __syncthreads();
    float *part = c.part + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * c.dim;
    constexpr int COLS = L * NB * 2 * P;
    for (int q = threadIdx.x; q < COLS; q += 256) {
        const int j = q % L, e = q / L % (2 * P), k = q / L / (2 * P);
        Block<P> of;
        of.place(c, j + k * L);
        const int i = e < P ? of.lo + e : of.hi + e - P;
        if (!of.on || i >= c.dim) continue;
        float sum = 0.0f;
#pragma unroll
        for (int y = 0; y < GROUPS; ++y) sum += sums[y * COLS + q];
        part[i] = sum;
    }
}

// The workgroups' sums of a side in their order: 32 threads take every 32nd of a
// column's, then their sums are added.
template <class DT>
__global__ __launch_bounds__(1024) void k_rot_join(RotCall c) {
    __shared__ float lds[32][33];
    const int which = blockIdx.y, x = threadIdx.x % 32, y = threadIdx.x / 32, i = blockIdx.x * 32 + x;
    const RotSide &s = c.side[which];
    const int cq = (c.side[0].heads + c.run - 1) / c.run, ck = (c.side[1].heads + c.run - 1) / c.run;
    const int n = (which ? ck : cq) * c.parts;
    const float *part = c.part + (which ? (size_t)cq * c.parts * c.dim : 0);
    float sum = 0.0f;
    if (i < c.dim)
#pragma unroll 8
        for (int p = y; p < n; p += 32) sum += part[(size_t)p * c.dim + i];
    lds[y][x] = sum;
    __syncthreads();
    if (y > 0 || i >= c.dim || !s.dw) return;
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) sum += lds[k][x];
    reinterpret_cast<typename DT::S *>(s.dw)[i] = round_to<DT>(sum);
}

template <class DT, int P, int L, int NB, bool BACK>
void run(const RotCall &c, hipStream_t s) {
    const int runs = (c.side[0].heads + c.run - 1) / c.run + (c.side[1].heads + c.run - 1) / c.run;
    const long long n = ((long long)c.T * c.B + 256 / L - 1) / (256 / L), most = BACK ? c.parts : 65536;
    RotCall d = c;
    d.parts = (int)(n < most ? n : most);
    if (P > 1 && c.pairs)
        hipLaunchKernelGGL((k_rot<DT, P, L, NB, true, BACK>), dim3(d.parts, runs), dim3(256), 0, s, d);
    else
        hipLaunchKernelGGL((k_rot<DT, P, L, NB, false, BACK>), dim3(d.parts, runs), dim3(256), 0, s, d);
    if (BACK && c.part)
        hipLaunchKernelGGL(k_rot_join<DT>, dim3((c.dim + 31) / 32, c.side[1].heads ? 2 : 1), dim3(1024), 0, s, d);
}

// Lanes of a row: as many as it has blocks (of 256 values at most).
template <class DT, int P, bool BACK, int L = 8>
void lanes(const RotCall &c, hipStream_t s) {
    const int n = (c.dim + 2 * P - 1) / (2 * P);
    if (n <= L)
        run<DT, P, L, 1, BACK>(c, s);
    else if constexpr (L < 64 && L * 2 * P < 256)
        lanes<DT, P, BACK, 2 * L>(c, s);
    else if constexpr (L * 2 * P < 256)
        run<DT, P, L, 2, BACK>(c, s);
}

// The widest piece that divides both halves of the turned part and of the rest.
template <class DT, bool BACK>
hipError_t pieces(const RotCall &c, hipStream_t s) {
    auto fits = [&](int p) { return c.rot / 2 % p == 0 && (c.dim - c.rot) % (2 * p) == 0; };
    if (DT::PER16 == 8 && fits(8))
        lanes<DT, DT::PER16, BACK>(c, s);
    else if (fits(4))
        lanes<DT, 4, BACK>(c, s);
    else if (fits(2))
        lanes<DT, 2, BACK>(c, s);
    else
        lanes<DT, 1, BACK>(c, s);
    return hipGetLastError();
}

}  // namespace

// Heads of a run: a token's angles are computed once a run, so the more the
// better, while there are about eight workgroups a CU (131072 tokens of 24 heads
// of 128 bf16: 358 us forward in runs of 8, 304 in runs of 16; 16 tokens: 8.2
// against 12.2 us).  Workgroups that keep sums of a run's weight gradients:
// enough to fill the card, few enough that joining their sums is cheap.
void rot_plan(long long tokens, int heads, int kv_heads, int dim, int *run, int *runs, int *parts) {
    const long long groups = tokens * (heads + kv_heads) * dim / 4096;  // of runs of one head
    *run = 32;
    while (*run > 4 && groups / *run < 2048) *run /= 2;
    *runs = (heads + *run - 1) / *run + (kv_heads + *run - 1) / *run;
    const int most = *runs < 16 ? 2048 / *runs : 128;
    *parts = tokens < most ? (int)tokens : most;
}

hipError_t launch_rot_forward(const RotCall &c, hipStream_t s) {
    return c.dtype == LSTM_BF16 ? pieces<BF16, false>(c, s) : pieces<F32, false>(c, s);
}
hipError_t launch_rot_backward(const RotCall &c, hipStream_t s) {
    return c.dtype == LSTM_BF16 ? pieces<BF16, true>(c, s) : pieces<F32, true>(c, s);
}

}  // namespace lstm_amd
