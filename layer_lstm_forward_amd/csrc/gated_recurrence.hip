// gated_recurrence.hip -- the gated linear recurrence, whole sequences forward
// and backward, and single tokens.
//     a = s(f),  z = s(-f) = 1 - a,  w = s(i) or z,  h_t = a h_{t-1} + w x_t
//     D_t = dy_t + E_{t+1},  E_t = a D_t  (E: what reaches h_{t-1})
//     dx = w D,  df = D (h_{t-1} - [w = z] x) z a,  di = D x w (1 - w)
// Three ways, chosen by an estimate of their times (gr_plan):
// k_gr_lanes: a thread walks the tokens of four neighbouring channels of a batch
// row, the next tokens' values under way meanwhile.  Bound by memory: 512 x 256 x
// 2048 bf16 316 us forward, 600 backward (5.1 and 5.4 TB/s, as a copy), 512 x 128 x
// 2048 fp32 297 and 622.
// k_gr_tile, for little work: a workgroup spreads a tile of tokens of 32 channels
// over its threads, composes their maps (carry -> A carry + B, A the product of
// the a), scans them and walks the tokens again from the carries that this
// gives: one launch, and memory is read once, but the steps of a tile wait for
// each other (333 x 5 x 1001 fp32 with an input gate: 13 + 20 us; 512 x 256 x
// 2048 bf16 730 + 1015).
// k_gr_tile in a chain, where channels are too few and tokens many: a workgroup a
// tile, which hands its map on, finds the carry that it begins with from the
// maps of the tiles before it, and hands on the carry that it ends with (a scan with
// look-back, as published for prefix sums in one pass).  One read of everything, and
// the results' bits do not depend on which tile is when (16384 x 1 x 2048 bf16 62 us
// forward, 127 backward, the memory's time 38 and 75; fp32 109 and 178; a launch for
// the maps of segments, one to join and one to walk them read it twice, and took 70
// and 113, fp32 122 and 319, when a gate cost fewer instructions).
#include <type_traits>

#include "blocks.h"
#include "device.h"
#include "ops_dev.h"

namespace lstm_amd {
namespace {

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
    __device__ void fill(float v) {
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] = round_to<DT>(v);
    }
    // Hides where the values come from: what is made of them before is made again
    // behind, instead of being kept in more registers than they take.
    __device__ void forget() {
        if constexpr (sizeof(s) % 4 == 0) {
            uint32_t w[sizeof(s) / 4];
            __builtin_memcpy(w, s, sizeof(s));
#pragma unroll
            for (unsigned i = 0; i < sizeof(s) / 4; ++i) asm volatile("" : "+v"(w[i]));
            __builtin_memcpy(s, w, sizeof(s));
        }
    }
};

template <class DT>
__device__ inline const char *gr_at(const GrView &v, int b, int ch, int t) {
    return v.p + (v.t * t + v.b * b + ch) * (long long)sizeof(typename DT::S);
}

__device__ inline int gr_length(const GrCall &c, int b) {
    return c.lengths ? min(max(c.lengths[b], 0), c.T) : c.T;
}

// s(f) and s(-f) of a logit, the smaller of them as precise as the larger, to (|f| + 3) 2^-23 of itself (0 below
// 2^-126).  What is kept of a value is taken from the smaller one, too: h - s(-f) h where the gate is near 1 and s(f) h
// where it is near 0; either form alone loses the digits of the other's end (s(f) 1e3 at f = -16 as 1e3 - s(16) 1e3 is
// off by 6%).
struct Gate {
    float f, small, big;
    __device__ explicit Gate(float logit) : f(logit) {
        const float e = __builtin_amdgcn_exp2f(fabsf(f) * -1.4426950408889634f);
        big = __builtin_amdgcn_rcpf(1.0f + e);
        small = e * big;
    }
    __device__ float on() const { return f < 0.0f ? small : big; }   // s(f)
    __device__ float off() const { return f > 0.0f ? small : big; }  // s(-f)
    __device__ float slope() const { return small * big; }           // s'(f)
    __device__ float share() const { return f > 0.0f ? -small : small; }
    // s(f) h; an infinite h stays what it is (h - part is 0 of finite ones).
    __device__ float keep(float h) const {
        const float part = __builtin_amdgcn_fmed3f(h, -3.4028235e38f, 3.4028235e38f);
        return fmaf(share(), part, f > 0.0f ? h : h - part);
    }
    // s(f) A of a map's factor, 0 < A <= 1.
    __device__ float keep_factor(float A) const { return fmaf(share(), A, f > 0.0f ? A : kLeast); }
    // Factors do not become 0, so that an infinite carry stays infinite however many gates lie between (2^-149 of a
    // finite one is 5e-7 at most).
    static constexpr float kLeast = 1.4e-45f;
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

// Backward the tokens count from the row's end.  Of bf16 without an input gate four waves a SIMD, for two spilled
// registers (256 x 512 x 2048 forward 315 us against 329 with 131 registers; with the gate three waves instead of two
// 440 against 422).
template <class DT, int V, bool INPUT, bool BACK>
__global__ __launch_bounds__(256, !BACK && !INPUT && sizeof(typename DT::S) == 2 ? 4 : 1) void k_gr_lanes(GrCall c) {
    // tokens loaded at a time, and as many under way: with more tensors fewer
    constexpr int U = BACK ? 4 : 8;
    int b, ch, own;
    if (!gr_place<V>(c, &b, &ch, &own)) return;
    const int count = gr_length(c, b);  // tokens that count
    const size_t at = (size_t)b * c.width + ch;
    const float *first = BACK ? c.ds1 : c.s0;
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = 0.0f;
    if (first) __builtin_memcpy(h, first + at, sizeof(h));
    struct Tokens {
        Raw<DT, V> x[U], f[U], g[U], d[U], p[U];
    } q[2];
    auto token = [&](int o) { return BACK ? count - 1 - o : o; };
    auto fetch = [&](Tokens &k, int o) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = token(min(o + u, count - 1));  // past the end: the last token again
            k.f[u].load(gr_at<DT>(c.f, b, ch, t));
            if (BACK) k.d[u].load(gr_at<DT>(c.dy, b, ch, t));
            k.x[u].load(gr_at<DT>(c.x, b, ch, t));
            if (INPUT) k.g[u].load(gr_at<DT>(c.i, b, ch, t));
            if (BACK) k.p[u].load(gr_at<DT>(c.y, b, ch, max(t - 1, 0)));
        }
    };
    auto walk = [&](Tokens &k, int o) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (o + u >= count) break;
            const int t = token(o + u);
            float r[3][V], was[V];
            if (BACK) {
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
                const Gate a(k.f[u].at(e));
                if (!BACK) {
                    const float w = INPUT ? sigmoid_f(k.g[u].at(e)) : a.off();
                    h[e] = fmaf(w, k.x[u].at(e), a.keep(h[e]));
                    r[0][e] = h[e];
                } else {
                    const float D = k.d[u].at(e) + h[e], x = k.x[u].at(e);
                    if (INPUT) {
                        const Gate w(k.g[u].at(e));
                        r[0][e] = w.on() * D;
                        r[1][e] = D * was[e] * a.slope();
                        r[2][e] = D * x * w.slope();
                    } else {
                        r[0][e] = a.off() * D;
                        r[1][e] = D * (was[e] - x) * a.slope();
                    }
                    h[e] = a.keep(D);
                }
            }
            if (!BACK) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), r[0], own);
            if (BACK) {
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
    const float zero[V] = {};
    for (int t = count; t < c.T; ++t) {
        if (!BACK) {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), zero, own);
        } else {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), zero, own);
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), zero, own);
            if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), zero, own);
        }
    }
    float *const last = BACK ? c.ds0 : c.s1;
    if (last) gr_store<F32, V>(reinterpret_cast<char *>(last + at), h, own);
}

// A tile's threads: LN lanes of V channels x TC runs of U tokens.  CHAIN: a
// workgroup takes one tile of a row, else all of them.
template <int LN_, int TC_, int U_, bool CHAIN_>
struct GrTile {
    static constexpr int LN = LN_, TC = TC_, U = U_, THREADS = LN * TC, WAVES = THREADS / 64;
    static constexpr bool CHAIN = CHAIN_;
};
// Of a chain: as many tokens a thread as its registers hold, at least kChainRun: a
// tile costs its workgroup 2.6 us that do not depend on its length (65536 x 1 x 2048
// bf16 309 us with 8 tokens a thread, 223 with 16, of 16 threads a channel; three
// workgroups a CU instead of two, whose registers spill, 313).  32 threads a channel
// halve the carry's way past the tiles (131072 x 1 x 256 bf16 100 -> 70 us, backward
// 238 -> 132), and cost what is bound by memory up to a tenth (65536 x 1 x 2048
// backward 423 -> 465, forward 231 now).
constexpr int kChainLanes = 16, kChainRuns = 32, kChainRun = 8;
template <class DT, bool INPUT, bool BACK>
using GrChain = GrTile<kChainLanes, kChainRuns, std::is_same_v<DT, BF16> && !INPUT && !BACK ? 16 : kChainRun, true>;
constexpr int chain_tiles(int T, int run) { return (T - 1) / (kChainRuns * run) + 1; }

// What the tiles of a chain hand on, a 64-bit word a channel, written and read at
// the coherence point and 0 when the launch begins: the tile's map, A with its
// sign set (A is not negative) beside B, and the carry after the tile, beside a 1.
enum { GR_MAP, GR_CARRY, GR_KINDS };
__device__ inline unsigned long long *gr_word(const GrCall &c, int kind, int tile, size_t at) {
    return c.words + ((size_t)kind * c.tiles + tile) * ((size_t)c.B * c.width) + at;
}

// Not 0 once a tile has given up its wait.
__device__ inline unsigned long long *gr_given_up(const GrCall &c) {
    return reinterpret_cast<unsigned long long *>(c.ticket) + 1;
}

__global__ __launch_bounds__(256) void k_gr_clear(u32x4 *p, size_t n) {
    for (size_t i = blockIdx.x * 256ull + threadIdx.x; i < n; i += gridDim.x * 256ull) p[i] = u32x4{0, 0, 0, 0};
}

// The carry that a tile begins with: that after the nearest tile before it which
// has handed its own on, taken through the maps of the tiles between.  Each run
// looks at one of the TC tiles before this one, again until one of them has
// (workgroups are numbered as they start, so those before this one run or are
// done, and the first waits for nobody).  Every tile's carry is its own map of the
// carry before it, so it does not matter which one is found: the bits are the same.
// A wait ends after c.patience ticks all the same (the words may have been cleared or
// written by another call on the same workspace), or once another tile's has: the
// carry is not a number then, and all workgroups come to their end.
// The first wave takes the maps in turn, hands on the carry after this tile (its
// map is P, Q), and tells the others.
template <int V, class TL>
__device__ inline void gr_carry_in(const GrCall &c, int tile, int l, int run, size_t at, int own, bool more,
                                   const float *P, const float *Q, float *carry) {
    constexpr int WINDOW = TL::TC, LN = TL::LN;
    static_assert(WINDOW <= 32, "a bit a tile");
    __shared__ float seen[WINDOW][LN][2][V];  // the map, or the carry in the place of B
    __shared__ int state[WINDOW][LN];         // 0: nothing yet, 1: the map, 2: the carry
    __shared__ float begin[LN][V];
    const int j = max(tile - 1 - run, 0);
    int st = 0, found = -1;
    unsigned spins = 0;
    long long since = 0;
    while (tile > 0) {
        if (__builtin_expect(c.patience < 0 || (++spins & 255) == 0, 0)) {
            const long long now = wall_clock64();
            if (spins == 256) since = now;
            const bool over = threadIdx.x == 0 && (now - since > c.patience || xload(gr_given_up(c)) != 0);
            if (__syncthreads_or(c.patience < 0 || over)) {
                found = 0;
                if (run == 0) {
                    xstore(gr_given_up(c), 1);
#pragma unroll
                    for (int e = 0; e < V; ++e) seen[0][l][1][e] = __builtin_nanf("");
                }
                __syncthreads();
                break;
            }
        }
        unsigned long long m[V], w[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[e] = xload(gr_word(c, GR_CARRY, j, at) + e);
            m[e] = st == 0 ? xload(gr_word(c, GR_MAP, j, at) + e) : 0;
        }
        bool map = run < tile && st == 0, all = run < tile;
#pragma unroll
        for (int e = 0; e < V; ++e) map = map && xtag(m[e]) != 0, all = all && xtag(w[e]) != 0;
        if (map && !all) {
            st = 1;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                seen[run][l][0][e] = fabsf(__uint_as_float(xtag(m[e])));
                seen[run][l][1][e] = __uint_as_float((uint32_t)m[e]);
            }
        }
        if (all) {
            st = 2;
#pragma unroll
            for (int e = 0; e < V; ++e) seen[run][l][1][e] = __uint_as_float((uint32_t)w[e]);
        }
        state[run][l] = st;
        __syncthreads();
        unsigned maps = 0, carries = 0;
#pragma unroll
        for (int back = 0; back < WINDOW; ++back) {
            const int s = state[back][l];
            maps |= (s == 1 ? 1u : 0u) << back;
            carries |= (s == 2 ? 1u : 0u) << back;
        }
        found = __ffs((int)carries) - 1;
        const unsigned nearer = carries ? (carries & -carries) - 1 : 0;
        if (__syncthreads_and(carries && (maps & nearer) == nearer)) break;
        __builtin_amdgcn_s_sleep(1);
    }
    if (threadIdx.x < 64) {
        if (tile > 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) carry[e] = seen[found][l][1][e];
#pragma unroll
            for (int back = WINDOW - 1; back >= 0; --back)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float next = fmaf(seen[back][l][0][e], carry[e], seen[back][l][1][e]);
                    carry[e] = back < found ? next : carry[e];
                }
        }
        if (run == 0) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (more && e >= own)
                    xstore(gr_word(c, GR_CARRY, tile, at) + e, xword(1, __float_as_uint(fmaf(P[e], carry[e], Q[e]))));
                begin[l][e] = carry[e];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) carry[e] = begin[l][e];
}

// Each thread composes the maps of its U tokens, the workgroup scans the
// threads' maps, and each thread walks its tokens again from the carry that it
// begins with.  Backward the tokens count from the row's end.
template <class DT, int V, bool INPUT, bool BACK, class TL>
__global__ __launch_bounds__(TL::THREADS) void k_gr_tile(GrCall c) {
    constexpr int U = TL::U, TC = TL::TC, LN = TL::LN, WAVES = TL::WAVES, TILE = TC * U;
    constexpr bool CHAIN = TL::CHAIN;
    __shared__ float maps[2][WAVES][LN][2 * V];  // the waves' maps of a tile, in turn
    const int l = threadIdx.x % LN, run = threadIdx.x / LN, wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int slabs = (c.width + LN * V - 1) / (LN * V);
    int group = blockIdx.x, tile = 0;
    if constexpr (CHAIN) {  // numbered as they start: all tiles before this one have started
        __shared__ unsigned number;
        if (threadIdx.x == 0) number = atomicAdd(c.ticket, 1u);
        __syncthreads();
        tile = (int)(number / (unsigned)(c.B * slabs));
        group = (int)(number % (unsigned)(c.B * slabs));
        if (tile >= c.tiles) return;  // only where another call counts on the same workspace
    }
    const int b = group / slabs;
    const int from = (group % slabs * LN + l) * V, ch = min(from, c.width - V), own = from - ch;
    const int count = gr_length(c, b);  // tokens that count
    const size_t at = (size_t)b * c.width + ch;
    const float *first = BACK ? c.ds1 : c.s0;
    float *const last = BACK ? c.ds0 : c.s1;
    float carry[V];
#pragma unroll
    for (int e = 0; e < V; ++e) carry[e] = 0.0f;
    if (first) __builtin_memcpy(carry, first + at, sizeof(carry));
    struct Tokens {
        Raw<DT, V> x[U], f[U], g[U], d[U], h[U];
    };
    // Token o + u of a walk is u steps from token o: pieces of whole rows and tiles
    // (plain) take their addresses from that alone.
    auto at_token = [&](const GrView &v, int o) { return gr_at<DT>(v, b, ch, BACK ? count - 1 - o : o); };
    auto step = [&](const GrView &v) { return (BACK ? -v.t : v.t) * (long long)sizeof(typename DT::S); };
    auto fetch = [&](auto plain, Tokens &q, int o) {
        auto get = [&](const GrView &v, Raw<DT, V> *to) {
            const char *p = at_token(v, decltype(plain)::value ? o : 0);
#pragma unroll
            for (int u = 0; u < U; ++u)  // past the end: the last token again
                to[u].load(p + (decltype(plain)::value ? u : min(o + u, count - 1)) * step(v));
        };
        get(c.f, q.f);
        if (BACK) get(c.dy, q.d);
        get(c.x, q.x);
        if (INPUT) get(c.i, q.g);
        if (BACK) {
            const char *p = at_token(c.y, o);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (decltype(plain)::value && u + 1 < U)
                    q.h[u].load(p + (u + 1) * step(c.y));
                else  // the first token has none before it
                    q.h[u].load(gr_at<DT>(c.y, b, ch, max(count - 2 - min(o + u, count - 1), 0)));
        }
    };
    int turn = 0;
    for (int o0 = tile * TILE; o0 < count; o0 += TILE, turn ^= 1) {
        const int mine = o0 + run * U;
        const bool plain = o0 + TILE <= count && c.width % V == 0;
        Tokens q;
        if (plain) {
            fetch(std::true_type{}, q, mine);
        } else {
            fetch(std::false_type{}, q, mine);
            // a token past the end changes nothing: z = 0 and x or dy = 0
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (mine + u >= count) {
                    q.f[u].fill(__builtin_huge_valf());
                    q.x[u].fill(0.0f);
                    if (INPUT) q.g[u].fill(0.0f);
                    if (BACK) q.d[u].fill(0.0f);
                }
        }
        // the thread's own map; forward also those up to each of its tokens
        float A[V], B[V], to[BACK ? 1 : U][2][V];
#pragma unroll
        for (int e = 0; e < V; ++e) A[e] = 1.0f, B[e] = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const Gate a(q.f[u].at(e));
                A[e] = a.keep_factor(A[e]);
                if (BACK) {
                    B[e] = a.keep(q.d[u].at(e) + B[e]);
                } else {
                    const float w = INPUT ? sigmoid_f(q.g[u].at(e)) : a.off();
                    B[e] = fmaf(w, q.x[u].at(e), a.keep(B[e]));
                    to[BACK ? 0 : u][0][e] = A[e];
                    to[BACK ? 0 : u][1][e] = B[e];
                }
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
                A[e] = on ? fmaf(A[e], a, Gate::kLeast) : A[e];
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
        if constexpr (CHAIN) {
            const bool more = o0 + TILE < count;
            float P[V], Q[V];
#pragma unroll
            for (int e = 0; e < V; ++e) P[e] = 1.0f, Q[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float a = maps[turn][w][l][e];
                    Q[e] = fmaf(a, Q[e], maps[turn][w][l][V + e]);
                    P[e] = fmaf(P[e], a, Gate::kLeast);
                }
            if (more && tile > 0 && run == 0)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (e >= own)
                        xstore(gr_word(c, GR_MAP, tile, at) + e,
                               xword(__float_as_uint(P[e]) | 0x80000000u, __float_as_uint(Q[e])));
            gr_carry_in<V, TL>(c, tile, l, run, at, own, more, P, Q, carry);
        }
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
        auto walk = [&](auto plain) {
            constexpr bool PLAIN = decltype(plain)::value;
            char *const p[3] = {const_cast<char *>(at_token(BACK ? c.dx : c.y, mine)),
                                const_cast<char *>(BACK ? at_token(c.df, mine) : nullptr),
                                const_cast<char *>(BACK && INPUT ? at_token(c.di, mine) : nullptr)};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!PLAIN && mine + u >= count) break;
                const int part = PLAIN ? 0 : own;
                if (!BACK) {
                    float y[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = fmaf(to[BACK ? 0 : u][0][e], h[e], to[BACK ? 0 : u][1][e]);
                    gr_store<DT, V>(p[0] + u * step(c.y), y, part);
                    if (last && (!PLAIN || u == U - 1) && mine + u == count - 1) gr_store<F32, V>(reinterpret_cast<char *>(last + at), y, part);
                } else {
                    q.f[u].forget();
                    q.d[u].forget();
                    float was[V], dx[V], df[V], di[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) was[e] = q.h[u].at(e);
                    if ((!PLAIN || u == U - 1) && mine + u == count - 1) {  // the row's first token
#pragma unroll
                        for (int e = 0; e < V; ++e) was[e] = 0.0f;
                        if (c.s0) __builtin_memcpy(was, c.s0 + at, sizeof(was));
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float D = q.d[u].at(e) + h[e], x = q.x[u].at(e);
                        const Gate a(q.f[u].at(e));
                        if (INPUT) {
                            const Gate w(q.g[u].at(e));
                            dx[e] = w.on() * D;
                            df[e] = D * was[e] * a.slope();
                            di[e] = D * x * w.slope();
                        } else {
                            dx[e] = a.off() * D;
                            df[e] = D * (was[e] - x) * a.slope();
                        }
                        h[e] = a.keep(D);
                    }
                    gr_store<DT, V>(p[0] + u * step(c.dx), dx, part);
                    gr_store<DT, V>(p[1] + u * step(c.df), df, part);
                    if (INPUT) gr_store<DT, V>(p[2] + u * step(c.di), di, part);
                    if (last && (!PLAIN || u == U - 1) && mine + u == count - 1) gr_store<F32, V>(reinterpret_cast<char *>(last + at), h, part);
                }
            }
        };
        if (plain)
            walk(std::true_type{});
        else
            walk(std::false_type{});
        if (CHAIN) break;
    }
    const float zero[V] = {};
    const int stop = CHAIN ? min(c.T, (tile + 1) * TILE) : c.T;
    for (int t = max(count, tile * TILE) + run; t < stop; t += TC) {
        if (!BACK) {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.y, b, ch, t)), zero, own);
        } else {
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.dx, b, ch, t)), zero, own);
            gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.df, b, ch, t)), zero, own);
            if (INPUT) gr_store<DT, V>(const_cast<char *>(gr_at<DT>(c.di, b, ch, t)), zero, own);
        }
    }
    if (last && count == 0 && run == 0 && tile == 0) gr_store<F32, V>(reinterpret_cast<char *>(last + at), carry, own);
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
        const Gate a(f[e]);
        const float w = INPUT ? sigmoid_f(g[e]) : a.off();
        h[e] = fmaf(w, x[e], a.keep(h[e]));
    }
    __builtin_memcpy(s, h, sizeof(h));
    gr_store<DT, V>(y, h);
}

// Channels of a thread: four, or one where the row is shorter.  (Of bf16 eight,
// 16 bytes, give half as many waves: 512 x 256 x 2048 backward 745 us against 598.)
int piece(int width) { return width >= 4 ? 4 : 1; }

long long groups_of(int B, int width, int lanes, int V) { return B * (long long)((width + lanes * V - 1) / (lanes * V)); }

template <class DT, int V, bool INPUT, bool BACK>
void run_piece(GrCall c, hipStream_t s) {
    auto tiles = [&](auto tile) {
        using TL = decltype(tile);
        c.tiles = TL::CHAIN ? chain_tiles(c.T, TL::U) : 1;
        const unsigned n = (unsigned)(groups_of(c.B, c.width, TL::LN, V) * c.tiles);
        if (TL::CHAIN) {
            const size_t pieces = 16 + (size_t)GR_KINDS * c.tiles * c.B * c.width / 2;  // of 16 bytes: counter, words
            hipLaunchKernelGGL(k_gr_clear, dim3((unsigned)(pieces < 256 * 1024 ? (pieces + 255) / 256 : 1024)), dim3(256),
                               0, s, reinterpret_cast<u32x4 *>(c.ticket), pieces);
        }
        hipLaunchKernelGGL((k_gr_tile<DT, V, INPUT, BACK, TL>), dim3(n), dim3(TL::THREADS), 0, s, c);
    };
    if (c.way == GR_CHAIN) {
        tiles(GrChain<DT, INPUT, BACK>{});
    } else if (c.way == GR_TILES) {
        if (c.T <= 32)
            tiles(GrTile<8, 8, 4, false>{});
        else if (c.T <= 128)
            tiles(GrTile<8, 32, 4, false>{});
        else
            tiles(GrTile<8, 64, 4, false>{});
    } else {
        const long long threads = (long long)c.B * ((c.width + V - 1) / V);
        hipLaunchKernelGGL((k_gr_lanes<DT, V, INPUT, BACK>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, c);
    }
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

// Bytes of a chain's workspace: the counter that numbers its workgroups, and its words.
size_t gr_words(int T, int B, int width) {
    return 256 + ((size_t)GR_KINDS * chain_tiles(T, kChainRun) * B * width * 8 + 255) / 256 * 256;
}

// The way with the least estimated time, by the bytes without an input gate (the
// workspace query does not know of one).
GrWay gr_plan(int T, int B, int width, int dtype, bool backward) {
    const int V = piece(width);
    const double lanes = (double)B * ((width + V - 1) / V);
    const double stream = (double)T * B * width * (dtype == LSTM_BF16 ? 2 : 4) * (backward ? 6 : 3) / 5e6;  // at 5 TB/s
    // Tiles of 256 tokens take 4 us alone and 9 where a CU has always one (6 and 15 backward).
    const double n = (T + 255) / 256, turns = groups_of(B, width, 8, V) * n / 256;
    const double alone = (backward ? 6.0 : 4.0) * n, busy = turns > 1 ? (backward ? 15.0 : 9.0) * turns : 0.0;
    double least = 3.0 + (alone > busy ? alone : busy);
    GrWay way = GR_TILES;
    // Lanes: 2.5 us for eight tokens that a thread waits for (4 backward), all of the memory's rate from 32768 on.
    const double wait = (T + 7) / 8 * (backward ? 4.0 : 2.5), rate = lanes < 32768 ? stream * 32768 / lanes : stream;
    const double walk = 3.0 + (wait > rate ? wait : rate);
    if (walk < least) {
        least = walk;
        way = GR_LANES;
    }
    // A chain: two launches, and the memory's time by 1.35, or 0.25 us for the carry's way past a tile; its grid holds
    // 2^23 workgroups (of 2^9 threads).
    const int parts = chain_tiles(T, kChainRun);
    const double chain = 14.0 + (1.35 * stream > 0.25 * parts ? 1.35 * stream : 0.25 * parts);
    if (parts > 1 && groups_of(B, width, kChainLanes, V) * parts < (1 << 23) && chain < least) way = GR_CHAIN;
    return way;
}

hipError_t launch_gr_forward(const GrCall &c, hipStream_t s) { return launch<false>(c, s); }
hipError_t launch_gr_backward(const GrCall &c, hipStream_t s) { return launch<true>(c, s); }

hipError_t launch_gr_step(const GrStep &c, hipStream_t s) {
    if (c.dtype == LSTM_BF16) return c.i.p ? run_step<BF16, true>(c, s) : run_step<BF16, false>(c, s);
    return c.i.p ? run_step<F32, true>(c, s) : run_step<F32, false>(c, s);
}

}  // namespace lstm_amd
