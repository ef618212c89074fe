// gated_mlp.hip -- the products of the gated feed-forward block, each with the
// elementwise work that follows it:
//     GATE   g = x Wg^T, u = x Wu^T, h = act(g) u
//     STORE  y = h Wd^T;  dx = dg Wg + du Wu;  dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//     DGATE  dh = dy Wd, dg = dh u act'(g), du = dh act(g)
// One kernel body runs all of them on v_mfma_f32_32x32x16_bf16.
#include <type_traits>

#include "blocks.h"
#include "device.h"
#include "ops_dev.h"

namespace lstm_amd {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int KS = 64;  // of the contraction, a stage

// The pairs of planes whose products make one product of fp32 matrices, the
// smallest first: what they leave out is below 2^-24 of each operand.
__device__ constexpr int kPairA[6] = {2, 1, 0, 1, 0, 0}, kPairB[6] = {0, 1, 2, 0, 1, 0};

// ------------------------------------------------------------- elementwise
struct Act {
    float a, slope;  // act(g), act'(g)
};

template <bool SLOPE>
__device__ inline Act activate(int kind, float g) {
    Act r;
    r.slope = 0.0f;
    if (kind == LSTM_ACT_GELU) {
        // g s(2t), t = k (g + c g^3); past |g| = 32 s is 0 or 1 in fp32, and
        // the clamp keeps 0 times infinity out of the slope
        constexpr float k = 0.7978845608028654f, c = 0.044715f;
        const float q = fminf(fmaxf(g, -32.0f), 32.0f), q2 = q * q;
        const float t = 2.0f * k * q * (1.0f + c * q2), p = sigmoid_f(t);
        r.a = g * p;
        if (SLOPE) r.slope = p + q * (p * sigmoid_f(-t)) * (2.0f * k * (1.0f + 3.0f * c * q2));
    } else {
        const float p = sigmoid_f(g), n = sigmoid_f(-g);
        if (kind == LSTM_ACT_SIGMOID) {
            r.a = p;
            if (SLOPE) r.slope = p * n;
        } else {
            r.a = g * p;
            if (SLOPE) r.slope = p + r.a * n;
        }
    }
    return r;
}

__device__ inline u32x4 pack8(const float *v) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = (uint32_t)round_to<BF16>(v[2 * i]) | (uint32_t)round_to<BF16>(v[2 * i + 1]) << 16;
    return o;
}

__device__ inline void unpack8(u32x4 x, float *v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(x[i] << 16);
        v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
}

// The first term of an fp32 value, to nearest; the largest finite values, whose
// nearest would be infinite, are cut.  The rest is exact in fp32.
__device__ inline float first_term(float v) {
    const float t = BF16::to_f(round_to<BF16>(v));
    return fabsf(t) <= 3.4e38f ? t : __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
}

// Eight values as an operand's planes at element `at`.
template <bool F32_>
__device__ inline void store_planes(const MlpOperand &o, size_t at, const float *v) {
    char *p = const_cast<char *>(o.p) + at * 2;
    if constexpr (!F32_) {
        *reinterpret_cast<u32x4 *>(p) = pack8(v);
    } else {
        float t[8], rest[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = first_term(v[i]), rest[i] = v[i] - t[i];
        *reinterpret_cast<u32x4 *>(p) = pack8(t);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = first_term(rest[i]), rest[i] -= t[i];
        *reinterpret_cast<u32x4 *>(p + o.plane) = pack8(t);
        *reinterpret_cast<u32x4 *>(p + 2 * o.plane) = pack8(rest);
    }
}

// Eight values of a matrix of the call's dtype, 16-byte aligned.
template <bool F32_>
__device__ inline void load8(const char *p, size_t at, float *v) {
    if constexpr (F32_) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(p + at * 4);
        const f32x4 x = q[0], y = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
    } else {
        unpack8(*reinterpret_cast<const u32x4 *>(p + at * 2), v);
    }
}

template <bool F32_>
__device__ inline void store8(char *p, size_t at, const float *v) {
    if constexpr (F32_) {
        f32x4 *q = reinterpret_cast<f32x4 *>(p + at * 4);
        q[0] = f32x4{v[0], v[1], v[2], v[3]};
        q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4 *>(p + at * 2) = pack8(v);
    }
}

// What follows a product: eight sums of one row, from column `col` (a multiple
// of 8, below N) on.  GATE: v are gate's and w up's.
template <int EPI, bool F32_>
__device__ inline void finish(const MlpCall &c, const MlpProduct &p, int row, int col, float *v, float *w) {
    if constexpr (EPI == MLP_STORE) {
        using DT = std::conditional_t<F32_, F32, BF16>;
        if (p.vec && col + 8 <= p.N) {
            store8<F32_>(p.out, (size_t)row * p.ldo + col, v);
        } else {
            auto *o = reinterpret_cast<typename DT::S *>(p.out) + (size_t)row * p.ldo + col;
            for (int i = 0; i < 8 && col + i < p.N; ++i) o[i] = round_to<DT>(v[i]);
        }
    } else if constexpr (EPI == MLP_GATE) {
        // columns past N are 0 (the operand's rows past N read as zeros), and
        // so are act(0) 0: the next product may run over them
        const size_t at = (size_t)row * c.ld + col;
        if (c.gate) {
            store8<F32_>(c.gate, at, v);
            store8<F32_>(c.up, at, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate<false>(c.act, v[i]).a * w[i];
        store_planes<F32_>(c.product, (size_t)row * c.product.ld + col, v);
    } else {
        float g[8], u[8];
        const size_t at = (size_t)row * c.ld + col;
        load8<F32_>(c.gate, at, g);
        load8<F32_>(c.up, at, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Act r = activate<true>(c.act, g[i]);
            const bool in = col + i < p.N;  // past N the sums are of another row's weights
            g[i] = in ? v[i] * u[i] * r.slope : 0.0f;
            u[i] = in ? v[i] * r.a : 0.0f;
        }
        store_planes<F32_>(c.dgate, (size_t)row * c.dgate.ld + col, g);
        store_planes<F32_>(c.dup, (size_t)row * c.dup.ld + col, u);
    }
}

// ------------------------------------------------------------------ operands
// One stage of an operand lies in LDS as ROWS rows of 64 values (k along the
// rows) or as 64 rows of ROWS values (k along the columns), filled by loads
// that write 64 16-byte pieces to consecutive places, so the place decides
// which piece a lane fetches.  Pieces are permuted inside a row such that the
// lanes of a fragment read fall on all banks:
//   rows of 64 values (128 bytes): piece p of row r lies at p ^ (r / 2 % 8);
//   columns: 64-byte groups g of row k lie at g ^ (k % 4), with 128-byte rows
//   (ROWS = 64) at g ^ (k / 2 % 2).
template <int ROWS, bool COLS, bool DUAL>
struct Side {
    static constexpr int PER = ROWS / 32;       // loads of a wave for a stage
    static constexpr int RB = COLS ? ROWS * 2 : 128;  // bytes of a row in LDS
    const char *seg[2];  // of this tile: first row (or column), k = 0
    long long ld2;       // bytes from row to row
    long long bytes[2];  // of the tile's part from seg on
    int K;
    unsigned off[PER];
    int kpiece;          // first k of the lane's piece (rows)

    __device__ void init(int ld, int K_, int lane, int w) {
        K = K_;
        ld2 = (long long)ld * 2;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int blk = w + 4 * i;
            if constexpr (COLS) {
                constexpr int PP = ROWS / 8;  // pieces a row
                const int k = blk * (64 / PP) + lane / PP, p = lane % PP;
                const int g = ROWS == 64 ? (p >> 2) ^ ((k >> 1) & 1) : (p >> 2) ^ (k & 3);
                off[i] = (unsigned)(k * ld2) + (g * 4 + (p & 3)) * 16;
            } else {
                // (two matrices side by side: the second's rows count anew)
                const int row = (DUAL ? blk % (ROWS / 16) : blk) * 8 + lane / 8;
                const int p = (lane & 7) ^ ((blk * 8 + lane / 8) >> 1 & 7);
                off[i] = (unsigned)(row * ld2) + p * 16;
                kpiece = p * 8;
            }
        }
    }
    // The operand's rows (columns) from `first` on, `width` in all.  Rows hold
    // whole pieces: what fills the last one is zeros (rows), or goes into sums
    // that are dropped (columns).
    __device__ void start(int which, const char *p, int first, int width) {
        if constexpr (COLS) {
            seg[which] = p + (long long)first * 2;
            bytes[which] = (K - 1) * ld2 + (long long)(((width + 7) & ~7) - first) * 2;
        } else {
            seg[which] = p + first * ld2;
            bytes[which] = (min(ROWS, width - first) - 1) * ld2 + (long long)((K + 7) & ~7) * 2;
        }
    }
    // Load i of the stage that begins at k0, to the tile at LDS byte `to`.
    __device__ void load(int i, int k0, unsigned to, int w) const {
        const int which = DUAL && i >= PER / 2;
        const long long skip = COLS ? k0 * ld2 : (long long)k0 * 2;
        const uint64_t p = (uint64_t)(seg[which] + skip);
        long long left = bytes[which] - skip;
        left = left < 0 ? 0 : left > 0x7FFFFFF0ll ? 0x7FFFFFF0ll : left;
        u32x4 r = {(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFFu, (uint32_t)left, 0x00020000u};
#pragma unroll
        for (int x = 0; x < 4; ++x) r[x] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[x]);
        unsigned o = off[i];
        if constexpr (!COLS) o = k0 + kpiece < K ? o : 0x80000000u;  // past K: zeros, as past the rows
        const unsigned at = to + (w + 4 * i) * 1024;
        // As the builtin for it, but unknown to the compiler's counting, which
        // would wait for every load under way before the next LDS read; the
        // waits are stage_barrier's.  Nothing else here reads m0 (the compiler
        // keeps no value in it).
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :
                     : "s"(__builtin_amdgcn_readfirstlane((int)at)), "v"(o), "s"(r)
                     : "memory");
    }
    // The part of a fragment's LDS offset that depends on the lane alone.
    // Fragment: lane l gets row (column) l % 32 of a 32-wide tile, k = 8 (l / 32) + 0..7.
    struct Lane {
        unsigned a, key;
    };
    static __device__ Lane lane_of(int lane) {
        Lane r;
        if constexpr (COLS) {
            const int m = lane % 16;
            r.a = (8 * (lane >> 5) + (m >> 2)) * RB + ((lane >> 4) & 1) * 32 + (m & 3) * 8;
            r.key = ROWS == 64 ? m >> 3 : m >> 2;  // of k = ... + m / 4
        } else {
            r.a = (lane & 31) * RB;
            r.key = ((lane & 31) >> 1) & 7;
        }
        return r;
    }
    // Rows (columns) row0.. (a multiple of 32) of the tile, k = 16 c + 0..15.
    static __device__ u32x4 frag(const char *tile, const Lane &l, int row0, int c, int lane) {
        if constexpr (COLS) {
            // two transposed reads of 4 k x 16 columns for each 16 lanes: lane
            // 4r+c of them names row r, columns 4c.., and receives column 4r+c
            // of all four rows
            u32x2 h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const unsigned at = l.a + (16 * c + 4 * k) * RB + (((unsigned)row0 / 32) ^ l.key) * 64;
                h[k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                     (__attribute__((address_space(3))) s16x4 *)(tile + at)));
            }
            return u32x4{h[0].x, h[0].y, h[1].x, h[1].y};
        } else {
            return *reinterpret_cast<const u32x4 *>(tile + l.a + row0 * RB + (((2 * c + (lane >> 5)) ^ l.key) * 16));
        }
    }
};

// Every load of this wave is in LDS and none of its LDS reads is under way;
// then the other waves'.
__device__ inline void stage_barrier() {
    __builtin_amdgcn_s_waitcnt(7 << 4);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Workgroups of consecutive numbers go to the 8 XCDs in turn: numbers are
// regrouped so that an XCD gets a run of consecutive tiles, and the tiles run
// down 8 rows of tiles before the next column, so the tiles under way on an XCD
// share their operands in its L2.
__device__ inline void tile_of(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int band = 8 * tiles_n, b = id / band, r = id % band;
    const int rows = min(8, tiles_m - 8 * b);
    tm = 8 * b + r % rows;
    tn = r / rows;
}

// -------------------------------------------------------------------- kernel
// A BM x BN tile of a product for 4 waves, a quadrant each, as 32 x 32 tiles.
// GATE: BN / 2 columns of gate and of up, each wave the same columns of both.
template <int BM, int BN, int EPI, bool ACOLS, bool BCOLS, bool F32_>
__global__ __launch_bounds__(256, BM == 256 ? 1 : 2) void k_mlp(MlpCall c) {
    constexpr bool DUAL = EPI == MLP_GATE;
    constexpr int TM = BM / 64, TN = BN / 64;           // 32 x 32 tiles of a wave
    constexpr unsigned ABYTES = BM * KS * 2, STAGE = (BM + BN) * KS * 2;
    constexpr int PAIRS = F32_ ? 6 : 1;
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = w >> 1, wn = w & 1;

    // the tile: numbers regrouped by XCD, then product by product
    int id;
    {
        const int n = gridDim.x, q = n >> 3, r = n & 7, x = blockIdx.x & 7;
        id = x * q + min(x, r) + (int)(blockIdx.x >> 3);
    }
    int which = 0;
    while (which + 1 < c.count && id >= c.p[which].tiles_m * c.p[which].tiles_n) {
        id -= c.p[which].tiles_m * c.p[which].tiles_n;
        ++which;
    }
    const MlpProduct &p = c.p[which];
    int tm, tn;
    tile_of(id, p.tiles_m, p.tiles_n, tm, tn);
    constexpr int NCOLS = DUAL ? BN / 2 : BN;
    const int m0 = tm * BM, n0 = tn * NCOLS;
    const int nk = max(1, (p.K + KS - 1) / KS), total = nk * PAIRS * p.lists;
    const int s0 = (int)((long long)total * blockIdx.y / c.splits);
    const int s1 = (int)((long long)total * (blockIdx.y + 1) / c.splits);

    Side<BM, ACOLS, false> sa;
    Side<BN, BCOLS, DUAL> sb;
    sa.init((int)p.a[0].ld, p.K, lane, w);
    sb.init((int)p.b[0].ld, p.K, lane, w);
    int seg = s0 / nk, kt = s0 - seg * nk;  // of the stage to be loaded next
    auto aim = [&]() {
        const int list = seg / PAIRS, pair = seg % PAIRS;
        const int pa = F32_ ? kPairA[pair] : 0, pb = F32_ ? kPairB[pair] : 0;
        sa.start(0, p.a[list].p + pa * p.a[list].plane, m0, p.M);
        sb.start(0, p.b[list].p + pb * p.b[list].plane, n0, p.N);
        if (DUAL) sb.start(1, p.b[1].p + pb * p.b[1].plane, n0, p.N);
    };
    aim();
    constexpr int LOADS = sa.PER + sb.PER;
    auto load = [&](int i, int k0, unsigned buf) {
        if (i < sa.PER)
            sa.load(i, k0, buf, w);
        else
            sb.load(i - sa.PER, k0, buf + ABYTES, w);
    };
    auto next = [&]() {
        if (++kt == nk) {
            kt = 0;
            ++seg;
            aim();
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
    const auto la = sa.lane_of(lane);
    const auto lb = sb.lane_of(lane);
    u32x4 fa[2][TM], fb[2][TN];
    auto frags = [&](const char *buf, int k, int to) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[to][i] = sa.frag(buf, la, wm * (BM / 2) + 32 * i, k, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int row = DUAL ? (j / (TN / 2)) * (BN / 2) + wn * (BN / 4) + 32 * (j % (TN / 2)) : wn * (BN / 2) + 32 * j;
            fb[to][j] = sb.frag(buf + ABYTES, lb, row, k, lane);
        }
    };

    if (s0 < s1) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load(i, kt * KS, lds0);
        if (s0 + 1 < s1) next();
        stage_barrier();
        frags(smem, 0, 0);
        for (int s = s0; s < s1; ++s) {
            const unsigned here = ((s - s0) & 1) * STAGE, there = STAGE - here;
            const bool more = s + 1 < s1;
            // The loads of the next stage go out behind the products of this
            // one, whose buffer the others have left at the last barrier.
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k < 3) {
                    frags(smem + here, k + 1, (k + 1) & 1);
                } else if (more) {
                    stage_barrier();
                    frags(smem + there, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    // (operands in turn: a lane gets four columns of one row)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = mma32_chunk(BF16{}, acc[i][j], fb[k & 1][j], fa[k & 1][i]);
                    constexpr int HALF = (LOADS + 2 * TM - 1) / (2 * TM);
                    if (k < 2 && more) {
#pragma unroll
                        for (int x = 0; x < HALF; ++x)
                            if ((k * TM + i) * HALF + x < LOADS)
                                load((k * TM + i) * HALF + x, kt * KS, lds0 + there);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (k == 1 && s + 2 < s1) next();
            }
        }
    }

    // The sums go through LDS in slabs of 32 rows of each row of waves, so that
    // a thread gets eight consecutive columns of a row.
    constexpr int PITCH = BN + 8;
    float *slab = reinterpret_cast<float *>(smem);
    static_assert(64 * PITCH * 4 <= 2 * STAGE, "slab");
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int col = DUAL ? (j / (TN / 2)) * (BN / 2) + wn * (BN / 4) + 32 * (j % (TN / 2)) : wn * (BN / 2) + 32 * j;
            float *to = slab + (wm * 32 + (lane & 31)) * PITCH + col + 4 * (lane >> 5);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                *reinterpret_cast<f32x4 *>(to + 8 * v) =
                    f32x4{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
        }
        __syncthreads();
        constexpr int TPR = NCOLS / 8;  // threads a row
#pragma unroll 2
        for (int r = threadIdx.x / TPR; r < 64; r += 256 / TPR) {
            const int row = m0 + (r >> 5) * (BM / 2) + 32 * i + (r & 31), col = n0 + (threadIdx.x % TPR) * 8;
            if (row >= p.M || col >= p.N) continue;
            const float *from = slab + r * PITCH + (threadIdx.x % TPR) * 8;
            float v[8], u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = from[e];
            if (DUAL)
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = from[BN / 2 + e];
            if (c.part) {
                const long long ldp = (p.N + 7) & ~7ll;
                float *o = c.part + ((long long)blockIdx.y * p.M + row) * ldp * (DUAL ? 2 : 1) + col;
                store8<true>(reinterpret_cast<char *>(o), 0, v);
                if (DUAL) store8<true>(reinterpret_cast<char *>(o + ldp), 0, u);
            } else {
                finish<EPI, F32_>(c, p, row, col, v, u);
            }
        }
    }
}

// The sums of a split contraction, in their order.
template <int EPI, bool F32_>
__global__ __launch_bounds__(256) void k_mlp_join(MlpCall c) {
    constexpr int D = EPI == MLP_GATE ? 2 : 1;
    const MlpProduct &p = c.p[0];
    const int ldp = (p.N + 7) & ~7, per = ldp / 8;
    const long long n = (long long)p.M * per, slice = (long long)p.M * ldp * D;
    for (long long t = blockIdx.x * 256ll + threadIdx.x; t < n; t += gridDim.x * 256ll) {
        const int row = (int)(t / per), col = (int)(t % per) * 8;
        const float *from = c.part + (long long)row * ldp * D + col;
        float v[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = u[e] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < c.splits; ++s) {
            float x[8];
            load8<true>(reinterpret_cast<const char *>(from + s * slice), 0, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += x[e];
            if (D == 2) {
                load8<true>(reinterpret_cast<const char *>(from + s * slice + ldp), 0, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] += x[e];
            }
        }
        finish<EPI, F32_>(c, p, row, col, v, u);
    }
}

template <bool F32_>
__global__ __launch_bounds__(256) void k_mlp_planes(const char *src, long long ld, long long rows, int cols,
                                                    MlpOperand to) {
    using DT = std::conditional_t<F32_, F32, BF16>;
    const int per = (int)to.ld / 8;
    const long long n = rows * per;
    for (long long t = blockIdx.x * 256ll + threadIdx.x; t < n; t += gridDim.x * 256ll) {
        const long long row = t / per;
        const int col = (int)(t - row * per) * 8;
        const typename DT::S *q = reinterpret_cast<const typename DT::S *>(src) + row * ld + col;
        typename DT::S s[8];
        float v[8];
        if (col + 8 <= cols) {
            __builtin_memcpy(s, q, sizeof(s));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = col + i < cols ? q[i] : (typename DT::S)0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = DT::to_f(s[i]);
        store_planes<F32_>(to, (size_t)(row * to.ld + col), v);
    }
}

constexpr int kTiles[3][2] = {{256, 256}, {128, 128}, {64, 64}};

unsigned blocks(long long n) {
    n = (n + 255) / 256;
    return (unsigned)(n < 1 ? 1 : n > 8192 ? 8192 : n);
}

template <int BM, int BN, int EPI, bool AC, bool BC, bool F32_>
hipError_t run(const MlpCall &c, int tiles, hipStream_t s) {
    constexpr int smem = 2 * (BM + BN) * KS * 2;
    const void *fn = reinterpret_cast<const void *>(&k_mlp<BM, BN, EPI, AC, BC, F32_>);
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_mlp<BM, BN, EPI, AC, BC, F32_>), dim3(tiles, c.splits), dim3(256), smem, s, c);
    if (c.part) {
        const MlpProduct &p = c.p[0];
        hipLaunchKernelGGL((k_mlp_join<EPI, F32_>), dim3(blocks((long long)p.M * ((p.N + 7) / 8))), dim3(256), 0, s,
                           c);
    }
    return hipGetLastError();
}

template <int EPI, bool AC, bool BC>
hipError_t launch(const MlpCall &c, int tile, int tiles, hipStream_t s) {
    const bool f = c.dtype == LSTM_F32;
    switch (tile) {
        case 0: return f ? run<256, 256, EPI, AC, BC, true>(c, tiles, s) : run<256, 256, EPI, AC, BC, false>(c, tiles, s);
        case 1: return f ? run<128, 128, EPI, AC, BC, true>(c, tiles, s) : run<128, 128, EPI, AC, BC, false>(c, tiles, s);
        default: {
            constexpr int BN = EPI == MLP_GATE ? 128 : 64;
            return f ? run<64, BN, EPI, AC, BC, true>(c, tiles, s) : run<64, BN, EPI, AC, BC, false>(c, tiles, s);
        }
    }
}

long long tiles_of(const MlpCall &c, int tile, MlpCall *to) {
    long long n = 0;
    // (gate and up side by side: half the columns; the smallest tile then is twice as wide)
    const int bn = c.epilogue == MLP_GATE ? (tile == 2 ? 64 : kTiles[tile][1] / 2) : kTiles[tile][1];
    for (int i = 0; i < c.count; ++i) {
        const long long tm = (c.p[i].M + kTiles[tile][0] - 1) / kTiles[tile][0], tn = (c.p[i].N + bn - 1) / bn;
        if (to) to->p[i].tiles_m = (int)tm, to->p[i].tiles_n = (int)tn;
        n += tm * tn;
    }
    return n;
}

}  // namespace

MlpPlan mlp_plan(const MlpCall &c) {
    MlpPlan r{0, 1, 0};
    // the largest tile that still gives most CUs one
    while (r.tile < 2 && tiles_of(c, r.tile, nullptr) < 200) ++r.tile;
    if (c.count == 1) {
        const MlpProduct &p = c.p[0];
        const long long n = tiles_of(c, r.tile, nullptr);
        const long long stages = (long long)((p.K + KS - 1) / KS) * p.lists * (c.dtype == LSTM_F32 ? 6 : 1);
        // few tiles of a long contraction: split it, eight stages a part at least
        long long k = n > 0 && n < 200 ? 512 / n : 1;
        if (k > stages / 8) k = stages / 8;
        if (k > 64) k = 64;
        if (k > 1) {
            r.splits = (int)k;
            r.floats = (size_t)k * p.M * ((p.N + 7) & ~7) * (c.epilogue == MLP_GATE ? 2 : 1);
        }
    }
    return r;
}

hipError_t launch_mlp(const MlpCall &call, hipStream_t s) {
    MlpCall c = call;
    const MlpPlan plan = mlp_plan(c);
    c.splits = plan.splits;
    if (plan.splits == 1) c.part = nullptr;
    const int tiles = (int)tiles_of(c, plan.tile, &c);
    if (tiles == 0) return hipSuccess;
    if (c.epilogue == MLP_GATE) return launch<MLP_GATE, false, false>(c, plan.tile, tiles, s);
    if (c.epilogue == MLP_DGATE) return launch<MLP_DGATE, false, true>(c, plan.tile, tiles, s);
    if (c.a_cols) return launch<MLP_STORE, true, true>(c, plan.tile, tiles, s);
    if (c.b_cols) return launch<MLP_STORE, false, true>(c, plan.tile, tiles, s);
    return launch<MLP_STORE, false, false>(c, plan.tile, tiles, s);
}

hipError_t launch_mlp_planes(int dtype, const void *src, long long ld, long long rows, int cols, const MlpOperand &to,
                             hipStream_t s) {
    const unsigned n = blocks(rows * (to.ld / 8));
    const char *p = static_cast<const char *>(src);
    if (dtype == LSTM_F32)
        hipLaunchKernelGGL(k_mlp_planes<true>, dim3(n), dim3(256), 0, s, p, ld, rows, cols, to);
    else
        hipLaunchKernelGGL(k_mlp_planes<false>, dim3(n), dim3(256), 0, s, p, ld, rows, cols, to);
    return hipGetLastError();
}

}  // namespace lstm_amd
