// gated_mlp.hip -- the products of the gated feed-forward block, each with the
// elementwise work that follows it:
//     GATE   g = x Wg^T, u = x Wu^T, h = act(g) u
//     STORE  y = h Wd^T;  dx = dg Wg + du Wu;  dWg = dg^T x, dWu = du^T x, dWd = dy^T h
//     DGATE  dh = dy Wd, dg = dh u act'(g), du = dh act(g)
// One kernel body, k_mlp, runs all of them on v_mfma_f32_32x32x16_bf16; few rows
// of a forward call go to k_mlp_few, which is bound by the weights' traffic.
//
// An fp32 matrix is three bf16 ones (its value rounded, the rest rounded, the
// rest), and its product the six largest of the nine between them (the published
// way to fp32 products on bf16 matrix cores), one after the other in the same sums:
// 121 to 128 TFLOP/s of fp32 products in a training step of 8191 x 512 x 1408,
// against 76 of the library's fp32 products there and 153 on large matrices; the
// fp32 matrix instructions end at 157.
//
// k_mlp is bound by the matrix cores and their power: with every load, LDS read
// and store taken out it gives 1410 to 1495 TFLOP/s on random values (the clock
// falls to 1.5 GHz), whole 1020 to 1040 for y, 1090 to 1170 for dx and 1130 to 1200
// for the weights' gradients at 16384 x 2048 x 5632, by card (the library 870 to 1190
// for the same products).  There the matrix cores are busy half of the time, and
// the waits for loads and barriers take a fifth.  Measured on the same sizes:
// 128 x 128 tiles, two workgroups a CU, 950 to 970; 256 x 128 in stages of 32, two workgroups a CU, 900 to 990;
// 256 x 256 in four stages of 32, 1020 to 1080; lines fetched into the L2 a
// stage ahead of their loads, 1030 to 1050.  GATE and DGATE lose to what they
// read and write with all CUs at once: 860 to 910 TFLOP/s with g and u kept, 1050
// without; 620 to 650 (each workgroup's results wait for nothing but are not hidden
// behind another's products; starting the XCDs apart did not help).
#include <type_traits>

#include "blocks.h"
#include "device.h"
#include "ops_dev.h"

namespace lstm_amd {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The pairs of planes whose products make one product of fp32 matrices, the
// smallest first: what they leave out is below 2^-24 of each operand.
__device__ constexpr int kPairA[6] = {2, 1, 0, 1, 0, 0}, kPairB[6] = {0, 1, 2, 0, 1, 0};

// ------------------------------------------------------------- elementwise
// act(g) and, with SLOPE, act'(g) of eight values.
template <bool SLOPE>
__device__ inline void activate(int kind, const float *g, float *a, float *slope) {
    if (kind == LSTM_ACT_GELU) {
        // g s(2t), t = k (g + c g^3); past |g| = 32 s is 0 or 1 in fp32, and
        // the clamp, which NaN passes, keeps 0 times infinity out of the slope
        constexpr float k = 0.7978845608028654f, c = 0.044715f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = g[i] > 32.0f ? 32.0f : g[i] < -32.0f ? -32.0f : g[i], q2 = q * q;
            const float t = 2.0f * k * q * (1.0f + c * q2), p = sigmoid_f(t);
            a[i] = g[i] * p;
            if (SLOPE) slope[i] = p + q * (p * sigmoid_f(-t)) * (2.0f * k * (1.0f + 3.0f * c * q2));
        }
    } else if (kind == LSTM_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = sigmoid_f(g[i]);
            if (SLOPE) slope[i] = a[i] * sigmoid_f(-g[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = sigmoid_f(g[i]);
            a[i] = g[i] * p;
            if (SLOPE) slope[i] = fmaf(a[i], 1.0f - p, p);
        }
    }
}

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ inline u32x4 pack8(const float *v) {
    const bf16x8 x = __builtin_convertvector(f32x8{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}, bf16x8);
    return __builtin_bit_cast(u32x4, x);
}

// The first term of an fp32 value, to nearest; the largest finite values, whose
// nearest would be infinite, are cut.  The rest is exact in fp32.
__device__ inline float first_term(float v) {
    const float t = BF16::to_f(round_to<BF16>(v));
    return fabsf(t) <= 3.4e38f ? t : __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
}

// Where a lane's eight values are in a matrix: element base (the same for all
// lanes of a wave, so that it costs scalar instructions only) + off.
struct Place {
    size_t base;
    unsigned off;
    template <class T>
    __device__ T *in(const char *p, int size) const {
        return reinterpret_cast<T *>(const_cast<char *>(p) + base * size + off * (unsigned)size);
    }
};

// Eight values as an operand's planes.
template <bool F32_>
__device__ inline void store_planes(const MlpOperand &o, Place at, const float *v) {
    char *p = at.in<char>(o.p, 2);
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

// Eight fp32 values, 16-byte aligned.
__device__ inline void load8f(const float *p, float *v) {
    const f32x4 x = reinterpret_cast<const f32x4 *>(p)[0], y = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
}
__device__ inline void store8f(float *p, const float *v) {
    reinterpret_cast<f32x4 *>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4 *>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}

// The bits of a value whose upper 24 are it rounded to them, halves to even; the
// finite values next to infinity are cut, infinities and NaN stay what they are.
// (Halves are frequent among sums of few products of 8 bits: away from zero, they
// leave 0.016 of a half step to one side.)
__device__ inline uint32_t rounded24(float v) {
    const uint32_t b = __float_as_uint(v);
    return fabsf(v) < 3.4027e38f ? b + 0x7F + (b >> 8 & 1) : b;
}

// g and u as they are kept for the backward call.  fp32 calls keep all bits,
// bf16 calls are rounded to the upper 24: 16, and eight more in a plane of bytes
// behind them.  (With 16 bits the gradients were off by 0.0031 of their size, rms,
// against 0.0024 from the operands' and the results' own roundings alone.)
template <bool F32_>
struct Kept {
    u32x4 w[F32_ ? 2 : 1];
    u32x2 low;
    __device__ void load(const MlpKept &k, Place at) {
        const u32x4 *q = at.in<const u32x4>(k.p, F32_ ? 4 : 2);
        w[0] = q[0];
        if constexpr (F32_)
            w[1] = q[1];
        else
            low = *at.in<const u32x2>(k.p + k.low, 1);
    }
    __device__ void values(float *v) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (F32_)
                v[i] = __uint_as_float(w[i / 4][i % 4]);
            else  // bytes: 0, byte i % 4 of low, both of the half
                v[i] = __uint_as_float(__builtin_amdgcn_perm(
                    w[0][i / 2], low[i / 4], (i % 2 ? 0x0706000Cu : 0x0504000Cu) | (uint32_t)(i % 4) << 8));
        }
    }
    static __device__ void store(const MlpKept &k, Place at, const float *v) {
        u32x4 *q = at.in<u32x4>(k.p, F32_ ? 4 : 2);
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = F32_ ? __float_as_uint(v[i]) : rounded24(v[i]);
        if constexpr (F32_) {
            q[0] = u32x4{b[0], b[1], b[2], b[3]};
            q[1] = u32x4{b[4], b[5], b[6], b[7]};
        } else {
            u32x4 x;
            u32x2 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __builtin_amdgcn_perm(b[2 * i + 1], b[2 * i], 0x07060302u);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                y[i] = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0C0C0501u) |
                       __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x05010C0Cu);
            q[0] = x;
            *at.in<u32x2>(k.p + k.low, 1) = y;
        }
    }
};

// What follows a product: eight sums of one row, the first `left` of which (at
// least one) are inside the matrix.  GATE: v are gate's and w up's.  DGATE: kg
// and ku are g and u.
template <int EPI, bool F32_>
__device__ inline void finish(const MlpCall &c, const MlpProduct &p, Place at, int left, float *v, float *w,
                              const Kept<F32_> &kg, const Kept<F32_> &ku) {
    if constexpr (EPI == MLP_STORE) {
        using DT = std::conditional_t<F32_, F32, BF16>;
        auto *o = at.in<typename DT::S>(p.out, sizeof(typename DT::S));
        if (p.vec && left >= 8) {
            if constexpr (F32_)
                store8f(o, v);
            else
                *reinterpret_cast<u32x4 *>(o) = pack8(v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) o[i] = round_to<DT>(v[i]);
        }
    } else if constexpr (EPI == MLP_GATE) {
        // columns past N are 0 (the operand's rows past N read as zeros), but for
        // rows of x that are not finite; the next product runs over them
        if (c.gate.p) {
            Kept<F32_>::store(c.gate, at, v);
            Kept<F32_>::store(c.up, at, w);
        }
        float a[8];
        activate<false>(c.act, v, a, nullptr);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? a[i] * w[i] : 0.0f;
        store_planes<F32_>(c.product, at, v);
    } else {
        float g[8], u[8], a[8], slope[8];
        kg.values(g);
        ku.values(u);
        activate<true>(c.act, g, a, slope);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = v[i] * u[i] * slope[i];
            u[i] = v[i] * a[i];
        }
        if (left < 8) {  // past N the sums are of another row's weights
#pragma unroll
            for (int i = 1; i < 8; ++i)
                if (i >= left) g[i] = u[i] = 0.0f;
        }
        store_planes<F32_>(c.dgate, at, g);
        store_planes<F32_>(c.dup, at, u);
    }
}

// ------------------------------------------------------------------ operands
// One stage, KS of the contraction, of an operand lies in LDS as ROWS rows of KS
// values (k along the rows) or as KS rows of ROWS values (k along the columns),
// filled by loads
// that write 64 16-byte pieces to consecutive places, so the place decides
// which piece a lane fetches.  Pieces are permuted inside a row such that the
// lanes of a fragment read fall on all banks:
//   rows (64 values, 128 bytes): piece p of row r lies at p ^ (r / 2 % 8);
//   columns: 64-byte groups g of row k lie at g ^ (k % 4), with 128-byte rows
//   (ROWS = 64) at g ^ (k / 2 % 2).
template <int ROWS, int KS, bool COLS, bool DUAL>
struct Side {
    static constexpr int PER = ROWS * KS / 2048;         // loads of a wave for a stage
    static constexpr int RB = COLS ? ROWS * 2 : KS * 2;  // bytes of a row in LDS
    static constexpr int PP = RB / 16;                   // pieces of a row
    static_assert(PER > 0 && KS == 64, "stage");
    static __device__ int key_of(int row) {
        if (COLS) return ROWS == 64 ? (row >> 1) & 1 : row & 3;  // of 64-byte groups
        return (row >> 1) & 7;
    }
    const char *seg[2];  // of this tile: first row (or column), k = 0
    long long ld2;       // bytes from row to row
    long long bytes[2];  // of the tile's part from seg on
    int K;
    unsigned off[PER];
    int kpiece;          // first k of the lane's piece (rows): the same in all its loads, whose rows are 32 apart

    __device__ void init(int ld, int K_, int lane, int w) {
        K = K_;
        ld2 = (long long)ld * 2;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int blk = w + 4 * i;
            if constexpr (COLS) {
                const int k = blk * (64 / PP) + lane / PP, p = lane % PP;
                off[i] = (unsigned)(k * ld2) + (((p >> 2) ^ key_of(k)) * 4 + (p & 3)) * 16;
            } else {
                // (two matrices side by side: the second's rows count anew)
                const int in = lane / PP, row = (DUAL ? blk % (ROWS * PP / 128) : blk) * (64 / PP) + in;
                const int p = (lane % PP) ^ key_of(blk * (64 / PP) + in);
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
    // Fragment: lane l gets row (column) l % 32 of a 32-wide tile, k = 8 (l / 32)
    // + 0..7.
    struct Lane {
        unsigned a, key;
    };
    static __device__ Lane lane_of(int lane) {
        Lane r;
        if constexpr (COLS) {
            const int m = lane % 16;
            r.a = (8 * (lane >> 5) + (m >> 2)) * RB + ((lane >> 4) & 1) * 32 + (m & 3) * 8;
            r.key = key_of(m >> 2);  // of k = 4 ... + m / 4
        } else {
            r.a = (lane & 31) * RB;
            r.key = key_of(lane & 31);
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

// All but LEFT of this wave's loads are in LDS and none of its LDS reads is under
// way; then the other waves'.
template <int LEFT = 0>
__device__ inline void stage_barrier() {
    static_assert(LEFT < 64, "vmcnt field");
    __builtin_amdgcn_s_waitcnt(7 << 4 | (LEFT & 15) | (LEFT >> 4) << 14);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// f(0), f(1), ... f(N - 1), each argument a constant: a loop that is unrolled
// however long its body is.
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<N, I + 1>(f);
    }
}

// Tile `id` of a call: which product's, and where.  Tiles run down 8 rows of
// tiles before the next column, so that neighbours share their operands.
__device__ inline int tile_of(const MlpCall &c, int id, int &tm, int &tn) {
    int which = 0;
    while (which + 1 < c.count && id >= c.p[which].tiles_m * c.p[which].tiles_n) {
        id -= c.p[which].tiles_m * c.p[which].tiles_n;
        ++which;
    }
    const int tiles_n = c.p[which].tiles_n, band = 8 * tiles_n, b = id / band, r = id % band;
    const int rows = min(8, c.p[which].tiles_m - 8 * b);
    tm = 8 * b + r % rows;
    tn = r / rows;
    return which;
}

// -------------------------------------------------------------------- kernel
// BM x BN tiles of the products for 4 waves, a quadrant each, as 32 x 32 tiles.
// GATE: BN / 2 columns of gate and of up, each wave the same columns of both.
// A workgroup takes one unit after the other: the first `whole` are tiles, the
// others the parts, in k, of the tiles that would not fill a last round.  The
// first loads of a unit go out before the one before it is finished off.
template <class TL, int EPI, bool ACOLS, bool BCOLS, bool F32_>
__global__ __launch_bounds__(256, TL::HELD > 1 ? 2 : 1) void k_mlp(MlpCall c) {
    constexpr int BM = TL::BM, BN = TL::BN, KS = TL::KS, KC = KS / 16, NBUF = TL::NBUF;
    constexpr bool DUAL = EPI == MLP_GATE;
    constexpr int TM = BM / 64, TN = BN / 64, TO = DUAL ? TN / 2 : TN;  // 32 x 32 tiles of a wave; of its results
    constexpr unsigned ABYTES = BM * KS * 2, STAGE = (BM + BN) * KS * 2;
    constexpr int PAIRS = F32_ ? 6 : 1, NCOLS = DUAL ? BN / 2 : BN;
    constexpr bool OWN_SLAB = TL::HELD == 1;  // LDS for the results besides the stages
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = w >> 1, wn = w & 1;
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)smem;

    Side<BM, KS, ACOLS, false> sa;
    Side<BN, KS, BCOLS, DUAL> sb;
    const auto la = sa.lane_of(lane);
    const auto lb = sb.lane_of(lane);
    constexpr int LOADS = sa.PER + sb.PER;

    struct Unit {
        int which, m0, n0, part, stages;  // part: number among the partial sums, or -1
    };
    int seg = 0, kt = 0, nk = 1;  // of the stage to be loaded next
    auto aim = [&](const Unit &t) {
        const MlpProduct &p = c.p[t.which];
        const int list = seg / PAIRS, pair = seg % PAIRS;
        const int pa = F32_ ? kPairA[pair] : 0, pb = F32_ ? kPairB[pair] : 0;
        sa.start(0, p.a[list].p + pa * p.a[list].plane, t.m0, p.M);
        sb.start(0, p.b[list].p + pb * p.b[list].plane, t.n0, p.N);
        if (DUAL) sb.start(1, p.b[1].p + pb * p.b[1].plane, t.n0, p.N);
    };
    auto open = [&](int id) {
        Unit t;
        int part = 0, parts = 1;
        t.part = id - c.whole;
        if (t.part >= 0) {
            parts = c.splits;
            part = t.part % parts;
            id = c.whole + t.part / parts;
        }
        int tm, tn;
        t.which = tile_of(c, id, tm, tn);
        t.m0 = tm * BM;
        t.n0 = tn * NCOLS;
        const MlpProduct &p = c.p[t.which];
        sa.init((int)p.a[0].ld, p.K, lane, w);
        sb.init((int)p.b[0].ld, p.K, lane, w);
        nk = max(1, (p.K + KS - 1) / KS);
        const long long total = (long long)nk * PAIRS * p.lists;
        const int s0 = (int)(total * part / parts);
        t.stages = (int)(total * (part + 1) / parts) - s0;
        seg = s0 / nk;
        kt = s0 - seg * nk;
        aim(t);
        return t;
    };
    auto next = [&](const Unit &t) {
        if (++kt == nk) {
            kt = 0;
            ++seg;
            aim(t);
        }
    };
    auto load = [&](int i, unsigned buf) {
        if (i < sa.PER)
            sa.load(i, kt * KS, buf, w);
        else
            sb.load(i - sa.PER, kt * KS, buf + ABYTES, w);
    };
    // the loads of the first NBUF - 1 stages and half of the next one's
    auto begin = [&](const Unit &t) {
#pragma unroll
        for (int s = 0; s < NBUF; ++s) {
            if (s >= t.stages) break;
            if (s > 0) next(t);
#pragma unroll
            for (int i = 0; i < (s == NBUF - 1 ? LOADS / 2 : LOADS); ++i) load(i, lds0 + s * STAGE);
        }
    };

    u32x4 fa[2][TM], fb[2][TN];
    auto frags = [&](const char *buf, int k, int to) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[to][i] = sa.frag(buf, la, wm * (BM / 2) + 32 * i, k, lane);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[to][j] = sb.frag(buf + ABYTES, lb, (j / TO) * (BN / 2) + wn * (32 * TO) + 32 * (j % TO), k, lane);
    };

    // Workgroups of consecutive numbers go to the 8 XCDs in turn: a round's
    // units are regrouped so that an XCD gets a run of consecutive ones, whose
    // operands it keeps in its L2.
    const int grid = gridDim.x;
    const int first = [&]() {
        const int q = grid >> 3, r = grid & 7, x = blockIdx.x & 7;
        return x * q + min(x, r) + (int)(blockIdx.x >> 3);
    }();
    Unit t = open(first);
    begin(t);
    for (int id = first;;) {
        f32x16 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

        // Loads run NBUF stages ahead: those of a stage go out as soon as its
        // buffer is free, behind the products of the last part of the stage that
        // had it and of the first part of the one after that.
        constexpr int HALF = LOADS - LOADS / 2, EACH = (HALF + TM - 1) / TM;
        stage_barrier();
        frags(smem, 0, 0);
        unsigned here = 0, last = (NBUF - 1) * STAGE;  // the buffers of stages s and s - 1
        for (int s = 0; s < t.stages; ++s) {
            const unsigned there = here == (NBUF - 1) * STAGE ? 0 : here + STAGE;
            const bool more = s + 1 < t.stages, late = s + NBUF - 1 < t.stages, early = s + NBUF < t.stages;
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                if (k < KC - 1) {
                    frags(smem + here, k + 1, (k + 1) & 1);
                } else if (more) {
                    if (NBUF > 2 && late)
                        stage_barrier<(NBUF - 2) * LOADS>();
                    else
                        stage_barrier();
                    frags(smem + there, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    // (operands in turn: a lane gets columns of one row)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = mma32_chunk(BF16{}, acc[i][j], fb[k & 1][j], fa[k & 1][i]);
                    if (k == 0 && late) {
#pragma unroll
                        for (int x = 0; x < EACH; ++x)
                            if (LOADS / 2 + i * EACH + x < LOADS) load(LOADS / 2 + i * EACH + x, lds0 + last);
                    }
                    if (k == KC - 1 && early) {
#pragma unroll
                        for (int x = 0; x < EACH; ++x)
                            if (i * EACH + x < LOADS / 2) load(i * EACH + x, lds0 + here);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (k == 0 && early) next(t);
            }
            last = here;
            here = there;
        }

        // The next unit's first loads, then this one's results (with the small
        // tiles, which keep no LDS besides the stages, the other way round).
        const Unit done = t;
        id += grid;
        const bool again = id < c.units;
        if (OWN_SLAB ? again : true) stage_barrier();  // every wave has read the last stage
        if (OWN_SLAB && again) {
            t = open(id);
            begin(t);
        }
        // A wave's 32 x 32 tiles go through LDS of its own, 64 columns at a time
        // (GATE: 32 of gate and of up), so that eight lanes (four) hold eight
        // columns each of a row and memory is written by whole lines.  Pieces of
        // four values of row r lie at p ^ (r % 16): all banks, both ways.
        const MlpProduct &p = c.p[done.which];
        constexpr int WIDE = TO > 1 && !DUAL ? 2 : 1, CPR = 4 * WIDE, ITS = CPR / 2;  // chunks of a row; of a lane
        constexpr int STEPS = TM * TO / WIDE;
        constexpr bool READS = EPI == MLP_DGATE;
        float *slab = reinterpret_cast<float *>(smem + (OWN_SLAB ? NBUF * STAGE : 0)) + w * 2048;
        const int r0 = lane / CPR, c0 = lane % CPR;
        // g and u of a step, of the next one, too, where registers allow
        constexpr int AHEAD = OWN_SLAB && !F32_ ? 1 : 0;
        Kept<F32_> kg[AHEAD + 1][READS ? ITS : 1], ku[AHEAD + 1][READS ? ITS : 1];
        const long long ld = EPI == MLP_STORE ? p.ldo : c.ld;
        const int mw = done.m0 + wm * (BM / 2), nw = done.n0 + wn * (32 * TO);  // the wave's rows and columns
        const size_t corner = (size_t)mw * ld + nw;
        const unsigned mine = r0 * (unsigned)ld + 8 * c0;
        const int rows = p.M - mw - r0, cols = p.N - nw - 8 * c0;  // inside, from the lane's first on
        auto row_of = [](int step, int it) { return 32 * (step / (TO / WIDE)) + it * (64 / CPR); };
        auto col_of = [](int step) { return 32 * WIDE * (step % (TO / WIDE)); };
        auto place = [&](int step, int it) { return Place{corner + (size_t)row_of(step, it) * ld + col_of(step), mine}; };
        auto fetch = [&](int step) {
#pragma unroll
            for (int it = 0; it < ITS; ++it)
                if (row_of(step, it) < rows && col_of(step) < cols) {
                    kg[step & AHEAD][it].load(c.gate, place(step, it));
                    ku[step & AHEAD][it].load(c.up, place(step, it));
                }
        };
        if constexpr (READS)
            if (AHEAD && done.part < 0) fetch(0);
        each<STEPS>([&](auto at) {
            constexpr int step = decltype(at)::value, i = step / (TO / WIDE), jw = step % (TO / WIDE);
#pragma unroll
            for (int h = 0; h < (DUAL ? 2 : WIDE); ++h)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const f32x16 &x = acc[i][DUAL ? jw + h * TO : jw * WIDE + h];
                    *reinterpret_cast<f32x4 *>(slab + (lane & 31) * 64 +
                                               4 * ((8 * h + 2 * v + (lane >> 5)) ^ (lane & 15))) =
                        f32x4{x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]};
                }
            if constexpr (READS)
                if (step + AHEAD < STEPS && done.part < 0) fetch(step + AHEAD);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            each<ITS>([&](auto ati) {
                constexpr int it = decltype(ati)::value;
                const int r = r0 + it * (64 / CPR);
                auto get = [&](int piece, float *v) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f32x4 x = *reinterpret_cast<const f32x4 *>(slab + r * 64 + 4 * ((piece + h) ^ (r & 15)));
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[4 * h + e] = x[e];
                    }
                };
                float v[8], u[8];
                get(2 * c0, v);
                if (DUAL) get(2 * c0 + 8, u);
                if (done.part >= 0) {
                    float *to = c.part + (size_t)done.part * (BM * BN) + (wm * (BM / 2) + row_of(step, it)) * BN +
                                wn * (32 * TO) + col_of(step) + (r0 * BN + 8 * c0);
                    store8f(to, v);
                    if (DUAL) store8f(to + BN / 2, u);
                } else if (row_of(step, it) < rows && col_of(step) < cols) {
                    finish<EPI, F32_>(c, p, place(step, it), cols - col_of(step), v, u, kg[step & AHEAD][READS ? it : 0],
                                      ku[step & AHEAD][READS ? it : 0]);
                }
                if constexpr (READS) __builtin_amdgcn_sched_barrier(0);
            });
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        });
        if (!again) break;
        if (!OWN_SLAB) {
            stage_barrier();
            t = open(id);
            begin(t);
        }
    }
}

// The sums of tiles whose contraction was split, in the parts' order.
template <class TL, int EPI, bool F32_>
__global__ __launch_bounds__(256) void k_mlp_join(MlpCall c) {
    constexpr int BM = TL::BM, BN = TL::BN;
    constexpr bool DUAL = EPI == MLP_GATE;
    constexpr int NCOLS = DUAL ? BN / 2 : BN, PER = BM * NCOLS / 8;
    int tm, tn;
    const MlpProduct &p = c.p[tile_of(c, c.whole + blockIdx.y, tm, tn)];
    const int t = blockIdx.x * 256 + threadIdx.x, r = t / (NCOLS / 8), q = t % (NCOLS / 8) * 8;
    const int row = tm * BM + r, col = tn * NCOLS + q;
    if (t >= PER || row >= p.M || col >= p.N) return;
    const float *from = c.part + (size_t)blockIdx.y * c.splits * (BM * BN) + r * BN + q;
    float v[8], u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u[e] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < c.splits; ++s, from += BM * BN) {
        float x[8];
        load8f(from, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += x[e];
        if (DUAL) {
            load8f(from + BN / 2, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] += x[e];
        }
    }
    Kept<F32_> kg, ku;
    const Place at{(size_t)row * (EPI == MLP_STORE ? p.ldo : c.ld) + col, 0};
    if constexpr (EPI == MLP_DGATE) {
        kg.load(c.gate, at);
        ku.load(c.up, at);
    }
    finish<EPI, F32_>(c, p, at, p.N - col, v, u, kg, ku);
}

// ------------------------------------------------------------------ few rows
// Up to 16 NT rows x: the weights' traffic is all that counts (4 x 1024 x 2816
// bf16: 5.4 + 7.2 us for 17 MB; the rule, few_rows, has both sides' times).  A workgroup
// takes 16 rows of a weight (GATE: of gate and of up), its NW waves every NW-th
// 128 bytes of k.  Weights go from memory to registers as fragments (lane (m, g):
// row m, 16 bytes at 16 g of each 64), several on their way at a time, and meet
// the rows of x, which stay in the caches, on 16 x 16 tiles.  fp32 runs on fp32
// matrix instructions: memory is slower than they are.
template <class DT>
__device__ inline u32x4 few_load(const char *row, int k, int K) {
    using S = typename DT::S;
    const S *q = reinterpret_cast<const S *>(row);
    S t[DT::PER16];
    if (k + DT::PER16 <= K) {
        __builtin_memcpy(t, q + k, 16);
    } else {
#pragma unroll
        for (int e = 0; e < DT::PER16; ++e) t[e] = k + e < K ? q[k + e] : (S)0;
    }
    return __builtin_bit_cast(u32x4, t);
}

template <class DT, int NT, bool GATE>
__global__ __launch_bounds__(GATE ? 512 : 1024) void k_mlp_few(MlpFew c) {
    constexpr bool F32_ = sizeof(typename DT::S) == 4;
    constexpr int NW = GATE ? 8 : 16, D = GATE ? 2 : 1, U = NT > 2 ? 2 : 4;  // U: fragments of each on their way
    __shared__ f32x4 sums[NW][D][NT][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    constexpr long long ES = sizeof(typename DT::S);
    const long long row = (long long)min(n0 + m, c.N - 1) * c.K * ES;  // past the last: it again, its sums are dropped
    const char *wa = c.w[0] + row, *wb = GATE ? c.w[1] + row : nullptr;
    const char *x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = c.x + min(16 * t + m, c.rows - 1) * c.xs * ES;
    f32x4 acc[D][NT];
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[d][t] = f32x4{0, 0, 0, 0};
    constexpr int LINE = 2 * DT::KC;  // k of a 128-byte line: two fragments
    for (int k0 = w * LINE; k0 < c.K; k0 += NW * LINE * (U / 2)) {
        u32x4 a[D][U], b[NT][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + (u / 2) * NW * LINE + (u % 2) * DT::KC + g * DT::PER16;
            a[0][u] = few_load<DT>(wa, k, c.K);
            if (GATE) a[D - 1][u] = few_load<DT>(wb, k, c.K);
#pragma unroll
            for (int t = 0; t < NT; ++t) b[t][u] = few_load<DT>(x[t], k, c.K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int d = 0; d < D; ++d) acc[d][t] = mma_chunk(DT{}, acc[d][t], a[d][u], b[t][u]);
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int t = 0; t < NT; ++t) sums[w][d][t][lane] = acc[d][t];
    __syncthreads();
    // thread (t, lane): the waves' sums in their order, of row 16 t + m and four columns
    if (threadIdx.x >= NT * 64) return;
    const int t = threadIdx.x >> 6, r = 16 * t + m, col = n0 + 4 * g;
    f32x4 v[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int d = 0; d < D; ++d)
        for (int i = 0; i < NW; ++i) v[d] += sums[i][d][t][lane];
    if (r >= c.rows) return;
    if constexpr (!GATE) {
        auto *o = reinterpret_cast<typename DT::S *>(c.out) + (long long)r * c.N + col;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e < c.N) o[e] = round_to<DT>(v[0][e]);
    } else {
        if (col >= c.ld) return;
        float h[4], gv[8], av[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) gv[e] = v[0][e % 4];
        activate<false>(c.act, gv, av, nullptr);
        const size_t at = (size_t)r * c.ld + col;
        uint32_t bits[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = col + e < c.N;  // up to ld zeros
            h[e] = in ? av[e] * v[1][e] : 0.0f;
            bits[0][e] = !in ? 0u : F32_ ? __float_as_uint(v[0][e]) : rounded24(v[0][e]);
            bits[1][e] = !in ? 0u : F32_ ? __float_as_uint(v[1][e]) : rounded24(v[1][e]);
        }
        typename DT::S s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = round_to<DT>(h[e]);
        __builtin_memcpy(c.out + at * ES, s, sizeof(s));
        if (!c.keep.p) return;
        // as Kept and store_planes write them
        const MlpKept *kept[2] = {&c.gate, &c.up};
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            if constexpr (F32_) {
                __builtin_memcpy(kept[d]->p + at * 4, bits[d], 16);
            } else {
                uint16_t high[4];
                unsigned char low[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) high[e] = bits[d][e] >> 16, low[e] = bits[d][e] >> 8 & 0xFF;
                __builtin_memcpy(kept[d]->p + at * 2, high, 8);
                __builtin_memcpy(kept[d]->p + kept[d]->low + at, low, 4);
            }
        }
        char *planes = const_cast<char *>(c.keep.p) + at * 2;
#pragma unroll
        for (int k = 0; k < (F32_ ? 3 : 1); ++k) {
            uint16_t q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float f = F32_ && k < 2 ? first_term(h[e]) : h[e];
                q[e] = round_to<BF16>(f);
                h[e] -= f;
            }
            __builtin_memcpy(planes + k * c.keep.plane, q, 8);
        }
    }
}

template <class DT, bool GATE>
hipError_t run_few(const MlpFew &c, hipStream_t s) {
    const dim3 grid(GATE ? (unsigned)((c.ld + 15) / 16) : (c.N + 15) / 16), block(GATE ? 512 : 1024);
    if (c.rows <= 16)
        hipLaunchKernelGGL((k_mlp_few<DT, 1, GATE>), grid, block, 0, s, c);
    else if (c.rows <= 32)
        hipLaunchKernelGGL((k_mlp_few<DT, 2, GATE>), grid, block, 0, s, c);
    else
        hipLaunchKernelGGL((k_mlp_few<DT, 4, GATE>), grid, block, 0, s, c);
    return hipGetLastError();
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
        store_planes<F32_>(to, Place{(size_t)(row * to.ld + col), 0}, v);
    }
}

// Tiles of BM x BN, stages of KS, NBUF of them in LDS, and HELD workgroups on a
// CU; a GATE tile has BN / 2 columns.
template <int BM_, int BN_, int KS_, int NBUF_, int HELD_>
struct MlpTile {
    static constexpr int BM = BM_, BN = BN_, KS = KS_, NBUF = NBUF_, HELD = HELD_;
    static constexpr int SLAB = HELD == 1 ? 32768 : 0, LDS = NBUF * (BM + BN) * KS * 2 + SLAB;
    static_assert(LDS * HELD <= 163840 && LDS >= 32768, "LDS");
};
using Tile0 = MlpTile<256, 256, 64, 2, 1>;
using Tile1 = MlpTile<128, 128, 64, 2, 2>;
using Tile2 = MlpTile<64, 128, 64, 3, 2>;

// Of each tile: the microseconds of 64 of the contraction in each workgroup when
// all run, and of a unit besides, as measured at 16384 x 2048 x 5632 (256 x 256:
// 168 us for 88 of them) and at 256 rows (64 x 128: 26 us for 32).
struct Tile {
    int m, n, held;
    float stage, unit;
};
template <class TL>
constexpr Tile tile_of_type(float stage, float unit) {
    return {TL::BM, TL::BN, TL::HELD, stage, unit};
}
constexpr int kTileCount = 3;
constexpr Tile kTiles[kTileCount] = {tile_of_type<Tile0>(1.9f, 7.0f), tile_of_type<Tile1>(1.1f, 5.0f),
                                     tile_of_type<Tile2>(0.7f, 4.0f)};
constexpr int kCus = 256;

unsigned blocks(long long n) {
    n = (n + 255) / 256;
    return (unsigned)(n < 1 ? 1 : n > 8192 ? 8192 : n);
}

template <class TL, int EPI, bool AC, bool BC, bool F32_>
hipError_t run(const MlpCall &c, const MlpPlan &plan, hipStream_t s) {
    const void *fn = reinterpret_cast<const void *>(&k_mlp<TL, EPI, AC, BC, F32_>);
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, TL::LDS);
    if (e != hipSuccess) return e;
    const int slots = kCus * TL::HELD;
    hipLaunchKernelGGL((k_mlp<TL, EPI, AC, BC, F32_>), dim3(c.units < slots ? c.units : slots), dim3(256), TL::LDS, s, c);
    if (plan.split_tiles) {
        constexpr int per = TL::BM * (EPI == MLP_GATE ? TL::BN / 2 : TL::BN) / 8;
        hipLaunchKernelGGL((k_mlp_join<TL, EPI, F32_>), dim3((per + 255) / 256, plan.split_tiles), dim3(256), 0, s, c);
    }
    return hipGetLastError();
}

template <int EPI, bool AC, bool BC, bool F32_>
hipError_t launch(const MlpCall &c, const MlpPlan &plan, hipStream_t s) {
    if (plan.tile == 0) return run<Tile0, EPI, AC, BC, F32_>(c, plan, s);
    if (plan.tile == 1) return run<Tile1, EPI, AC, BC, F32_>(c, plan, s);
    return run<Tile2, EPI, AC, BC, F32_>(c, plan, s);
}

template <int EPI, bool AC, bool BC>
hipError_t launch(const MlpCall &c, const MlpPlan &plan, hipStream_t s) {
    return c.dtype == LSTM_F32 ? launch<EPI, AC, BC, true>(c, plan, s) : launch<EPI, AC, BC, false>(c, plan, s);
}

long long tiles_of(const MlpCall &c, int tile, MlpCall *to) {
    long long n = 0;
    const int bn = c.epilogue == MLP_GATE ? kTiles[tile].n / 2 : kTiles[tile].n;
    for (int i = 0; i < c.count; ++i) {
        const long long tm = (c.p[i].M + kTiles[tile].m - 1) / kTiles[tile].m, tn = (c.p[i].N + bn - 1) / bn;
        if (to) to->p[i].tiles_m = (int)tm, to->p[i].tiles_n = (int)tn;
        n += tm * tn;
    }
    return n;
}

}  // namespace

// The tile and the split of the last round with the least estimated time:
// rounds of units, and the partial sums' way to memory and back at 4 TB/s with
// a launch to join them.
MlpPlan mlp_plan(const MlpCall &c) {
    MlpPlan best{};
    double least = 1e30;
    double stages = 0;  // of 64, of a tile (the longest product's)
    for (int i = 0; i < c.count; ++i) {
        const double n = (double)((c.p[i].K + 63) / 64) * c.p[i].lists * (c.dtype == LSTM_F32 ? 6 : 1);
        if (n > stages) stages = n;
    }
    for (int tile = 0; tile < kTileCount; ++tile) {
        const Tile &t = kTiles[tile];
        const long long n = tiles_of(c, tile, nullptr), slots = kCus * t.held, rem = n % slots;
        const double area = (double)t.m * t.n * sizeof(float);
        auto offer = [&](long long whole, long long splits) {
            const long long split_tiles = splits > 1 ? n - whole : 0;
            double us = 0;
            // (alone on its CU a workgroup of a small tile takes two thirds of that)
            auto units = [&](long long n, double stages) {
                const long long last = n % slots;
                const double one = stages * t.stage + t.unit;
                return n / slots * one + (last == 0 ? 0.0 : last <= kCus && t.held > 1 ? one * 0.67 : one);
            };
            us += units(whole, stages);
            if (split_tiles) us += units(split_tiles * splits, stages / splits) + 4.0 + 2 * split_tiles * splits * area / 4e6;
            if (us < least) {
                least = us;
                best.tile = tile;
                best.whole = (int)whole;
                best.splits = (int)splits;
                best.split_tiles = (int)split_tiles;
                best.units = (int)(whole + split_tiles * splits);
                best.floats = (size_t)(split_tiles * splits) * (size_t)(area / sizeof(float));
            }
        };
        offer(n, 1);
        // split the tiles of the last round so that they fill it, in one or two rounds of parts
        for (int k = 2; rem && k <= 64 && stages / k >= 4; ++k)
            if (rem * k <= 2 * slots) offer(n - rem, k);
    }
    return best;
}

hipError_t launch_mlp(const MlpCall &call, hipStream_t s) {
    MlpCall c = call;
    const MlpPlan plan = mlp_plan(c);
    c.whole = plan.whole;
    c.splits = plan.splits;
    c.units = plan.units;
    (void)tiles_of(c, plan.tile, &c);
    if (c.units == 0) return hipSuccess;
    if (c.epilogue == MLP_GATE) return launch<MLP_GATE, false, false>(c, plan, s);
    if (c.epilogue == MLP_DGATE) return launch<MLP_DGATE, false, true>(c, plan, s);
    if (c.a_cols) return launch<MLP_STORE, true, true>(c, plan, s);
    if (c.b_cols) return launch<MLP_STORE, false, true>(c, plan, s);
    return launch<MLP_STORE, false, false>(c, plan, s);
}

hipError_t launch_mlp_few(const MlpFew &c, hipStream_t s) {
    if (c.w[1]) return c.dtype == LSTM_F32 ? run_few<F32, true>(c, s) : run_few<BF16, true>(c, s);
    return c.dtype == LSTM_F32 ? run_few<F32, false>(c, s) : run_few<BF16, false>(c, s);
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
