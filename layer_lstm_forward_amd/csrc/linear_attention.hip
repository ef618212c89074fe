// linear_attention.hip -- linear attention with a decay for each head:
//     S_t = gamma S_{t-1} + b_t c_t^T,   o_t = a_t S_t
// for whole sequences, chunk by chunk on the matrix cores, and for single
// tokens.
//
// A chunk of C tokens, with the matrix S before it, local indices i and j:
//     O  = diag(gamma^(i+e)) A S + ((A B^T) . W) Cv,   W_ij = gamma^(i-j) for i >= j, else 0
//     S' = gamma^C S + B^T diag(gamma^(C-j-e)) Cv
// with e = 1; in a reversed pass e = 0 and tokens count from the row's end.
// Every power has an exponent of at least 0, so that nothing overflows however
// small gamma is, but for a gamma near 1 (2^(+-20/128) at most), whose S is
// carried as S / gamma^lag, lag up to 128: values above 2^108 leave the fp32
// range there.
#include "device.h"
#include "ops.h"
#include "ops_dev.h"

namespace lstm_amd {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;

// log2 gamma, finite: gamma = 0 (log decay -infinity) becomes 2^-1e30, whose
// power 0 is 1 and whose other powers are 0.  NaN stays.
__device__ inline float la_log2(float log_decay) {
    const float g = log_decay * kLog2e;
    return g < -1e30f ? -1e30f : g;
}
__device__ inline float la_pow(float g2, int n) { return __builtin_amdgcn_exp2f((float)n * g2); }

__device__ inline int la_len(const int *lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : n > T ? T : n;
}

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

// N neighbouring columns of a token; unless all are known to be, `left` of them
// are in range.
template <class DT, int N, bool ALL, class V>
__device__ inline void la_write(char *o, bool f32, V v, int left) {
    if (sizeof(typename DT::S) == 4 || f32) {
        float *q = reinterpret_cast<float *>(o);
        if (ALL || left >= N)
            __builtin_memcpy(q, &v, sizeof(v));
        else
#pragma unroll
            for (int x = 0; x < N; ++x)
                if (x < left) q[x] = v[x];
    } else {
        typename DT::S *q = reinterpret_cast<typename DT::S *>(o), tmp[N];
#pragma unroll
        for (int x = 0; x < N; ++x) tmp[x] = round_to<DT>(v[x]);
        if (ALL || left >= N)
            __builtin_memcpy(q, tmp, sizeof(tmp));
        else
#pragma unroll
            for (int x = 0; x < N; ++x)
                if (x < left) q[x] = tmp[x];
    }
}

// Shape of a workgroup's tile.  A wave owns NT column tiles of 16 of S (all of
// its DA rows, in accumulators) for the whole sequence, so S never leaves the
// registers: the accumulator layout of S (rows 4g+r of a tile, g = lane / 16)
// is, read as an operand over the row axis, a fragment.  bf16 fragments hold 8
// consecutive values of a 32-long axis, that is rows 8g..8g+7: the row tiles
// 2u and 2u+1 take the rows 32u + 8g + r and 32u + 8g + 4 + r (row_of), so a
// pair of accumulators is the fragment of 32u + 8g.. without a move between
// lanes.  The same holds for the chunk's products A B^T, whose tiles become
// the operand of the product with Cv.
template <class DT, int DA_, int NW_, int NT_>
struct LaTile {
    static constexpr int DA = DA_, NW = NW_, NT = NT_;
    static constexpr int PER = DT::PER16, KC = DT::KC, TPK = KC / 16;
    static constexpr int C = 32;                               // tokens of a chunk
    static constexpr int NU = DA / KC, JU = C / KC, AT = DA / 16;
    static constexpr int COLS = NW * 16 * NT;                  // columns of a workgroup
    static constexpr int THREADS = 64 * NW;
    static constexpr int RA = DA / PER, RC = COLS / PER;       // 16-byte pieces of a row in LDS
    static constexpr int PA = C * RA > THREADS ? C * RA / THREADS : 1;  // pieces a thread moves
    static constexpr int PC = C * RC > THREADS ? C * RC / THREADS : 1;
    static constexpr int ELEMS = C * (2 * DA + COLS);          // a chunk's three tensors in LDS
    static constexpr int P_ELEMS = C * C;                      // and its (A B^T) . W
    // 32 rows of S pass through a chunk's buffer on their way from and to memory
    static constexpr int LD = COLS + 4;                        // floats of such a row
    static constexpr int ROWS_ELEMS = 32 * LD * 4 / (int)sizeof(typename DT::S);
    static constexpr int BUF_ELEMS = ELEMS > ROWS_ELEMS ? ELEMS : (ROWS_ELEMS + 511) / 512 * 512;
    static constexpr int PT = NW < 4 ? 4 / NW : 1;             // tiles of A B^T a wave computes
    // chunks in the LDS of a workgroup such that 8 waves, and two workgroups, share a CU's 160 KB
    static constexpr int FIT = (160 * 1024 / (NW < 4 ? 4 : 2) / (int)sizeof(typename DT::S) - P_ELEMS) / BUF_ELEMS;
    // chunk buffers where the loads go through registers (a second one saves a barrier a chunk) ...
    static constexpr int BUFS = FIT >= 2 ? 2 : 1;
    // ... and where they write to LDS themselves, two chunks ahead of the products if it fits
    static constexpr int RING = FIT >= 3 ? 3 : 2;
    static_assert(THREADS % RA == 0 && THREADS % RC == 0, "tile");

    // row (of the 16-row tile `tile`) that accumulator row 4g + r stands for
    __device__ static int row_of(int tile, int g, int r) {
        return TPK == 2 ? 32 * (tile / 2) + 8 * g + 4 * (tile % 2) + r : 16 * tile + 4 * g + r;
    }
    // column (of a wave's NT tiles) that position m of tile n stands for
    __device__ static int col_of(int n, int m) {
        return TPK == 2 && NT == 2 ? 8 * (m / 4) + 4 * n + m % 4 : 16 * n + m;
    }
    // Piece p of LDS row j lies at p ^ key(j): the 16 rows that a fragment
    // read touches, and the 4 rows x 4 pieces of a transposed read, then all
    // fall on different places of 16 bytes.  A transposed read takes the same
    // 8 bytes of every place, half of the 64 banks, so it lasts twice its
    // minimum: conflicts are counted in half of the LDS cycles of the pass that
    // reads only so (k_la with STATE_ONLY), which LDS does not bound.
    template <int R>
    __device__ static int key(int j) {
        if (TPK == 1) return j & 15;
        return R >= 16 ? ((j & 3) << 2) | ((j >> 3) & 3) : (((j >> 1) & 1) << 2) | ((j >> 3) & 3);
    }
    template <int R>
    __device__ static int at(int j, int p) {
        return (j * R + (p ^ key<R>(j))) * PER;
    }
};

// How a call's rows are read, by its dims (LaEdge).  No path branches around a
// load (a branch makes the compiler wait for the load where the paths join):
// tokens past the end read the last valid one again, whose weight is 0.
//   WHOLE  every 16-byte piece of a tile lies in the row (fp32)
//   EDGES  a piece that reaches past the row's end is read further left, so
//          that it ends with the row, and shifted into place (zeros follow)
//   SHORT  a dim below one piece: element by element
// No alignment is assumed: the hardware splits what is not aligned.
//   DIRECT_LDS  as WHOLE, bf16, rows 16-byte aligned: loads that write to LDS
enum LaEdge { WHOLE = 0, EDGES = 1, SHORT = 2, DIRECT_LDS = 3 };

// v shifted down by n bits (0..128, a multiple of the element's bits).
__device__ inline u32x4 la_shift(u32x4 v, int n) {
    const int w = n >> 5, b = n & 31;
    const u32x4 x = w & 1 ? u32x4{v.y, v.z, v.w, 0} : v;
    const u32x4 y = w & 2 ? u32x4{x.z, x.w, 0, 0} : x;
    const u32x4 z = w & 4 ? u32x4{0, 0, 0, 0} : y;
    return u32x4{__builtin_amdgcn_alignbit(z.y, z.x, b), __builtin_amdgcn_alignbit(z.z, z.y, b),
                 __builtin_amdgcn_alignbit(z.w, z.z, b), z.w >> b};
}

// Tokens of one tensor on their way from memory to LDS: piece p of a thread is
// row tid / R + p * (THREADS / R), 16-byte piece tid % R.
template <class DT, class TL, int R, int P, int EDGE>
struct LaStage {
    using S = typename DT::S;
    static constexpr int RS = TL::THREADS / R;
    const char *base;  // the row's first token in the pass's order
    int step;          // bytes between tokens, signed by direction
    int row, piece, off, shift, dim;
    u32x4 v[P];

    __device__ void init(const LaTensor &x, int b, int h, int t0, int dir, int d0, int dim_) {
        row = threadIdx.x / R;
        piece = threadIdx.x % R;
        dim = dim_ - d0;
        step = (int)(x.t * (long long)sizeof(S)) * dir;
        base = x.p + ((long long)t0 * x.t + (long long)b * x.b + (long long)(h / x.hdiv) * x.h + d0) *
                         (long long)sizeof(S);
        const int d = piece * TL::PER, rest = dim - d;
        off = d * (int)sizeof(S);
        shift = 0;
        if (EDGE == EDGES && rest < TL::PER) {
            off = (dim - TL::PER) * (int)sizeof(S);
            shift = rest > 0 ? (TL::PER - rest) * 8 * (int)sizeof(S) : 128;
        }
    }
    // tokens i0.. of which n >= 1 are valid
    __device__ void load(int i0, int n) {
        const char *at = base + (long long)i0 * step;
        if (EDGE != SHORT) at += off;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const char *q = at + (long long)min(row + p * RS, n - 1) * step;
            if constexpr (EDGE != SHORT) {
                __builtin_memcpy(&v[p], q, 16);
            } else {
                S tmp[TL::PER];
#pragma unroll
                for (int e = 0; e < TL::PER; ++e) {
                    const int d = piece * TL::PER + e;
                    // (a slab past this tensor's columns has dim <= 0: still in the row)
                    const S x = reinterpret_cast<const S *>(q)[min(d, dim - 1)];
                    tmp[e] = d < dim ? x : (S)0;
                }
                v[p] = __builtin_bit_cast(u32x4, tmp);
            }
        }
    }
    __device__ void store(S *lds) const {
        if (RS > TL::C && row >= TL::C) return;  // more threads than pieces
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<u32x4 *>(lds + TL::template at<R>(row + p * RS, piece)) =
                EDGE == EDGES ? la_shift(v[p], shift) : v[p];
    }
};

// The same without registers between: each wave's load writes 64 pieces of 16
// bytes to consecutive LDS places, so the place decides which piece of which
// row a lane fetches.  Block w + NW * i of a tensor's pieces is wave w's load i.
// Needs whole pieces, 16-byte alignment and rows of a chunk within 32-bit
// offsets of each other.
template <class DT, class TL, int R>
struct LaDirect {
    using S = typename DT::S;
    static constexpr int BLOCKS = TL::C * R / 64;  // of 64 pieces
    // loads of a wave; with fewer blocks than waves some load the same block
    static constexpr int N = BLOCKS > TL::NW ? BLOCKS / TL::NW : 1;
    const char *base;
    int step;
    unsigned full[N];  // offsets of a chunk of C valid tokens

    __device__ unsigned offset(int i, int n) const {
        const int at = (threadIdx.x / 64 + TL::NW * i) % BLOCKS * 64 + threadIdx.x % 64, j = at / R;
        const unsigned piece = (at % R) ^ TL::template key<R>(j);
        const int k = min(j, n - 1);  // past the end: the last token again, whose weight is 0
        return (unsigned)(step >= 0 ? k : n - 1 - k) * (unsigned)abs(step) + piece * 16u;
    }
    __device__ void init(const LaTensor &x, int b, int h, int t0, int dir, int d0) {
        step = (int)(x.t * (long long)sizeof(S)) * dir;
        base = x.p + ((long long)t0 * x.t + (long long)b * x.b + (long long)(h / x.hdiv) * x.h + d0) *
                         (long long)sizeof(S);
#pragma unroll
        for (int i = 0; i < N; ++i) full[i] = offset(i, TL::C);
    }
    __device__ void load(S *lds, int i0, int n) const {
        const long long low = (long long)(step >= 0 ? i0 : i0 + n - 1) * step;
        const uint64_t p = (uint64_t)(base + low);
        u32x4 r = {(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFFu, 0xFFFFFFFFu, 0x00020000u};
#pragma unroll
        for (int x = 0; x < 4; ++x) r[x] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[x]);
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const unsigned o = n == TL::C ? full[i] : offset(i, n);
            const uint32_t to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) S *)lds +
                                (wave + TL::NW * i) % BLOCKS * 1024;
            // As the builtin for it, but unknown to the compiler's counting:
            // with the builtin it waits for every load under way before the
            // next transposed LDS read.  The waits are la_barrier's.  Nothing
            // else here reads m0 (it is reserved: the compiler keeps no value
            // in it).
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                         :
                         : "s"(to), "v"(o), "s"(r)
                         : "memory");
        }
    }
};

// Waits until at most VM of this wave's memory operations and none of its LDS
// operations are under way, then for the other waves.  (The fence of
// __syncthreads would wait for the loads of later chunks too.)
template <int VM>
__device__ inline void la_barrier() {
    static_assert(VM < 64, "vmcnt field");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Fragment of rows: lane (m, g) gets row tile_row(m), values KC*u + PER*g ...
template <class DT, class TL, int R>
__device__ inline u32x4 la_frag(const typename DT::S *lds, int tile, int u, int lane) {
    const int m = lane % 16, g = lane / 16;
    return *reinterpret_cast<const u32x4 *>(lds + TL::template at<R>(TL::row_of(tile, m / 4, m % 4), 4 * u + g));
}

// Fragment of columns over the tokens KC*ju..: lane (m, g) gets column
// col(m), tokens KC*ju + PER*g + 0..PER-1.  col4(c) is the first of the four
// columns that positions 4c..4c+3 stand for.  bf16: two transposed reads of 4
// tokens x 16 columns for each 16 lanes (lane 4r+c of them names row r, columns
// col4(c).., and receives column 4r+c of all four rows).
template <class DT, class TL, int R, class F>
__device__ inline u32x4 la_cols(const typename DT::S *lds, int ju, F col4, int lane) {
    const int m = lane % 16, g = lane / 16;
    if constexpr (TL::TPK == 2) {
        u32x2 h[2];
        const int c = col4(m % 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = 32 * ju + 8 * g + 4 * k + m / 4;
            auto p = (__attribute__((address_space(3))) s16x4 *)(lds + TL::template at<R>(j, c / 8) + c % 8);
            h[k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
        }
        return u32x4{h[0].x, h[0].y, h[1].x, h[1].y};
    } else {
        const int c = col4(m / 4) + m % 4;
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = *reinterpret_cast<const uint32_t *>(lds + TL::template at<R>(16 * ju + 4 * g + e, c / 4) + c % 4);
        return v;
    }
}

// Accumulators of TPK row tiles as one fragment.  bf16: S is rounded here, once,
// as an operand; the sum itself stays fp32.  With the rounding of (A B^T) . W
// this takes o's error from 0.0017 of its size, rms (its own rounding), to 0.0023;
// two terms for each operand would be 20 more matrix instructions to a chunk's 56.
template <class DT, class TL>
__device__ inline u32x4 la_pack(const f32x4 *acc, int stride) {
    if constexpr (TL::TPK == 2) {
        const f32x4 x = acc[0], y = acc[stride];
        const bf16x8 v = __builtin_convertvector(f32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}, bf16x8);
        return __builtin_bit_cast(u32x4, v);
    } else {
        return __builtin_bit_cast(u32x4, acc[0]);
    }
}

// The state update's operand: column fragments times their tokens' weights.
// bf16: the weighted value is kept as a sum of bf16 terms, rounded, so that S
// keeps what fp32 arithmetic would.  Two terms leave 2^-17 of a value (2.7e-6
// rms, measured against fp64), enough where S only enters bf16 results; a
// state that is returned in fp32 and carried from call to call gets the third
// (4e-7; fp32 products have 3e-7).
template <class DT, class TL>
struct LaWeighted {
    static constexpr int TERMS = TL::TPK == 2 ? 3 : 1;
    u32x4 part[TERMS][TL::NT][TL::JU];
    __device__ void make(const u32x4 (*cf)[TL::JU], const float (*weight)[TL::PER], bool third) {
#pragma unroll
        for (int ju = 0; ju < TL::JU; ++ju) {
            const float *w = weight[ju];
#pragma unroll
            for (int t = 0; t < TL::NT; ++t) {
                if constexpr (TL::TPK == 2) {
                    const bf16x8 v = __builtin_bit_cast(bf16x8, cf[t][ju]);
                    f32x8 f = __builtin_convertvector(v, f32x8);
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[x] *= w[x];
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        if (k == 2 && !third) break;
                        const bf16x8 h = __builtin_convertvector(f, bf16x8);
                        part[k][t][ju] = __builtin_bit_cast(u32x4, h);
                        if (k < 2) f -= __builtin_convertvector(h, f32x8);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        part[0][t][ju][x] = __float_as_uint(__uint_as_float(cf[t][ju][x]) * w[x]);
                }
            }
        }
    }
};

// Where a workgroup is: pass, batch row, head, segment, column slab.
struct LaWhere {
    int pass, b, h, seg, slab;
};

// Workgroups that share operands (the slabs of a head, the passes of a
// gradient, the heads of a group) get neighbouring numbers; the number is
// spread so that each of the 8 XCDs, which take workgroups in turn, gets a run
// of neighbours and finds them in its L2.
__device__ inline LaWhere la_where(const LaCall &c, int slabs) {
    const unsigned n = gridDim.x, x = blockIdx.x % 8, i = blockIdx.x / 8;
    unsigned id = x * (n / 8) + (x < n % 8 ? x : n % 8) + i;
    LaWhere w;
    w.slab = id % slabs;
    id /= slabs;
    w.pass = id % c.npass;
    id /= c.npass;
    w.h = id % c.H;
    id /= c.H;
    w.seg = id % c.grid_seg;
    w.b = id / c.grid_seg;
    return w;
}

// Offset of a wave's part of a segment's matrix in the workspace: fragment
// order [segment][row][slab][wave][tile][n][lane], 4 rows each.
template <class TL>
__device__ inline size_t la_seg_at(const LaCall &c, const LaWhere &w, int slabs, int wave, int lane) {
    const size_t row = ((size_t)w.seg * c.B + w.b) * c.H + w.h;
    return (((row * slabs + w.slab) * TL::NW + wave) * (TL::AT * TL::NT) * 64 + lane) * 4;
}

// One workgroup: the columns of a slab of one (pass, batch row, head), one
// segment of its tokens, chunk by chunk; STATE_ONLY: only the segment's own
// matrix, from zero, into the workspace.
//
// What bounds it.  bf16, heads of 128, 512 x 256 tokens with a state in and out
// (2.7 GB): 552 us, 4.9 TB/s, what a large copy reaches.  A chunk of 32 tokens
// costs a wave about 380 vector and 56 matrix instructions (72 where the state
// is returned), which with two waves a SIMD is two thirds of that time; the
// loads run two chunks ahead.  Chunks of 64 spilled (2.65 ms); every wave
// computing all of A B^T instead of its quarter took 1.5 times as many matrix
// instructions.  fp32: the matrix instructions themselves, 401 us for 512 x 64
// tokens of 16 heads of 128, about 140 of the 157 TFLOP/s with the products
// inside the chunks counted.
template <class DT, class TL, int EDGE, bool STATE_ONLY>
__global__ __launch_bounds__(TL::THREADS, 2) void k_la(LaCall c, int slabs) {
    using S_t = typename DT::S;
    constexpr bool DIRECT = EDGE == DIRECT_LDS;
    constexpr int BUFS = DIRECT ? TL::RING : TL::BUFS;
    __shared__ __align__(1024) S_t tiles[BUFS][TL::BUF_ELEMS];
    __shared__ __align__(16) S_t ps[STATE_ONLY ? 1 : 2 * TL::JU][64][TL::PER];  // fragments [it][ju] of (A B^T) . W
    const LaWhere at = la_where(c, slabs);
    const LaPass &p = c.pass[at.pass];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, m = lane % 16, g = lane / 16;
    const int len = la_len(c.lengths, at.b, c.T);
    const int i0 = at.seg * c.seg_tokens, i1 = min(len, i0 + c.seg_tokens);  // this segment's tokens
    const int dir = p.reverse ? -1 : 1, first = p.reverse ? len - 1 : 0, e = p.reverse ? 0 : 1;
    const float g2 = la_log2(c.log_decay[at.h]);
    const int slab0 = at.slab * TL::COLS, col0 = slab0 + wave * 16 * TL::NT;
    const bool busy = col0 < p.dc;  // else the wave only moves data and takes its part in A B^T

    // the matrix is a result: after the last segment here, or joined from the segments' own
    const bool keep = p.s1 && at.seg == c.nseg - 1, third = STATE_ONLY ? p.s1 != nullptr : keep, f32 = p.o.f32;
    const float chunk_scale = p.row_scale * p.sum_scale;
    const int osize = f32 ? 4 : (int)sizeof(S_t);
    // where this lane's columns of the chunk's two tokens go
    const int col_at = TL::TPK == 2 && TL::NT == 2 ? 8 * g : 4 * g;
    const long long ostep = p.o.t * dir * osize;
    char *op[2];
#pragma unroll
    for (int it = 0; it < 2; ++it)
        op[it] = p.o.p +
                 ((long long)first * p.o.t + (long long)at.b * p.o.b + (long long)at.h * p.o.h + col0 + col_at) * osize +
                 (i0 + TL::row_of(it, m / 4, m % 4)) * ostep;
    const int cols = p.dc - col0;
    // where a chunk's tensors lie in its buffer
    constexpr int AT_B = TL::C * TL::DA, AT_C = 2 * TL::C * TL::DA;
    LaStage<DT, TL, TL::RA, TL::PA, EDGE> sa, sb;
    LaStage<DT, TL, TL::RC, TL::PC, EDGE> sc;
    LaDirect<DT, TL, TL::RA> da, db;
    LaDirect<DT, TL, TL::RC> dc;
    constexpr int LOADS = (STATE_ONLY ? 1 : 2) * LaDirect<DT, TL, TL::RA>::N + LaDirect<DT, TL, TL::RC>::N;
    if constexpr (DIRECT) {
        if (!STATE_ONLY) da.init(p.a, at.b, at.h, first, dir, 0);
        db.init(p.b, at.b, at.h, first, dir, 0);
        dc.init(p.c, at.b, at.h, first, dir, slab0);
    } else {
        if (!STATE_ONLY) sa.init(p.a, at.b, at.h, first, dir, 0, p.da);
        sb.init(p.b, at.b, at.h, first, dir, 0, p.da);
        sc.init(p.c, at.b, at.h, first, dir, slab0, p.dc);
    }
    auto issue = [&](int i, int buf) {  // DIRECT: chunk i into its buffer
        const int n = min(TL::C, i1 - i);
        S_t *t = tiles[buf];
        if (!STATE_ONLY) da.load(t, i, n);
        db.load(t + AT_B, i, n);
        dc.load(t + AT_C, i, n);
    };
    auto fetch = [&](int i) {  // else: into registers,
        const int n = i1 - i;
        if (!STATE_ONLY) sa.load(i, n);
        sb.load(i, n);
        sc.load(i, n);
    };
    auto put = [&](S_t *t) {  // and from there
        if (!STATE_ONLY) sa.store(t);
        sb.store(t + AT_B);
        sc.store(t + AT_C);
    };
    if (i0 < i1) {
        if constexpr (DIRECT) {
#pragma unroll
            for (int k = 0; k < TL::RING - 1; ++k)
                if (i0 + k * TL::C < i1) issue(i0 + k * TL::C, k);
        } else {
            fetch(i0);
        }
    }
    f32x4 S[TL::AT * TL::NT];
#pragma unroll
    for (int x = 0; x < TL::AT * TL::NT; ++x) S[x] = f32x4{0, 0, 0, 0};
    // S from and to memory: 32 rows at a time through LDS, so that lanes take
    // neighbouring addresses (each lane fetching its own rows and columns took
    // 1.2 TB/s).  The matrix may lie transposed (srow = 1).
    constexpr int W4 = EDGE == WHOLE || DIRECT ? 4 : 1;  // neighbours in memory that a thread moves at once
    constexpr int PART = 8 * TL::NT / W4;                // such moves of a thread for 32 rows
    constexpr int ALL32 = (int)sizeof(tiles) / (32 * TL::LD * 4) < TL::DA / 32 ? (int)sizeof(tiles) / (32 * TL::LD * 4)
                                                                              : TL::DA / 32;  // that fit LDS at once
    float *const rows32 = reinterpret_cast<float *>(tiles[BUFS - 1]);
    const int across = p.srow == 1 ? TL::LD : 1;         // floats between a thread's neighbours in LDS
    auto place = [&](int y, int *row, int *col) {
        const int x = (y * TL::THREADS + tid) * W4;
        *row = p.srow == 1 ? x % 32 : x / TL::COLS;
        *col = p.srow == 1 ? x / 32 : x % TL::COLS;
    };
    const size_t own = ((size_t)at.b * c.H + at.h) * p.da * p.dc;
    if constexpr (!STATE_ONLY) {
        if (p.seg) {
            if (busy) {
                const float *src = p.seg + la_seg_at<TL>(c, at, slabs, wave, lane);
#pragma unroll
                for (int x = 0; x < TL::AT * TL::NT; ++x) S[x] = *reinterpret_cast<const f32x4 *>(src + x * 256);
            }
        } else if (p.s0) {
            float raw[TL::DA / 32][PART][W4];
            // (through a buffer resource, which reads 0 past the matrix: a
            // condition on a load becomes a branch and a wait for each)
            const unsigned bytes = (unsigned)(p.da * p.dc) * 4u;
            const __amdgpu_buffer_rsrc_t src = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<float *>(p.s0 + own), (short)0, (int)bytes, 0x00020000);
#pragma unroll
            for (int k = 0; k < TL::DA / 32; ++k)
#pragma unroll
                for (int y = 0; y < PART; ++y) {
                    int row, col;
                    place(y, &row, &col);
                    row += 32 * k;
                    col += slab0;
                    const unsigned off = (unsigned)(row * p.srow + col * p.scol) * 4u;
                    if constexpr (W4 == 4) {
                        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(src, (int)off, 0, 0);
#pragma unroll
                        for (int e = 0; e < 4; ++e) raw[k][y][e] = __uint_as_float(v[e]);
                    } else {
                        const int at0 = row < p.da && col < p.dc ? (int)off : (int)bytes;
                        const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(src, at0, 0, 0);
                        raw[k][y][0] = __uint_as_float(v);
                    }
                }
#pragma unroll
            for (int k = 0; k < TL::DA / 32; ++k) {
                if (k) la_barrier<63>();  // the rows before have been read
#pragma unroll
                for (int y = 0; y < PART; ++y) {
                    int row, col;
                    place(y, &row, &col);
#pragma unroll
                    for (int e = 0; e < W4; ++e) rows32[row * TL::LD + col + e * across] = raw[k][y][e];
                }
                la_barrier<63>();
#pragma unroll
                for (int t = 2 * k; t < 2 * k + 2; ++t)
#pragma unroll
                    for (int x = 0; x < TL::NT; ++x)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            S[t * TL::NT + x][r] =
                                rows32[(TL::row_of(t, g, r) - 32 * k) * TL::LD + wave * 16 * TL::NT + TL::col_of(x, m)];
            }
            la_barrier<63>();  // before the buffer takes tokens
        }
    }
    if (!DIRECT && i0 < i1) put(tiles[0]);

    int buf = 0;
    f32x4 O[2][TL::NT];
    // O's columns of its 2 x 16 tokens, n of the 32 valid; on to the next chunk
    auto flush = [&](int n) {
#pragma unroll
        for (int it = 0; it < 2; ++it) {
            char *const o = op[it];
            op[it] += TL::C * ostep;
            if (TL::row_of(it, m / 4, m % 4) >= n) continue;
            if constexpr (TL::TPK == 2 && TL::NT == 2) {  // 8 neighbouring columns
                const f32x8 v = __builtin_shufflevector(O[it][0], O[it][1], 0, 1, 2, 3, 4, 5, 6, 7);
                la_write<DT, 8, EDGE == WHOLE || DIRECT>(o, f32, v, cols - col_at);
            } else {
#pragma unroll
                for (int t = 0; t < TL::NT; ++t)
                    la_write<DT, 4, EDGE == WHOLE || DIRECT>(o + 16 * t * osize, f32, O[it][t], cols - 16 * t - col_at);
            }
        }
    };
    // S is kept as S / gamma^lag while gamma^128 lies within 2^-20 and 2^20: its
    // products with gamma then come due every fourth chunk only, and the powers
    // of gamma stand with the tokens' weights, which are multiplied anyway.
    // (A gamma far above 1 would take the weights to 0 and gamma^128 to infinity.)
    const bool slow = fabsf(g2) <= 20.0f / 128.0f;
    int lag = 0;
    // gamma^(i+e) of this lane's tokens, gamma^(i-j) of its part of W, and the
    // weights of the tokens j in the state's update over a whole chunk:
    // gamma^-(j+e) where gamma is slow, else gamma^(C-j-e)
    float row_w[2], mask_w[TL::PT][4], tok_w[TL::JU][TL::PER];
#pragma unroll
    for (int it = 0; it < 2; ++it) row_w[it] = la_pow(g2, TL::row_of(it, m / 4, m % 4) + e) * p.row_scale;
#pragma unroll
    for (int x = 0; x < TL::PT; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int it = wave % 2, jt = TL::NW == 2 ? x : wave / 2 % 2;
            mask_w[x][r] = la_pow(g2, max(TL::row_of(it, m / 4, m % 4) - TL::row_of(jt, g, r), 0)) * chunk_scale;
        }
#pragma unroll
    for (int ju = 0; ju < TL::JU; ++ju)
#pragma unroll
        for (int x = 0; x < TL::PER; ++x) {
            const int j = TL::KC * ju + TL::PER * g + x;
            tok_w[ju][x] = la_pow(g2, slow ? -(j + e) : TL::C - j - e) * p.sum_scale;
        }
    for (int i = i0; i < i1; i += TL::C) {
        const int n = min(TL::C, i1 - i);
        const bool more = i + TL::C < i1;
        if constexpr (DIRECT) {
            // this chunk lies in LDS once at most the later chunk's loads are
            // under way (the stores of the chunk before last come before them)
            if (TL::RING > 2 && more)
                la_barrier<LOADS *(TL::RING - 2)>();
            else
                la_barrier<0>();
            if (!STATE_ONLY && i > i0 && busy) flush(TL::C);
            const int next = i + (TL::RING - 1) * TL::C;
            if (next < i1) issue(next, buf == 0 ? TL::RING - 1 : buf - 1);
        } else {
            if (more) fetch(i + TL::C);
            __syncthreads();  // this chunk lies in LDS
        }
        const S_t *la = tiles[buf], *lb = la + AT_B, *lc = la + AT_C;

        // bf16: fragments are read well before their products, all at once (left
        // to itself the compiler reads a few, waits for LDS, and so on: about
        // 20 round trips a chunk).
        constexpr bool AHEAD = TL::TPK == 2 && TL::NU <= 4;
        u32x4 pa[TL::NU], pb[TL::NU], af[2][TL::NU], cf[TL::NT][TL::JU], bt[TL::AT];
        auto read_cf = [&]() {
#pragma unroll
            for (int t = 0; t < TL::NT; ++t)
#pragma unroll
                for (int ju = 0; ju < TL::JU; ++ju)
                    cf[t][ju] = la_cols<DT, TL, TL::RC>(
                        lc, ju, [&](int x) { return wave * 16 * TL::NT + TL::col_of(t, 4 * x); }, lane);
        };
        auto read_bt = [&](int t, int ju) {
            return la_cols<DT, TL, TL::RA>(lb, ju, [&](int x) { return TL::row_of(t, x, 0); }, lane);
        };
        if constexpr (AHEAD) {
            if constexpr (!STATE_ONLY) {
                const int it = wave % 2, jt = wave / 2 % 2;
#pragma unroll
                for (int u = 0; u < TL::NU; ++u) {
                    pb[u] = la_frag<DT, TL, TL::RA>(lb, jt, u, lane);
                    pa[u] = la_frag<DT, TL, TL::RA>(la, it, u, lane);
                }
#pragma unroll
                for (int u = 0; u < TL::NU; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) af[k][u] = la_frag<DT, TL, TL::RA>(la, k, u, lane);
            }
            read_cf();
            __builtin_amdgcn_sched_barrier(0);
        }

        // This wave's tiles of four of B A^T (rows: tokens j), weighted, as parts of
        // the fragments that the product with Cv reads.
        if constexpr (!STATE_ONLY) {
#pragma unroll
            for (int x = 0; x < TL::PT; ++x) {
                if (TL::NW > 4 && wave >= 4) break;
                const int it = wave % 2, jt = TL::NW == 2 ? x : wave / 2;
                f32x4 P = {0, 0, 0, 0};
                if (TL::TPK == 2 || jt <= it) {
#pragma unroll
                    for (int u = 0; u < TL::NU; ++u) {
                        // (x: a second tile of the same rows)
                        const u32x4 b = AHEAD && x == 0 ? pb[u] : la_frag<DT, TL, TL::RA>(lb, jt, u, lane);
                        P = mma_chunk(DT{}, P, b, AHEAD ? pa[u] : la_frag<DT, TL, TL::RA>(la, it, u, lane));
                    }
                    const int ri = TL::row_of(it, m / 4, m % 4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        P[r] = ri >= TL::row_of(jt, g, r) ? P[r] * mask_w[x][r] : 0.0f;
                    }
                }
                if constexpr (TL::TPK == 2)  // rounded here, once, as S is in la_pack
                    *reinterpret_cast<bf16x4 *>(&ps[it][lane][4 * jt]) = __builtin_convertvector(P, bf16x4);
                else
                    *reinterpret_cast<f32x4 *>(&ps[it * 2 + jt][lane][0]) = P;
            }
        }

        if (busy) {
            if constexpr (!STATE_ONLY) {
                // O = diag(gamma^(i+e)) A S, held transposed (rows: columns of
                // Cv), so that a lane ends with neighbouring columns of a token
#pragma unroll
                for (int it = 0; it < 2; ++it)
#pragma unroll
                    for (int t = 0; t < TL::NT; ++t) O[it][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int u = 0; u < TL::NU; ++u) {
                    if constexpr (!AHEAD)
#pragma unroll
                        for (int it = 0; it < 2; ++it) af[it][u] = la_frag<DT, TL, TL::RA>(la, it, u, lane);
#pragma unroll
                    for (int t = 0; t < TL::NT; ++t) {
                        const u32x4 sf = la_pack<DT, TL>(&S[u * TL::TPK * TL::NT + t], TL::NT);
#pragma unroll
                        for (int it = 0; it < 2; ++it) O[it][t] = mma_chunk(DT{}, O[it][t], sf, af[it][u]);
                    }
                }
                const float lag_w = la_pow(g2, lag);
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const float w = row_w[it] * lag_w;
#pragma unroll
                    for (int t = 0; t < TL::NT; ++t) O[it][t] *= w;
                }
            }
            if (!AHEAD) read_cf();
            // the state after the chunk, unless nothing reads it
            if (STATE_ONLY || more || keep) {
                if constexpr (AHEAD) {
#pragma unroll
                    for (int t = 0; t < TL::AT; ++t) bt[t] = read_bt(t, 0);
                    __builtin_amdgcn_sched_barrier(0);
                }
                const bool due = !slow || lag >= 3 * TL::C;
                float w[TL::JU][TL::PER];
                const float by = due ? la_pow(g2, n) : la_pow(g2, -lag);
#pragma unroll
                for (int ju = 0; ju < TL::JU; ++ju)
#pragma unroll
                    for (int x = 0; x < TL::PER; ++x) w[ju][x] = slow ? tok_w[ju][x] * by : tok_w[ju][x];
                if (n < TL::C)  // the last chunk
#pragma unroll
                    for (int ju = 0; ju < TL::JU; ++ju)
#pragma unroll
                        for (int x = 0; x < TL::PER; ++x) {
                            const int j = TL::KC * ju + TL::PER * g + x;
                            if (!slow) w[ju][x] = la_pow(g2, max(n - j - e, 0)) * p.sum_scale;
                            if (j >= n) w[ju][x] = 0.0f;
                        }
                LaWeighted<DT, TL> cw;
                cw.make(cf, w, third);
                if (due) {
                    const float whole = la_pow(g2, lag + n);
#pragma unroll
                    for (int x = 0; x < TL::AT * TL::NT; ++x) S[x] *= whole;
                    lag = 0;
                } else {
                    lag += n;
                }
#pragma unroll
                for (int t = 0; t < TL::AT; ++t) {
#pragma unroll
                    for (int ju = 0; ju < TL::JU; ++ju) {
                        const u32x4 kf = AHEAD ? bt[t] : read_bt(t, ju);
#pragma unroll
                        for (int x = 0; x < TL::NT; ++x) {
                            S[t * TL::NT + x] = mma_chunk(DT{}, S[t * TL::NT + x], kf, cw.part[0][x][ju]);
                            if constexpr (TL::TPK == 2)
                                S[t * TL::NT + x] = mma_chunk(DT{}, S[t * TL::NT + x], kf, cw.part[1][x][ju]);
                        }
                        if (TL::TPK == 2 && third)
#pragma unroll
                            for (int x = 0; x < TL::NT; ++x)
                                S[t * TL::NT + x] = mma_chunk(DT{}, S[t * TL::NT + x], kf,
                                                              cw.part[LaWeighted<DT, TL>::TERMS - 1][x][ju]);
                    }
                }
            }
        }

        if constexpr (!STATE_ONLY) {
            // the fragments of (A B^T) . W lie in LDS
            if constexpr (DIRECT)
                la_barrier<63>();
            else
                __syncthreads();
            if (busy) {
#pragma unroll
                for (int it = 0; it < 2; ++it) {
#pragma unroll
                    for (int ju = 0; ju < TL::JU; ++ju) {
                        if (TL::TPK == 1 && ju > it) continue;
                        const u32x4 pf = *reinterpret_cast<const u32x4 *>(&ps[it * TL::JU + ju][lane][0]);
#pragma unroll
                        for (int t = 0; t < TL::NT; ++t) O[it][t] = mma_chunk(DT{}, O[it][t], cf[t][ju], pf);
                    }
                }
                // DIRECT: the stores wait for the next chunk, behind whose
                // barrier they precede loads that nobody waits for yet
                if (!DIRECT || !more) flush(n);
            }
        }
        if constexpr (!DIRECT) {
            if (BUFS == 1 && more) __syncthreads();  // the chunk has been read
            if (more) put(tiles[BUFS == 2 ? buf ^ 1 : 0]);
        }
        buf = buf + 1 < BUFS ? buf + 1 : 0;
    }

    const float rest = la_pow(g2, lag);
    if constexpr (STATE_ONLY) {
        if (!busy) return;
        float *dst = p.seg + la_seg_at<TL>(c, at, slabs, wave, lane);
#pragma unroll
        for (int x = 0; x < TL::AT * TL::NT; ++x) *reinterpret_cast<f32x4 *>(dst + x * 256) = S[x] * rest;
    } else {
        if (keep) {
            float *dst = p.s1 + own, *rows = reinterpret_cast<float *>(tiles);
#pragma unroll
            for (int k0 = 0; k0 < TL::DA / 32; k0 += ALL32) {
                la_barrier<63>();  // the buffers' last readers are through
#pragma unroll
                for (int t = 2 * k0; t < 2 * (k0 + ALL32) && t < TL::AT; ++t)
#pragma unroll
                    for (int x = 0; x < TL::NT; ++x)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            rows[(TL::row_of(t, g, r) - 32 * k0) * TL::LD + wave * 16 * TL::NT + TL::col_of(x, m)] =
                                S[t * TL::NT + x][r] * rest;
                la_barrier<63>();
#pragma unroll
                for (int k = k0; k < k0 + ALL32 && k < TL::DA / 32; ++k)
#pragma unroll
                    for (int y = 0; y < PART; ++y) {
                        int row, col;
                        place(y, &row, &col);
                        const float *v = rows + (row + 32 * (k - k0)) * TL::LD + col;
                        row += 32 * k;
                        col += slab0;
                        float *q = dst + row * p.srow + col * p.scol;
                        if constexpr (W4 == 4) {
                            const f32x4 w = {v[0], v[across], v[2 * across], v[3 * across]};
                            __builtin_memcpy(q, &w, 16);
                        } else if (row < p.da && col < p.dc) {
                            *q = *v;
                        }
                    }
            }
        }
        if (!busy) return;
        // tokens past the row's end, by the segment of their own position
        const int width = min(16 * TL::NT, p.dc - col0), t1 = min(c.T, i0 + c.seg_tokens);
        for (int t = max(len, i0) + lane / 16; t < t1; t += 4)
            for (int d = m; d < width; d += 16) la_put<DT>(p.o, t, at.b, at.h, col0 + d, 0.0f);
    }
}

// Segments' own matrices -> the matrix before each segment, in place:
//     run = S0;  for each s: (seg_s, run) = (run, gamma^(tokens of s) run + seg_s)
// A thread keeps 4 rows of one column.
template <class DT, class TL>
__global__ __launch_bounds__(256) void k_la_join(LaCall c, int slabs) {
    const LaPass &p = c.pass[blockIdx.y];
    constexpr int PER_ROW = TL::AT * TL::NT * 64;  // threads for a wave's part
    const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x;
    const size_t row_size = (size_t)slabs * TL::NW * PER_ROW, rows = (size_t)c.B * c.H;
    if (id >= rows * row_size) return;
    const int bh = (int)(id / row_size), x = (int)(id % row_size);
    const int lane = x % 64, tile = x / 64 % (TL::AT * TL::NT), wave = x / PER_ROW % TL::NW;
    const int slab = x / PER_ROW / TL::NW;
    const int b = bh / c.H, h = bh % c.H, n = tile % TL::NT;
    const int col = slab * TL::COLS + wave * 16 * TL::NT + TL::col_of(n, lane % 16);
    const int row = TL::row_of(tile / TL::NT, lane / 16, 0);  // rows row .. row + 3
    if (col >= p.dc || row >= p.da) {
        // never read back into a result: the operands are zero there
        for (int s = 0; s < c.nseg; ++s)
            *reinterpret_cast<f32x4 *>(p.seg + (s * rows * row_size + id) * 4) = f32x4{0, 0, 0, 0};
        return;
    }
    const int len = la_len(c.lengths, b, c.T);
    const float g2 = la_log2(c.log_decay[h]);
    const size_t own = (size_t)bh * p.da * p.dc;
    f32x4 run = {0, 0, 0, 0};
    if (p.s0)
        for (int r = 0; r < 4 && row + r < p.da; ++r)
            run[r] = p.s0[own + (row + r) * p.srow + col * p.scol];
    constexpr int AHEAD = 8;  // segments read before the first is written
    const size_t step = rows * row_size * 4;
    float *q = p.seg + id * 4;
    for (int s = 0; s < c.nseg; s += AHEAD) {
        f32x4 add[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)  // the last segment has none (and is read for nothing)
            add[k] = *reinterpret_cast<const f32x4 *>(q + min(s + k, c.nseg - 1) * step);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (s + k >= c.nseg) break;
            *reinterpret_cast<f32x4 *>(q + (s + k) * step) = run;
            run = run * la_pow(g2, min(max(len - (s + k) * c.seg_tokens, 0), c.seg_tokens)) + add[k];
        }
    }
}

// Shared heads: out head g = the sum, in order, of the fp32 partial sums of
// its `per` query heads.  VEC neighbouring elements a thread; a workgroup takes
// `rows` tokens; blockIdx.y chooses between the two tensors.
template <class DT, int VEC>
__global__ __launch_bounds__(256) void k_la_share(LaShare a, LaShare b, int T, int B, int G, int per, int rows) {
    const LaShare &x = blockIdx.y ? b : a;
    const unsigned D = (unsigned)x.D / VEC, row_items = D * G, items = row_items * rows;
    const long long first = (long long)blockIdx.x * rows, all = (long long)T * B;
    for (unsigned i = threadIdx.x; i < items; i += 256) {
        const unsigned d = i % D * VEC, g = i / D % G;
        const long long row = first + i / row_items;  // b * T + t
        if (row >= all) return;
        const float *p = x.part + (row * G + g) * per * x.D + d;
        float sum[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] = p[e];
        for (int j = 1; j < per; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[e] += p[(size_t)j * x.D + e];
        const long long t = row % T, bt = row / T;
        typename DT::S *o = reinterpret_cast<typename DT::S *>(x.out.p) + t * x.out.t + bt * x.out.b + g * x.out.h + d;
        typename DT::S w[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = round_to<DT>(sum[e]);
        __builtin_memcpy(o, w, sizeof(w));
    }
}

// One token.  The state is read and written once, which is all the time goes
// into: a workgroup takes TX * VEC columns of one (request, head), TX lanes to
// a row, and has RB rows a thread on their way before it needs the first.  o
// is summed over a thread's rows, then over the row groups through LDS, in
// fixed order.
template <class DT, int VEC, int TX>
__global__ __launch_bounds__(256) void k_la_step(LaStep c, int slabs) {
    constexpr int TY = 256 / TX, RB = 16;
    __shared__ float qs[256], ks[256], part[TY][TX * VEC];
    const int tid = threadIdx.x, x = tid % TX, y = tid / TX;
    const int slab = blockIdx.x % slabs, h = blockIdx.x / slabs % c.H, b = blockIdx.x / slabs / c.H;
    const int col = (slab * TX + x) * VEC;
    const int slot = c.slots ? c.slots[b] : b;
    const bool live = slot >= 0 && slot < c.n_slots, on = live && col < c.Dv;  // VEC divides Dv
    float o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = 0.0f;
    if (live) {
        const float gamma = la_pow(la_log2(c.log_decay[h]), 1);
        float *s = c.pool + ((size_t)slot * c.H + h) * c.Dk * c.Dv + col;
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = on ? la_get<DT>(c.v, 0, b, h, col + e) : 0.0f;
        if (tid < c.Dk) {
            qs[tid] = la_get<DT>(c.q, 0, b, h, tid);
            ks[tid] = la_get<DT>(c.k, 0, b, h, tid);
        }
        for (int d0 = y; d0 < c.Dk || d0 == y; d0 += TY * RB) {
            float st[RB][VEC];
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if (on && d0 + r * TY < c.Dk) __builtin_memcpy(st[r], s + (size_t)(d0 + r * TY) * c.Dv, VEC * 4);
            if (d0 == y) __syncthreads();  // q and k lie in LDS
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int d = d0 + r * TY;
                if (!on || d >= c.Dk) continue;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    st[r][e] = st[r][e] * gamma + ks[d] * v[e];
                    o[e] += qs[d] * st[r][e];
                }
                __builtin_memcpy(s + (size_t)d * c.Dv, st[r], VEC * 4);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[y][x * VEC + e] = o[e];
    __syncthreads();
    const int out = slab * TX * VEC + tid;
    if (tid >= TX * VEC || out >= c.Dv) return;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < TY; ++k) sum += part[k][tid];
    la_put<DT>(c.o, 0, b, h, out, sum * c.scale);
}

}  // namespace

namespace {

// Tile of a call: the contraction dim padded to 64, 128 or 256, the waves of a
// workgroup, and the 16-column tiles of a wave.  bf16 takes two tiles a wave:
// every wave reads all of A and B from LDS, which one tile a wave makes twice
// as much of (512 x 256 tokens, heads of 128: 505 us against 630).  fp32 is
// bound by its matrix instructions and by registers, and takes one (64 x 512
// tokens: 423 us against 530, which spilled).  Few and short sequences of bf16
// take one too, half a head a workgroup, so that more CUs share the work: 128
// rows of 1024 tokens 57 us against 70, 64 rows 45 against 51; 128 rows of 2048
// would lose (119 against 107, in segments).  fp32 does the same at any length
// (30 rows of 333 tokens 40 us against 47, 64 of 512 61 against 73; the three
// passes of 64 rows lost, 110 against 97).
struct LaPlan {
    int DA, NW, NT;
    int cols() const { return NW * NT * 16; }
};
LaPlan la_plan(int da, int dc, int dtype, long long rows, int T) {
    const int DA = da <= 64 ? 64 : da <= 128 ? 128 : 256;
    if (dtype != LSTM_BF16) return LaPlan{DA, dc <= 64 || rows <= 128 ? 4 : 8, 1};
    if (DA == 256) return LaPlan{DA, 4, 1};
    if (DA == 128 && dc > 64 && rows <= 192 && T <= 1024) return LaPlan{DA, 4, 1};
    return LaPlan{DA, DA == 64 && dc <= 64 ? 2 : 4, 2};
}

template <class DT, class TL, int EDGE>
hipError_t la_launch(const LaCall &c, int slabs, hipStream_t s) {
    const long long blocks = (long long)slabs * c.npass * c.H * c.B * c.nseg;
    if (blocks > 0xFFFFFFFFll / TL::THREADS) return hipErrorInvalidValue;
    if (c.nseg > 1) {
        LaCall own = c;  // the last segment's own matrix is the last pass's business
        own.grid_seg = c.nseg - 1;
        hipLaunchKernelGGL((k_la<DT, TL, EDGE, true>), dim3((unsigned)(blocks / c.nseg * own.grid_seg)),
                           dim3(TL::THREADS), 0, s, own, slabs);
        const size_t n = (size_t)c.B * c.H * slabs * TL::NW * TL::AT * TL::NT * 64;
        hipLaunchKernelGGL((k_la_join<DT, TL>), dim3((unsigned)((n + 255) / 256), c.npass), dim3(256), 0, s, c, slabs);
    }
    hipLaunchKernelGGL((k_la<DT, TL, EDGE, false>), dim3((unsigned)blocks), dim3(TL::THREADS), 0, s, c, slabs);
    return hipGetLastError();
}

// Every row begins on 16 bytes, and a chunk's rows lie within 32-bit offsets.
bool la_aligned(const LaTensor &x) {
    return (uintptr_t)x.p % 16 == 0 && x.t % 8 == 0 && x.b % 8 == 0 && x.h % 8 == 0 && x.t < (1 << 25) &&
           x.t > -(1 << 25);
}

template <class DT, int DA, int NW, int NT>
hipError_t la_go(const LaCall &c, int dc, hipStream_t s) {
    using TL = LaTile<DT, DA, NW, NT>;
    const int slabs = (dc + TL::COLS - 1) / TL::COLS;
    bool whole = true, pieces = true;
    for (int i = 0; i < c.npass; ++i) {
        whole = whole && c.pass[i].da == DA && c.pass[i].dc % TL::COLS == 0 && c.pass[i].dc == dc;
        pieces = pieces && c.pass[i].da >= TL::PER && c.pass[i].dc >= TL::PER;
    }
    if constexpr (TL::TPK == 2) {
        bool direct = whole;
        for (int i = 0; i < c.npass; ++i)
            direct = direct && la_aligned(c.pass[i].a) && la_aligned(c.pass[i].b) && la_aligned(c.pass[i].c);
        if (direct) return la_launch<DT, TL, DIRECT_LDS>(c, slabs, s);
    } else {
        if (whole) return la_launch<DT, TL, WHOLE>(c, slabs, s);
    }
    return pieces ? la_launch<DT, TL, EDGES>(c, slabs, s) : la_launch<DT, TL, SHORT>(c, slabs, s);
}

template <class DT>
hipError_t la_any(const LaCall &c, hipStream_t s) {
    const int da = c.npass > 1 ? max(c.pass[0].da, c.pass[0].dc) : c.pass[0].da;
    const int dc = c.npass > 1 ? da : c.pass[0].dc;
    const LaPlan t = la_plan(da, dc, c.dtype, (long long)c.B * c.H * c.npass, c.T);
    if constexpr (sizeof(typename DT::S) == 2) {
        if (t.DA == 64) return t.NW == 2 ? la_go<DT, 64, 2, 2>(c, dc, s) : la_go<DT, 64, 4, 2>(c, dc, s);
        if (t.DA == 128) return t.NT == 1 ? la_go<DT, 128, 4, 1>(c, dc, s) : la_go<DT, 128, 4, 2>(c, dc, s);
        return la_go<DT, 256, 4, 1>(c, dc, s);
    } else {
        if (t.DA == 64) return t.NW == 4 ? la_go<DT, 64, 4, 1>(c, dc, s) : la_go<DT, 64, 8, 1>(c, dc, s);
        if (t.DA == 128) return t.NW == 4 ? la_go<DT, 128, 4, 1>(c, dc, s) : la_go<DT, 128, 8, 1>(c, dc, s);
        return t.NW == 4 ? la_go<DT, 256, 4, 1>(c, dc, s) : la_go<DT, 256, 8, 1>(c, dc, s);
    }
}

}  // namespace

void la_segments(int T, long long rows, int npass, int da, int dc, int dtype, int *nseg, int *seg_tokens,
                 size_t *seg_floats) {
    if (npass > 1) da = dc = da > dc ? da : dc;
    const LaPlan t = la_plan(da, dc, dtype, rows * npass, T);
    constexpr int C = 32;
    const long long slabs = (dc + t.cols() - 1) / t.cols(), blocks = rows * npass * slabs;
    const int chunks = (T + C - 1) / C;
    // Microseconds, measured on heads of 128 x 128: a chunk takes `one` in the
    // pass that writes outputs and `own` in the one that sums a segment's own
    // matrix, however many workgroups run up to two a CU; cutting costs two
    // more launches and moves each segment's matrix three times.  16 rows of
    // 16384 tokens: 922 uncut, 111 in 16 segments, 100 in 32; 64 rows of 1024:
    // 65 uncut, 43 in 4, 49 in 8; 128 rows of 512: 39 uncut, 44 in 2.
    const double one = dtype == LSTM_BF16 ? 1.8 : 4.5, own = dtype == LSTM_BF16 ? 1.0 : 2.5;
    const double move = blocks * (double)t.DA * t.cols() * 12 / 5e6;
    double best = one * chunks;
    int per = chunks;  // chunks of a segment
    for (int n = 2; n <= chunks && n * blocks <= 512; ++n) {
        const int p = (chunks + n - 1) / n;
        const double time = (one + own) * p + 12 + move * n;
        if (time < best) best = time, per = p;
    }
    *nseg = (chunks + per - 1) / per;
    *seg_tokens = per * C;
    *seg_floats = (size_t)t.DA * slabs * t.cols();
}

hipError_t launch_la(const LaCall &call, hipStream_t s) {
    LaCall c = call;
    c.grid_seg = c.nseg;
    return c.dtype == LSTM_BF16 ? la_any<BF16>(c, s) : la_any<F32>(c, s);
}

hipError_t launch_la_share(const LaShare &a, const LaShare &b, int T, int B, int H, int G, int dtype, hipStream_t s) {
    const bool vec = a.D % 4 == 0 && b.D % 4 == 0;
    const int wide = G * (a.D > b.D ? a.D : b.D) / (vec ? 4 : 1), rows = wide >= 1024 ? 1 : 1024 / wide;
    const long long all = (long long)T * B, blocks = (all + rows - 1) / rows;
    if (blocks > 0xFFFFFFFFll / 256) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks, 2);
    const auto k = dtype == LSTM_BF16 ? (vec ? k_la_share<BF16, 4> : k_la_share<BF16, 1>)
                                      : (vec ? k_la_share<F32, 4> : k_la_share<F32, 1>);
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a, b, T, B, G, H / G, rows);
    return hipGetLastError();
}

namespace {

template <class DT, int VEC, int TX>
void la_step_go(const LaStep &c, hipStream_t s) {
    const int slabs = (c.Dv + TX * VEC - 1) / (TX * VEC);
    hipLaunchKernelGGL((k_la_step<DT, VEC, TX>), dim3((unsigned)slabs * c.B * c.H), dim3(256), 0, s, c, slabs);
}

template <class DT>
void la_step_any(const LaStep &c, hipStream_t s) {
    // 16-byte accesses where rows allow them; narrow column slabs while there
    // are fewer states than two for each CU
    const bool vec = c.Dv % 4 == 0 && (uintptr_t)c.pool % 16 == 0, few = (long long)c.B * c.H < 512;
    if (vec)
        few || c.Dv <= 32 ? la_step_go<DT, 4, 8>(c, s) : la_step_go<DT, 4, 32>(c, s);
    else
        la_step_go<DT, 1, 32>(c, s);
}

}  // namespace

hipError_t launch_la_step(const LaStep &c, hipStream_t s) {
    c.dtype == LSTM_BF16 ? la_step_any<BF16>(c, s) : la_step_any<F32>(c, s);
    return hipGetLastError();
}

}  // namespace lstm_amd
