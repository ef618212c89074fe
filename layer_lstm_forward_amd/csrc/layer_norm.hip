// layer_norm.hip -- layer norm with its residual sum, forward and backward.
//     z = x + residual,  u = (z - mean) rstd,  y = u w + b
//     dz = rstd (g - mean(g) - u mean(g u)) + dsum  with g = dy w
//     dw = sum over rows of dy u,  db = sum over rows of dy
// Both directions are bound by memory: a row is read once, into registers,
// and its sums are taken from there (the variance from the differences, in a
// second look at the registers).  131072 rows of 2048 bf16 with a residual:
// forward 397 us, backward 396 + 5 us, 5.4 TB/s each, as a copy.  A wave a row
// needs no barrier: with a workgroup a row the backward took 722 us.
#include "device.h"
#include "ops.h"
#include "ops_dev.h"

namespace lstm_amd {

// Two workgroups a CU keep the partial sums of the weight gradients; of rows
// that take 1024 threads only one is resident, and half the partial sums are
// half the traffic (2048 rows of 8192 bf16: 37 us against 48).
int ln_parts(long long rows, int width) {
    const int most = width > 4096 ? 256 : 512;
    return (int)(rows < most ? rows : most);
}

namespace {

// Sum over the 256 threads, the same value in each; fixed order.
__device__ inline float block_sum(float v, float *lds) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

// A row lies over TPR threads, NV 16-byte pieces each: piece v of thread t is
// the row's piece v * TPR + t.  A workgroup holds 256 / TPR rows at a time
// (TPR = 1024: one row over 1024 threads).
template <class DT, int TPR_, int NV_>
struct LnTile {
    static constexpr int TPR = TPR_, NV = NV_, PER = DT::PER16;
    static constexpr int THREADS = TPR > 256 ? TPR : 256, ROWS = THREADS / TPR;
    static constexpr int WIDTH = TPR * NV * PER;  // widest row
};

// Sum over the TPR threads of a row, the same value in each, in fixed order.
template <class TL>
__device__ inline float row_sum(float v, float *lds) {
#pragma unroll
    for (int o = (TL::TPR < 64 ? TL::TPR : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (TL::TPR > 64) {
        __syncthreads();
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TL::TPR / 64; ++i) v += lds[i];
    }
    return v;
}

// One 16-byte piece widened, zeros past the row's end, or with PAST that value
// in the storage type; any alignment.
template <class DT, bool PAST = false>
__device__ inline void ln_load(const typename DT::S *p, int i, int W, float *f, float past = 0.0f) {
    using S = typename DT::S;
    S t[DT::PER16];
    if (i + DT::PER16 <= W) {
        __builtin_memcpy(t, p + i, 16);
    } else {
        // (bf16: not rounded ahead, which would wait for it before any load)
        if (PAST && sizeof(S) == 2) asm volatile("" : "+v"(past));
#pragma unroll
        for (int e = 0; e < DT::PER16; ++e) t[e] = i + e < W ? p[i + e] : PAST ? round_to<DT>(past) : (S)0;
    }
#pragma unroll
    for (int e = 0; e < DT::PER16; ++e) f[e] = DT::to_f(t[e]);
}

template <class DT>
__device__ inline void ln_store(typename DT::S *p, int i, int W, const float *f) {
    using S = typename DT::S;
    S t[DT::PER16];
#pragma unroll
    for (int e = 0; e < DT::PER16; ++e) t[e] = round_to<DT>(f[e]);
    if (i + DT::PER16 <= W)
        __builtin_memcpy(p + i, t, 16);
    else
#pragma unroll
        for (int e = 0; e < DT::PER16; ++e)
            if (i + e < W) p[i + e] = t[e];
}

template <class DT, class TL>
__global__ __launch_bounds__(TL::THREADS) void k_ln_forward(LnForward c) {
    using S = typename DT::S;
    constexpr int PER = TL::PER;
    __shared__ float lds[16];
    const int W = c.width, t = threadIdx.x % TL::TPR;
    const float inv = 1.0f / (float)W;
    float w[TL::NV][PER], bias[TL::NV][PER];  // kept for all rows of the workgroup
#pragma unroll
    for (int v = 0; v < TL::NV; ++v) {
        const int i = (v * TL::TPR + t) * PER;
#pragma unroll
        for (int e = 0; e < PER; ++e) w[v][e] = 1.0f, bias[v][e] = 0.0f;
        if (c.w) ln_load<DT>(reinterpret_cast<const S *>(c.w), i, W, w[v]);
        if (c.bias) ln_load<DT>(reinterpret_cast<const S *>(c.bias), i, W, bias[v]);
    }
    for (long long r0 = (long long)blockIdx.x * TL::ROWS; r0 < c.rows; r0 += (long long)gridDim.x * TL::ROWS) {
        const long long r = r0 + threadIdx.x / TL::TPR;
        const bool on = r < c.rows;  // every thread takes part in the sums
        const S *x = reinterpret_cast<const S *>(c.x) + (on ? r : 0) * c.xs;
        const S *res = c.res ? reinterpret_cast<const S *>(c.res) + (on ? r : 0) * c.rs : nullptr;
        float z[TL::NV][PER], s = 0.0f;
#pragma unroll
        for (int v = 0; v < TL::NV; ++v) ln_load<DT>(x, (v * TL::TPR + t) * PER, W, z[v]);
        if (res) {
            float y[TL::NV][PER];
#pragma unroll
            for (int v = 0; v < TL::NV; ++v) ln_load<DT>(res, (v * TL::TPR + t) * PER, W, y[v]);
#pragma unroll
            for (int v = 0; v < TL::NV; ++v)
#pragma unroll
                for (int e = 0; e < PER; ++e) z[v][e] = DT::to_f(round_to<DT>(z[v][e] + y[v][e]));
        }
#pragma unroll
        for (int v = 0; v < TL::NV; ++v)
#pragma unroll
            for (int e = 0; e < PER; ++e) s += z[v][e];
        const float mean = row_sum<TL>(s, lds) * inv;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < TL::NV; ++v)
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const float d = z[v][e] - mean;
                if ((v * TL::TPR + t) * PER + e < W) s += d * d;
            }
        const float rstd = 1.0f / sqrtf(row_sum<TL>(s, lds) * inv + c.eps);
        if (!on) continue;
        if (t == 0) {
            if (c.mean) c.mean[r] = mean;
            if (c.rstd) c.rstd[r] = rstd;
        }
#pragma unroll
        for (int v = 0; v < TL::NV; ++v) {
            const int i = (v * TL::TPR + t) * PER;
            if (c.sum) ln_store<DT>(reinterpret_cast<S *>(c.sum) + r * W, i, W, z[v]);
#pragma unroll
            for (int e = 0; e < PER; ++e) z[v][e] = (z[v][e] - mean) * rstd * w[v][e] + bias[v][e];
            ln_store<DT>(reinterpret_cast<S *>(c.y) + r * W, i, W, z[v]);
        }
    }
}

// dz, and the workgroup's own sums of dy u and dy over its rows, which stay in
// registers until the last row: the weight gradients cost no second pass over
// dy and z.
template <class DT, class TL>
__global__ __launch_bounds__(TL::THREADS) void k_ln_backward(LnBackward c) {
    using S = typename DT::S;
    constexpr int PER = TL::PER;
    __shared__ float lds[16];
    __shared__ float joint[TL::ROWS > 1 ? TL::ROWS * TL::WIDTH : 1];
    const int W = c.width, t = threadIdx.x % TL::TPR, mine = threadIdx.x / TL::TPR;
    const float inv = 1.0f / (float)W;
    float w[TL::NV][PER], dw[TL::NV][PER], db[TL::NV][PER];
#pragma unroll
    for (int v = 0; v < TL::NV; ++v) {
#pragma unroll
        for (int e = 0; e < PER; ++e) w[v][e] = 1.0f, dw[v][e] = db[v][e] = 0.0f;
        if (c.w) ln_load<DT>(reinterpret_cast<const S *>(c.w), (v * TL::TPR + t) * PER, W, w[v]);
    }
    for (long long r0 = (long long)blockIdx.x * TL::ROWS; r0 < c.rows; r0 += (long long)gridDim.x * TL::ROWS) {
        const long long r = r0 + mine;
        const bool on = r < c.rows;
        const long long q = on ? r : 0;
        const S *dy = reinterpret_cast<const S *>(c.dy) + q * c.ys, *z = reinterpret_cast<const S *>(c.z) + q * c.zs;
        const S *ds = c.dsum ? reinterpret_cast<const S *>(c.dsum) + q * W : nullptr;
        const float mean = c.mean[q], rstd = c.rstd[q];
        float g[TL::NV][PER], u[TL::NV][PER], add[TL::NV][PER], s = 0.0f, su = 0.0f;
#pragma unroll
        for (int v = 0; v < TL::NV; ++v) {
            const int i = (v * TL::TPR + t) * PER;
            ln_load<DT>(dy, i, W, g[v]);
            // (The mean past the end, not 0: a constant row of large values has an
            // infinite mean rstd, whose product with a dy of 0 would be NaN.)
            ln_load<DT, true>(z, i, W, u[v], mean);
#pragma unroll
            for (int e = 0; e < PER; ++e) add[v][e] = 0.0f;
            if (ds) ln_load<DT>(ds, i, W, add[v]);
        }
#pragma unroll
        for (int v = 0; v < TL::NV; ++v)
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                u[v][e] = (u[v][e] - mean) * rstd;  // past the row's end: times a dy of 0
                if (on) {
                    dw[v][e] += g[v][e] * u[v][e];
                    db[v][e] += g[v][e];
                }
                g[v][e] *= w[v][e];
                s += g[v][e];
                su += g[v][e] * u[v][e];
            }
        const float m = row_sum<TL>(s, lds) * inv, mu = row_sum<TL>(su, lds) * inv;
        if (!on) continue;
#pragma unroll
        for (int v = 0; v < TL::NV; ++v) {
#pragma unroll
            for (int e = 0; e < PER; ++e) g[v][e] = rstd * (g[v][e] - m - u[v][e] * mu) + add[v][e];
            ln_store<DT>(reinterpret_cast<S *>(c.dx) + r * W, (v * TL::TPR + t) * PER, W, g[v]);
        }
    }
    if (!c.part) return;
    float *part = c.part + (size_t)blockIdx.x * 2 * W;
#pragma unroll
    for (int k = 0; k < 2; ++k, part += W) {
        if constexpr (TL::ROWS == 1) {
#pragma unroll
            for (int v = 0; v < TL::NV; ++v)
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const int i = (v * TL::TPR + t) * PER + e;
                    if (i < W) part[i] = k ? db[v][e] : dw[v][e];
                }
        } else {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < TL::NV; ++v)
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    joint[mine * TL::WIDTH + (v * TL::TPR + t) * PER + e] = k ? db[v][e] : dw[v][e];
            __syncthreads();
            for (int i = threadIdx.x; i < W; i += TL::THREADS) {
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < TL::ROWS; ++j) sum += joint[j * TL::WIDTH + i];
                part[i] = sum;
            }
        }
    }
}

// Rows too wide for the registers of a workgroup: read again for each sum.
// (Already the widest tile, above 8192 values, has 37 values of each thread of
// the backward in scratch: 1024 rows of 16384 bf16 61 us, 1.6 TB/s.)
template <class DT>
__global__ __launch_bounds__(256) void k_ln_forward_wide(LnForward c) {
    using S = typename DT::S;
    __shared__ float lds[4];
    const int W = c.width;
    for (long long r = blockIdx.x; r < c.rows; r += gridDim.x) {
        const S *x = reinterpret_cast<const S *>(c.x) + r * c.xs;
        const S *res = c.res ? reinterpret_cast<const S *>(c.res) + r * c.rs : nullptr;
        S *y = reinterpret_cast<S *>(c.y) + r * W, *z = c.sum ? reinterpret_cast<S *>(c.sum) + r * W : nullptr;
        auto at = [&](int i) {
            const float v = DT::to_f(x[i]);
            return res ? DT::to_f(round_to<DT>(v + DT::to_f(res[i]))) : v;
        };
        float s = 0.0f;
        for (int i = threadIdx.x; i < W; i += 256) s += at(i);
        const float mean = block_sum(s, lds) / (float)W;
        s = 0.0f;
        for (int i = threadIdx.x; i < W; i += 256) s += (at(i) - mean) * (at(i) - mean);
        const float rstd = 1.0f / sqrtf(block_sum(s, lds) / (float)W + c.eps);
        if (threadIdx.x == 0) {
            if (c.mean) c.mean[r] = mean;
            if (c.rstd) c.rstd[r] = rstd;
        }
        for (int i = threadIdx.x; i < W; i += 256) {
            const float v = at(i);
            const float w = c.w ? DT::to_f(reinterpret_cast<const S *>(c.w)[i]) : 1.0f;
            const float b = c.bias ? DT::to_f(reinterpret_cast<const S *>(c.bias)[i]) : 0.0f;
            if (z) z[i] = round_to<DT>(v);
            y[i] = round_to<DT>((v - mean) * rstd * w + b);
        }
    }
}

template <class DT>
__global__ __launch_bounds__(256) void k_ln_dx_wide(LnBackward c) {
    using S = typename DT::S;
    __shared__ float lds[4];
    const int W = c.width;
    for (long long r = blockIdx.x; r < c.rows; r += gridDim.x) {
        const S *dy = reinterpret_cast<const S *>(c.dy) + r * c.ys, *z = reinterpret_cast<const S *>(c.z) + r * c.zs;
        const S *ds = c.dsum ? reinterpret_cast<const S *>(c.dsum) + r * W : nullptr;
        S *dx = reinterpret_cast<S *>(c.dx) + r * W;
        const float mean = c.mean[r], rstd = c.rstd[r];
        auto g = [&](int i) {
            return DT::to_f(dy[i]) * (c.w ? DT::to_f(reinterpret_cast<const S *>(c.w)[i]) : 1.0f);
        };
        float s = 0.0f, sx = 0.0f;
        for (int i = threadIdx.x; i < W; i += 256) {
            s += g(i);
            sx += g(i) * (DT::to_f(z[i]) - mean) * rstd;
        }
        const float m = block_sum(s, lds) / (float)W, mx = block_sum(sx, lds) / (float)W;
        for (int i = threadIdx.x; i < W; i += 256) {
            const float unit = (DT::to_f(z[i]) - mean) * rstd;
            dx[i] = round_to<DT>(rstd * (g(i) - m - unit * mx) + (ds ? DT::to_f(ds[i]) : 0.0f));
        }
    }
}

// Workgroup p sums the rows p, p + parts, ... of every column.
template <class DT>
__global__ __launch_bounds__(256) void k_ln_dw_wide(LnBackward c) {
    using S = typename DT::S;
    const int W = c.width;
    for (int i = threadIdx.x; i < W; i += 256) {
        float w = 0.0f, b = 0.0f;
        for (long long r = blockIdx.x; r < c.rows; r += gridDim.x) {
            const float dy = DT::to_f(reinterpret_cast<const S *>(c.dy)[r * c.ys + i]);
            const float z = DT::to_f(reinterpret_cast<const S *>(c.z)[r * c.zs + i]);
            w += dy * (z - c.mean[r]) * c.rstd[r];
            b += dy;
        }
        c.part[(size_t)blockIdx.x * 2 * W + i] = w;
        c.part[((size_t)blockIdx.x * 2 + 1) * W + i] = b;
    }
}

// The workgroups' partial sums, in their order: 8 threads take every eighth of
// a column's, then their sums are added.  A grid holds fewer than 2^32 threads,
// which the widest rows would need here, so workgroups go on to further columns.
constexpr unsigned kJoinBlocks = 1 << 20;
template <class DT>
__global__ __launch_bounds__(256) void k_ln_join(LnBackward c, int parts) {
    using S = typename DT::S;
    __shared__ float lds[8][32];
    const int W2 = 2 * c.width, x = threadIdx.x % 32, y = threadIdx.x / 32;
    for (int i0 = blockIdx.x * 32; i0 < W2; i0 += gridDim.x * 32) {
        const int i = i0 + x;
        float sum = 0.0f;
        if (i < W2)
#pragma unroll 8
            for (int p = y; p < parts; p += 8) sum += c.part[(size_t)p * W2 + i];
        if (i0 != (int)blockIdx.x * 32) __syncthreads();  // the sums before have been read
        lds[y][x] = sum;
        __syncthreads();
        if (y > 0 || i >= W2) continue;
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += lds[k][x];
        S *out = reinterpret_cast<S *>(i < c.width ? c.dw : c.db);
        if (out) out[i < c.width ? i : i - c.width] = round_to<DT>(sum);
    }
}

// The smallest tile that a row fits: f(LnTile) for it, else wide().
template <class DT, class F, class G>
void ln_tile(int W, F f, G wide) {
    constexpr int P = DT::PER16;
    if (W <= 16 * P)
        f(LnTile<DT, 16, 1>{});
    else if (W <= 32 * P)
        f(LnTile<DT, 16, 2>{});
    else if (W <= 64 * P)
        f(LnTile<DT, 64, 1>{});
    else if (W <= 128 * P)
        f(LnTile<DT, 64, 2>{});
    else if (W <= 256 * P)
        f(LnTile<DT, 64, 4>{});
    else if (W <= 512 * P)
        f(LnTile<DT, 256, 2>{});
    else if (W <= 1024 * P)
        f(LnTile<DT, 1024, 1>{});
    else if (W <= 2048 * P)
        f(LnTile<DT, 1024, 2>{});
    else if (P == 4 && W <= 4096 * P)
        f(LnTile<DT, 1024, P == 4 ? 4 : 2>{});
    else
        wide();
}

unsigned blocks_of(long long rows, int per, long long most) {
    const long long n = (rows + per - 1) / per;
    return (unsigned)(n < most ? n : most);
}

template <class DT>
hipError_t ln_forward(const LnForward &c, hipStream_t s) {
    ln_tile<DT>(
        c.width,
        [&](auto tile) {
            using TL = decltype(tile);
            hipLaunchKernelGGL((k_ln_forward<DT, TL>), dim3(blocks_of(c.rows, TL::ROWS, 2048)), dim3(TL::THREADS), 0, s,
                               c);
        },
        [&]() { hipLaunchKernelGGL(k_ln_forward_wide<DT>, dim3(blocks_of(c.rows, 1, 65536)), dim3(256), 0, s, c); });
    return hipGetLastError();
}

template <class DT>
hipError_t ln_backward(const LnBackward &c, hipStream_t s) {
    int parts = 0;
    if (c.rows > 0)
        ln_tile<DT>(
            c.width,
            [&](auto tile) {
                using TL = decltype(tile);
                parts = (int)blocks_of(c.rows, TL::ROWS, ln_parts(c.rows, c.width));
                hipLaunchKernelGGL((k_ln_backward<DT, TL>), dim3(parts), dim3(TL::THREADS), 0, s, c);
            },
            [&]() {
                parts = ln_parts(c.rows, c.width);
                // the sums first: dx may lie over dy
                if (c.part) hipLaunchKernelGGL(k_ln_dw_wide<DT>, dim3(parts), dim3(256), 0, s, c);
                hipLaunchKernelGGL(k_ln_dx_wide<DT>, dim3(blocks_of(c.rows, 1, 65536)), dim3(256), 0, s, c);
            });
    if (c.dw || c.db)
        hipLaunchKernelGGL(k_ln_join<DT>, dim3(blocks_of(2ll * c.width, 32, kJoinBlocks)), dim3(256), 0, s, c, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ln_forward(const LnForward &c, hipStream_t s) {
    return c.dtype == LSTM_BF16 ? ln_forward<BF16>(c, s) : ln_forward<F32>(c, s);
}

hipError_t launch_ln_backward(const LnBackward &c, hipStream_t s) {
    return c.dtype == LSTM_BF16 ? ln_backward<BF16>(c, s) : ln_backward<F32>(c, s);
}

}  // namespace lstm_amd
