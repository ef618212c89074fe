// layer_norm.hip -- layer norm with its residual sum, forward and backward.
#include "device.h"
#include "ops.h"
#include "ops_dev.h"

namespace lstm_amd {

int ln_parts(long long rows, int width) {
    (void)width;
    return (int)(rows < 256 ? rows : 256);
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

// One workgroup per row.
template <class DT>
__global__ __launch_bounds__(256) void k_ln_forward(LnForward c) {
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
__global__ __launch_bounds__(256) void k_ln_dx(LnBackward c) {
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
__global__ __launch_bounds__(256) void k_ln_dw(LnBackward c) {
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

template <class DT>
__global__ __launch_bounds__(256) void k_ln_join(LnBackward c, int parts) {
    using S = typename DT::S;
    const int W = c.width, i = blockIdx.x * 256 + threadIdx.x;
    if (i >= W) return;
    float w = 0.0f, b = 0.0f;
    for (int p = 0; p < parts; ++p) {
        w += c.part[(size_t)p * 2 * W + i];
        b += c.part[((size_t)p * 2 + 1) * W + i];
    }
    if (c.dw) reinterpret_cast<S *>(c.dw)[i] = round_to<DT>(w);
    if (c.db) reinterpret_cast<S *>(c.db)[i] = round_to<DT>(b);
}

template <class DT>
hipError_t ln_backward(const LnBackward &c, hipStream_t s) {
    const int parts = ln_parts(c.rows, c.width);
    if (c.rows > 0)
        hipLaunchKernelGGL(k_ln_dx<DT>, dim3((unsigned)(c.rows < 65536 ? c.rows : 65536)), dim3(256), 0, s, c);
    if (c.dw || c.db) {
        if (parts) hipLaunchKernelGGL(k_ln_dw<DT>, dim3(parts), dim3(256), 0, s, c);
        hipLaunchKernelGGL(k_ln_join<DT>, dim3((c.width + 255) / 256), dim3(256), 0, s, c, parts);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ln_forward(const LnForward &c, hipStream_t s) {
    const dim3 grid((unsigned)(c.rows < 65536 ? c.rows : 65536));
    if (c.dtype == LSTM_BF16)
        hipLaunchKernelGGL(k_ln_forward<BF16>, grid, dim3(256), 0, s, c);
    else
        hipLaunchKernelGGL(k_ln_forward<F32>, grid, dim3(256), 0, s, c);
    return hipGetLastError();
}

hipError_t launch_ln_backward(const LnBackward &c, hipStream_t s) {
    return c.dtype == LSTM_BF16 ? ln_backward<BF16>(c, s) : ln_backward<F32>(c, s);
}

}  // namespace lstm_amd
