// adamw.hip -- one AdamW step over a list of tensors.
#include "device.h"
#include "ops.h"
#include "ops_dev.h"

namespace lstm_amd {

namespace {

constexpr int kBlock = LSTM_ADAMW_BLOCK;

// Up to kMaxEntries tensors travel in the kernel's arguments, so that a call
// needs no device table and no copy, and reads every pointer afresh.
constexpr int kMaxEntries = 44;
struct AdamwTable {
    lstm_adamw_tensor t[kMaxEntries];
    unsigned first[kMaxEntries + 1];  // first state block of each tensor, and their end
    int count;
};
static_assert(sizeof(AdamwTable) + sizeof(AdamwHyper) <= 4096, "kernel arguments");

// 32 bits for an element, from its index (low 32 bits) and the seed: two
// rounds of xor-shift and multiply by odd constants.
__device__ inline unsigned dither(unsigned i, unsigned seed) {
    unsigned x = i + seed * 0x9E3779B1u;
    x ^= x >> 16;
    x *= 0x6C9F52D5u;
    x ^= x >> 15;
    x *= 0xB5297A4Du;
    return x ^ (x >> 16);
}

// The code of |x| = y * scale, y below 256: rounded up where the dropped
// fraction plus 16 random bits carries.  Below 2^-6 the codes are multiples of
// 2^-9; above, they are the float's own bits without the low 20.
__device__ inline unsigned code_of(float y, unsigned bits16) {
#pragma clang fp contract(off)
    const unsigned r = (bits16 << 4) | 8u;
    if (!(y < __builtin_inff())) return 0x7Fu;  // infinity or NaN: the format's NaN
    if (y >= 0.015625f) return ((__float_as_uint(y) + r) >> 20) - (120u << 3);
    return (unsigned)(y * 512.0f + (float)r * 0x1p-20f);
}

__device__ inline float value_of(unsigned code) {
    const unsigned e = (code >> 3) & 15u, f = code & 7u;
    float v = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : (float)f * 0x1p-9f;
    if ((code & 0x7Fu) == 0x7Fu) v = __builtin_nanf("");
    return code & 0x80u ? -v : v;
}

// One workgroup per block of 256 elements, one element a thread.
template <class DT, bool EIGHT>
__global__ __launch_bounds__(256) void k_adamw(AdamwTable tab, AdamwHyper h) {
    using S = typename DT::S;
    __shared__ unsigned top[2][4];
    int e = 0;
    while (blockIdx.x >= tab.first[e + 1]) ++e;
    const lstm_adamw_tensor &t = tab.t[e];
    const unsigned blk = blockIdx.x - tab.first[e];
    const long long i = (long long)blk * kBlock + threadIdx.x;
    const bool on = i < t.n;
    float m = 0.0f, v = 0.0f, root = 0.0f;
    if (on) {
#pragma clang fp contract(off)
        float g = DT::to_f(static_cast<const S *>(t.grad)[i]);
        if (h.grad_scale) g = g * *h.grad_scale;
        if (EIGHT) {
            m = value_of(static_cast<const unsigned char *>(t.m)[i]) * t.m_scale[blk];
            root = value_of(static_cast<const unsigned char *>(t.v)[i]) * t.v_scale[blk];
            v = root * root;
        } else {
            m = static_cast<const float *>(t.m)[i];
            v = static_cast<const float *>(t.v)[i];
        }
        m = m * h.beta1 + g * h.one_beta1;
        v = v * h.beta2 + (g * g) * h.one_beta2;
        root = sqrtf(v);
        const float step = m * h.inv_bc1 / (root * h.inv_sqrt_bc2 + h.eps);
        S *p = static_cast<S *>(t.param) + i;
        const float w = (t.master ? t.master[i] : DT::to_f(*p)) * (1.0f - t.lr * t.weight_decay) - t.lr * step;
        if (t.master) t.master[i] = w;
        *p = round_to<DT>(w);
    }
    if (!EIGHT) {
        if (on) {
            static_cast<float *>(t.m)[i] = m;
            static_cast<float *>(t.v)[i] = v;
        }
        return;
    }
    // the block's largest exponents; what is not finite does not count
    unsigned am = __float_as_uint(m) & 0x7FFFFFFFu, av = __float_as_uint(root) & 0x7FFFFFFFu;
    if (am >= 0x7F800000u) am = 0;
    if (av >= 0x7F800000u) av = 0;
    for (int o = 32; o > 0; o >>= 1) {
        am = max(am, (unsigned)__shfl_xor((int)am, o));
        av = max(av, (unsigned)__shfl_xor((int)av, o));
    }
    if (threadIdx.x % 64 == 0) {
        top[0][threadIdx.x / 64] = am;
        top[1][threadIdx.x / 64] = av;
    }
    __syncthreads();
    am = max(max(top[0][0], top[0][1]), max(top[0][2], top[0][3]));
    av = max(max(top[1][0], top[1][1]), max(top[1][2], top[1][3]));
    const unsigned em = max((int)(am >> 23) - 7, 1), ev = max((int)(av >> 23) - 7, 1);
    if (on) {
        const unsigned bits = dither((unsigned)i, h.seed);
        const float im = __uint_as_float((254u - em) << 23), iv = __uint_as_float((254u - ev) << 23);
        unsigned cm = code_of(fabsf(m) * im, bits & 0xFFFFu), cv = code_of(root * iv, bits >> 16);
        if (cv == 0 && root > 0.0f) cv = 1;
        static_cast<unsigned char *>(t.m)[i] = (unsigned char)(cm | (m < 0.0f ? 0x80u : 0u));
        static_cast<unsigned char *>(t.v)[i] = (unsigned char)cv;
    }
    if (threadIdx.x == 0) {
        t.m_scale[blk] = __uint_as_float(em << 23);
        t.v_scale[blk] = __uint_as_float(ev << 23);
    }
}

template <class DT>
void adamw_go(const AdamwTable &tab, bool eight, const AdamwHyper &h, hipStream_t s) {
    const dim3 grid(tab.first[tab.count]);
    if (eight)
        hipLaunchKernelGGL((k_adamw<DT, true>), grid, dim3(kBlock), 0, s, tab, h);
    else
        hipLaunchKernelGGL((k_adamw<DT, false>), grid, dim3(kBlock), 0, s, tab, h);
}

}  // namespace

hipError_t launch_adamw(int dtype, int bits, const lstm_adamw_tensor *t, int count, const AdamwHyper &h,
                        hipStream_t s) {
    // A tensor of more blocks than a grid holds goes in parts.
    constexpr long long kGrid = 1 << 23;
    AdamwTable tab{};
    auto flush = [&]() {
        if (!tab.count) return hipSuccess;
        if (dtype == LSTM_BF16)
            adamw_go<BF16>(tab, bits == 8, h, s);
        else
            adamw_go<F32>(tab, bits == 8, h, s);
        tab.count = 0;
        tab.first[0] = 0;
        return hipGetLastError();
    };
    for (int i = 0; i < count; ++i) {
        const long long blocks = (t[i].n + kBlock - 1) / kBlock;
        if (blocks == 0) continue;
        if (blocks > kGrid) return hipErrorInvalidValue;
        if (tab.count == kMaxEntries || tab.first[tab.count] + blocks > kGrid) {
            const hipError_t e = flush();
            if (e != hipSuccess) return e;
        }
        tab.t[tab.count] = t[i];
        tab.first[tab.count + 1] = tab.first[tab.count] + (unsigned)blocks;
        ++tab.count;
    }
    return flush();
}

}  // namespace lstm_amd
