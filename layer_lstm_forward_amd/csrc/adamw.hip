// adamw.hip -- one AdamW step over a list of tensors.
#include "device.h"
#include "ops.h"
#include "ops_dev.h"

namespace lstm_amd {

namespace {

constexpr int kBlock = LSTM_ADAMW_BLOCK;

// Up to kMaxEntries tensors travel in the kernel's arguments, so that a call
// needs no device table and no copy, and reads every pointer afresh.
struct AdamwEntry {
    void *param;
    const void *grad;
    void *m, *v;
    float *m_scale, *v_scale, *master;
    long long n;
    float lr, weight_decay;
    unsigned index0;  // index of element 0 in its tensor (a part of one that is cut)
    int aligned;      // every array allows the widest accesses
};
constexpr int kMaxEntries = 46;
struct AdamwTable {
    AdamwEntry t[kMaxEntries];
    unsigned first[kMaxEntries + 1];  // first workgroup of each entry, and their end
    int count;
};
static_assert(sizeof(AdamwTable) + sizeof(AdamwHyper) <= 4096, "kernel arguments");

// 32 bits for an element, from its index (low 32 bits) and the seed: two
// rounds of xor-shift and multiply, as in published integer hashes.  Any odd
// multipliers of mixed bits serve: 0x9E3779B1 is Knuth's for multiplicative
// hashing, 0xB5297A4D is known from noise generators (Eiserloh 2017).  Over 200000
// draws each bit of index or seed flips each result bit in 49.4 to 50.6%, and
// neighbouring indices, seeds and halves correlate by less than 0.002.
__device__ inline unsigned dither(unsigned i, unsigned seed) {
    unsigned x = i + seed * 0x9E3779B1u;
    x ^= x >> 16;
    x *= 0x6C9F52D5u;
    x ^= x >> 15;
    x *= 0xB5297A4Du;
    return x ^ (x >> 16);
}

// The code of |x| = y * scale, y finite and below 256: rounded up where the
// dropped fraction plus 16 random bits carries.  Below 2^-6 the codes are
// multiples of 2^-9 (y * 512 is exact, so the fused sum rounds once); above,
// they are the float's own bits without the low 20.
__device__ inline unsigned code_of(float y, unsigned bits16) {
    const unsigned r = (bits16 << 4) | 8u;
    const unsigned normal = ((__float_as_uint(y) + r) >> 20) - (120u << 3);
    const unsigned small = (unsigned)fmaf(y, 512.0f, (float)r * 0x1p-20f);
    return y >= 0.015625f ? normal : small;
}

// The values of N codes.  The hardware's conversion reads this very format.
template <int N>
__device__ inline void values_of(const unsigned char *c, float *f) {
#pragma unroll
    for (int x = 0; x < N; x += 4) {
        unsigned q;
        __builtin_memcpy(&q, c + x, 4);
        f[x] = __builtin_amdgcn_cvt_f32_fp8((int)q, 0);
        f[x + 1] = __builtin_amdgcn_cvt_f32_fp8((int)q, 1);
        f[x + 2] = __builtin_amdgcn_cvt_f32_fp8((int)q, 2);
        f[x + 3] = __builtin_amdgcn_cvt_f32_fp8((int)q, 3);
    }
}

// sqrt(v) for v >= 2^-96 or 0: the hardware's reciprocal root and one Newton
// step on the remainder v - s^2, half the instructions of the full sqrtf,
// which also serves the smallest floats.  0, infinity and NaN are their own
// roots (the Newton step would make infinity, which a g^2 past the fp32 range
// leaves in v, a NaN).
__device__ inline float root_of(float v) {
    const float y = __builtin_amdgcn_rsqf(v), s = v * y;
    constexpr int kPositive = 1 << 7 | 1 << 8;  // and finite: denormal, normal
    return __builtin_amdgcn_classf(v, kPositive) ? fmaf(fmaf(-s, s, v), 0.5f * y, s) : v;
}

// The states' update, each operation rounded by itself: a state that is stored
// in 8 bits is then the same whatever the compiler fuses around it.
__device__ inline void adamw_element(float g, const AdamwHyper &h, float &m, float &v) {
#pragma clang fp contract(off)
    m = m * h.beta1 + g * h.one_beta1;
    v = v * h.beta2 + (g * g) * h.one_beta2;
}

// What a lane loads and stores at once: VEC elements, so that 16 bytes of
// parameters move with each instruction.  VEC lanes' worth of a block of 256:
// its scale is a maximum over 256 / VEC lanes of one wave.
template <class DT>
struct AdamwVec {
    static constexpr int VEC = DT::PER16, LANES = kBlock / VEC;
};

template <class T, int N>
__device__ inline void load_n(const void *p, long long i, int left, bool whole, T *x) {
    const T *q = static_cast<const T *>(p) + i;
    if (whole)
        __builtin_memcpy(x, __builtin_assume_aligned(q, N * sizeof(T) < 16 ? N * sizeof(T) : 16), N * sizeof(T));
    else
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = e < left ? q[e] : (T)0;
}
template <class T, int N>
__device__ inline void store_n(void *p, long long i, int left, bool whole, const T *x) {
    T *q = static_cast<T *>(p) + i;
    if (whole)
        __builtin_memcpy(__builtin_assume_aligned(q, N * sizeof(T) < 16 ? N * sizeof(T) : 16), x, N * sizeof(T));
    else
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) q[e] = x[e];
}

// K pieces of 256 * VEC elements from element c0.  WHOLE: all of them lie in
// the tensor and its arrays are aligned, which every load of the piece then
// knows (a condition on each load would make each wait for the one before).
template <class DT, bool EIGHT, int K, bool WHOLE>
__device__ inline void adamw_part(const AdamwEntry &t, const AdamwHyper &h, long long c0, float keep, float scale) {
    using S = typename DT::S;
    constexpr int VEC = AdamwVec<DT>::VEC, LANES = AdamwVec<DT>::LANES;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const long long i = c0 + (k * 256 + threadIdx.x) * VEC;
        const long long rest = t.n - i;
        const int left = WHOLE ? VEC : rest < VEC ? (rest < 0 ? 0 : (int)rest) : VEC;
        constexpr bool whole = WHOLE;
        const long long blk = i / kBlock;
        S pv[VEC], gv[VEC];
        float m[VEC], v[VEC], root[VEC], w[VEC], least = 1.0f;
        unsigned char cm[VEC], cv[VEC];
        load_n<S, VEC>(t.grad, i, left, whole, gv);
        if (t.master)
            load_n<float, VEC>(t.master, i, left, whole, w);
        else
            load_n<S, VEC>(t.param, i, left, whole, pv);
        if constexpr (EIGHT) {
            load_n<unsigned char, VEC>(t.m, i, left, whole, cm);
            load_n<unsigned char, VEC>(t.v, i, left, whole, cv);
            const float sm = left ? t.m_scale[blk] : 0.0f, sv = left ? t.v_scale[blk] : 0.0f;
            values_of<VEC>(cm, m);
            values_of<VEC>(cv, root);
#pragma unroll
            for (int x = 0; x < VEC; ++x) {
                m[x] *= sm;
                root[x] = fminf(root[x] * sv, INFINITY);  // (NaN becomes infinity)
                v[x] = root[x] * root[x];
            }
        } else {
            load_n<float, VEC>(t.m, i, left, whole, m);
            load_n<float, VEC>(t.v, i, left, whole, v);
        }
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            if (!t.master) w[x] = DT::to_f(pv[x]);
            adamw_element(DT::to_f(gv[x]) * scale, h, m[x], v[x]);
            least = fminf(least, v[x] > 0.0f ? v[x] : 1.0f);
            root[x] = root_of(v[x]);
        }
        if (__any(least < 0x1p-96f))
#pragma unroll
            for (int x = 0; x < VEC; ++x) root[x] = sqrtf(v[x]);
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
            const float step = m[x] * __builtin_amdgcn_rcpf(fmaf(root[x], h.inv_sqrt_bc2, h.eps)) * h.inv_bc1;
            w[x] = w[x] * keep - t.lr * step;
            pv[x] = round_to<DT>(w[x]);
        }
        if (t.master) store_n<float, VEC>(t.master, i, left, whole, w);
        store_n<S, VEC>(t.param, i, left, whole, pv);
        if constexpr (EIGHT) {
            // the block's largest magnitudes
            unsigned am = 0, av = 0;
#pragma unroll
            for (int x = 0; x < VEC; ++x) {
                if (x < left) {
                    am = max(am, __float_as_uint(m[x]) & 0x7FFFFFFFu);
                    av = max(av, __float_as_uint(root[x]) & 0x7FFFFFFFu);
                }
            }
            const bool odd = __any(max(am, av) >= 0x7F800000u);
            if (odd) {  // what is not finite does not count
                am = av = 0;
#pragma unroll
                for (int x = 0; x < VEC; ++x) {
                    const unsigned bm = __float_as_uint(m[x]) & 0x7FFFFFFFu;
                    const unsigned bv = __float_as_uint(root[x]) & 0x7FFFFFFFu;
                    if (x < left && bm < 0x7F800000u) am = max(am, bm);
                    if (x < left && bv < 0x7F800000u) av = max(av, bv);
                }
            }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) {
                am = max(am, (unsigned)__shfl_xor((int)am, o));
                av = max(av, (unsigned)__shfl_xor((int)av, o));
            }
            const unsigned em = max((int)(am >> 23) - 7, 1), ev = max((int)(av >> 23) - 7, 1);
            const float im = __uint_as_float((254u - em) << 23), iv = __uint_as_float((254u - ev) << 23);
#pragma unroll
            for (int x = 0; x < VEC; ++x) {
                const unsigned bits = dither((unsigned)(i + x) + t.index0, h.seed);
                const unsigned a = code_of(fabsf(m[x]) * im, bits & 0xFFFFu);
                const unsigned b = max(code_of(root[x] * iv, bits >> 16), root[x] > 0.0f ? 1u : 0u);
                cm[x] = (unsigned char)(a | ((__float_as_uint(m[x]) >> 24) & 0x80u));
                cv[x] = (unsigned char)b;
            }
            if (odd)  // infinity or NaN: the format's NaN (which it reads as infinity for sqrt(v))
#pragma unroll
                for (int x = 0; x < VEC; ++x) {
                    if ((__float_as_uint(m[x]) & 0x7FFFFFFFu) >= 0x7F800000u) cm[x] = 0x7F;
                    if ((__float_as_uint(root[x]) & 0x7FFFFFFFu) >= 0x7F800000u) cv[x] = 0x7F;
                }
            store_n<unsigned char, VEC>(t.m, i, left, whole, cm);
            store_n<unsigned char, VEC>(t.v, i, left, whole, cv);
            if (left && threadIdx.x % LANES == 0) {
                t.m_scale[blk] = __uint_as_float(em << 23);
                t.v_scale[blk] = __uint_as_float(ev << 23);
            }
        } else {
            store_n<float, VEC>(t.m, i, left, whole, m);
            store_n<float, VEC>(t.v, i, left, whole, v);
        }
    }
}

// A workgroup takes K * 256 * VEC elements of one tensor.  Every byte is read and
// written once: 28 bytes an element for fp32 with 32-bit states (3.7 M elements:
// 18.6 us, 5.5 TB/s), 10 for bf16 with 8-bit states (134 M: 281 us, 4.8 TB/s;
// with IEEE roots and quotients and conditions on each load it took 425).
template <class DT, bool EIGHT, int K>
__global__ __launch_bounds__(256) void k_adamw(AdamwTable tab, AdamwHyper h) {
    constexpr int VEC = AdamwVec<DT>::VEC;
    // the entry, by all lanes at once: a loop would wait for memory each time
    const int lane = threadIdx.x % 64;
    const bool past = lane < tab.count && blockIdx.x >= tab.first[lane + 1];
    const int e = __popcll(__ballot(past));
    const AdamwEntry &t = tab.t[e];
    const long long c0 = (long long)(blockIdx.x - tab.first[e]) * (K * 256 * VEC);
    const float keep = 1.0f - t.lr * t.weight_decay, scale = h.grad_scale ? *h.grad_scale : 1.0f;
    if (t.aligned && c0 + K * 256 * VEC <= t.n)
        adamw_part<DT, EIGHT, K, true>(t, h, c0, keep, scale);
    else
        adamw_part<DT, EIGHT, K, false>(t, h, c0, keep, scale);
}

template <class DT, int K>
void adamw_go(const AdamwTable &tab, bool eight, const AdamwHyper &h, hipStream_t s) {
    const dim3 grid(tab.first[tab.count]);
    if (eight)
        hipLaunchKernelGGL((k_adamw<DT, true, K>), grid, dim3(256), 0, s, tab, h);
    else
        hipLaunchKernelGGL((k_adamw<DT, false, K>), grid, dim3(256), 0, s, tab, h);
}

}  // namespace

hipError_t launch_adamw(int dtype, int bits, const lstm_adamw_tensor *t, int count, const AdamwHyper &h,
                        hipStream_t s) {
    // a larger tensor goes in parts (of whole chunks, so of whole blocks too)
    constexpr long long kPart = (long long)1 << 31, kGrid = (long long)1 << 22, kFew = (long long)1 << 23;
    constexpr int kLong = 4;
    const bool eight = bits == 8, bf = dtype == LSTM_BF16;
    const size_t ps = bf ? 2 : 4, ss = eight ? 1 : 4, wide = bf ? 8 : 4;  // elements of a lane's access
    // few elements: one access a thread, so that every CU gets its share
    long long all = 0;
    for (int i = 0; i < count; ++i) all += t[i].n;
    const bool few = all < kFew;
    const int chunk = (bf ? 2048 : 1024) * (few ? 1 : kLong);  // elements of a workgroup
    AdamwTable tab{};
    auto flush = [&]() {
        if (!tab.count) return hipSuccess;
        if (bf)
            few ? adamw_go<BF16, 1>(tab, eight, h, s) : adamw_go<BF16, kLong>(tab, eight, h, s);
        else
            few ? adamw_go<F32, 1>(tab, eight, h, s) : adamw_go<F32, kLong>(tab, eight, h, s);
        tab.count = 0;
        tab.first[0] = 0;
        return hipGetLastError();
    };
    for (int i = 0; i < count; ++i) {
        for (long long at = 0; at < t[i].n; at += kPart) {
            const long long n = t[i].n - at < kPart ? t[i].n - at : kPart, chunks = (n + chunk - 1) / chunk;
            if (tab.count == kMaxEntries || tab.first[tab.count] + chunks > kGrid) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
            }
            AdamwEntry &o = tab.t[tab.count];
            o.param = static_cast<char *>(t[i].param) + at * ps;
            o.grad = static_cast<const char *>(t[i].grad) + at * ps;
            o.m = static_cast<char *>(t[i].m) + at * ss;
            o.v = static_cast<char *>(t[i].v) + at * ss;
            o.m_scale = eight ? t[i].m_scale + at / kBlock : nullptr;
            o.v_scale = eight ? t[i].v_scale + at / kBlock : nullptr;
            o.master = t[i].master ? t[i].master + at : nullptr;
            o.n = n;
            o.lr = t[i].lr;
            o.weight_decay = t[i].weight_decay;
            o.index0 = (unsigned)at;
            const uintptr_t state = wide * ss < 16 ? wide * ss : 16;
            o.aligned = ((uintptr_t)o.param | (uintptr_t)o.grad) % 16 == 0 &&
                        ((uintptr_t)o.m | (uintptr_t)o.v) % state == 0 && (uintptr_t)o.master % 16 == 0;
            tab.first[tab.count + 1] = tab.first[tab.count] + (unsigned)chunks;
            ++tab.count;
        }
    }
    return flush();
}

}  // namespace lstm_amd
