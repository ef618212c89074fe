// ops.h -- launchers of the operators of include/lstm_ops.h (host side).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>

#include "../../include/lstm_ops.h"

namespace lstm_amd {

// ---------------------------------------------------------- linear attention
// One pass of the operator over every (batch row, head):
//     out_i = row_scale gamma^(i + e) a_i S0 + chunk_scale sum over j <= i of gamma^(i-j) (a_i . b_j) c_j
// in token order (e = 1), or, reversed, in the order of falling token index
// (i counts from the row's last token, e = 0: the carried state then is the
// gradient that arrives at a token from the one after it).  The carried
// matrix is S [da][dc], the decayed S0 and sum_scale times the b_j c_j^T, and
// chunk_scale = row_scale sum_scale.  Forward: (a, b, c) = (q, k, v).  The
// gradients are three more passes: dq from (do, v, k), dk reversed from (v,
// do, q), dv reversed from (k, q, do).  The call's scale stands with what
// reads the state in the forward and in dq (row_scale), and with what is added
// to its gradient in the other two (sum_scale): S is in the state's own units
// in every pass, for any scale.
struct LaTensor {
    const char *p;
    long long t, b, h;  // strides in elements
    int hdiv;           // query heads that share a head of this tensor
};
struct LaOut {
    char *p;
    long long t, b, h;
    int f32;  // fp32 elements (partial sums of a shared head), else the call's dtype
};
struct LaPass {
    LaTensor a, b, c;
    LaOut o;
    int da, dc;           // contraction and column dims of the carried matrix
    const float *s0;      // [B][H][Dk][Dv] or null; element (r, c) at r * srow + c * scol
    float *s1;            // the carried matrix after the last token, or null
    int srow, scol;
    float row_scale, sum_scale;
    int reverse;
    float *seg;           // matrices before the segments (workspace), or null (one segment)
};
struct LaCall {
    LaPass pass[3];
    int npass;
    const float *log_decay;
    const int *lengths;   // or null
    int T, B, H, dtype;
    int nseg, seg_tokens; // segments of the sequence, tokens in each
    int grid_seg;         // segments a launch covers (set by launch_la)
};

// Segments a sequence of each of `rows` (batch row, head) pairs is cut into,
// their tokens (a multiple of the chunk), and the floats of one matrix in the
// workspace.
void la_segments(int T, long long rows, int npass, int da, int dc, int dtype, int *nseg, int *seg_tokens,
                 size_t *seg_floats);
hipError_t launch_la(const LaCall &c, hipStream_t s);
// Partial sums [B][T][H][D] of the gradients of shared heads, and where their sums go.
struct LaShare {
    const float *part;
    LaOut out;
    int D;
};
hipError_t launch_la_share(const LaShare &a, const LaShare &b, int T, int B, int H, int G, int dtype, hipStream_t s);

struct LaStep {
    LaTensor q, k, v;
    LaOut o;
    const float *log_decay;
    const int *slots;
    float *pool;
    int n_slots, B, H, Dk, Dv, dtype;
    float scale;
};
hipError_t launch_la_step(const LaStep &c, hipStream_t s);

// ----------------------------------------------------------------- layer norm
struct LnForward {
    const char *x, *res, *w, *bias;
    char *y, *sum;
    float *mean, *rstd;
    long long xs, rs, rows;
    int width, dtype;
    float eps;
};
hipError_t launch_ln_forward(const LnForward &c, hipStream_t s);

struct LnBackward {
    const char *dy, *z, *w, *dsum;
    const float *mean, *rstd;
    char *dx, *dw, *db;
    float *part;  // [ln_parts][2][width]
    long long ys, zs, rows;
    int width, dtype;
};
// workgroups that keep partial sums of the weight and bias gradients
int ln_parts(long long rows, int width);
hipError_t launch_ln_backward(const LnBackward &c, hipStream_t s);

// ---------------------------------------------------------------------- AdamW
struct AdamwHyper {
    // step = m / (sqrt(v) inv_sqrt_bc2 + eps) inv_bc1; the last three may carry a common factor
    float beta1, beta2, one_beta1, one_beta2, eps, inv_bc1, inv_sqrt_bc2;
    const float *grad_scale;
    unsigned seed;
};
hipError_t launch_adamw(int dtype, int bits, const lstm_adamw_tensor *t, int count, const AdamwHyper &h,
                        hipStream_t s);

}  // namespace lstm_amd
