// blocks.h -- launchers of the operators of include/lstm_blocks.h (host side).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>

#include "../../include/lstm_blocks.h"

namespace lstm_amd {

// ----------------------------------------------------------- gated recurrence
// A [T, B, width] tensor: element strides of time and batch, channels dense.
struct GrView {
    char *p;
    long long t, b;
};
struct GrCall {
    GrView x, f, i, y;     // i.p null: the input gate is 1 - the forget gate's
    GrView dy, dx, df, di; // backward only
    const int *lengths;    // or null
    const float *s0;       // state before the first token, or null
    float *s1;             // state after the last, or null
    const float *ds1;      // gradient of s1, or null
    float *ds0;            // gradient of s0, or null
    unsigned *ticket;            // GR_CHAIN: workspace, gr_words bytes: a counter, 8 bytes on the word that says a
    unsigned long long *words;   // wait was given up, 256 bytes on the words
    long long patience;          // GR_CHAIN: clock ticks that a tile waits at most; below 0 none waits
    int T, B, width, dtype;
    int way, tiles;        // GrWay; tiles of a chain (set by its launch)
};
enum GrWay { GR_TILES = 0, GR_LANES = 1, GR_CHAIN = 2 };
GrWay gr_plan(int T, int B, int width, int dtype, bool backward);
size_t gr_words(int T, int B, int width);
hipError_t launch_gr_forward(const GrCall &c, hipStream_t s);
hipError_t launch_gr_backward(const GrCall &c, hipStream_t s);

struct GrStep {
    GrView x, f, i, y;
    const int *slots;
    float *pool;
    int n_slots, B, width, dtype;
};
hipError_t launch_gr_step(const GrStep &c, hipStream_t s);

// --------------------------------------------------------------------- rotary
// A [T, B, heads, dim] tensor: element strides, the last axis dense.
struct RotView {
    char *p;
    long long t, b, h;
};
struct RotSide {  // queries or keys
    RotView x, y;   // forward: input and output; backward: input and gradient of the output
    RotView dx;     // backward
    const char *w;  // norm weight or null
    char *dw;       // backward: its gradient or null
    int heads;
};
struct RotCall {
    RotSide side[2];
    const double *freq;      // [rot / 2] radians a position
    const int *pos;          // or null: the token's index
    long long pos_t, pos_b;
    float *part;             // backward: [runs][parts][dim] sums of the weight gradients, or null
    int T, B, dim, rot, pairs, norm, dtype, run, parts;
    float eps, scale;
};
// Heads that a workgroup takes of a token, how many runs of these a token has, and workgroups that keep sums of a run's
// weight gradients.
void rot_plan(long long tokens, int heads, int kv_heads, int dim, int *run, int *runs, int *parts);
hipError_t launch_rot_forward(const RotCall &c, hipStream_t s);
hipError_t launch_rot_backward(const RotCall &c, hipStream_t s);

// ------------------------------------------------------------------ gated MLP
// Operands of the products are bf16: a bf16 matrix itself, or three bf16
// matrices (planes) whose sum is an fp32 matrix to 2^-24.
struct MlpOperand {
    const char *p;     // first plane
    size_t plane;      // bytes from plane to plane
    long long ld;      // elements from row to row
};
// g or u as the forward keeps it: [rows][ld] fp32, or the upper 16 bits of each
// value and `low` bytes further on eight more.
struct MlpKept {
    char *p;
    size_t low;
};
// One product C[m][n] = sum over k of A[m][k] B[n][k], k running over `lists`
// pairs of operands one after the other.  An operand is stored with k along
// its rows (a[m][k]) or along its columns (a[k][m]), which the launch says.
struct MlpProduct {
    MlpOperand a[2], b[2];
    int M, N, K, lists;
    char *out;         // STORE: [M][ldo] of the call's dtype
    long long ldo;
    int vec;           // STORE: rows of out are 16-byte aligned
    int tiles_m, tiles_n;
};
enum MlpEpilogue { MLP_STORE = 0, MLP_GATE = 1, MLP_DGATE = 2 };
struct MlpCall {
    MlpProduct p[3];
    int count, dtype, act;
    int epilogue, a_cols, b_cols;  // a_cols: A is stored as a[k][m]
    // MLP_GATE: b[0] and b[1] are the weights of gate and up, products of one
    // pass.  product receives act(g) u in planes, gate and up g and u (null: not kept).
    // MLP_DGATE: gate and up are read, dgate and dup receive the gradients in planes.
    MlpKept gate, up;
    MlpOperand product, dgate, dup;
    long long ld;      // elements from row to row of all of these
    float *part;       // partial sums where the contraction is split
    int whole, splits, units;  // set by launch_mlp, as in MlpPlan
};
// How a launch is cut up: its tile, the first `whole` tiles as they are, each of
// the other split_tiles in `splits` parts; workgroups take `units` of these.
struct MlpPlan {
    int tile, whole, splits, split_tiles, units;
    size_t floats;  // partial sums
};
MlpPlan mlp_plan(const MlpCall &c);
hipError_t launch_mlp(const MlpCall &c, hipStream_t s);
// The products of the forward call for few rows, MLP_FEW at most, from the matrices as
// they are: w[0] and w[1] gate and up, out receives h [rows][ld] of the call's
// dtype, zeros past N; or w[0] alone, out receives [rows][N].
constexpr int MLP_FEW = 64;
struct MlpFew {
    const char *x, *w[2];  // w [N][K]
    long long xs;          // elements from row to row of x
    int rows, N, K, dtype, act;
    char *out;
    long long ld;
    MlpKept gate, up;      // kept for the backward call where keep.p is set
    MlpOperand keep;       // h as an operand
};
hipError_t launch_mlp_few(const MlpFew &c, hipStream_t s);
// src [rows][cols] of dtype (ld elements from row to row) as bf16 planes (one, or three for fp32) of rows `to.ld`
// long, the columns past cols 0.
hipError_t launch_mlp_planes(int dtype, const void *src, long long ld, long long rows, int cols, const MlpOperand &to,
                             hipStream_t s);

}  // namespace lstm_amd
