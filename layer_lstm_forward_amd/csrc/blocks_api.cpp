// blocks_api.cpp -- the C ABI declared in include/lstm_blocks.h: argument
// checks, workspace carve-up and the kernel launches.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/lstm_blocks.h"
#include "blocks.h"
#include "ops_host.h"

using namespace lstm_amd;

namespace {

bool aligned(const void *p) { return (uintptr_t)p % 16 == 0; }

bool dtype_ok(int d) { return d == LSTM_F32 || d == LSTM_BF16; }

// ----------------------------------------------------------- gated recurrence
constexpr int kMaxTokens = 1 << 30;
constexpr int kMaxChannels = 1 << 20;

lstm_status gr_check(const lstm_gated_recurrence_shape *s) {
    if (!s) return LSTM_ERR_ARG;
    if (!dtype_ok(s->dtype)) return LSTM_ERR_DTYPE;
    if (s->T < 1 || s->T > kMaxTokens || s->B < 1 || s->width < 1 || s->width > kMaxChannels) return LSTM_ERR_SHAPE;
    // a grid holds fewer than 2^32 threads
    if ((long long)s->B * s->width > INT_MAX) return LSTM_ERR_SHAPE;
    return LSTM_OK;
}

GrView gr_view(const lstm_view *v) {
    return v ? GrView{static_cast<char *>(v->data), v->time, v->batch} : GrView{nullptr, 0, 0};
}

lstm_status gr_size(const lstm_gated_recurrence_shape *s, bool backward, GrCall *c, size_t *bytes) {
    const lstm_status rc = gr_check(s);
    if (rc != LSTM_OK) return rc;
    if (!bytes) return LSTM_ERR_ARG;
    c->way = gr_plan(s->T, s->B, s->width, s->dtype, backward);
    *bytes = c->way == GR_CHAIN ? gr_words(s->T, s->B, s->width) : 0;
    return LSTM_OK;
}

void gr_workspace(GrCall *c, void *workspace, int dev) {
    c->ticket = static_cast<unsigned *>(workspace);
    c->words = reinterpret_cast<unsigned long long *>(static_cast<char *>(workspace) + 256);
    if (c->way != GR_CHAIN) return;
    int khz = 0;
    if (hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, dev) != hipSuccess) (void)hipGetLastError();
    c->patience = (khz > 0 ? khz : 100000) * 1000ll * 5;  // five seconds
}

// ------------------------------------------------------------------- rotary
constexpr int kMaxHeads = 1 << 16;
constexpr int kMaxDim = 256;

lstm_status rot_check(const lstm_rotary_shape *s) {
    if (!s) return LSTM_ERR_ARG;
    if (!dtype_ok(s->dtype)) return LSTM_ERR_DTYPE;
    if (s->heads < 1 || s->kv_heads < 0 || s->heads > kMaxHeads || s->kv_heads > kMaxHeads) return LSTM_ERR_ARG;
    if (s->dim < 1 || s->dim > kMaxDim || s->rotary_dim < 0 || s->rotary_dim > s->dim || s->rotary_dim % 2)
        return LSTM_ERR_ARG;
    if ((s->interleaved != 0 && s->interleaved != 1) || (s->norm != 0 && s->norm != 1)) return LSTM_ERR_ARG;
    if (!(s->eps >= 0.0f) || !std::isfinite(s->eps) || !std::isfinite(s->scale)) return LSTM_ERR_ARG;
    if (s->T < 1 || s->B < 1 || (long long)s->T * s->B > INT_MAX) return LSTM_ERR_SHAPE;
    return LSTM_OK;
}

RotView rot_view(const lstm_view *v) {
    return v ? RotView{static_cast<char *>(v->data), v->time, v->batch, v->head} : RotView{nullptr, 0, 0, 0};
}

lstm_status rot_size(const lstm_rotary_shape *s, size_t *bytes) {
    *bytes = 0;
    if (!s->norm) return LSTM_OK;
    int run, runs, parts;
    rot_plan((long long)s->T * s->B, s->heads, s->kv_heads, s->dim, &run, &runs, &parts);
    return add_bytes(bytes, (size_t)runs, (size_t)parts, (size_t)s->dim, sizeof(float)) ? LSTM_OK : LSTM_ERR_SHAPE;
}

RotCall rot_call(const lstm_rotary_shape *s, const void *wq, const void *wk, const double *freq,
                 const lstm_positions *pos) {
    RotCall c{};
    c.side[0].heads = s->heads;
    c.side[1].heads = s->kv_heads;
    c.side[0].w = static_cast<const char *>(wq);
    c.side[1].w = static_cast<const char *>(wk);
    c.freq = freq;
    if (pos && pos->data) c.pos = pos->data, c.pos_t = pos->time, c.pos_b = pos->batch;
    c.T = s->T;
    c.B = s->B;
    c.dim = s->dim;
    c.rot = s->rotary_dim;
    c.pairs = s->interleaved;
    c.norm = s->norm;
    c.dtype = s->dtype;
    c.eps = s->eps;
    c.scale = s->scale;
    int runs;
    rot_plan((long long)s->T * s->B, s->heads, s->kv_heads, s->dim, &c.run, &runs, &c.parts);
    return c;
}

// ---------------------------------------------------------------- gated MLP
constexpr int kMaxFeatures = 1 << 18;
constexpr int kMaxTokensMlp = 1 << 30;     // rows: the kernels count tiles of them in int
constexpr long long kMaxProduct = 1ll << 38;  // elements of a matrix: 2^22 tiles of 256 x 256

lstm_status mlp_check(const lstm_gated_mlp_shape *s) {
    if (!s) return LSTM_ERR_ARG;
    if (!dtype_ok(s->dtype)) return LSTM_ERR_DTYPE;
    if (s->activation < LSTM_ACT_SILU || s->activation > LSTM_ACT_SIGMOID) return LSTM_ERR_ARG;
    if (s->rows < 0 || s->rows > kMaxTokensMlp || s->in < 1 || s->hidden < 1 || s->out < 1) return LSTM_ERR_SHAPE;
    if (s->in > kMaxFeatures || s->hidden > kMaxFeatures || s->out > kMaxFeatures) return LSTM_ERR_SHAPE;
    const long long wide = s->in > s->hidden ? (s->in > s->out ? s->in : s->out) : (s->hidden > s->out ? s->hidden : s->out);
    if (s->rows * wide > kMaxProduct) return LSTM_ERR_SHAPE;
    return LSTM_OK;
}

long long padded(long long n) { return (n + 7) / 8 * 8; }
int planes(const lstm_gated_mlp_shape *s) { return s->dtype == LSTM_F32 ? 3 : 1; }

// Takes the next part of a memory block; without one (size queries) only counts.
struct Carver {
    char *base;
    size_t used = 0;
    bool ok = true;
    char *take(size_t a, size_t b, size_t c) {
        char *p = base ? base + used : nullptr;
        ok = add_bytes(&used, a, b, c, 1) && ok;
        return p;
    }
    // planes of a [rows][cols] matrix
    MlpOperand operand(const lstm_gated_mlp_shape *s, size_t rows, long long cols) {
        MlpOperand o;
        o.ld = padded(cols);
        size_t one = 0;
        ok = add_bytes(&one, rows, (size_t)o.ld, 2, 1) && ok;
        o.plane = one;
        o.p = take(one, (size_t)planes(s), 1);
        return o;
    }
};

struct Reserve {
    MlpKept gate, up;
    MlpOperand product;
    size_t bytes;
    bool ok;
};
Reserve reserve_of(const lstm_gated_mlp_shape *s, const void *at) {
    Carver k{static_cast<char *>(const_cast<void *>(at))};
    Reserve r;
    auto kept = [&]() {
        MlpKept o;
        const size_t ld = (size_t)padded(s->hidden);
        const size_t before = k.used;
        o.p = k.take((size_t)s->rows, ld, elem(s->dtype));
        o.low = k.used - before;
        if (s->dtype == LSTM_BF16) (void)k.take((size_t)s->rows, ld, 1);
        return o;
    };
    r.gate = kept();
    r.up = kept();
    r.product = k.operand(s, (size_t)s->rows, s->hidden);
    r.bytes = k.used;
    r.ok = k.ok;
    return r;
}

// A bf16 matrix that the products can read where it lies: whole 16-byte pieces in every row.
bool in_place(const lstm_gated_mlp_shape *s, const void *p, long long ld, long long cols) {
    return s->dtype == LSTM_BF16 && (uintptr_t)p % 16 == 0 && ld % 8 == 0 && cols % 8 == 0 && ld < (1 << 21);
}

// Operands of a call: where they lie, or planes in the workspace that launch() fills.
struct Operands {
    const lstm_gated_mlp_shape *s;
    Carver *k;
    struct Copy {
        const void *src;
        long long ld, rows;
        int cols;
        MlpOperand to;
    } copy[5];
    int n = 0;
    // `dense`: a weight, whose place is known to be aligned, so that the size
    // query knows whether it is copied; an activation's is not, and room for
    // its copy is always there.  Filled only where a launch of the call reads it.
    MlpOperand add(const void *p, long long ld, long long rows, int cols, bool dense, bool read) {
        const bool sizes = k->base == nullptr;
        if (dense ? s->dtype == LSTM_BF16 && cols % 8 == 0 : !sizes && in_place(s, p, ld, cols)) {
            if (!dense) (void)k->operand(s, (size_t)rows, cols);
            MlpOperand o;
            o.p = static_cast<const char *>(p);
            o.plane = 0;
            o.ld = ld;
            return o;
        }
        const MlpOperand o = k->operand(s, (size_t)rows, cols);
        if (!sizes && read) copy[n++] = Copy{p, ld, rows, cols, o};
        return o;
    }
    hipError_t launch(hipStream_t st) const {
        for (int i = 0; i < n; ++i) {
            if (copy[i].rows == 0) continue;
            const hipError_t e =
                launch_mlp_planes(s->dtype, copy[i].src, copy[i].ld, copy[i].rows, copy[i].cols, copy[i].to, st);
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    }
};

MlpProduct product(const MlpOperand &a, const MlpOperand &b, int M, int N, int K) {
    MlpProduct p{};
    p.a[0] = p.a[1] = a;
    p.b[0] = p.b[1] = b;
    p.M = M;
    p.N = N;
    p.K = K;
    p.lists = 1;
    return p;
}

// A product whose result is the caller's dense [M][N].
MlpProduct stored(const lstm_gated_mlp_shape *s, const MlpOperand &a, const MlpOperand &b, int M, int N, int K,
                  void *out) {
    MlpProduct p = product(a, b, M, N, K);
    p.out = static_cast<char *>(out);
    p.ldo = N;
    p.vec = (uintptr_t)out % 16 == 0 && N % (s->dtype == LSTM_F32 ? 4 : 8) == 0;
    return p;
}

MlpCall mlp_call(const lstm_gated_mlp_shape *s, int epilogue, int a_cols, int b_cols) {
    MlpCall c{};
    c.count = 1;
    c.dtype = s->dtype;
    c.act = s->activation;
    c.epilogue = epilogue;
    c.a_cols = a_cols;
    c.b_cols = b_cols;
    c.ld = padded(s->hidden);
    return c;
}

size_t most(size_t a, size_t b) { return a > b ? a : b; }

// Forward calls of few rows go to the kernel that reads the weights as they are; its time grows with the rows, that of
// the tiles hardly.  Whole calls, in x hidden, us in this kernel / in tiles:
//     rows                 16           32           48           64
//     bf16  1024 x 2816    18 / 24      18 / 24      21 / 25      24 / 25
//           1536 x 4224    23 / 27      30 / 28      36 / 28      41 / 29
//           2048 x 2816    18 / 26      22 / 26      27 / 27      30 / 28
//           2048 x 5632    28 / 32      37 / 32      47 / 33      53 / 33
//     fp32  1024 x 2816    24 / 60      35 / 61      47 / 61      52 / 62
//           2048 x 5632    52 / 141     80 / 144    120 / 146    130 / 148
// (of 17 and of 33 rows as of the next 16).
bool few_rows(const lstm_gated_mlp_shape *s) {
    if (s->dtype == LSTM_F32 || s->rows <= 16) return s->rows <= MLP_FEW;
    return s->rows <= MLP_FEW && (long long)s->rows * (s->hidden + s->out) <= 240 * 1024;
}

// The launches of a forward call and its workspace.
struct Forward {
    bool few;
    MlpFew few_gate, few_down;
    Operands ops;
    MlpCall gate, down;
    size_t bytes;
    bool ok;
};
Forward forward_of(const lstm_gated_mlp_shape *s, const void *x, long long xs, const void *wg, const void *wu,
                   const void *wd, void *y, void *reserve, void *workspace) {
    Carver k{static_cast<char *>(workspace)};
    Forward f{};
    f.few = few_rows(s);
    const Reserve r = reserve_of(s, reserve);
    if (f.few) {
        const long long ld = padded(s->hidden);
        char *h = k.take((size_t)s->rows, (size_t)ld, elem(s->dtype));
        f.few_gate = MlpFew{static_cast<const char *>(x), {static_cast<const char *>(wg), static_cast<const char *>(wu)},
                            xs, s->rows, s->hidden, s->in, s->dtype, s->activation, h, ld, {}, {}, {}};
        if (reserve) {
            f.few_gate.gate = r.gate;
            f.few_gate.up = r.up;
            f.few_gate.keep = r.product;
        }
        f.few_down = MlpFew{h, {static_cast<const char *>(wd), nullptr}, ld, s->rows, s->out, s->hidden, s->dtype,
                            s->activation, static_cast<char *>(y), s->out, {}, {}, {}};
        f.bytes = k.used;
        f.ok = k.ok;
        return f;
    }
    f.ops.s = s;
    f.ops.k = &k;
    const MlpOperand ox = f.ops.add(x, xs, s->rows, s->in, false, true);
    const MlpOperand og = f.ops.add(wg, s->in, s->hidden, s->in, true, true);
    const MlpOperand ou = f.ops.add(wu, s->in, s->hidden, s->in, true, true);
    const MlpOperand od = f.ops.add(wd, s->hidden, s->out, s->hidden, true, true);
    f.gate = mlp_call(s, MLP_GATE, 0, 0);
    f.gate.p[0] = product(ox, og, s->rows, s->hidden, s->in);
    f.gate.p[0].b[1] = ou;
    f.gate.product = k.operand(s, (size_t)s->rows, s->hidden);
    if (reserve) {
        f.gate.gate = r.gate;
        f.gate.up = r.up;
        f.gate.product = r.product;
    }
    f.down = mlp_call(s, MLP_STORE, 0, 0);
    f.down.p[0] = stored(s, f.gate.product, od, s->rows, s->out, s->hidden, y);
    const size_t floats = most(mlp_plan(f.gate).floats, mlp_plan(f.down).floats);
    f.gate.part = f.down.part = reinterpret_cast<float *>(k.take(floats, sizeof(float), 1));
    f.bytes = k.used;
    f.ok = k.ok;
    f.ops.k = nullptr;
    return f;
}

struct Backward {
    Operands ops;
    MlpCall hidden, dx, dw;
    bool want_hidden, want_dx;  // whether these are launched
    size_t bytes;
    bool ok;
};
Backward backward_of(const lstm_gated_mlp_shape *s, const void *x, long long xs, const void *wg, const void *wu,
                     const void *wd, const void *reserve, const void *dy, long long ys, void *dx, void *dwg, void *dwu,
                     void *dwd, void *workspace) {
    Carver k{static_cast<char *>(workspace)};
    Backward f{};
    f.ops.s = s;
    f.ops.k = &k;
    f.want_hidden = s->rows && (dx || dwg || dwu);
    f.want_dx = s->rows && dx;
    const MlpOperand ox = f.ops.add(x, xs, s->rows, s->in, false, dwg || dwu);
    const MlpOperand oy = f.ops.add(dy, ys, s->rows, s->out, false, true);
    const MlpOperand og = f.ops.add(wg, s->in, s->hidden, s->in, true, f.want_dx);
    const MlpOperand ou = f.ops.add(wu, s->in, s->hidden, s->in, true, f.want_dx);
    const MlpOperand od = f.ops.add(wd, s->hidden, s->out, s->hidden, true, f.want_hidden);
    const Reserve r = reserve_of(s, reserve);
    f.hidden = mlp_call(s, MLP_DGATE, 0, 1);
    f.hidden.p[0] = product(oy, od, s->rows, s->hidden, s->out);
    f.hidden.gate = r.gate;
    f.hidden.up = r.up;
    f.hidden.dgate = k.operand(s, (size_t)s->rows, s->hidden);
    f.hidden.dup = k.operand(s, (size_t)s->rows, s->hidden);
    f.dx = mlp_call(s, MLP_STORE, 0, 1);
    f.dx.p[0] = stored(s, f.hidden.dgate, og, s->rows, s->in, s->hidden, dx);
    f.dx.p[0].a[1] = f.hidden.dup;
    f.dx.p[0].b[1] = ou;
    f.dx.p[0].lists = 2;
    f.dw = mlp_call(s, MLP_STORE, 1, 1);
    f.dw.count = 0;
    const bool sizes = !dx && !dwg && !dwu && !dwd;  // a call wants something (its workspace may be of no bytes)
    if (dwg || sizes) f.dw.p[f.dw.count++] = stored(s, f.hidden.dgate, ox, s->hidden, s->in, s->rows, dwg);
    if (dwu || sizes) f.dw.p[f.dw.count++] = stored(s, f.hidden.dup, ox, s->hidden, s->in, s->rows, dwu);
    if (dwd || sizes) f.dw.p[f.dw.count++] = stored(s, oy, r.product, s->out, s->hidden, s->rows, dwd);
    size_t floats = most(mlp_plan(f.hidden).floats, mlp_plan(f.dx).floats);
    // whichever of the weights' gradients a call asks for
    MlpCall some = f.dw;
    for (int wanted = 1; wanted < 8 && sizes; ++wanted) {
        some.count = 0;
        for (int i = 0; i < 3; ++i)
            if (wanted >> i & 1) some.p[some.count++] = f.dw.p[i];
        floats = most(floats, mlp_plan(some).floats);
    }
    if (f.dw.count) floats = most(floats, mlp_plan(f.dw).floats);
    f.hidden.part = f.dx.part = f.dw.part = reinterpret_cast<float *>(k.take(floats, sizeof(float), 1));
    f.bytes = k.used;
    f.ok = k.ok;
    f.ops.k = nullptr;
    return f;
}

}  // namespace

extern "C" {

lstm_status lstm_gated_recurrence_workspace_size(const lstm_gated_recurrence_shape *s, size_t *bytes) {
    GrCall c{};
    return gr_size(s, false, &c, bytes);
}

lstm_status lstm_gated_recurrence_backward_workspace_size(const lstm_gated_recurrence_shape *s, size_t *bytes) {
    GrCall c{};
    return gr_size(s, true, &c, bytes);
}

lstm_status lstm_gated_recurrence_forward(const lstm_gated_recurrence_shape *s, const lstm_view *x,
                                          const lstm_view *forget, const lstm_view *input, const int *lengths,
                                          const float *state, const lstm_view *y, float *state_out, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    GrCall c{};
    size_t need = 0;
    lstm_status rc = gr_size(s, false, &c, &need);
    if (rc != LSTM_OK) return rc;
    if (!view_ok(x) || !view_ok(forget) || (input && !input->data) || !view_ok(y)) return LSTM_ERR_ARG;
    if (need && (!workspace || workspace_bytes < need)) return LSTM_ERR_WORKSPACE;
    if (need && !aligned(workspace)) return LSTM_ERR_ARG;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {x->data, forget->data, input ? input->data : nullptr, y->data, lengths, state, state_out,
                          need ? workspace : nullptr};
    if (!all_on_device(ptrs, 8, dev)) return LSTM_ERR_DEVICE;
    c.x = gr_view(x);
    c.f = gr_view(forget);
    c.i = gr_view(input);
    c.y = gr_view(y);
    c.lengths = lengths;
    c.s0 = state;
    c.s1 = state_out;
    gr_workspace(&c, workspace, dev);
    c.T = s->T;
    c.B = s->B;
    c.width = s->width;
    c.dtype = s->dtype;
    return launched(launch_gr_forward(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_gated_recurrence_backward(const lstm_gated_recurrence_shape *s, const lstm_view *x,
                                           const lstm_view *forget, const lstm_view *input, const int *lengths,
                                           const float *state, const lstm_view *y, const lstm_view *dy,
                                           const float *dstate_out, const lstm_view *dx, const lstm_view *dforget,
                                           const lstm_view *dinput, float *dstate, void *workspace,
                                           size_t workspace_bytes, void *stream) {
    GrCall c{};
    size_t need = 0;
    lstm_status rc = gr_size(s, true, &c, &need);
    if (rc != LSTM_OK) return rc;
    if (!view_ok(x) || !view_ok(forget) || (input && !input->data) || !view_ok(y) || !view_ok(dy) || !view_ok(dx) ||
        !view_ok(dforget) || (dinput && !dinput->data) || (input != nullptr) != (dinput != nullptr))
        return LSTM_ERR_ARG;
    if (need && (!workspace || workspace_bytes < need)) return LSTM_ERR_WORKSPACE;
    if (need && !aligned(workspace)) return LSTM_ERR_ARG;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {x->data, forget->data, input ? input->data : nullptr, y->data, dy->data, dx->data,
                          dforget->data, dinput ? dinput->data : nullptr, lengths, state, dstate_out, dstate,
                          need ? workspace : nullptr};
    if (!all_on_device(ptrs, 13, dev)) return LSTM_ERR_DEVICE;
    c.x = gr_view(x);
    c.f = gr_view(forget);
    c.i = gr_view(input);
    c.y = gr_view(y);
    c.dy = gr_view(dy);
    c.dx = gr_view(dx);
    c.df = gr_view(dforget);
    c.di = gr_view(dinput);
    c.lengths = lengths;
    c.s0 = state;
    c.ds1 = dstate_out;
    c.ds0 = dstate;
    gr_workspace(&c, workspace, dev);
    c.T = s->T;
    c.B = s->B;
    c.width = s->width;
    c.dtype = s->dtype;
    return launched(launch_gr_backward(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_gated_recurrence_step(const lstm_gated_recurrence_shape *s, const lstm_view *x,
                                       const lstm_view *forget, const lstm_view *input, const int *slots, int n_slots,
                                       float *pool, const lstm_view *y, void *stream) {
    lstm_status rc = gr_check(s);
    if (rc != LSTM_OK) return rc;
    if (!view_ok(x) || !view_ok(forget) || (input && !input->data) || !view_ok(y) || !pool) return LSTM_ERR_ARG;
    if (s->T != 1 || n_slots < 1 || (!slots && n_slots < s->B)) return LSTM_ERR_SHAPE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {x->data, forget->data, input ? input->data : nullptr, y->data, slots, pool};
    if (!all_on_device(ptrs, 6, dev)) return LSTM_ERR_DEVICE;
    const GrStep c{gr_view(x), gr_view(forget), gr_view(input), gr_view(y), slots, pool, n_slots, s->B, s->width,
                   s->dtype};
    return launched(launch_gr_step(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_rotary_forward(const lstm_rotary_shape *s, const lstm_view *q, const lstm_view *k,
                                const void *q_weight, const void *k_weight, const double *frequencies,
                                const lstm_positions *positions, const lstm_view *q_out, const lstm_view *k_out,
                                void *stream) {
    lstm_status rc = rot_check(s);
    if (rc != LSTM_OK) return rc;
    const bool keys = s->kv_heads > 0;
    if (!view_ok(q) || !view_ok(q_out) || (keys && (!view_ok(k) || !view_ok(k_out)))) return LSTM_ERR_ARG;
    if ((!s->norm && (q_weight || (keys && k_weight))) || (s->rotary_dim && !frequencies)) return LSTM_ERR_ARG;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {q->data, q_out->data, keys ? k->data : nullptr, keys ? k_out->data : nullptr, q_weight,
                          keys ? k_weight : nullptr, s->rotary_dim ? frequencies : nullptr,
                          positions ? positions->data : nullptr};
    if (!all_on_device(ptrs, 8, dev)) return LSTM_ERR_DEVICE;
    RotCall c = rot_call(s, q_weight, k_weight, frequencies, positions);
    c.side[0].x = rot_view(q);
    c.side[0].y = rot_view(q_out);
    if (keys) {
        c.side[1].x = rot_view(k);
        c.side[1].y = rot_view(k_out);
    }
    return launched(launch_rot_forward(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_rotary_backward_workspace_size(const lstm_rotary_shape *s, size_t *bytes) {
    const lstm_status rc = rot_check(s);
    if (rc != LSTM_OK) return rc;
    if (!bytes) return LSTM_ERR_ARG;
    return rot_size(s, bytes);
}

lstm_status lstm_rotary_backward(const lstm_rotary_shape *s, const lstm_view *q, const lstm_view *k,
                                 const void *q_weight, const void *k_weight, const double *frequencies,
                                 const lstm_positions *positions, const lstm_view *dq_out, const lstm_view *dk_out,
                                 const lstm_view *dq, const lstm_view *dk, void *dq_weight, void *dk_weight,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    lstm_status rc = rot_check(s);
    if (rc != LSTM_OK) return rc;
    const bool keys = s->kv_heads > 0;
    if (!view_ok(dq_out) || !view_ok(dq) || (keys && (!view_ok(dk_out) || !view_ok(dk)))) return LSTM_ERR_ARG;
    if (s->norm && (!view_ok(q) || (keys && !view_ok(k)))) return LSTM_ERR_ARG;
    if (!s->norm && (q_weight || dq_weight || (keys && (k_weight || dk_weight)))) return LSTM_ERR_ARG;
    if (s->rotary_dim && !frequencies) return LSTM_ERR_ARG;
    const bool sums = dq_weight || (keys && dk_weight);
    size_t need = 0;
    if ((rc = rot_size(s, &need)) != LSTM_OK) return rc;
    if (sums && (!workspace || workspace_bytes < need)) return LSTM_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {s->norm ? q->data : nullptr, s->norm && keys ? k->data : nullptr, dq_out->data,
                          keys ? dk_out->data : nullptr, dq->data, keys ? dk->data : nullptr, q_weight,
                          keys ? k_weight : nullptr, s->rotary_dim ? frequencies : nullptr,
                          positions ? positions->data : nullptr, dq_weight, keys ? dk_weight : nullptr,
                          sums ? workspace : nullptr};
    if (!all_on_device(ptrs, 13, dev)) return LSTM_ERR_DEVICE;
    RotCall c = rot_call(s, q_weight, k_weight, frequencies, positions);
    if (s->norm) c.side[0].x = rot_view(q);
    c.side[0].y = rot_view(dq_out);
    c.side[0].dx = rot_view(dq);
    c.side[0].dw = static_cast<char *>(dq_weight);
    if (keys) {
        if (s->norm) c.side[1].x = rot_view(k);
        c.side[1].y = rot_view(dk_out);
        c.side[1].dx = rot_view(dk);
        c.side[1].dw = static_cast<char *>(dk_weight);
    }
    c.part = sums ? static_cast<float *>(workspace) : nullptr;
    return launched(launch_rot_backward(c, static_cast<hipStream_t>(stream)));
}

lstm_status lstm_gated_mlp_workspace_size(const lstm_gated_mlp_shape *s, size_t *bytes) {
    const lstm_status rc = mlp_check(s);
    if (rc != LSTM_OK) return rc;
    if (!bytes) return LSTM_ERR_ARG;
    const Forward f = forward_of(s, nullptr, s->in, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
    if (!f.ok) return LSTM_ERR_SHAPE;
    *bytes = f.bytes;
    return LSTM_OK;
}

lstm_status lstm_gated_mlp_reserve_size(const lstm_gated_mlp_shape *s, size_t *bytes) {
    const lstm_status rc = mlp_check(s);
    if (rc != LSTM_OK) return rc;
    if (!bytes) return LSTM_ERR_ARG;
    const Reserve r = reserve_of(s, nullptr);
    if (!r.ok) return LSTM_ERR_SHAPE;
    *bytes = r.bytes;
    return LSTM_OK;
}

lstm_status lstm_gated_mlp_backward_workspace_size(const lstm_gated_mlp_shape *s, size_t *bytes) {
    const lstm_status rc = mlp_check(s);
    if (rc != LSTM_OK) return rc;
    if (!bytes) return LSTM_ERR_ARG;
    const Backward f = backward_of(s, nullptr, s->in, nullptr, nullptr, nullptr, nullptr, nullptr, s->out, nullptr,
                                   nullptr, nullptr, nullptr, nullptr);
    if (!f.ok) return LSTM_ERR_SHAPE;
    *bytes = f.bytes;
    return LSTM_OK;
}

lstm_status lstm_gated_mlp_forward(const lstm_gated_mlp_shape *s, const void *x, long long x_stride,
                                   const void *w_gate, const void *w_up, const void *w_down, void *y, void *reserve,
                                   size_t reserve_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0, keep = 0;
    lstm_status rc = lstm_gated_mlp_workspace_size(s, &need);
    if (rc != LSTM_OK) return rc;
    if ((rc = lstm_gated_mlp_reserve_size(s, &keep)) != LSTM_OK) return rc;
    if (x_stride < s->in) return LSTM_ERR_SHAPE;
    if (s->rows == 0) return LSTM_OK;
    if (!x || !w_gate || !w_up || !w_down || !y) return LSTM_ERR_ARG;
    if (!aligned(w_gate) || !aligned(w_up) || !aligned(w_down) || !aligned(workspace) || !aligned(reserve))
        return LSTM_ERR_ARG;
    if (!workspace || workspace_bytes < need || (reserve && reserve_bytes < keep)) return LSTM_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {x, w_gate, w_up, w_down, y, reserve, workspace};
    if (!all_on_device(ptrs, 7, dev)) return LSTM_ERR_DEVICE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Forward f = forward_of(s, x, x_stride, w_gate, w_up, w_down, y, reserve, workspace);
    if (f.few) {
        if ((rc = launched(launch_mlp_few(f.few_gate, st))) != LSTM_OK) return rc;
        return launched(launch_mlp_few(f.few_down, st));
    }
    if ((rc = launched(f.ops.launch(st))) != LSTM_OK) return rc;
    if ((rc = launched(launch_mlp(f.gate, st))) != LSTM_OK) return rc;
    return launched(launch_mlp(f.down, st));
}

lstm_status lstm_gated_mlp_backward(const lstm_gated_mlp_shape *s, const void *x, long long x_stride,
                                    const void *w_gate, const void *w_up, const void *w_down, const void *reserve,
                                    size_t reserve_bytes, const void *dy, long long dy_stride, void *dx, void *dw_gate,
                                    void *dw_up, void *dw_down, void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0, keep = 0;
    lstm_status rc = lstm_gated_mlp_backward_workspace_size(s, &need);
    if (rc != LSTM_OK) return rc;
    if ((rc = lstm_gated_mlp_reserve_size(s, &keep)) != LSTM_OK) return rc;
    if (x_stride < s->in || dy_stride < s->out) return LSTM_ERR_SHAPE;
    if (!w_gate || !w_up || !w_down || (s->rows && (!x || !dy || !reserve))) return LSTM_ERR_ARG;
    if (!aligned(w_gate) || !aligned(w_up) || !aligned(w_down) || !aligned(workspace) || !aligned(reserve))
        return LSTM_ERR_ARG;
    if ((need && (!workspace || workspace_bytes < need)) || (s->rows && reserve_bytes < keep))
        return LSTM_ERR_WORKSPACE;
    int dev = 0;
    if ((rc = current_device(&dev)) != LSTM_OK) return rc;
    const void *ptrs[] = {s->rows ? x : nullptr, w_gate, w_up, w_down, s->rows ? reserve : nullptr,
                          s->rows ? dy : nullptr, dx, dw_gate, dw_up, dw_down, need ? workspace : nullptr};
    if (!all_on_device(ptrs, 11, dev)) return LSTM_ERR_DEVICE;
    if (!dx && !dw_gate && !dw_up && !dw_down) return LSTM_OK;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Backward f = backward_of(s, x, x_stride, w_gate, w_up, w_down, reserve, dy, dy_stride, dx, dw_gate, dw_up,
                                   dw_down, workspace);
    if ((rc = launched(f.ops.launch(st))) != LSTM_OK) return rc;
    if (f.want_hidden)
        if ((rc = launched(launch_mlp(f.hidden, st))) != LSTM_OK) return rc;
    if (f.want_dx)
        if ((rc = launched(launch_mlp(f.dx, st))) != LSTM_OK) return rc;
    return f.dw.count ? launched(launch_mlp(f.dw, st)) : LSTM_OK;
}

}  // extern "C"
