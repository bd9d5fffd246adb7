// block_api.cpp -- the C ABI of the gated linear recurrence, of q/k norms with rotary positions and of the short convolution:
// argument checks (host only, before any HIP call), workspaces and dispatch.  See include/lconv.h for the contract.
#include "lconv.h"

#include "block_kernels.h"
#include "mixer_checks.h"

using namespace lcv;

namespace {

constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;      // workgroups of 256 threads: threads along a grid stay below 2^32

// An operand [B][N][C] with contiguous channels; NULL strides: dense.  B, N, C > 0 here.
lconv_status_t tokens(const void* p, const lconv_strides_t* given, int64_t B, int64_t N, int64_t C, lconv_dtype_t dt,
                      bool written, TokOperand* o, Range* r) {
    int64_t b, n, tb, tn;
    if (given) {
        b = given->b;
        n = given->n;
    } else {
        n = C;
        if (!mul_ok(N, C, &b)) return LCONV_ERR_INVALID_SHAPE;
    }
    if (B == 1) b = 0;
    if (N == 1) n = 0;
    if (b < 0 || n < 0 || !mul_ok(B - 1, b, &tb) || !mul_ok(N - 1, n, &tn)) return LCONV_ERR_INVALID_SHAPE;
    if (tb > INT64_MAX / 32 || tn > INT64_MAX / 32 || C > INT64_MAX / 32) return LCONV_ERR_INVALID_SHAPE;
    if (written) {      // rows apart: the smaller stride clears a row, the larger one all rows along the other
        const bool nin = B == 1 || (N > 1 && n <= b);
        const int64_t inner = nin ? n : b, span = (nin ? tn : tb) + C, count = nin ? N : B;
        if (count > 1 && inner < C) return LCONV_ERR_INVALID_SHAPE;
        if (B > 1 && N > 1 && (nin ? b : n) < span) return LCONV_ERR_INVALID_SHAPE;
    }
    if (!p) return LCONV_ERR_NULL_POINTER;
    const size_t es = dtype_size(dt);
    if ((uintptr_t)p % es) return LCONV_ERR_MISALIGNED;      // channels of any width: a token may begin at any element
    *o = TokOperand{p, b, n};
    *r = Range{p, (size_t)(tb + tn + C) * es, 0, 0};
    const int64_t step = N > 1 ? n : b;          // slices of one token-major buffer
    if ((N > 1 || B > 1) && step >= C && (N == 1 || B == 1 || b % step == 0)) {
        r->foot = (size_t)C * es;
        r->step = (size_t)step * es;
    }
    return LCONV_SUCCESS;
}

bool scan_flags_ok(int flags) {
    const int gate = flags & 3, mix = flags & ~3;
    return gate <= LCONV_GATE_RATE && (mix == LCONV_MIX_PLAIN || mix == LCONV_MIX_CONVEX || mix == LCONV_MIX_NORM);
}

// sizes that the kernels' indices hold: channels and segments in 32 bits, marks and states in 64
bool scan_sizes_ok(int64_t B, int64_t N, int64_t C) {
    int64_t t;
    if (N >= ((int64_t)1 << 31) || C > ((int64_t)1 << 24) || B > ((int64_t)1 << 24) || !mul_ok(B, C, &t)) return false;
    return mul_ok(t, (N + kScanMark - 1) / kScanMark, &t) && t <= INT64_MAX / 16;
}

// and those that a launch has threads for, which differ by type, as 16-bit calls may have two channels to a lane
bool scan_dims_ok(int64_t B, int64_t N, int64_t C, lconv_dtype_t dtype) {
    if (!scan_sizes_ok(B, N, C)) return false;
    // workgroups of 1024 threads (gradients: 512), and single tokens
    const ScanPlan p = scan_plan(B, N > 0 ? N : 1, C, dtype, false), g = scan_plan(B, N > 0 ? N : 1, C, dtype, true);
    return B * p.cblocks * p.nseg <= kMaxGrid / 4 && B * g.cblocks * g.nseg <= kMaxGrid / 2 && B * ((C + 511) / 256) <= kMaxGrid;
}

size_t seg_bytes(const ScanPlan& p, int64_t B, int64_t C) {
    return p.nseg > 1 ? round256((size_t)(B * p.nseg) * (size_t)C * 12) : 0;
}

void set_plan(ScanArgs* a, const ScanPlan& p) {
    a->vec = p.vec; a->cblocks = p.cblocks; a->nseg = p.nseg; a->seg_len = p.seg_len; a->waves = p.waves;
}

}  // namespace

extern "C" {

size_t lconv_gated_scan_marks_bytes(int64_t B, int64_t N, int64_t C) {
    if (B <= 0 || N <= 0 || C <= 0 || !scan_sizes_ok(B, N, C)) return 0;      // whatever a launch of some type takes
    return (size_t)(B * ((N + kScanMark - 1) / kScanMark)) * (size_t)C * 4;
}

size_t lconv_gated_scan_workspace_bytes(int64_t B, int64_t N, int64_t C, lconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B <= 0 || N <= 0 || C <= 0 || !scan_dims_ok(B, N, C, dtype)) return 0;
    return seg_bytes(scan_plan(B, N, C, dtype, false), B, C);
}

size_t lconv_gated_scan_bwd_workspace_bytes(int64_t B, int64_t N, int64_t C, int flags, lconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B <= 0 || N <= 0 || C <= 0 || !scan_flags_ok(flags) || !scan_dims_ok(B, N, C, dtype)) return 0;
    const ScanPlan p = scan_plan(B, N, C, dtype, true);
    return seg_bytes(p, B, C) + ((flags & 3) == LCONV_GATE_RATE ? round256((size_t)(B * p.nseg) * (size_t)C * 4) : 0);
}

lconv_status_t lconv_gated_scan_fwd(const void* x, const lconv_strides_t* x_strides, const void* z,
                                    const lconv_strides_t* z_strides, const void* input_gate,
                                    const lconv_strides_t* input_gate_strides, const float* rate, const float* state_in,
                                    const int32_t* lengths, void* y, const lconv_strides_t* y_strides, float* state_out,
                                    float* marks, int64_t B, int64_t N, int64_t C, int flags, lconv_dtype_t dtype,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype) || !scan_flags_ok(flags)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || N < 0 || C < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || C == 0) return LCONV_SUCCESS;
    if (!scan_dims_ok(B, N, C, dtype)) return LCONV_ERR_UNSUPPORTED;
    if (!aligned16(state_in) || !aligned16(state_out) || !aligned16(marks) || !aligned16(rate)) return LCONV_ERR_MISALIGNED;
    const Range rsi = buffer(state_in, B * C, 4), rso = buffer(state_out, B * C, 4);
    if (state_in != state_out && overlap(rsi, rso)) return LCONV_ERR_ALIASING;
    if (N == 0) return state_out && state_in != state_out ? hip_status(launch_row_state(state_in, state_out, B * C, stream)) : LCONV_SUCCESS;
    ScanArgs a{};
    TokOperand yo{};
    Range rx, rz, ri{}, ry;
    lconv_status_t st;
    if ((st = tokens(x, x_strides, B, N, C, dtype, false, &a.x, &rx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(z, z_strides, B, N, C, dtype, false, &a.z, &rz)) != LCONV_SUCCESS) return st;
    if (input_gate && (st = tokens(input_gate, input_gate_strides, B, N, C, dtype, false, &a.i, &ri)) != LCONV_SUCCESS) return st;
    if ((st = tokens(y, y_strides, B, N, C, dtype, true, &yo, &ry)) != LCONV_SUCCESS) return st;
    const bool rated = (flags & 3) == LCONV_GATE_RATE;
    if (rated && !rate) return LCONV_ERR_NULL_POINTER;
    const Range rr = buffer(rated ? rate : nullptr, C, 4), rl = buffer(lengths, B, 4);
    const Range rm = buffer(marks, (int64_t)lconv_gated_scan_marks_bytes(B, N, C), 1);
    if (clash({ry, rso, rm}, {rx, rz, ri, rr, rl}) || overlap(ry, rsi) || overlap(rm, rsi)) return LCONV_ERR_ALIASING;
    const ScanPlan p = scan_plan(B, N, C, dtype, false);
    const size_t need = seg_bytes(p, B, C);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rx, rz, ri, ry, rsi, rso, rr, rl, rm})) return LCONV_ERR_ALIASING;
    }
    a.rate = rated ? rate : nullptr; a.state_in = state_in; a.lengths = lengths;
    a.y = y; a.yb = yo.b; a.yn = yo.n; a.state_out = state_out; a.marks = marks; a.seg = (float*)workspace;
    a.B = B; a.N = N; a.C = C; a.gate = flags & 3; a.mix = flags & ~3;
    set_plan(&a, p);
    return hip_status(launch_scan_fwd(dtype, a, stream));
}

lconv_status_t lconv_gated_scan_bwd(const void* dy, const lconv_strides_t* dy_strides, const void* x,
                                    const lconv_strides_t* x_strides, const void* z, const lconv_strides_t* z_strides,
                                    const void* input_gate, const lconv_strides_t* input_gate_strides, const float* rate,
                                    const float* marks, const float* dstate_out, const int32_t* lengths, void* dx,
                                    const lconv_strides_t* dx_strides, void* dz, const lconv_strides_t* dz_strides,
                                    void* dinput_gate, const lconv_strides_t* dinput_gate_strides, float* drate,
                                    float* dstate_in, int64_t B, int64_t N, int64_t C, int flags, lconv_dtype_t dtype,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype) || !scan_flags_ok(flags)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || N < 0 || C < 0) return LCONV_ERR_INVALID_SHAPE;
    if (C == 0) return LCONV_SUCCESS;
    if (!scan_dims_ok(B, N, C, dtype)) return LCONV_ERR_UNSUPPORTED;
    const bool rated = (flags & 3) == LCONV_GATE_RATE;
    if (!rated) drate = nullptr;
    if (!aligned16(marks) || !aligned16(rate) || !aligned16(drate) || !aligned16(dstate_in) || !aligned16(dstate_out))
        return LCONV_ERR_MISALIGNED;
    const Range rso = buffer(dstate_out, B * C, 4), rsi = buffer(dstate_in, B * C, 4), rdr = buffer(drate, C, 4);
    if ((dstate_in != dstate_out && overlap(rsi, rso)) || overlap(rdr, rsi) || overlap(rdr, rso)) return LCONV_ERR_ALIASING;
    if (B == 0 || N == 0) {     // no tokens: the state's gradient passes through, the rate has none
        if (B > 0 && dstate_in && dstate_in != dstate_out && launch_row_state(dstate_out, dstate_in, B * C, stream) != hipSuccess)
            return LCONV_ERR_HIP;
        return drate ? hip_status(launch_row_state(nullptr, drate, C, stream)) : LCONV_SUCCESS;
    }
    ScanArgs a{};
    TokOperand ox{}, oz{}, oi{};
    Range rdy, rx, rz, ri{}, rdx, rdz, rdi{};
    lconv_status_t st;
    if ((st = tokens(dy, dy_strides, B, N, C, dtype, false, &a.dy, &rdy)) != LCONV_SUCCESS) return st;
    if ((st = tokens(x, x_strides, B, N, C, dtype, false, &a.x, &rx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(z, z_strides, B, N, C, dtype, false, &a.z, &rz)) != LCONV_SUCCESS) return st;
    if ((st = tokens(dx, dx_strides, B, N, C, dtype, true, &ox, &rdx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(dz, dz_strides, B, N, C, dtype, true, &oz, &rdz)) != LCONV_SUCCESS) return st;
    if (input_gate) {
        if ((st = tokens(input_gate, input_gate_strides, B, N, C, dtype, false, &a.i, &ri)) != LCONV_SUCCESS) return st;
        if ((st = tokens(dinput_gate, dinput_gate_strides, B, N, C, dtype, true, &oi, &rdi)) != LCONV_SUCCESS) return st;
    }
    if (!marks || (rated && !rate)) return LCONV_ERR_NULL_POINTER;
    const Range rr = buffer(rated ? rate : nullptr, C, 4), rl = buffer(lengths, B, 4);
    const Range rm = buffer(marks, (int64_t)lconv_gated_scan_marks_bytes(B, N, C), 1);
    if (clash({rdx, rdz, rdi, rsi, rdr}, {rdy, rx, rz, ri, rr, rl, rm}) || overlap(rdx, rso) || overlap(rdz, rso) || overlap(rdi, rso))
        return LCONV_ERR_ALIASING;
    const ScanPlan p = scan_plan(B, N, C, dtype, true);
    const size_t need = lconv_gated_scan_bwd_workspace_bytes(B, N, C, flags, dtype);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rdy, rx, rz, ri, rdx, rdz, rdi, rso, rsi, rdr, rr, rl, rm})) return LCONV_ERR_ALIASING;
    }
    a.rate = rated ? rate : nullptr; a.state_in = dstate_out; a.lengths = lengths;
    a.dx = dx; a.dxb = ox.b; a.dxn = ox.n; a.dz = dz; a.dzb = oz.b; a.dzn = oz.n; a.di = dinput_gate; a.dib = oi.b; a.din = oi.n;
    a.state_out = dstate_in; a.marks = const_cast<float*>(marks); a.seg = (float*)workspace;
    a.part = drate ? (float*)((char*)workspace + seg_bytes(p, B, C)) : nullptr; a.drate = drate;
    a.B = B; a.N = N; a.C = C; a.gate = flags & 3; a.mix = flags & ~3;
    set_plan(&a, p);
    return hip_status(launch_scan_bwd(dtype, a, stream));
}

lconv_status_t lconv_gated_scan_step(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const void* input_gate,
                                     int64_t input_gate_stride, const float* rate, float* state, const int32_t* slots,
                                     void* y, int64_t y_stride, int64_t B, int64_t C, int64_t nslots, int flags,
                                     lconv_dtype_t dtype, hipStream_t stream) {
    if (!dtype_ok(dtype) || !scan_flags_ok(flags)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || C < 0 || nslots < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || C == 0) return LCONV_SUCCESS;
    if (!scan_dims_ok(B, 1, C, dtype)) return LCONV_ERR_UNSUPPORTED;
    int64_t states;
    if ((!slots && nslots < B) || !mul_ok(nslots, 4 * C, &states)) return LCONV_ERR_INVALID_SHAPE;
    ScanStepArgs a{};
    TokOperand yo{};
    Range rx, rz, ri{}, ry;
    const lconv_strides_t sx{x_stride, 0, 0}, sz{z_stride, 0, 0}, si{input_gate_stride, 0, 0}, sy{y_stride, 0, 0};
    lconv_status_t st;
    if ((st = tokens(x, &sx, B, 1, C, dtype, false, &a.x, &rx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(z, &sz, B, 1, C, dtype, false, &a.z, &rz)) != LCONV_SUCCESS) return st;
    if (input_gate && (st = tokens(input_gate, &si, B, 1, C, dtype, false, &a.i, &ri)) != LCONV_SUCCESS) return st;
    if ((st = tokens(y, &sy, B, 1, C, dtype, true, &yo, &ry)) != LCONV_SUCCESS) return st;
    const bool rated = (flags & 3) == LCONV_GATE_RATE;
    if ((rated && !rate) || (!state && nslots > 0)) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(state) || !aligned16(rate)) return LCONV_ERR_MISALIGNED;
    if (clash({ry, buffer(state, states, 1)}, {rx, rz, ri, buffer(rated ? rate : nullptr, C, 4), buffer(slots, B, 4)}))
        return LCONV_ERR_ALIASING;
    a.rate = rate; a.state = state; a.slots = slots; a.y = y; a.yb = yo.b;
    a.B = B; a.C = C; a.nslots = nslots; a.gate = flags & 3; a.mix = flags & ~3;
    return hip_status(launch_scan_step(dtype, a, stream));
}

}  // extern "C"

namespace {

constexpr int kQkFlags = LCONV_ROTARY_INTERLEAVED | LCONV_QKNORM_CENTRED;

bool qk_dims_ok(int64_t B, int64_t H, int64_t G, int64_t N, int64_t D, int64_t rot, int flags) {
    int64_t tokens, t;
    if (D < 8 || D > LCONV_QKNORM_MAX_D || D % 8 || rot > D || rot % 2 || (flags & ~kQkFlags)) return false;
    if (H >= (1 << 20) || G >= (1 << 20) || !mul_ok(B, N, &tokens) || !mul_ok(tokens, H + G, &t)) return false;
    if (tokens == 0 || H + G == 0) return true;
    if (tokens >= ((int64_t)1 << 31)) return false;
    const QkPlan p = qk_plan(tokens, D, rot, (int)(H + G));
    return p.items < ((int64_t)1 << 31) && (p.items * p.lanes + 255) / 256 <= kMaxGrid;
}

// positions, frequencies and weights: their ranges
struct QkSides { Range pos, freq, w[2]; };
lconv_status_t qk_sides(QkArgs* a, const int32_t* positions, int64_t pos_stride, const float* inv_freq, const void* q_weight,
                        const void* k_weight, int64_t B, int64_t N, int64_t D, int64_t rot, lconv_dtype_t dtype, QkSides* r) {
    int64_t t;
    if (rot > 0 && !inv_freq) return LCONV_ERR_NULL_POINTER;
    if (!mul_ok(B - 1, pos_stride, &t) || t > INT64_MAX / 8 - N) return LCONV_ERR_INVALID_SHAPE;
    if (!aligned16(q_weight) || !aligned16(k_weight)) return LCONV_ERR_MISALIGNED;
    r->pos = buffer(positions, t + N, 4);
    r->freq = buffer(rot > 0 ? inv_freq : nullptr, rot / 2, 4);
    r->w[0] = buffer(q_weight, D, dtype_size(dtype));
    r->w[1] = buffer(k_weight, D, dtype_size(dtype));
    a->w[0] = q_weight; a->w[1] = k_weight;
    a->positions = positions; a->pos_stride = pos_stride; a->inv_freq = inv_freq;
    return LCONV_SUCCESS;
}

bool same_place(const void* x, const lconv_strides_t& xs, const void* y, const lconv_strides_t& ys) {
    return x == y && xs.b == ys.b && xs.h == ys.h && xs.n == ys.n;
}

}  // namespace

extern "C" {

lconv_status_t lconv_qknorm_rotary_fwd(const void* q, const lconv_strides_t* q_strides, const void* k,
                                       const lconv_strides_t* k_strides, const void* q_weight, const void* k_weight,
                                       const int32_t* positions, int64_t pos_stride, const float* inv_freq, float magnitude,
                                       float eps, void* yq, const lconv_strides_t* yq_strides, void* yk,
                                       const lconv_strides_t* yk_strides, int64_t B, int64_t H, int64_t G, int64_t N, int64_t D,
                                       int64_t rot, int flags, lconv_dtype_t dtype, hipStream_t stream) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || G < 0 || N < 0 || D < 0 || rot < 0 || pos_stride < 0) return LCONV_ERR_INVALID_SHAPE;
    if (!k && !yk) G = 0;
    if (B == 0 || N == 0 || H + G == 0) return LCONV_SUCCESS;
    if (!qk_dims_ok(B, H, G, N, D, rot, flags)) return LCONV_ERR_UNSUPPORTED;
    QkArgs a{};
    QkSides side{};
    lconv_status_t st = qk_sides(&a, positions, pos_stride, inv_freq, q_weight, k_weight, B, N, D, rot, dtype, &side);
    if (st != LCONV_SUCCESS) return st;
    const int64_t heads[2] = {H, G};
    const void* const in[2] = {q, k};
    const lconv_strides_t *const is[2] = {q_strides, k_strides}, *const os[2] = {yq_strides, yk_strides};
    void* const out[2] = {yq, yk};
    Range rx[2]{}, ry[2]{};
    bool inplace[2] = {false, false};
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        if ((st = operand(in[i], is[i], B, heads[i], N, D, dtype, false, &a.xs[i], &rx[i])) != LCONV_SUCCESS) return st;
        if ((st = operand(out[i], os[i], B, heads[i], N, D, dtype, true, &a.ys[i], &ry[i])) != LCONV_SUCCESS) return st;
        a.x[i] = in[i]; a.y[i] = out[i]; a.heads[i] = (int)heads[i];
        inplace[i] = same_place(in[i], a.xs[i], out[i], a.ys[i]);
    }
    if (clash({ry[0], ry[1]}, {side.pos, side.freq, side.w[0], side.w[1]}) || overlap(ry[0], rx[1]) || overlap(ry[1], rx[0]) ||
        (overlap(ry[0], rx[0]) && !inplace[0]) || (overlap(ry[1], rx[1]) && !inplace[1]))
        return LCONV_ERR_ALIASING;
    a.magnitude = magnitude; a.eps = eps; a.B = B; a.N = N; a.D = (int)D; a.rot = (int)rot; a.flags = flags;
    return hip_status(launch_qknorm_fwd(dtype, a, stream));
}

size_t lconv_qknorm_rotary_bwd_workspace_bytes(int64_t B, int64_t H, int64_t G, int64_t N, int64_t D, int64_t rot) {
    if (B <= 0 || H < 0 || G < 0 || H + G <= 0 || N <= 0 || rot < 0 || !qk_dims_ok(B, H, G, N, D, rot, 0)) return 0;
    const QkGradPlan g = qk_grad_plan(B * N, D, rot, H, G);
    return (size_t)(g.parts[0] + g.parts[1]) * (size_t)D * 4;
}

lconv_status_t lconv_qknorm_rotary_bwd(const void* dyq, const lconv_strides_t* dyq_strides, const void* dyk,
                                       const lconv_strides_t* dyk_strides, const void* q, const lconv_strides_t* q_strides,
                                       const void* k, const lconv_strides_t* k_strides, const void* q_weight,
                                       const void* k_weight, const int32_t* positions, int64_t pos_stride,
                                       const float* inv_freq, float magnitude, float eps, void* dq,
                                       const lconv_strides_t* dq_strides, void* dk, const lconv_strides_t* dk_strides,
                                       float* dq_weight, float* dk_weight, int64_t B, int64_t H, int64_t G, int64_t N, int64_t D,
                                       int64_t rot, int flags, lconv_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || G < 0 || N < 0 || D < 0 || rot < 0 || pos_stride < 0) return LCONV_ERR_INVALID_SHAPE;
    if (!k && !dyk && !dk) G = 0;
    if (!qk_dims_ok(B, H, G, N, D, rot, flags)) return LCONV_ERR_UNSUPPORTED;
    if (!aligned16(dq_weight) || !aligned16(dk_weight)) return LCONV_ERR_MISALIGNED;
    const Range rdw[2] = {buffer(dq_weight, D, 4), buffer(dk_weight, D, 4)};
    if (overlap(rdw[0], rdw[1])) return LCONV_ERR_ALIASING;
    QkArgs a{};
    a.dw[0] = dq_weight; a.dw[1] = dk_weight; a.D = (int)D;
    const int64_t heads[2] = {H, G};
    if (B == 0 || N == 0 || H + G == 0) return hip_status(launch_qknorm_bwd(dtype, a, stream));    // zeros to the weights' gradients
    QkSides side{};
    lconv_status_t st = qk_sides(&a, positions, pos_stride, inv_freq, q_weight, k_weight, B, N, D, rot, dtype, &side);
    if (st != LCONV_SUCCESS) return st;
    const void *const in[2] = {q, k}, *const grad[2] = {dyq, dyk};
    const lconv_strides_t *const is[2] = {q_strides, k_strides}, *const gs[2] = {dyq_strides, dyk_strides},
                          *const os[2] = {dq_strides, dk_strides};
    void* const out[2] = {dq, dk};
    Range rx[2]{}, rg[2]{}, ry[2]{};
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        if ((st = operand(grad[i], gs[i], B, heads[i], N, D, dtype, false, &a.dys[i], &rg[i])) != LCONV_SUCCESS) return st;
        if ((st = operand(in[i], is[i], B, heads[i], N, D, dtype, false, &a.xs[i], &rx[i])) != LCONV_SUCCESS) return st;
        if ((st = operand(out[i], os[i], B, heads[i], N, D, dtype, true, &a.ys[i], &ry[i])) != LCONV_SUCCESS) return st;
        a.x[i] = in[i]; a.dy[i] = grad[i]; a.y[i] = out[i]; a.heads[i] = (int)heads[i];
    }
    if (clash({ry[0], ry[1], rdw[0], rdw[1]}, {rx[0], rx[1], rg[0], rg[1], side.pos, side.freq, side.w[0], side.w[1]}))
        return LCONV_ERR_ALIASING;
    if (dq_weight || dk_weight) {
        const size_t need = lconv_qknorm_rotary_bwd_workspace_bytes(B, H, G, N, D, rot);
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rx[0], rx[1], rg[0], rg[1], ry[0], ry[1], rdw[0], rdw[1], side.pos,
                                                          side.freq, side.w[0], side.w[1]}))
            return LCONV_ERR_ALIASING;
        a.part = (float*)workspace;
    }
    a.magnitude = magnitude; a.eps = eps; a.B = B; a.N = N; a.rot = (int)rot; a.flags = flags;
    return hip_status(launch_qknorm_bwd(dtype, a, stream));
}

}  // extern "C"

namespace {

bool conv_dims_ok(int64_t B, int64_t N, int64_t C, int64_t K) {
    int64_t t;
    if (K < 2 || K > LCONV_SHORTCONV_MAX_TAPS || N >= ((int64_t)1 << 31) || C > ((int64_t)1 << 24) || B > ((int64_t)1 << 24)) return false;
    if (!mul_ok(B, C, &t) || t > INT64_MAX / 64) return false;
    if (B == 0 || N == 0 || C == 0) return true;
    for (bool inplace : {false, true}) {
        const ConvPlan p = conv_plan(B, N, C, K, false, inplace);
        if (B * p.runs >= ((int64_t)1 << 31) || (int64_t)p.cgroups * p.groups > kMaxGrid) return false;
    }
    return B * ((C + 511) / 256) <= kMaxGrid;      // single tokens
}

void set_plan(ConvArgs* a, const ConvPlan& p) {
    a->vec = p.vec; a->cgroups = p.cgroups; a->runs = p.runs; a->groups = p.groups; a->run = p.run;
}

}  // namespace

extern "C" {

lconv_status_t lconv_shortconv_fwd(const void* x, const lconv_strides_t* x_strides, const void* weight, const void* bias,
                                   const void* state_in, const int32_t* lengths, void* y, const lconv_strides_t* y_strides,
                                   void* state_out, int64_t B, int64_t N, int64_t C, int64_t K, int flags, lconv_dtype_t dtype,
                                   hipStream_t stream) {
    if (!dtype_ok(dtype) || (flags & ~LCONV_SHORTCONV_SILU)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || N < 0 || C < 0 || K < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || C == 0) return LCONV_SUCCESS;
    if (!conv_dims_ok(B, N, C, K)) return LCONV_ERR_UNSUPPORTED;
    if (!aligned16(weight) || !aligned16(bias) || !aligned16(state_in) || !aligned16(state_out)) return LCONV_ERR_MISALIGNED;
    const size_t es = dtype_size(dtype);
    const int64_t states = B * (K - 1) * C;
    const Range rsi = buffer(state_in, states, es), rso = buffer(state_out, states, es);
    if (state_in != state_out && overlap(rsi, rso)) return LCONV_ERR_ALIASING;
    if (N == 0)
        return state_out && state_in != state_out ? hip_status(launch_conv_state(dtype, state_in, state_out, states, stream)) : LCONV_SUCCESS;
    ConvArgs a{};
    TokOperand yo{};
    Range rx, ry;
    lconv_status_t st;
    if ((st = tokens(x, x_strides, B, N, C, dtype, false, &a.x, &rx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(y, y_strides, B, N, C, dtype, true, &yo, &ry)) != LCONV_SUCCESS) return st;
    if (!weight) return LCONV_ERR_NULL_POINTER;
    if (clash({ry, rso}, {rx, buffer(weight, C * K, es), buffer(bias, C, es), buffer(lengths, B, 4)}) || overlap(ry, rsi))
        return LCONV_ERR_ALIASING;
    a.w = weight; a.bias = bias; a.state_in = state_in; a.lengths = lengths; a.y = y; a.yb = yo.b; a.yn = yo.n; a.state_out = state_out;
    a.B = B; a.N = N; a.C = C; a.K = (int)K; a.silu = flags & LCONV_SHORTCONV_SILU;
    set_plan(&a, conv_plan(B, N, C, K, false, state_in && state_in == state_out));
    return hip_status(launch_conv_fwd(dtype, a, stream));
}

size_t lconv_shortconv_bwd_workspace_bytes(int64_t B, int64_t N, int64_t C, int64_t K) {
    if (B <= 0 || N <= 0 || C <= 0 || !conv_dims_ok(B, N, C, K)) return 0;
    return (size_t)conv_plan(B, N, C, K, true, false).groups * (size_t)(K + 1) * (size_t)C * 4;
}

lconv_status_t lconv_shortconv_bwd(const void* dy, const lconv_strides_t* dy_strides, const void* x,
                                   const lconv_strides_t* x_strides, const void* weight, const void* bias, const void* state_in,
                                   const void* dstate_out, const int32_t* lengths, void* dx, const lconv_strides_t* dx_strides,
                                   float* dweight, float* dbias, void* dstate_in, int64_t B, int64_t N, int64_t C, int64_t K,
                                   int flags, lconv_dtype_t dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype) || (flags & ~LCONV_SHORTCONV_SILU)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || N < 0 || C < 0 || K < 0) return LCONV_ERR_INVALID_SHAPE;
    if (C == 0) return LCONV_SUCCESS;
    if (!conv_dims_ok(B, N, C, K)) return LCONV_ERR_UNSUPPORTED;
    if (!aligned16(weight) || !aligned16(bias) || !aligned16(state_in) || !aligned16(dstate_out) || !aligned16(dstate_in) ||
        !aligned16(dweight) || !aligned16(dbias))
        return LCONV_ERR_MISALIGNED;
    const size_t es = dtype_size(dtype);
    const int64_t states = B * (K - 1) * C;
    const Range rsi = buffer(state_in, states, es), rdso = buffer(dstate_out, states, es), rdsi = buffer(dstate_in, states, es);
    const Range rdw = buffer(dweight, C * K, 4), rdb = buffer(dbias, C, 4);
    if (clash({rdsi, rdw, rdb}, {rsi, rdso})) return LCONV_ERR_ALIASING;
    ConvArgs a{};
    a.dw = dweight; a.db = dbias; a.K = (int)K; a.C = C; a.B = B; a.N = N; a.silu = flags & LCONV_SHORTCONV_SILU;
    if (B == 0 || N == 0) {     // no tokens: the state's gradient passes through, the weights have none
        if (B > 0 && dstate_in && launch_conv_state(dtype, dstate_out, dstate_in, states, stream) != hipSuccess) return LCONV_ERR_HIP;
        return hip_status(launch_conv_bwd(dtype, a, stream));
    }
    TokOperand xo{};
    Range rdy, rx, rdx;
    lconv_status_t st;
    if ((st = tokens(dy, dy_strides, B, N, C, dtype, false, &a.dy, &rdy)) != LCONV_SUCCESS) return st;
    if ((st = tokens(x, x_strides, B, N, C, dtype, false, &a.x, &rx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(dx, dx_strides, B, N, C, dtype, true, &xo, &rdx)) != LCONV_SUCCESS) return st;
    if (!weight) return LCONV_ERR_NULL_POINTER;
    const Range rw = buffer(weight, C * K, es), rb = buffer(bias, C, es), rl = buffer(lengths, B, 4);
    if (clash({rdx, rdsi, rdw, rdb}, {rdy, rx, rw, rb, rl, rsi, rdso})) return LCONV_ERR_ALIASING;
    const ConvPlan p = conv_plan(B, N, C, K, true, false);
    if (dweight || dbias) {
        const size_t need = lconv_shortconv_bwd_workspace_bytes(B, N, C, K);
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rdy, rx, rdx, rw, rb, rl, rsi, rdso, rdsi, rdw, rdb})) return LCONV_ERR_ALIASING;
        a.part = (float*)workspace;
    }
    a.w = weight; a.bias = bias; a.state_in = state_in; a.dstate_out = dstate_out; a.lengths = lengths;
    a.y = dx; a.yb = xo.b; a.yn = xo.n; a.state_out = dstate_in;
    set_plan(&a, p);
    return hip_status(launch_conv_bwd(dtype, a, stream));
}

lconv_status_t lconv_shortconv_step(const void* x, int64_t x_stride, const void* weight, const void* bias, void* state,
                                    const int32_t* slots, void* y, int64_t y_stride, int64_t B, int64_t C, int64_t K,
                                    int64_t nslots, int flags, lconv_dtype_t dtype, hipStream_t stream) {
    if (!dtype_ok(dtype) || (flags & ~LCONV_SHORTCONV_SILU)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || C < 0 || K < 0 || nslots < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || C == 0) return LCONV_SUCCESS;
    if (!conv_dims_ok(B, 1, C, K)) return LCONV_ERR_UNSUPPORTED;
    const size_t es = dtype_size(dtype);
    int64_t states;
    if ((!slots && nslots < B) || !mul_ok(nslots, (K - 1) * C * (int64_t)es, &states)) return LCONV_ERR_INVALID_SHAPE;
    ConvStepArgs a{};
    TokOperand yo{};
    Range rx, ry;
    const lconv_strides_t sx{x_stride, 0, 0}, sy{y_stride, 0, 0};
    lconv_status_t st;
    if ((st = tokens(x, &sx, B, 1, C, dtype, false, &a.x, &rx)) != LCONV_SUCCESS) return st;
    if ((st = tokens(y, &sy, B, 1, C, dtype, true, &yo, &ry)) != LCONV_SUCCESS) return st;
    if (!weight || (!state && nslots > 0)) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(weight) || !aligned16(bias) || !aligned16(state)) return LCONV_ERR_MISALIGNED;
    if (clash({ry, buffer(state, states, 1)}, {rx, buffer(weight, C * K, es), buffer(bias, C, es), buffer(slots, B, 4)}))
        return LCONV_ERR_ALIASING;
    a.w = weight; a.bias = bias; a.state = state; a.slots = slots; a.y = y; a.yb = yo.b;
    a.B = B; a.C = C; a.nslots = nslots; a.K = (int)K; a.silu = flags & LCONV_SHORTCONV_SILU;
    return hip_status(launch_conv_step(dtype, a, stream));
}

}  // extern "C"
