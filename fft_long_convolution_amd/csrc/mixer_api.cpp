// mixer_api.cpp -- the C ABI of linear attention, rotary positions and layer norm: argument checks
// (host only, before any HIP call), workspaces and dispatch.  See include/lconv.h for the contract.
#include "lconv.h"

#include <initializer_list>

#include "api_checks.h"
#include "mixer_kernels.h"
#include "mixer_plan.h"

using namespace lcv;

namespace {

// The address range of one buffer; with a token-major footprint where it is a strided operand.
struct Range {
    const void* p;
    size_t bytes;
    // strided operands: the elements of one token lie within `foot` bytes, tokens are `step` bytes
    // apart and batch rows a multiple of that (step 0: not of this form)
    size_t foot, step;
};

Range buffer(const void* p, int64_t n, size_t es) { return Range{p, (size_t)n * es, 0, 0}; }

bool overlap(const Range& a, const Range& b) {
    if (!lcv::overlap(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.step == 0 || a.step != b.step) return true;
    // slices of one token-major buffer: b's footprint modulo the token step, seen from a's start
    const intptr_t d = (intptr_t)((uintptr_t)b.p - (uintptr_t)a.p);
    const intptr_t st = (intptr_t)a.step;
    const size_t at = (size_t)(((d % st) + st) % st);
    return !(at >= a.foot && at + b.foot <= a.step);
}

// Strides of an operand [B][H][N][D]: resolves NULL to dense and checks them; `r` gets its range.
// B, H, N > 0 here.  A dimension of length one may come with any stride; it leaves with 0, since the kernels also form
// addresses a chunk away from a row's ends (the gradients' 31 tokens before a single one, which no lane then reads).
lconv_status_t operand(const void* p, const lconv_strides_t* given, int64_t B, int64_t H, int64_t N, int64_t D,
                       lconv_dtype_t dt, bool written, lconv_strides_t* s, Range* r) {
    const int64_t es = (int64_t)dtype_size(dt);
    if (given) {
        *s = *given;
    } else {
        int64_t t;
        s->n = D;
        if (!mul_ok(N, D, &s->h) || !mul_ok(H, s->h, &s->b) || !mul_ok(B, s->b, &t)) return LCONV_ERR_INVALID_SHAPE;
    }
    if (B == 1) s->b = 0;
    if (H == 1) s->h = 0;
    if (N == 1) s->n = 0;
    struct Dim { int64_t n, st; } dim[3] = {{B, s->b}, {H, s->h}, {N, s->n}};
    int64_t last = D, t;                 // elements from the start to the end of the last row
    for (const Dim& d : dim) {
        if (d.n == 1) continue;
        if (d.st < 0 || !mul_ok(d.n - 1, d.st, &t) || t > INT64_MAX / 8 - last) return LCONV_ERR_INVALID_SHAPE;
        last += t;
        if (d.st * es % 16) return LCONV_ERR_MISALIGNED;
    }
    if (written) {
        // rows must be apart: taken from the smallest stride up, each step clears what lies below it
        int64_t span = D;
        bool used[3] = {false, false, false};
        for (int k = 0; k < 3; ++k) {
            int m = -1;
            for (int i = 0; i < 3; ++i)
                if (!used[i] && (m < 0 || dim[i].st < dim[m].st || (dim[i].st == dim[m].st && dim[i].n < dim[m].n))) m = i;
            used[m] = true;
            if (dim[m].n == 1) continue;
            if (dim[m].st < span) return LCONV_ERR_INVALID_SHAPE;
            span += (dim[m].n - 1) * dim[m].st;
        }
    }
    if (!p) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(p)) return LCONV_ERR_MISALIGNED;
    *r = Range{p, (size_t)last * (size_t)es, 0, 0};
    const int64_t foot = (H == 1 ? 0 : (H - 1) * s->h) + D;
    // one token's step: the n stride, or for single tokens the batch row's
    const int64_t step = N > 1 ? s->n : s->b;
    if ((N > 1 || B > 1) && step >= foot && (B == 1 || s->b % step == 0)) {
        r->foot = (size_t)(foot * es);
        r->step = (size_t)(step * es);
    }
    return LCONV_SUCCESS;
}

// no output meets an input or another output
bool clash(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* a = outs.begin(); a != outs.end(); ++a) {
        for (const Range& b : ins)
            if (overlap(*a, b)) return true;
        for (const Range* b = a + 1; b != outs.end(); ++b)
            if (overlap(*a, *b)) return true;
    }
    return false;
}

bool linattn_dims_ok(int64_t B, int64_t H, int64_t G, int64_t N, int64_t Dk, int64_t Dv) {
    if (G < 1 || H % G || N >= ((int64_t)1 << 31)) return false;
    if (Dk < 8 || Dk > LCONV_LINATTN_MAX_D || Dk % 8 || Dv < 8 || Dv > LCONV_LINATTN_MAX_D || Dv % 8) return false;
    int64_t rows;
    return mul_ok(B, H, &rows) && rows <= kMaxWorkgroups;     // a launch has a workgroup to a (b, h) at least
}

// whether the forward's launches fit a grid: at most three roles of four column blocks to a row, and few rows in segments
constexpr int64_t kRowsThatFit = (int64_t)1 << 20;
bool linattn_fwd_fits(int64_t B, int64_t H, int64_t N, int64_t Dk, int64_t Dv, lconv_dtype_t dtype) {
    return B * H <= kRowsThatFit || linattn_workgroups(linattn_plan(B * H, 1, N, Dk, Dv, dtype), B * H, 1) <= kMaxWorkgroups;
}

// The chunk kernel reaches a chunk's 32 tokens by 32-bit byte offsets from its first: 31 strides have to fit.
constexpr int64_t kTokenStrideBytes = (int64_t)1 << 27;
bool far_apart(int64_t N, lconv_dtype_t dt, std::initializer_list<lconv_strides_t> all) {
    for (const lconv_strides_t& s : all)
        if (N > 1 && s.n > kTokenStrideBytes / (int64_t)dtype_size(dt)) return true;
    return false;
}

// fp32 gradients of each query head, before the sum over the heads that share a k/v head
size_t head_grads_bytes(int64_t B, int64_t H, int64_t G, int64_t N, int64_t D) {
    return H == G ? 0 : round256((size_t)(B * H) * (size_t)N * (size_t)D * 4);
}

void set_plan(LinJob* a, const LinPlan& p) {
    a->kt = p.kt; a->nw = p.nw; a->ncb = p.ncb; a->nseg = p.nseg; a->seg_len = p.seg_len;
}

// whether the gradients' launches fit a grid, the decay's (which is on or not) among them
bool linattn_bwd_fits(int64_t B, int64_t H, int64_t N, int64_t Dk, int64_t Dv, lconv_dtype_t dtype) {
    if (B * H <= kRowsThatFit) return true;
    const LinBwdPlan p = linattn_bwd_plan(B * H, N, Dk, Dv, dtype);
    for (int i = 0; i < p.launches; ++i)
        if (linattn_workgroups(p.plan[i], B * H, p.roles[i]) > kMaxWorkgroups) return false;
    return linattn_tan_workgroups(B * H, N, Dv) <= kMaxWorkgroups;
}

// the decay's gradient: partial sums, and the segments' states
size_t tan_part_bytes(int64_t rows, int64_t N, int64_t Dv) {
    return round256((size_t)(rows * linattn_tan_plan(rows, N, Dv).nseg) * (size_t)linattn_tan_blocks(Dv) * 4);
}
size_t tan_bytes(int64_t rows, int64_t N, int64_t Dk, int64_t Dv) {
    const int nseg = linattn_tan_plan(rows, N, Dv).nseg;
    return tan_part_bytes(rows, N, Dv) + (nseg > 1 ? round256((size_t)(rows * nseg) * 2 * (size_t)(Dk * Dv) * 4) : 0);
}

}  // namespace

extern "C" {

size_t lconv_linattn_workspace_bytes(int64_t B, int64_t H, int64_t G, int64_t N, int64_t Dk, int64_t Dv,
                                     lconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B <= 0 || H <= 0 || N <= 0 || !linattn_dims_ok(B, H, G, N, Dk, Dv) ||
        !linattn_fwd_fits(B, H, N, Dk, Dv, dtype))
        return 0;
    return linattn_states_bytes(linattn_plan(B * H, 1, N, Dk, Dv, dtype), B * H);
}

lconv_status_t lconv_linattn_fwd(const void* q, const lconv_strides_t* q_strides, const void* k,
                                 const lconv_strides_t* k_strides, const void* v, const lconv_strides_t* v_strides,
                                 const float* log_decay, float scale, const float* state_in, const int32_t* lengths,
                                 void* y, const lconv_strides_t* y_strides, float* state_out, int64_t B, int64_t H,
                                 int64_t G, int64_t N, int64_t Dk, int64_t Dv, lconv_dtype_t dtype, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || G < 0 || N < 0 || Dk < 0 || Dv < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || H == 0) return LCONV_SUCCESS;
    if (!linattn_dims_ok(B, H, G, N, Dk, Dv) || (N > 0 && !linattn_fwd_fits(B, H, N, Dk, Dv, dtype))) return LCONV_ERR_UNSUPPORTED;
    if (!aligned16(state_in) || !aligned16(state_out)) return LCONV_ERR_MISALIGNED;
    const int64_t states = B * H * Dk * Dv;
    const Range rsi = buffer(state_in, states, 4), rso = buffer(state_out, states, 4);
    if (state_in != state_out && overlap(rso, rsi)) return LCONV_ERR_ALIASING;
    if (N == 0) return state_out && state_in != state_out ? hip_status(launch_copy_state(state_in, state_out, states, stream)) : LCONV_SUCCESS;
    LinJob a{};
    LinRole& r = a.r[0];
    Range rq, rk, rv, ry;
    lconv_status_t st;
    if ((st = operand(q, q_strides, B, H, N, Dk, dtype, false, &r.Q.s, &rq)) != LCONV_SUCCESS) return st;
    if ((st = operand(k, k_strides, B, G, N, Dk, dtype, false, &r.K.s, &rk)) != LCONV_SUCCESS) return st;
    if ((st = operand(v, v_strides, B, G, N, Dv, dtype, false, &r.V.s, &rv)) != LCONV_SUCCESS) return st;
    if ((st = operand(y, y_strides, B, H, N, Dv, dtype, true, &r.o, &ry)) != LCONV_SUCCESS) return st;
    if (far_apart(N, dtype, {r.Q.s, r.K.s, r.V.s, r.o})) return LCONV_ERR_UNSUPPORTED;
    if (!log_decay) return LCONV_ERR_NULL_POINTER;
    const Range rld = buffer(log_decay, H, 4), rlen = buffer(lengths, B, 4);
    if (clash({ry, rso}, {rq, rk, rv, rld, rlen}) || overlap(ry, rsi)) return LCONV_ERR_ALIASING;
    const size_t need = lconv_linattn_workspace_bytes(B, H, G, N, Dk, Dv, dtype);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rq, rk, rv, ry, rsi, rso, rld, rlen})) return LCONV_ERR_ALIASING;
    }
    r.Q.p = q; r.Q.share = 1;
    r.K.p = k; r.K.share = (int)(H / G);
    r.V.p = v; r.V.share = (int)(H / G);
    r.O = y;
    r.DK = (int)Dk; r.DV = (int)Dv;
    r.s_in = state_in; r.s_out = state_out; r.s_row = (int)Dv; r.s_col = 1;
    r.states = (float*)workspace;
    r.s_q = scale; r.s_kv = 1.f;
    a.nroles = 1;
    a.exact = state_out != nullptr;
    a.log_decay = log_decay; a.lengths = lengths;
    a.B = B; a.H = (int)H; a.N = N;
    set_plan(&a, linattn_plan(B * H, 1, N, Dk, Dv, dtype));
    return hip_status(launch_linattn(dtype, a, stream));
}

size_t lconv_linattn_bwd_workspace_bytes(int64_t B, int64_t H, int64_t G, int64_t N, int64_t Dk, int64_t Dv,
                                         lconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B <= 0 || H <= 0 || N <= 0 || !linattn_dims_ok(B, H, G, N, Dk, Dv) ||
        !linattn_bwd_fits(B, H, N, Dk, Dv, dtype))
        return 0;
    return head_grads_bytes(B, H, G, N, Dk) + head_grads_bytes(B, H, G, N, Dv) + tan_bytes(B * H, N, Dk, Dv) +
           linattn_bwd_plan(B * H, N, Dk, Dv, dtype).total;
}

lconv_status_t lconv_linattn_bwd(const void* dy, const lconv_strides_t* dy_strides, const void* q,
                                 const lconv_strides_t* q_strides, const void* k, const lconv_strides_t* k_strides,
                                 const void* v, const lconv_strides_t* v_strides, const float* log_decay, float scale,
                                 const float* state_in, const float* dstate_out, const int32_t* lengths, void* dq,
                                 const lconv_strides_t* dq_strides, void* dk, const lconv_strides_t* dk_strides,
                                 void* dv, const lconv_strides_t* dv_strides, float* dstate_in, float* dlog_decay,
                                 int64_t B, int64_t H, int64_t G, int64_t N, int64_t Dk, int64_t Dv,
                                 lconv_dtype_t dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || G < 0 || N < 0 || Dk < 0 || Dv < 0) return LCONV_ERR_INVALID_SHAPE;
    if (H == 0) return LCONV_SUCCESS;
    if (!linattn_dims_ok(B, H, G, N, Dk, Dv) || (B > 0 && N > 0 && !linattn_bwd_fits(B, H, N, Dk, Dv, dtype)))
        return LCONV_ERR_UNSUPPORTED;
    if (!aligned16(state_in) || !aligned16(dstate_out) || !aligned16(dstate_in) || !aligned16(dlog_decay))
        return LCONV_ERR_MISALIGNED;
    const int64_t states = B * H * Dk * Dv;
    const Range rsi = buffer(state_in, states, 4), rdso = buffer(dstate_out, states, 4);
    const Range rdsi = buffer(dstate_in, states, 4), rdl = buffer(dlog_decay, H, 4);
    if (clash({rdsi, rdl}, {rsi, rdso})) return LCONV_ERR_ALIASING;
    if (B == 0 || N == 0) {  // no tokens: the state's gradient passes through, the decay has none
        if (B > 0 && dstate_in && launch_copy_state(dstate_out, dstate_in, states, stream) != hipSuccess) return LCONV_ERR_HIP;
        return dlog_decay ? hip_status(launch_copy_state(nullptr, dlog_decay, H, stream)) : LCONV_SUCCESS;
    }
    LinOperand oq{q, {}, 1}, ok{k, {}, (int)(H / G)}, ov{v, {}, (int)(H / G)}, ody{dy, {}, 1};
    lconv_strides_t sdq, sdk, sdv;
    Range rdy, rq, rk, rv, rdq, rdk, rdv;
    lconv_status_t st;
    if ((st = operand(dy, dy_strides, B, H, N, Dv, dtype, false, &ody.s, &rdy)) != LCONV_SUCCESS) return st;
    if ((st = operand(q, q_strides, B, H, N, Dk, dtype, false, &oq.s, &rq)) != LCONV_SUCCESS) return st;
    if ((st = operand(k, k_strides, B, G, N, Dk, dtype, false, &ok.s, &rk)) != LCONV_SUCCESS) return st;
    if ((st = operand(v, v_strides, B, G, N, Dv, dtype, false, &ov.s, &rv)) != LCONV_SUCCESS) return st;
    if ((st = operand(dq, dq_strides, B, H, N, Dk, dtype, true, &sdq, &rdq)) != LCONV_SUCCESS) return st;
    if ((st = operand(dk, dk_strides, B, G, N, Dk, dtype, true, &sdk, &rdk)) != LCONV_SUCCESS) return st;
    if ((st = operand(dv, dv_strides, B, G, N, Dv, dtype, true, &sdv, &rdv)) != LCONV_SUCCESS) return st;
    if (far_apart(N, dtype, {ody.s, oq.s, ok.s, ov.s, sdq, sdk, sdv})) return LCONV_ERR_UNSUPPORTED;
    if (!log_decay) return LCONV_ERR_NULL_POINTER;
    const Range rld = buffer(log_decay, H, 4), rlen = buffer(lengths, B, 4);
    if (clash({rdq, rdk, rdv, rdsi, rdl}, {rdy, rq, rk, rv, rld, rlen, rsi, rdso})) return LCONV_ERR_ALIASING;
    const size_t need = lconv_linattn_bwd_workspace_bytes(B, H, G, N, Dk, Dv, dtype);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rdy, rq, rk, rv, rdq, rdk, rdv, rsi, rdso, rdsi, rdl, rld, rlen}))
            return LCONV_ERR_ALIASING;
    }
    char* ws = (char*)workspace;
    const int share = (int)(H / G);
    float* gk = share > 1 ? (float*)ws : nullptr;
    ws += head_grads_bytes(B, H, G, N, Dk);
    float* gv = share > 1 ? (float*)ws : nullptr;
    ws += head_grads_bytes(B, H, G, N, Dv);

    const LinBwdPlan plan = linattn_bwd_plan(B * H, N, Dk, Dv, dtype);
    float* const tan = (float*)ws;
    float* const tan_states = (float*)(ws + tan_part_bytes(B * H, N, Dv));
    ws += tan_bytes(B * H, N, Dk, Dv);

    LinJob a{};
    a.log_decay = log_decay; a.lengths = lengths;
    a.B = B; a.H = (int)H; a.N = N;

    // dq: dy, v, k in the places of q, k, v, with the state transposed
    LinRole role[3] = {};
    LinRole &rdq_ = role[0], &rdk_ = role[1], &rdv_ = role[2];
    rdq_.Q = ody; rdq_.K = ov; rdq_.V = ok;
    rdq_.O = dq; rdq_.o = sdq;
    rdq_.DK = (int)Dv; rdq_.DV = (int)Dk;
    rdq_.s_in = state_in; rdq_.s_row = 1; rdq_.s_col = (int)Dv;
    rdq_.s_q = scale; rdq_.s_kv = 1.f;

    // dk: v, dy, q from the last token to the first
    rdk_ = rdq_;
    rdk_.Q = ov; rdk_.K = ody; rdk_.V = oq;
    rdk_.O = share > 1 ? (void*)gk : dk;
    rdk_.wide = share > 1;
    rdk_.o = share > 1 ? lconv_strides_t{H * N * Dk, N * Dk, Dk} : sdk;
    rdk_.s_in = dstate_out;
    rdk_.s_q = 1.f; rdk_.s_kv = scale; rdk_.reverse = 1;

    // dv and the gradient of the state that entered: k, q, dy
    rdv_ = rdk_;
    rdv_.Q = ok; rdv_.K = oq; rdv_.V = ody;
    rdv_.O = share > 1 ? (void*)gv : dv;
    rdv_.o = share > 1 ? lconv_strides_t{H * N * Dv, N * Dv, Dv} : sdv;
    rdv_.DK = (int)Dk; rdv_.DV = (int)Dv;
    rdv_.s_out = dstate_in; rdv_.s_row = (int)Dv; rdv_.s_col = 1;

    for (int i = 0; i < plan.launches; ++i) {
        a.nroles = plan.roles[i];
        for (int j = 0; j < a.nroles; ++j) {
            a.r[j] = role[plan.first[i] + j];
            a.r[j].states = (float*)ws;
            ws += plan.states[i];
        }
        a.exact = dstate_in && plan.first[i] + plan.roles[i] == 3;
        set_plan(&a, plan.plan[i]);
        if (launch_linattn(dtype, a, stream) != hipSuccess) return LCONV_ERR_HIP;
    }
    if (dlog_decay) {
        const LinTanPlan p = linattn_tan_plan(B * H, N, Dv);
        LinTanArgs t{};
        t.q = oq; t.k = ok; t.v = ov; t.dy = ody;
        t.s_in = state_in; t.ds_out = dstate_out;
        t.log_decay = log_decay; t.lengths = lengths;
        t.states = tan_states; t.part = tan; t.scale = scale;
        t.B = B; t.N = N; t.seg_len = p.seg_len; t.nseg = p.nseg;
        t.H = (int)H; t.DK = (int)Dk; t.DV = (int)Dv;
        if (launch_linattn_tan(dtype, t, dlog_decay, stream) != hipSuccess) return LCONV_ERR_HIP;
    }
    if (share > 1) {
        const HeadSumArgs s{{gk, gv}, {dk, dv}, {sdk, sdv}, {(int)Dk, (int)Dv}, B, N, (int)G, share};
        if (launch_head_sum(dtype, s, stream) != hipSuccess) return LCONV_ERR_HIP;
    }
    return LCONV_SUCCESS;
}

lconv_status_t lconv_linattn_step(const void* q, const lconv_strides_t* q_strides, const void* k,
                                  const lconv_strides_t* k_strides, const void* v, const lconv_strides_t* v_strides,
                                  const float* log_decay, float scale, float* state, const int32_t* slots, void* y,
                                  const lconv_strides_t* y_strides, int64_t B, int64_t H, int64_t G, int64_t Dk,
                                  int64_t Dv, int64_t nslots, lconv_dtype_t dtype, hipStream_t stream) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || G < 0 || Dk < 0 || Dv < 0 || nslots < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || H == 0) return LCONV_SUCCESS;
    if (!linattn_dims_ok(B, H, G, 1, Dk, Dv) || linattn_step_workgroups(B * H, Dv) > kMaxWorkgroups) return LCONV_ERR_UNSUPPORTED;
    int64_t states;
    if (!slots && nslots < B) return LCONV_ERR_INVALID_SHAPE;
    if (!mul_ok(nslots, H * Dk * Dv, &states) || !mul_ok(states, 4, &states)) return LCONV_ERR_INVALID_SHAPE;
    LinStepArgs a{};
    Range rq, rk, rv, ry;
    lconv_status_t st;
    if ((st = operand(q, q_strides, B, H, 1, Dk, dtype, false, &a.q.s, &rq)) != LCONV_SUCCESS) return st;
    if ((st = operand(k, k_strides, B, G, 1, Dk, dtype, false, &a.k.s, &rk)) != LCONV_SUCCESS) return st;
    if ((st = operand(v, v_strides, B, G, 1, Dv, dtype, false, &a.v.s, &rv)) != LCONV_SUCCESS) return st;
    if ((st = operand(y, y_strides, B, H, 1, Dv, dtype, true, &a.ys, &ry)) != LCONV_SUCCESS) return st;
    if (!log_decay || (!state && nslots > 0)) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(state)) return LCONV_ERR_MISALIGNED;
    if (clash({ry, buffer(state, states, 1)}, {rq, rk, rv, buffer(log_decay, H, 4), buffer(slots, B, 4)}))
        return LCONV_ERR_ALIASING;
    const int share = (int)(H / G);
    a.q.p = q; a.q.share = 1;
    a.k.p = k; a.k.share = share;
    a.v.p = v; a.v.share = share;
    a.y = y; a.log_decay = log_decay; a.state = state; a.slots = slots; a.scale = scale;
    a.B = B; a.nslots = nslots; a.H = (int)H; a.DK = (int)Dk; a.DV = (int)Dv;
    return hip_status(launch_linattn_step(dtype, a, stream));
}

lconv_status_t lconv_rotary(const void* q, const lconv_strides_t* q_strides, const void* k,
                            const lconv_strides_t* k_strides, const int32_t* positions, int64_t pos_stride,
                            const float* inv_freq, float magnitude, void* yq, const lconv_strides_t* yq_strides,
                            void* yk, const lconv_strides_t* yk_strides, int64_t B, int64_t H, int64_t G, int64_t N,
                            int64_t D, int64_t rot, int flags, lconv_dtype_t dtype, hipStream_t stream) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (B < 0 || H < 0 || G < 0 || N < 0 || D < 0 || rot < 0 || pos_stride < 0) return LCONV_ERR_INVALID_SHAPE;
    if (B == 0 || N == 0 || (H == 0 && (G == 0 || (!k && !yk)))) return LCONV_SUCCESS;
    if (D < 8 || D > 1024 || D % 8 || rot < 2 || rot > D || rot % 2 || (flags & ~3)) return LCONV_ERR_UNSUPPORTED;
    int64_t rows, t;
    const bool on[2] = {H > 0, G > 0 && (k || yk)};
    if (!mul_ok(B, N, &rows) || !mul_ok(rows, D, &t) || t >= ((int64_t)1 << 39) || H >= (1 << 20) || G >= (1 << 20) ||
        rotary_plan(rows, D, rot, (int)((on[0] ? H : 0) + (on[1] ? G : 0))).threads > 256 * kMaxWorkgroups)
        return LCONV_ERR_UNSUPPORTED;  // threads of one launch
    if (!inv_freq) return LCONV_ERR_NULL_POINTER;
    if (!mul_ok(B - 1, pos_stride, &t) || t > INT64_MAX / 8 - N) return LCONV_ERR_INVALID_SHAPE;
    const Range rp = buffer(positions, t + N, 4), rf = buffer(inv_freq, rot / 2, 4);
    RotaryArgs a{};
    Range rx[2]{}, ry[2]{};
    lconv_status_t st;
    if (on[0]) {
        if ((st = operand(q, q_strides, B, H, N, D, dtype, false, &a.q.s, &rx[0])) != LCONV_SUCCESS) return st;
        if ((st = operand(yq, yq_strides, B, H, N, D, dtype, true, &a.yqs, &ry[0])) != LCONV_SUCCESS) return st;
    }
    if (on[1]) {
        if ((st = operand(k, k_strides, B, G, N, D, dtype, false, &a.k.s, &rx[1])) != LCONV_SUCCESS) return st;
        if ((st = operand(yk, yk_strides, B, G, N, D, dtype, true, &a.yks, &ry[1])) != LCONV_SUCCESS) return st;
    }
    // an output is apart from everything but, in place, its own input
    const auto same = [](const void* x, const lconv_strides_t& xs, const void* y, const lconv_strides_t& ys) {
        return x == y && xs.b == ys.b && xs.h == ys.h && xs.n == ys.n;
    };
    const bool inplace[2] = {on[0] && same(q, a.q.s, yq, a.yqs), on[1] && same(k, a.k.s, yk, a.yks)};
    for (int i = 0; i < 2; ++i) {
        if (!on[i]) continue;
        if (overlap(ry[i], rp) || overlap(ry[i], rf)) return LCONV_ERR_ALIASING;
        for (int j = 0; j < 2; ++j)
            if (on[j] && ((overlap(ry[i], rx[j]) && !(i == j && inplace[i])) || (j > i && overlap(ry[i], ry[j]))))
                return LCONV_ERR_ALIASING;
    }
    a.q.p = on[0] ? q : nullptr; a.q.share = 1;
    a.k.p = on[1] ? k : nullptr; a.k.share = 1;
    a.yq = yq; a.yk = yk;
    a.positions = positions; a.pos_stride = pos_stride; a.inv_freq = inv_freq; a.magnitude = magnitude;
    a.B = B; a.N = N; a.H = (int)(on[0] ? H : 0); a.G = (int)(on[1] ? G : 0);
    a.D = (int)D; a.rot = (int)rot; a.flags = flags;
    return hip_status(launch_rotary(dtype, a, stream));
}

}  // extern "C"

namespace {

constexpr int64_t kNormMaxC = 65536;

// rows of C elements `stride` apart, from a 16-byte aligned start
lconv_status_t norm_rows(const void* p, int64_t stride, int64_t rows, int64_t C, lconv_dtype_t dt, Range* r) {
    int64_t t;
    if (rows > 1 && (stride < C || !mul_ok(rows - 1, stride, &t) || t > INT64_MAX / 8 - C)) return LCONV_ERR_INVALID_SHAPE;
    if (!p) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(p)) return LCONV_ERR_MISALIGNED;
    const int64_t es = (int64_t)dtype_size(dt);
    *r = Range{p, (size_t)(((rows > 1 ? (rows - 1) * stride : 0) + C) * es), 0, 0};
    if (rows > 1) {
        r->foot = (size_t)(C * es);
        r->step = (size_t)(stride * es);
    }
    return LCONV_SUCCESS;
}

lconv_status_t norm_dims(int64_t rows, int64_t C, lconv_dtype_t dtype) {
    if (!dtype_ok(dtype)) return LCONV_ERR_UNSUPPORTED;
    if (rows < 0 || C < 0) return LCONV_ERR_INVALID_SHAPE;
    if (C > kNormMaxC || rows >= ((int64_t)1 << 31)) return LCONV_ERR_UNSUPPORTED;
    return LCONV_SUCCESS;
}

}  // namespace

extern "C" {

lconv_status_t lconv_layernorm_fwd(const void* x, int64_t x_stride, const void* weight, const void* bias, void* y,
                                   int64_t y_stride, float* mean, float* rstd, int64_t rows, int64_t C, float eps,
                                   lconv_dtype_t dtype, hipStream_t stream) {
    lconv_status_t st = norm_dims(rows, C, dtype);
    if (st != LCONV_SUCCESS) return st;
    if (rows == 0 || C == 0) return LCONV_SUCCESS;
    Range rx, ry;
    if ((st = norm_rows(x, x_stride, rows, C, dtype, &rx)) != LCONV_SUCCESS) return st;
    if ((st = norm_rows(y, y_stride, rows, C, dtype, &ry)) != LCONV_SUCCESS) return st;
    if (!aligned16(weight) || !aligned16(bias) || !aligned16(mean) || !aligned16(rstd)) return LCONV_ERR_MISALIGNED;
    const size_t es = dtype_size(dtype);
    const Range rw = buffer(weight, C, es), rb = buffer(bias, C, es), rm = buffer(mean, rows, 4), rr = buffer(rstd, rows, 4);
    const bool inplace = x == y && (rows == 1 || x_stride == y_stride);
    if ((overlap(ry, rx) && !inplace) || clash({ry, rm, rr}, {rw, rb}) || overlap(rm, rx) || overlap(rr, rx))
        return LCONV_ERR_ALIASING;
    NormArgs a{};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.xs = x_stride; a.ys = y_stride;
    a.mean = mean; a.rstd = rstd; a.rows = rows; a.C = C; a.eps = eps;
    return hip_status(launch_layernorm_fwd(dtype, a, stream));
}

size_t lconv_layernorm_bwd_workspace_bytes(int64_t rows, int64_t C) {
    if (rows <= 0 || C <= 0 || C > kNormMaxC || rows >= ((int64_t)1 << 31)) return 0;
    return (size_t)layernorm_parts(rows, C) * (size_t)C * 8;
}

lconv_status_t lconv_layernorm_bwd(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                   const void* weight, const float* mean, const float* rstd, void* dx,
                                   int64_t dx_stride, float* dweight, float* dbias, int64_t rows, int64_t C,
                                   lconv_dtype_t dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    lconv_status_t st = norm_dims(rows, C, dtype);
    if (st != LCONV_SUCCESS) return st;
    if (C == 0) return LCONV_SUCCESS;
    const size_t es = dtype_size(dtype);
    const Range rw = buffer(weight, C, es), rdw = buffer(dweight, C, 4), rdb = buffer(dbias, C, 4);
    if (!aligned16(weight) || !aligned16(dweight) || !aligned16(dbias)) return LCONV_ERR_MISALIGNED;
    NormArgs a{};
    a.dweight = dweight; a.dbias = dbias; a.C = C;
    if (rows == 0) {
        if (overlap(rdw, rdb)) return LCONV_ERR_ALIASING;
        return hip_status(launch_layernorm_bwd(dtype, a, stream));
    }
    Range rdy, rx, rdx;
    if ((st = norm_rows(dy, dy_stride, rows, C, dtype, &rdy)) != LCONV_SUCCESS) return st;
    if ((st = norm_rows(x, x_stride, rows, C, dtype, &rx)) != LCONV_SUCCESS) return st;
    if ((st = norm_rows(dx, dx_stride, rows, C, dtype, &rdx)) != LCONV_SUCCESS) return st;
    if (!mean || !rstd) return LCONV_ERR_NULL_POINTER;
    if (!aligned16(mean) || !aligned16(rstd)) return LCONV_ERR_MISALIGNED;
    const Range rm = buffer(mean, rows, 4), rr = buffer(rstd, rows, 4);
    if ((overlap(rdx, rdy) && !(dx == dy && (rows == 1 || dx_stride == dy_stride))) ||
        (overlap(rdx, rx) && !(dx == x && (rows == 1 || dx_stride == x_stride))) || overlap(rdx, rw) || overlap(rdx, rm) ||
        overlap(rdx, rr) || clash({rdw, rdb}, {rdy, rx, rdx, rw, rm, rr}))
        return LCONV_ERR_ALIASING;
    if (dweight || dbias) {
        const size_t need = lconv_layernorm_bwd_workspace_bytes(rows, C);
        if (!workspace || workspace_bytes < need) return LCONV_ERR_WORKSPACE;
        if (!aligned16(workspace)) return LCONV_ERR_MISALIGNED;
        if (clash({buffer(workspace, (int64_t)need, 1)}, {rdy, rx, rdx, rw, rm, rr, rdw, rdb})) return LCONV_ERR_ALIASING;
    }
    a.dy = dy; a.x = x; a.weight = weight; a.y = dx; a.dys = dy_stride; a.xs = x_stride; a.ys = dx_stride;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.part = dweight || dbias ? (float*)workspace : nullptr;
    a.rows = rows;
    return hip_status(launch_layernorm_bwd(dtype, a, stream));
}

}  // extern "C"
