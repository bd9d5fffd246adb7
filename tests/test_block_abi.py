"""Refusals of the C ABI and torch wrappers of the gated recurrence, the q/k norms and the short convolution, all on the host
before any HIP call."""
import pytest

torch = pytest.importorskip("torch")

from fft_long_convolution_amd import lconv  # noqa: E402

F32, F16, BF16 = lconv.F32, lconv.F16, lconv.BF16
OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, WSERR = range(7)
# fake, 16-byte aligned "device" addresses far apart: never touched
A = [0x10000000 * (i + 1) for i in range(24)]


def st(b, n):
    return lconv.Strides(b, 0, n)


def sf(x=A[0], z=A[1], g=None, r=A[3], si=None, ln=None, y=A[4], so=None, m=None, B=2, N=8, C=12, fl=2 | 8, dt=BF16, xs=None, ys=None,
       ws=A[19], wsb=1 << 40):
    return lconv.lconv_gated_scan_fwd(x, xs, z, None, g, None, r, si, ln, y, ys, so, m, B, N, C, fl, dt, ws, wsb, None)


def sb(dy=A[0], x=A[1], z=A[2], g=None, r=A[3], m=A[4], ds=None, ln=None, dx=A[5], dz=A[6], dg=None, dr=A[7], dsi=None, B=2, N=8, C=12,
       fl=2 | 8, dt=BF16, ws=A[19], wsb=1 << 40, dxs=None):
    return lconv.lconv_gated_scan_bwd(dy, None, x, None, z, None, g, None, r, m, ds, ln, dx, dxs, dz, None, dg, None, dr, dsi, B, N, C,
                                      fl, dt, ws, wsb, None)


def ss(x=A[0], xst=12, z=A[1], g=None, r=A[2], s=A[3], sl=None, y=A[4], yst=12, B=2, C=12, ns=2, fl=2, dt=BF16):
    return lconv.lconv_gated_scan_step(x, xst, z, 12, g, 12, r, s, sl, y, yst, B, C, ns, fl, dt, None)


def test_scan_refusals():
    assert sf(dt=3) == UNSUP and sf(fl=3) == UNSUP and sf(fl=12) == UNSUP and sf(fl=16) == UNSUP and sf(fl=-1) == UNSUP
    for bad in (dict(B=-1), dict(N=-1), dict(C=-8)):
        assert sf(**bad) == SHAPE
    assert sf(N=2 ** 31) == UNSUP and sf(C=2 ** 24 + 1) == UNSUP and sf(B=2 ** 24, C=2 ** 20) == UNSUP
    for name in ("x", "z", "r", "y"):
        assert sf(**{name: None}) == NULLP
    assert sf(x=A[0] + 1) == MISAL and sf(dt=F32, y=A[4] + 2) == MISAL
    for bad in (dict(si=A[5] + 4), dict(so=A[6] + 8), dict(m=A[7] + 8), dict(r=A[3] + 4)):
        assert sf(**bad) == MISAL
    assert sf(xs=st(-96, 12)) == SHAPE and sf(xs=st(2 ** 62, 2 ** 62)) == SHAPE
    # an output whose rows meet: tokens inside one another, batch rows inside the tokens
    assert sf(ys=st(96, 11)) == SHAPE and sf(ys=st(12, 12)) == SHAPE and sf(ys=st(0, 12)) == SHAPE and sf(ys=st(90, 12)) == SHAPE
    for bad in (dict(y=A[0]), dict(y=A[1] + 16), dict(so=A[1]), dict(m=A[0]), dict(si=A[5], y=A[5]), dict(si=A[5], so=A[5] + 16),
                dict(si=A[5], m=A[5]), dict(g=A[4]), dict(ln=A[4] + 16), dict(so=A[3]), dict(so=A[4]), dict(m=A[4] + 16)):
        assert sf(**bad) == ALIAS, bad
    need = lconv.lconv_gated_scan_workspace_bytes(1, 4096, 12, BF16)
    assert need > 0 and lconv.lconv_gated_scan_workspace_bytes(8, 8, 12, BF16) == 0
    big = dict(B=1, N=4096)
    assert sf(ws=None, **big) == WSERR and sf(wsb=need - 1, **big) == WSERR and sf(ws=A[19] + 8, **big) == MISAL
    assert sf(ws=A[4], **big) == ALIAS
    assert lconv.lconv_gated_scan_workspace_bytes(1, 4096, 12, 7) == 0 and lconv.lconv_gated_scan_marks_bytes(2, 65, 12) == 2 * 2 * 12 * 4


def test_scan_bwd_refusals():
    assert sb(dt=-1) == UNSUP and sb(fl=3) == UNSUP and sb(N=-2) == SHAPE
    for name in ("dy", "x", "z", "r", "m", "dx", "dz"):
        assert sb(**{name: None}) == NULLP
    assert sb(g=A[8]) == NULLP                                       # a gate without a place for its gradient
    assert sb(dr=A[7] + 4) == MISAL and sb(dsi=A[9] + 8) == MISAL and sb(dxs=st(0, 0)) == SHAPE
    for bad in (dict(dx=A[1]), dict(dz=A[5]), dict(dr=A[3]), dict(dsi=A[4]), dict(g=A[8], dg=A[8]), dict(dx=A[4]), dict(dz=A[0] + 16),
                dict(ds=A[9], dx=A[9]), dict(ds=A[9], dsi=A[9] + 16), dict(dr=A[9], ds=A[9])):
        assert sb(**bad) == ALIAS, bad
    need = lconv.lconv_gated_scan_bwd_workspace_bytes(2, 8, 12, 2, BF16)
    assert need > 0 and lconv.lconv_gated_scan_bwd_workspace_bytes(2, 8, 12, 1, BF16) == 0
    assert sb(ws=None) == WSERR and sb(wsb=need - 1) == WSERR and sb(ws=A[5]) == ALIAS
    assert lconv.lconv_gated_scan_bwd_workspace_bytes(2, 8, 12, 3, BF16) == 0


def test_scan_step_refusals():
    assert ss(dt=4) == UNSUP and ss(fl=3) == UNSUP and ss(B=-1) == SHAPE and ss(ns=1) == SHAPE and ss(ns=-1) == SHAPE and ss(yst=11) == SHAPE
    for name in ("x", "z", "r", "s", "y"):
        assert ss(**{name: None}) == NULLP
    assert ss(s=A[3] + 8) == MISAL and ss(x=A[0] + 1) == MISAL
    assert ss(y=A[3]) == ALIAS and ss(s=A[0]) == ALIAS and ss(sl=A[3] + 16) == ALIAS and ss(g=A[4]) == ALIAS


def qf(q=A[0], k=A[1], wq=A[2], wk=A[3], p=A[4], ps=8, f=A[5], yq=A[6], yk=A[7], B=2, H=4, G=2, N=8, D=32, r=16, fl=0, dt=BF16, qs=None,
       yqs=None):
    return lconv.lconv_qknorm_rotary_fwd(q, qs, k, None, wq, wk, p, ps, f, 1.0, 1e-6, yq, yqs, yk, None, B, H, G, N, D, r, fl, dt, None)


def qb(dq=A[0], dk=A[1], q=A[2], k=A[3], wq=A[4], wk=A[5], p=A[6], f=A[7], oq=A[8], ok=A[9], gq=A[10], gk=A[11], B=2, H=4, G=2, N=8, D=32,
       r=16, fl=0, dt=BF16, ws=A[19], wsb=1 << 40):
    return lconv.lconv_qknorm_rotary_bwd(dq, None, dk, None, q, None, k, None, wq, wk, p, 8, f, 1.0, 1e-6, oq, None, ok, None, gq, gk, B, H,
                                         G, N, D, r, fl, dt, ws, wsb, None)


def test_qknorm_refusals():
    assert qf(dt=9) == UNSUP
    for bad in (dict(D=12), dict(D=520, r=2), dict(r=15), dict(r=34), dict(fl=2), dict(fl=8), dict(B=2 ** 20, N=2 ** 12)):
        assert qf(**bad) == UNSUP, bad
    assert qf(N=-1) == SHAPE and qf(ps=-1) == SHAPE and qf(r=-2) == SHAPE
    for name in ("q", "f", "yq", "k", "yk"):
        assert qf(**{name: None}) == NULLP
    assert qf(q=A[0] + 8) == MISAL and qf(wq=A[2] + 2) == MISAL
    assert qf(qs=lconv.Strides(1024, 32, 130)) == MISAL
    for bad in (dict(yq=A[1]), dict(yq=A[0] + 16), dict(yk=A[6]), dict(yq=A[5]), dict(yq=A[4]), dict(yk=A[2]),
                dict(yq=A[0], yqs=lconv.Strides(8 * 4 * 32, 32, 4 * 32))):
        assert qf(**bad) == ALIAS, bad
    assert qb(dt=9) == UNSUP and qb(D=12) == UNSUP and qb(H=-1) == SHAPE
    for name in ("dq", "dk", "q", "k", "f", "oq", "ok"):
        assert qb(**{name: None}) == NULLP
    assert qb(gq=A[10] + 4) == MISAL
    for bad in (dict(oq=A[0]), dict(oq=A[2]), dict(ok=A[8]), dict(gq=A[11]), dict(gk=A[8]), dict(gq=A[4])):
        assert qb(**bad) == ALIAS, bad
    need = lconv.lconv_qknorm_rotary_bwd_workspace_bytes(2, 4, 2, 8, 32, 16)
    assert need > 0 and qb(ws=None) == WSERR and qb(wsb=need - 1) == WSERR and qb(ws=A[19] + 8) == MISAL and qb(ws=A[8]) == ALIAS
    assert lconv.lconv_qknorm_rotary_bwd_workspace_bytes(2, 4, 2, 8, 33, 16) == 0


def cf(x=A[0], w=A[1], b=A[2], si=None, ln=None, y=A[3], so=None, B=2, N=8, C=12, K=4, fl=0, dt=BF16, ys=None):
    return lconv.lconv_shortconv_fwd(x, None, w, b, si, ln, y, ys, so, B, N, C, K, fl, dt, None)


def cb(dy=A[0], x=A[1], w=A[2], b=A[3], si=None, ds=None, ln=None, dx=A[4], dw=A[5], db=A[6], dsi=None, B=2, N=8, C=12, K=4, fl=0, dt=BF16,
       ws=A[19], wsb=1 << 40):
    return lconv.lconv_shortconv_bwd(dy, None, x, None, w, b, si, ds, ln, dx, None, dw, db, dsi, B, N, C, K, fl, dt, ws, wsb, None)


def cs(x=A[0], w=A[1], b=A[2], s=A[3], sl=None, y=A[4], yst=12, B=2, C=12, K=4, ns=2, fl=0, dt=BF16):
    return lconv.lconv_shortconv_step(x, 12, w, b, s, sl, y, yst, B, C, K, ns, fl, dt, None)


def test_shortconv_refusals():
    for bad in (dict(dt=3), dict(fl=2), dict(K=1), dict(K=9), dict(N=2 ** 31), dict(C=2 ** 24 + 1)):
        assert cf(**bad) == UNSUP, bad
    assert cf(N=-1) == SHAPE and cf(K=-1) == SHAPE and cf(ys=st(96, 11)) == SHAPE
    for name in ("x", "w", "y"):
        assert cf(**{name: None}) == NULLP
    assert cf(x=A[0] + 1) == MISAL and cf(w=A[1] + 2) == MISAL and cf(si=A[5] + 2) == MISAL
    for bad in (dict(y=A[0]), dict(y=A[1]), dict(so=A[0]), dict(si=A[5], so=A[5] + 16), dict(si=A[5], y=A[5]), dict(so=A[3]), dict(ln=A[3])):
        assert cf(**bad) == ALIAS, bad
    assert cb(dt=3) == UNSUP and cb(K=9) == UNSUP and cb(C=-1) == SHAPE
    for name in ("dy", "x", "w", "dx"):
        assert cb(**{name: None}) == NULLP
    for bad in (dict(dx=A[0]), dict(dx=A[1] + 16), dict(dw=A[6]), dict(dw=A[2]), dict(ds=A[7], dsi=A[7]), dict(si=A[7], dsi=A[7]), dict(db=A[4])):
        assert cb(**bad) == ALIAS, bad
    need = lconv.lconv_shortconv_bwd_workspace_bytes(2, 8, 12, 4)
    assert need > 0 and cb(ws=None) == WSERR and cb(wsb=need - 1) == WSERR and cb(ws=A[4]) == ALIAS
    assert lconv.lconv_shortconv_bwd_workspace_bytes(2, 8, 12, 9) == 0
    assert cs(dt=3) == UNSUP and cs(K=1) == UNSUP and cs(ns=1) == SHAPE and cs(yst=11) == SHAPE
    for name in ("x", "w", "s", "y"):
        assert cs(**{name: None}) == NULLP
    assert cs(s=A[3] + 2) == MISAL and cs(y=A[3]) == ALIAS and cs(s=A[1]) == ALIAS and cs(sl=A[3]) == ALIAS


def test_empty_calls_need_no_pointers():
    assert sf(B=0, x=None) == OK and sf(C=0, x=None) == OK and sf(N=0, x=None, y=None) == OK
    assert sb(C=0, x=None) == OK and sb(B=0, x=None, dr=None) == OK and sb(N=0, dx=None, dr=None) == OK
    assert ss(B=0, x=None, ns=0, s=None) == OK
    assert qf(B=0, q=None) == OK and qf(N=0, yq=None) == OK and qf(H=0, G=0, q=None) == OK
    assert qb(B=0, q=None, gq=None, gk=None) == OK
    assert cf(B=0, x=None) == OK and cf(N=0, x=None, y=None) == OK
    assert cb(C=0, x=None) == OK and cb(N=0, x=None, dw=None, db=None) == OK
    assert cs(B=0, x=None, ns=0, s=None) == OK


def test_slices_of_one_buffer_do_not_alias():
    """y beside x in a token-major buffer is apart; one that meets its columns is not.  (An acceptable call would launch: only on a
    host without a device.)"""
    row = 3 * 16
    call = lambda off: lconv.lconv_gated_scan_fwd(A[0], st(8 * row, row), A[1], None, None, None, None, None, None,  # noqa: E731
                                                  A[0] + 2 * off, st(8 * row, row), None, None, 2, 8, 16, 1, BF16, None, 0, None)
    assert call(0) == ALIAS and call(15) == ALIAS and call(40) == ALIAS
    if not torch.cuda.is_available():
        assert call(16) in (OK, 7) and call(32) in (OK, 7)


def raises(match, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **kw)


def test_wrapper_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    x, f = z(2, 8, 12), lconv.gated_scan
    rate = z(12, dt=torch.float32)
    raises("GPU tensor", f, x, x)
    raises("3-D", f, x[0], x[0])
    raises("dtype", f, x.double(), x.double())
    raises("dtype", f, x, x.float())
    raises("shape", f, x, x[:, :7])
    raises("unknown gate", f, x, x, "tanh")
    raises("unknown gate", f, x, x, "log", "other")
    raises("rate goes with", f, x, x, "rate")
    raises("rate goes with", f, x, x, "log", rate=rate)
    raises("rate has dtype", f, x, x, "rate", rate=z(12))
    raises("last dimension", f, x, z(2, 12, 8).transpose(1, 2))
    raises("state has shape", f, x, x, state=z(2, 11, dt=torch.float32))
    raises("state has dtype", f, x, x, state=z(2, 12))
    raises("lengths", f, x, x, lengths=torch.zeros(2, dtype=torch.int64))
    raises("input_gate has shape", f, x, x, input_gate=x[:1])
    raises("marks has shape", lconv.gated_scan_bwd, x, x, x, z(3, dt=torch.float32))
    raises("dy has shape", lconv.gated_scan_bwd, x[:1], x, x, z(24, dt=torch.float32))
    g = lconv.gated_scan_step
    raises("GPU tensor", g, x[:, 0], x[:, 0], z(2, 12, dt=torch.float32))
    raises("slots are needed", g, x[:, 0], x[:, 0], z(1, 12, dt=torch.float32))
    raises("state must", g, x[:, 0], x[:, 0], z(2, dt=torch.float32))
    raises("2-D", g, x, x, z(2, 12, dt=torch.float32))

    q, k, w, inv = z(2, 4, 8, 16), z(2, 2, 8, 16), z(16), z(8, dt=torch.float32)
    n = lconv.qk_norm_rotary
    raises("GPU tensor", n, q, k, w, w, None, inv)
    raises("q_weight has shape", n, q, k, z(8), w, None, inv)
    raises("k_weight has dtype", n, q, k, w, w.float(), None, inv)
    raises("without k", n, q, None, w, w, None, inv)
    raises("without k", n, q, None, w, None, None, inv, out=(q, k))
    raises("int32", n, q, k, w, w, torch.zeros(2, 8, dtype=torch.int64), inv)
    raises("positions has shape", n, q, k, w, w, torch.zeros(8, 2, dtype=torch.int32), inv)
    raises("dtype", n, q, k, w, w, None, inv.double())
    raises("goes with k", lconv.qk_norm_rotary_bwd, q, None, q, k, w, w, None, inv)
    raises("dyq has shape", lconv.qk_norm_rotary_bwd, k, k, q, k, w, w, None, inv)

    c, wt = lconv.short_conv, z(12, 4)
    raises("GPU tensor", c, x, wt)
    raises("weight has shape", c, x, z(11, 4))
    raises("taps", c, x, z(12, 9))
    raises("taps", c, x, z(12, 1))
    raises("2-D", c, x, z(12))
    raises("unknown activation", c, x, wt, activation="gelu")
    raises("bias has shape", c, x, wt, z(11))
    raises("state has shape", c, x, wt, state=z(2, 4, 12))
    raises("state has dtype", c, x, wt, state=z(2, 3, 12, dt=torch.float32))
    raises("dy has dtype", lconv.short_conv_bwd, x.float(), x, wt)
    raises("slots are needed", lconv.short_conv_step, x[:, 0], wt, z(1, 3, 12))
    raises("state has shape", lconv.short_conv_step, x[:, 0], wt, z(2, 2, 12))
