"""Refusals of the mixer operators' C ABI and torch wrappers, all on the host before any HIP call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from fft_long_convolution_amd import lconv  # noqa: E402

F32, F16, BF16 = lconv.F32, lconv.F16, lconv.BF16
OK, NULLP, SHAPE, UNSUP, MISAL, ALIAS, WSERR = range(7)
# fake, 16-byte aligned "device" addresses far apart: never touched
A = [0x10000000 * (i + 1) for i in range(20)]


def st(b, h, n):
    return lconv.Strides(b, h, n)


def fwd(q=A[0], k=A[1], v=A[2], ld=A[3], si=None, ln=None, y=A[4], so=None, B=2, H=4, G=2, N=8, Dk=16, Dv=24, dt=BF16,
        qs=None, ks=None, vs=None, ys=None, ws=A[19], wsb=1 << 40):
    return lconv.lconv_linattn_fwd(q, qs, k, ks, v, vs, ld, 1.0, si, ln, y, ys, so, B, H, G, N, Dk, Dv, dt, ws, wsb, None)


def test_linattn_fwd_refusals():
    assert fwd(dt=3) == UNSUP
    for bad in (dict(B=-1), dict(N=-1), dict(Dk=-8), dict(G=-2)):
        assert fwd(**bad) == SHAPE
    for bad in (dict(Dk=12), dict(Dv=264), dict(Dk=0), dict(G=3), dict(G=0), dict(N=2 ** 31), dict(B=2 ** 26)):
        assert fwd(**bad) == UNSUP
    for name in ("q", "k", "v", "ld", "y"):
        assert fwd(**{name: None}) == NULLP
    for bad in (dict(q=A[0] + 8), dict(y=A[4] + 2), dict(si=A[5] + 4), dict(so=A[6] + 8)):
        assert fwd(**bad) == MISAL
    assert fwd(qs=st(512, 128, 20)) == MISAL and fwd(qs=st(512, 130, 16)) == MISAL
    assert fwd(ks=st(512, -128, 16)) == SHAPE
    assert fwd(vs=st(2 ** 62, 2 ** 62, 2 ** 62)) == SHAPE
    # an output whose rows meet: a zero stride, tokens inside one another, heads inside the tokens
    assert fwd(ys=st(0, 24 * 8, 24)) == SHAPE
    assert fwd(ys=st(1024, 24 * 8, 16)) == SHAPE
    assert fwd(ys=st(4096, 32, 64)) == SHAPE
    assert fwd(y=A[0]) == ALIAS and fwd(y=A[2] + 64) == ALIAS and fwd(so=A[1]) == ALIAS
    assert fwd(si=A[5], y=A[5]) == ALIAS and fwd(so=A[4]) == ALIAS and fwd(si=A[5], so=A[5] + 64) == ALIAS
    assert fwd(ln=A[4] + 16) == ALIAS


@pytest.mark.parametrize("dt,size", [(F32, 4), (F16, 2), (BF16, 2)])
def test_linattn_refuses_tokens_too_far_apart(dt, size):
    """Offsets within 32 tokens are 32-bit: token strides past 2^27 bytes are refused, and only for N > 1."""
    far = 2 ** 27 // size + 16 // size
    big = [1 << 44, 1 << 45, 1 << 46, 1 << 47]
    for name in ("qs", "ks", "vs", "ys"):
        s = st(8 * 8 * far, 8 * far, far)
        assert fwd(q=big[0], k=big[1], v=big[2], y=big[3], dt=dt, **{name: s}) == UNSUP
    assert bwd(dq=big[3], dt=dt, dqs=st(8 * 8 * far, 8 * far, far)) == UNSUP
    # the limit itself passes on to the next check
    s = st(8 * 8 * (far - 16 // size), 8 * (far - 16 // size), far - 16 // size)
    assert fwd(q=big[0], dt=dt, qs=s, ld=None) == NULLP
    assert fwd(q=big[0], dt=dt, N=1, qs=st(4 * far, far, far), ld=None) == NULLP


def test_linattn_slices_of_one_buffer_do_not_alias():
    """y between q and k in a token-major buffer is apart; one that meets q's columns is not."""
    B, H, N, D = 2, 4, 8, 16
    row = 3 * H * D
    s = lambda: st(N * row, D, row)  # noqa: E731
    need = lconv.lconv_linattn_workspace_bytes(B, H, H, N, D, D, BF16)
    call = lambda off: lconv.lconv_linattn_fwd(A[0], s(), A[1], None, A[2], None, A[3], 1.0, None, None,  # noqa: E731
                                               A[0] + off, s(), None, B, H, H, N, D, D, BF16, None if need else A[19],
                                               0, None)
    fine = WSERR if need else lconv.lconv_linattn_workspace_bytes(B, H, H, N, D, D, BF16)
    assert call(0) == ALIAS and call(2 * (H * D - 8)) == ALIAS and call(2 * (2 * H * D + 16)) == ALIAS
    # an acceptable call would launch: only checked where it stops at the missing workspace, or on a host
    # without a device
    if not torch.cuda.is_available():
        assert call(2 * H * D) in (fine, 7) and call(2 * 2 * H * D) in (fine, 7)


def bwd(dy=A[0], q=A[1], k=A[2], v=A[3], ld=A[4], si=None, ds=None, ln=None, dq=A[5], dk=A[6], dv=A[7], dsi=None, dl=None,
        B=2, H=4, G=2, N=8, Dk=16, Dv=24, dt=BF16, dqs=None, ws=A[19], wsb=1 << 40):
    return lconv.lconv_linattn_bwd(dy, None, q, None, k, None, v, None, ld, 1.0, si, ds, ln, dq, dqs, dk, None, dv, None,
                                   dsi, dl, B, H, G, N, Dk, Dv, dt, ws, wsb, None)


def test_linattn_bwd_refusals():
    assert bwd(dt=-1) == UNSUP and bwd(G=3) == UNSUP and bwd(Dv=20) == UNSUP
    assert bwd(N=-2) == SHAPE
    for name in ("dy", "q", "k", "v", "ld", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == NULLP
    assert bwd(dk=A[6] + 8) == MISAL and bwd(dsi=A[8] + 4) == MISAL
    assert bwd(dqs=st(0, 0, 0)) == SHAPE
    for bad in (dict(dq=A[1]), dict(dk=A[5]), dict(dv=A[0]), dict(si=A[8], dsi=A[8]), dict(ds=A[8], dsi=A[8]), dict(dl=A[4]),
                dict(dsi=A[5])):
        assert bwd(**bad) == ALIAS
    need = lconv.lconv_linattn_bwd_workspace_bytes(2, 4, 2, 8, 16, 24, BF16)
    assert need > 0
    assert bwd(ws=None) == WSERR and bwd(wsb=need - 1) == WSERR and bwd(ws=A[19] + 8) == MISAL
    assert bwd(ws=A[5]) == ALIAS
    assert lconv.lconv_linattn_bwd_workspace_bytes(2, 4, 3, 8, 16, 24, BF16) == 0


def step(q=A[0], k=A[1], v=A[2], ld=A[3], s=A[4], sl=None, y=A[5], B=2, H=4, G=2, Dk=16, Dv=24, ns=2, dt=BF16, qs=None):
    return lconv.lconv_linattn_step(q, qs, k, None, v, None, ld, 1.0, s, sl, y, None, B, H, G, Dk, Dv, ns, dt, None)


def test_linattn_step_refusals():
    assert step(dt=4) == UNSUP and step(G=3) == UNSUP and step(Dk=4) == UNSUP
    assert step(ns=1) == SHAPE and step(ns=-1) == SHAPE and step(B=-1) == SHAPE
    for name in ("q", "k", "v", "ld", "s", "y"):
        assert step(**{name: None}) == NULLP
    assert step(s=A[4] + 8) == MISAL and step(qs=st(20, 16, 0)) == MISAL
    assert step(y=A[4]) == ALIAS and step(s=A[0]) == ALIAS and step(sl=A[4] + 16) == ALIAS


def rot(q=A[0], k=A[1], p=A[2], ps=8, f=A[3], yq=A[4], yk=A[5], B=2, H=4, G=2, N=8, D=32, r=16, fl=0, dt=BF16, qs=None, yqs=None):
    return lconv.lconv_rotary(q, qs, k, None, p, ps, f, 1.0, yq, yqs, yk, None, B, H, G, N, D, r, fl, dt, None)


def test_rotary_refusals():
    assert rot(dt=9) == UNSUP
    for bad in (dict(D=12), dict(D=1032, r=2), dict(r=15), dict(r=34), dict(r=0), dict(fl=4)):
        assert rot(**bad) == UNSUP
    assert rot(N=-1) == SHAPE and rot(ps=-1) == SHAPE
    for name in ("q", "f", "yq", "k", "yk"):
        assert rot(**{name: None}) == NULLP
    assert rot(q=A[0] + 8) == MISAL
    assert rot(yq=A[1]) == ALIAS and rot(yq=A[0] + 16) == ALIAS and rot(yk=A[4]) == ALIAS and rot(yq=A[3]) == ALIAS
    assert rot(yq=A[2]) == ALIAS
    # in place with other strides is not in place
    assert rot(yq=A[0], yqs=st(8 * 4 * 32, 32, 4 * 32)) == ALIAS


def nf(x=A[0], xs=40, w=A[1], b=A[2], y=A[3], ys=40, m=A[4], r=A[5], rows=6, C=40, dt=BF16):
    return lconv.lconv_layernorm_fwd(x, xs, w, b, y, ys, m, r, rows, C, 1e-5, dt, None)


def nb(dy=A[0], dys=40, x=A[1], xs=40, w=A[2], m=A[3], r=A[4], dx=A[5], dxs=40, dw=A[6], db=A[7], rows=6, C=40, dt=BF16,
       ws=A[8], wsb=1 << 40):
    return lconv.lconv_layernorm_bwd(dy, dys, x, xs, w, m, r, dx, dxs, dw, db, rows, C, dt, ws, wsb, None)


def test_layernorm_refusals():
    assert nf(dt=5) == UNSUP and nf(C=65537, xs=65537, ys=65537) == UNSUP and nf(rows=2 ** 31) == UNSUP
    assert nf(rows=-1) == SHAPE and nf(xs=39) == SHAPE and nf(ys=0) == SHAPE
    assert nf(x=None) == NULLP and nf(y=None) == NULLP
    assert nf(x=A[0] + 2) == MISAL and nf(w=A[1] + 4) == MISAL and nf(m=A[4] + 4) == MISAL
    assert nf(y=A[0] + 16) == ALIAS and nf(y=A[1]) == ALIAS and nf(m=A[0]) == ALIAS and nf(r=A[4]) == ALIAS
    assert nf(y=A[0], ys=48) == ALIAS
    assert nb(dt=5) == UNSUP and nb(dxs=39) == SHAPE
    for name in ("dy", "x", "m", "r", "dx"):
        assert nb(**{name: None}) == NULLP
    assert nb(dw=A[6] + 4) == MISAL
    assert nb(dx=A[2]) == ALIAS and nb(dw=A[5]) == ALIAS and nb(db=A[6]) == ALIAS and nb(dx=A[0] + 16) == ALIAS
    need = lconv.lconv_layernorm_bwd_workspace_bytes(6, 40)
    assert need > 0 and nb(ws=None) == WSERR and nb(wsb=need - 1) == WSERR and nb(ws=A[6]) == ALIAS
    assert lconv.lconv_layernorm_bwd_workspace_bytes(0, 40) == 0


def test_empty_calls_need_no_pointers():
    assert fwd(B=0, q=None) == OK and fwd(H=0, G=0, q=None) == OK and fwd(N=0, q=None, y=None) == OK
    assert bwd(B=0, q=None) == OK and bwd(N=0, dq=None) == OK
    assert step(B=0, q=None, ns=0, s=None) == OK
    assert rot(B=0, q=None) == OK and rot(N=0, yq=None) == OK
    assert nf(rows=0, x=None) == OK and nf(C=0, xs=0, ys=0, x=None) == OK


def raises(match, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **kw)


def test_wrapper_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    q, k, v, ld = z(2, 4, 8, 16), z(2, 2, 8, 16), z(2, 2, 8, 24), z(4, dt=torch.float32)
    f = lconv.linear_attention
    raises("GPU tensor", f, q, k, v, ld)
    raises("4-D", f, q[0], k, v, ld)
    raises("dtype", f, q.double(), k, v, ld)
    raises("dtype", f, q, k.float(), v, ld)
    raises("shape", f, q, k, v[:, :, :7], ld)
    raises("multiple", f, z(2, 3, 8, 16), k, v, z(3, dt=torch.float32))
    raises("dtype", f, q, k, v, ld.bfloat16())
    raises("last dimension", f, q.transpose(2, 3).contiguous().transpose(2, 3), k, v, ld)
    raises("state has shape", f, q, k, v, ld, state=z(2, 4, 16, 16, dt=torch.float32))
    raises("state has dtype", f, q, k, v, ld, state=z(2, 4, 16, 24))
    raises("lengths", f, q, k, v, ld, lengths=torch.zeros(2, dtype=torch.int64))
    raises("GPU tensor", lconv.linear_attention_bwd, z(2, 4, 8, 24), q, k, v, ld)
    raises("dy has shape", lconv.linear_attention_bwd, z(2, 4, 8, 16), q, k, v, ld)
    s = z(2, 4, 16, 24, dt=torch.float32)
    g = lconv.linear_attention_step
    raises("GPU tensor", g, q[:, :, 0], k[:, :, 0], v[:, :, 0], ld, s)
    raises("slots are needed", g, q[:, :, 0], k[:, :, 0], v[:, :, 0], ld, s[:1])
    raises("state must", g, q[:, :, 0], k[:, :, 0], v[:, :, 0], ld, s[0])
    inv = z(8, dt=torch.float32)
    raises("GPU tensor", lconv.rotary, q, k, None, inv)
    raises("int32", lconv.rotary, q, k, torch.zeros(2, 8, dtype=torch.int64), inv)
    raises("positions has shape", lconv.rotary, q, k, torch.zeros(8, 2, dtype=torch.int32), inv)
    raises("dtype", lconv.rotary, q, k, None, inv.double())
    raises("without k", lconv.rotary, q, None, None, inv, out=(q, k))
    raises("even", lconv.rotary_frequencies, 7)
    raises("unknown scaling", lconv.rotary_frequencies, 8, scaling="other")
    x = z(6, 40)
    raises("GPU tensor", lconv.layer_norm, x)
    raises("weight has shape", lconv.layer_norm, x, z(41))
    raises("contiguous", lconv.layer_norm, z(40, 6).t())
    raises("dtype", lconv.layer_norm, x.double())
    raises("mean has shape", lconv.layer_norm_bwd, x, x, None, z(5, dt=torch.float32), z(6, dt=torch.float32))


def test_strides_struct_is_three_int64():
    assert ctypes.sizeof(lconv.Strides) == 24
