"""The operators around the scan without a GPU: invalid requests are rejected on the host before any
HIP call, by the C ABI (placeholder addresses, never dereferenced) and by the binding (shapes, types
and strides of CPU tensors)."""

import ctypes

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block, libssd

OK, INVALID, UNSUPPORTED, NO_DEVICE = 0, 1, 2, 3
BASE, SPAN = 1 << 40, 1 << 34

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="placeholder-pointer checks run only without a visible GPU")


def addr(i, extra=0):
    return BASE + i * SPAN + extra


def tokens(**kw):
    t = dict(batch=2, seqlen=50, channels=64, nseq=2, seq_starts=None, io_dtype=1, reserved=0)
    t.update(kw)
    return block.SSDTokens(*(t[n] for n, _ in block.SSDTokens._fields_))


PACKED = dict(batch=1, nseq=3, seq_starts=addr(60))


def ptr3(*p):
    return (ctypes.c_void_p * 3)(*p)


def len3(*n):
    return (ctypes.c_int64 * 3)(*n)


class Conv:
    """A valid call of ssd_conv, ssd_conv_step or ssd_conv_backward, with fields to spoil."""

    def __init__(self, **kw):
        self.t = tokens()
        self.x, self.xs, self.w, self.b, self.width, self.silu = addr(0), 0, addr(1), addr(2), 4, 1
        self.init, self.fin = addr(3), addr(4)
        self.y, self.split = [addr(5), addr(6), addr(7)], [48, 8, 8]
        self.dy_dtype, self.df, self.dx, self.dw, self.db = 1, addr(8), addr(9), addr(10), addr(11)
        self.di, self.ws, self.n = addr(12), addr(13), 1 << 30
        self.__dict__.update(kw)

    def forward(self):
        return block._function("ssd_conv")(
            ctypes.byref(self.t), self.x, self.xs, self.w, self.b, self.width, self.silu,
            self.init, ptr3(*self.y), len3(*self.split), self.fin, None)

    def step(self):
        return block._function("ssd_conv_step")(
            ctypes.byref(self.t), self.x, self.xs, self.w, self.b, self.width, self.silu,
            self.init, self.fin, ptr3(*self.y), len3(*self.split), None)

    def backward(self):
        return block._function("ssd_conv_backward")(
            ctypes.byref(self.t), self.x, self.xs, self.w, self.b, self.width, self.silu,
            self.init, ptr3(*self.y), len3(*self.split), self.dy_dtype, self.df, self.dx, self.dw,
            self.db, self.di, self.ws, self.n, None)


def one(**kw):
    return tokens(seqlen=1, **kw)


@no_gpu
def test_conv_valid_requests_report_no_device():
    assert Conv().forward() == Conv().backward() == NO_DEVICE
    assert Conv(t=tokens(**PACKED)).forward() == Conv(t=tokens(**PACKED)).backward() == NO_DEVICE
    assert Conv(t=one()).step() == NO_DEVICE
    assert Conv(t=one(), fin=addr(3)).step() == NO_DEVICE  # in place
    assert Conv(b=None, init=None, fin=None, xs=128).forward() == NO_DEVICE
    assert Conv(b=None, init=None, df=None, db=None, di=None, dy_dtype=0).backward() == NO_DEVICE
    assert Conv(y=[addr(5), None, None], split=[64, 0, 0]).forward() == NO_DEVICE


@no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(t=tokens(batch=0)), INVALID), (dict(t=tokens(seqlen=0)), INVALID),
    (dict(t=tokens(channels=0)), INVALID), (dict(t=tokens(nseq=3)), INVALID),
    (dict(t=tokens(io_dtype=2)), INVALID), (dict(t=tokens(reserved=1)), INVALID),
    (dict(t=tokens(batch=2, nseq=2, seq_starts=addr(60))), INVALID),
    (dict(t=tokens(batch=1, nseq=0, seq_starts=addr(60))), INVALID),
    (dict(t=tokens(batch=1, nseq=3, seq_starts=addr(60, 2))), INVALID),
    (dict(t=tokens(channels=60), split=[44, 8, 8]), UNSUPPORTED),
    (dict(t=tokens(batch=1 << 20, seqlen=1 << 12, nseq=1 << 20)), UNSUPPORTED),
    (dict(width=0), INVALID), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x=addr(0, 8)), INVALID),
    (dict(w=addr(1, 4)), INVALID), (dict(b=addr(2, 4)), INVALID), (dict(init=addr(3, 8)), INVALID),
    (dict(xs=56), INVALID), (dict(xs=68), INVALID), (dict(xs=-64), INVALID),
    (dict(split=[48, 8, 0]), INVALID), (dict(split=[40, 8, 8]), INVALID),
    (dict(split=[44, 12, 8]), INVALID), (dict(split=[72, -8, 0]), INVALID),
    (dict(y=[addr(5), addr(6), None]), INVALID), (dict(y=[addr(5), addr(6, 8), addr(7)]), INVALID),
    (dict(y=[addr(0), addr(6), addr(7)]), INVALID), (dict(y=[addr(5), addr(5, 64), addr(7)]), INVALID),
    (dict(fin=addr(3)), INVALID), (dict(fin=addr(5)), INVALID), (dict(fin=addr(4, 4)), INVALID),
])
def test_conv_rejects(kw, status):
    assert Conv(**kw).forward() == status


@no_gpu
@pytest.mark.parametrize("kw", [dict(t=tokens()), dict(t=one(), init=None), dict(t=one(), fin=None),
                                dict(t=tokens(**{**PACKED, "seqlen": 1})),
                                dict(t=one(), fin=addr(3, 64)), dict(t=one(), fin=addr(5))])
def test_conv_step_rejects(kw):
    assert Conv(**kw).step() == INVALID


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(dx=None), dict(dw=None), dict(dx=addr(0)), dict(dx=addr(5)), dict(dw=addr(1)),
    dict(db=addr(10)), dict(di=addr(8)), dict(dy_dtype=3), dict(t=tokens(io_dtype=0)),
    dict(ws=None), dict(n=16), dict(ws=addr(13, 8)), dict(ws=addr(9)), dict(df=addr(8, 4))])
def test_conv_backward_rejects(kw):
    assert Conv(**kw).backward() == INVALID


class Selective:
    def __init__(self, **kw):
        self.t = tokens()
        self.q = dict(dstate=16, ngroups=2, x=addr(0), dt=addr(1), B=addr(2), C=addr(3), z=addr(4),
                      x_stride=0, dt_stride=0, b_stride=0, c_stride=0, z_stride=0, A=addr(5),
                      D=addr(6), dt_bias=addr(7), initial_state=addr(8), dt_softplus=1, reserved=0)
        self.y, self.fin, self.dy, self.df, self.ws, self.n = (addr(9), addr(10), addr(11),
                                                               addr(12), addr(13), 1 << 33)
        self.g = dict(dx=addr(20), ddt=addr(21), dz=addr(22), dB=addr(23), dC=addr(24),
                      dA=addr(25), dD=addr(26), ddt_bias=addr(27), dinitial_state=addr(28))
        for k, v in kw.items():
            if k in self.q:
                self.q[k] = v
            elif k in self.g:
                self.g[k] = v
            else:
                setattr(self, k, v)

    def _q(self):
        return ctypes.byref(block.SSDSelective(*(self.q[n] for n, _ in
                                                 block.SSDSelective._fields_)))

    def forward(self):
        return block._function("ssd_selective_scan")(ctypes.byref(self.t), self._q(), self.y,
                                                     self.fin, self.ws, self.n, None)

    def step(self):
        return block._function("ssd_selective_step")(ctypes.byref(self.t), self._q(), self.fin,
                                                     self.y, None)

    def backward(self):
        g = block.SSDSelectiveGrads(*(self.g[n] for n, _ in block.SSDSelectiveGrads._fields_))
        return block._function("ssd_selective_backward")(
            ctypes.byref(self.t), self._q(), self.dy, self.df, ctypes.byref(g), self.ws, self.n,
            None)


@no_gpu
def test_selective_valid_requests_report_no_device():
    assert Selective().forward() == Selective().backward() == NO_DEVICE
    none = dict(z=None, D=None, dt_bias=None, initial_state=None)
    assert Selective(fin=None, ws=None, n=0, **none).forward() == NO_DEVICE
    assert Selective(df=None, dz=None, dD=None, ddt_bias=None, dinitial_state=None,
                     **none).backward() == NO_DEVICE
    assert Selective(t=tokens(**PACKED), b_stride=100, c_stride=36, B=addr(2, 8)).forward() == \
        NO_DEVICE
    assert Selective(t=one()).step() == NO_DEVICE
    assert Selective(t=one(), fin=addr(8)).step() == NO_DEVICE  # in place


@no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(dstate=0), INVALID), (dict(ngroups=0), INVALID), (dict(ngroups=3), INVALID),
    (dict(ngroups=16), UNSUPPORTED), (dict(dstate=18), UNSUPPORTED), (dict(dstate=68), UNSUPPORTED),
    (dict(reserved=1), INVALID), (dict(x=None), INVALID), (dict(dt=None), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(C=None), INVALID), (dict(y=None), INVALID),
    (dict(x=addr(0, 8)), INVALID), (dict(z=addr(4, 2)), INVALID), (dict(B=addr(2, 4)), INVALID),
    (dict(A=addr(5, 8)), INVALID), (dict(dt_bias=addr(7, 4)), INVALID),
    (dict(x_stride=60), INVALID), (dict(z_stride=68), INVALID), (dict(b_stride=34), INVALID),
    (dict(y=addr(0)), INVALID), (dict(y=addr(4)), INVALID), (dict(fin=addr(8)), INVALID),
    (dict(fin=addr(9)), INVALID), (dict(y=addr(9, 8)), INVALID),
    (dict(t=tokens(nseq=1)), INVALID), (dict(t=tokens(channels=24), ngroups=2), UNSUPPORTED),
])
def test_selective_rejects(kw, status):
    assert Selective(**kw).forward() == status


@no_gpu
@pytest.mark.parametrize("kw", [dict(t=tokens()), dict(t=one(), initial_state=None),
                                dict(t=one(), fin=None), dict(t=one(), fin=addr(8, 64)),
                                dict(t=one(), y=addr(8)), dict(t=tokens(**{**PACKED, "seqlen": 1}))])
def test_selective_step_rejects(kw):
    assert Selective(**kw).step() == INVALID


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(dx=None), dict(ddt=None), dict(dB=None), dict(dC=None), dict(dA=None),
    dict(dz=None), dict(z=None), dict(dx=addr(0)), dict(dx=addr(21)), dict(dA=addr(5)),
    dict(ws=None), dict(n=64), dict(ws=addr(20)), dict(df=addr(12, 4)), dict(dD=addr(26, 4))])
def test_selective_backward_rejects(kw):
    assert Selective(**kw).backward() == INVALID


@no_gpu
def test_norms_valid_and_rejected():
    t = tokens(seqlen=7)
    G, GB = block._function("ssd_gated_norm"), block._function("ssd_gated_norm_backward")
    R, RB = block._function("ssd_residual_norm"), block._function("ssd_residual_norm_backward")

    def gated(t=t, x=addr(0), xs=0, z=addr(1), zs=0, w=addr(2), g=2, eps=1e-5, y=addr(3)):
        return G(ctypes.byref(t), x, xs, z, zs, w, g, eps, 0, y, None)

    def gated_backward(z=addr(1), dy=addr(4), dx=addr(5), dz=addr(6), dw=addr(7), ws=addr(8),
                       n=1 << 30):
        return GB(ctypes.byref(t), addr(0), 0, z, 0, addr(2), 2, 1e-5, 1, dy, dx, dz, dw, ws, n,
                  None)

    def residual(res=addr(1), rt=0, scale=addr(2), w=addr(3), y=addr(4), out=addr(5)):
        return R(ctypes.byref(t), addr(0), 0, res, rt, scale, w, 1e-5, y, out, None)

    def residual_backward(r=addr(1), x=addr(0), scale=addr(2), dy=addr(4), dx=addr(5),
                          dr=addr(6), dw=addr(7), ds=addr(8), ws=addr(9), n=1 << 30):
        return RB(ctypes.byref(t), r, 0, x, 0, scale, addr(3), 1e-5, dy, None, dx, dr, dw, ds, ws,
                  n, None)

    assert gated() == gated(z=None) == gated(xs=128, zs=72) == gated(eps=0.0) == NO_DEVICE
    assert gated_backward() == gated_backward(z=None, dz=None) == NO_DEVICE
    assert residual() == residual(res=None, scale=None, rt=1) == NO_DEVICE
    assert residual_backward() == residual_backward(x=None, scale=None, ds=None, dr=None) == \
        NO_DEVICE
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(g=0), dict(g=3), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(xs=32), dict(zs=68),
               dict(y=addr(0)), dict(y=addr(1)), dict(y=addr(3, 8)),
               dict(t=tokens(**PACKED))):
        assert gated(**kw) == INVALID, kw
    assert gated(g=16) == gated(t=tokens(channels=8200), g=1) == UNSUPPORTED
    for kw in (dict(dy=None), dict(dx=None), dict(dw=None), dict(dz=None), dict(z=None),
               dict(dx=addr(0)), dict(dz=addr(5)), dict(ws=None), dict(n=8)):
        assert gated_backward(**kw) == INVALID, kw
    for kw in (dict(w=None), dict(y=None), dict(out=None), dict(rt=5), dict(out=addr(1)),
               dict(y=addr(5))):
        assert residual(**kw) == INVALID, kw
    for kw in (dict(r=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(ds=None),
               dict(x=None), dict(scale=None), dict(dr=addr(5)), dict(ws=None), dict(n=8)):
        assert residual_backward(**kw) == INVALID, kw


def test_workspace_queries():
    n = ctypes.c_int64()
    t = tokens(batch=1, nseq=1, seqlen=1000)
    f = block._function("ssd_conv_backward_workspace")
    assert f(ctypes.byref(t), 4, ctypes.byref(n)) == OK and n.value > 0 and n.value % 4 == 0
    assert f(ctypes.byref(t), 4, None) == INVALID and f(None, 4, ctypes.byref(n)) == INVALID
    f = block._function("ssd_gated_norm_backward_workspace")
    assert f(ctypes.byref(t), 1, ctypes.byref(n)) == OK and n.value > 0
    f = block._function("ssd_residual_norm_backward_workspace")
    assert f(ctypes.byref(t), ctypes.byref(n)) == OK and n.value > 0
    s = Selective()
    f = block._function("ssd_selective_backward_workspace")
    assert f(ctypes.byref(t), s._q(), ctypes.byref(n)) == OK and n.value > 0


def test_exports_are_declared():
    assert set(block.EXPORTS) <= set(libssd.EXPORTS)


# ---- the binding -----------------------------------------------------------------------------------

Bt, L, C = 2, 6, 16


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_rejects_shapes_and_types():
    x, w = z(Bt, L, C), z(C, 4)
    cu = torch.zeros(3, dtype=torch.int32)
    ab = dict(A=z(C, 16), B=z(Bt, L, 1, 16), C=z(Bt, L, 1, 16))
    sel = lambda **k: ssd.selective_scan(  # noqa: E731
        k.get("x", x), k.get("dt", x), k.get("A", ab["A"]), k.get("B", ab["B"]),
        k.get("C", ab["C"]), k.get("D"), k.get("z"), k.get("h0"))
    for match, call in (
            ("x must be", lambda: ssd.conv(x[0], w)),
            ("unsupported io dtype", lambda: ssd.conv(x.half(), w)),
            ("weight has shape", lambda: block._conv_params(z(C + 1, 4), None, C, x.device)),
            ("weight has shape", lambda: block._conv_params(z(C), None, C, x.device)),
            ("split must be", lambda: block._split_sizes((8, 4), C)),
            ("split must be", lambda: block._split_sizes((8, 4, 2, 2), C)),
            ("x must be a device", lambda: ssd.conv(x, w)),
            ("batch 1", lambda: ssd.conv(x, w, cu_seqlens=cu)),
            ("cu_seqlens must be", lambda: ssd.conv(x[:1], w, cu_seqlens=cu[:1])),
            ("unknown activation", lambda: block._silu("relu")),
            ("values of a token", lambda: block._rows(z(Bt, C, L).mT, "x", x.shape, x.dtype,
                                                      x.device)),
            ("x must be a device", lambda: sel()),
            ("B must be", lambda: sel(B=z(Bt, L, 16))),
            ("x must be", lambda: ssd.selective_step(z(Bt, C, 16), x, x, ab["A"], ab["B"], ab["C"])),
            ("state must be", lambda: ssd.selective_step(None, x[:, 0], x[:, 0], ab["A"],
                                                         ab["B"][:, 0], ab["C"][:, 0])),
            ("x must be a device", lambda: ssd.gated_norm(x, x, z(C))),
            ("residual_dtype must be", lambda: block._res_dtype(x.half(), "residual_dtype", x))):
        with pytest.raises(ValueError, match=match):
            call()
