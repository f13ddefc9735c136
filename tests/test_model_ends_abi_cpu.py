"""Host-side checks of the head, norm and embedding entry points that need no
GPU: struct layouts, scratch sizes, and every refusal before anything is enqueued."""
import ctypes

import pytest
import torch

A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000
BIG = 1 << 40


def test_struct_layouts(zs):
    assert ctypes.sizeof(zs.Head) == 72 and zs.Head.type.offset == 56 and zs.Head.inv_temperature.offset == 64
    assert ctypes.sizeof(zs.Norm) == 64 and zs.Norm.type.offset == 48 and zs.Norm.eps.offset == 56
    assert ctypes.sizeof(zs.Embed) == 64 and zs.Embed.type.offset == 48 and zs.Embed.scale.offset == 56


def test_work_bytes(zs):
    L, arg = zs.lib(), zs.ZS_ERR_ARG
    for bad in ((-1, 64, 100, 0, 0), ((1 << 24) + 1, 64, 100, 0, 0), (4, 7, 100, 0, 0), (4, 0, 100, 0, 0),
                (4, 65544, 100, 0, 0), (4, 64, 0, 0, 0), (4, 64, (1 << 24) + 1, 0, 0), (4, 64, 100, -1, 1), (4, 64, 100, 0, 2)):
        assert L.zero_head_work_bytes(*bad) == arg, bad
    for rows, width, vocab in ((0, 8, 1), (1, 64, 1000), (8192, 4096, 131072), (1 << 24, 65536, 1 << 24)):
        one = [L.zero_head_work_bytes(rows, width, vocab, piece, 1) for piece in (256, 4096, 0)]
        assert 0 < one[0] <= one[1] and one[0] <= one[2]
        assert L.zero_head_work_bytes(rows, width, vocab, 0, 0) > 0
        assert L.zero_head_work_bytes(rows, width, vocab, 100, 1) == one[0]
        whole = L.zero_head_work_bytes(rows, width, vocab, vocab, 1)
        assert all(L.zero_head_work_bytes(rows, width, vocab, p, 1) == whole for p in (vocab + 1, 1 << 40, (1 << 63) - 1))
    # a large batch's scratch stays far below its logits: one piece of them, and fp32 sums of dhidden
    assert L.zero_head_work_bytes(8192, 4096, 131072, 0, 1) < 2 * 8192 * 131072
    for bad in ((-1, 4), (1 << 31, 4), (1, 0), (1, (1 << 24) + 1)):
        assert L.zero_layer_norm_work_bytes(*bad) == arg
    for bad in ((-1, 4), ((1 << 28) + 1, 4), (1, 0), (1, (1 << 24) + 1)):
        assert L.zero_embed_work_bytes(*bad) == arg
    assert L.zero_layer_norm_work_bytes(0, 1) > 0 and L.zero_embed_work_bytes(0, 1) > 0
    assert L.zero_embed_work_bytes(1 << 28, 1 << 24) > 0 and L.zero_layer_norm_work_bytes((1 << 31) - 1, 1 << 24) > 0
    with pytest.raises(zs.ZeroShardError):
        zs.new_head_work(4, 63, 100, device="cpu")


def _head(zs, **kw):
    v = dict(hidden=A, weight=B, rows=4, vocab=100, width=64, hidden_stride=64, weight_stride=64, type=zs.ZS_BF16, reserved=0,
             inv_temperature=1.0)
    v.update(kw)
    return zs.Head(*[v[n] for n, _ in zs.Head._fields_])


def test_head_refusals(zs):
    L, arg, align = zs.lib(), zs.ZS_ERR_ARG, zs.ZS_ERR_ALIGN

    def logp(h, labels=C, out=D, saved=None, work=A, size=BIG):
        return L.zero_head_logp_async(None if h is None else ctypes.byref(h), labels, out, saved, work, size, None)

    def grad(h, labels=C, saved=C, dlogp=C, ctrl=None, dh=D, dhs=64, dw=B, dws=64, work=A, size=BIG):
        return L.zero_head_logp_grad_async(None if h is None else ctypes.byref(h), labels, saved, dlogp, ctrl, dh, dhs, dw, dws,
                                           work, size, None)

    for call in (logp, grad):
        assert call(None) == arg
        for kw in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(width=0),
                   dict(width=63), dict(width=1 << 17), dict(type=zs.ZS_F32), dict(type=3), dict(type=-1), dict(reserved=1),
                   dict(inv_temperature=0.0), dict(inv_temperature=float("nan")), dict(inv_temperature=float("inf")),
                   dict(hidden=None), dict(weight=None), dict(hidden_stride=56), dict(weight_stride=56),
                   dict(hidden_stride=(1 << 40) + 8), dict(hidden_stride=-64)):
            assert call(_head(zs, **kw)) == arg, kw
        for kw in (dict(hidden=A + 8), dict(weight=B + 2), dict(hidden_stride=68), dict(weight_stride=65)):
            assert call(_head(zs, **kw)) == align, kw
        for kw in (dict(labels=None), dict(work=None), dict(size=0), dict(size=-1), dict(size=-(1 << 63)), dict(size=1000)):
            assert call(_head(zs), **kw) == arg, kw
        assert call(_head(zs), labels=C + 4) == align and call(_head(zs), work=A + 64) == align
        assert call(_head(zs), saved=C + 2) == align
    assert logp(_head(zs), out=None) == arg and logp(_head(zs), out=D + 1) == align
    assert logp(_head(zs), size=L.zero_head_work_bytes(4, 64, 100, 0, 0) - 1) == arg
    assert logp(_head(zs, rows=0, hidden=None), labels=None, out=None, work=None, size=0) == zs.ZS_OK
    for kw in (dict(saved=None), dict(dlogp=None), dict(dh=None, dw=None), dict(dhs=56), dict(dws=56),
               dict(size=L.zero_head_work_bytes(4, 64, 100, 256, 1) - 1), dict(dhs=(1 << 40) + 8)):
        assert grad(_head(zs), **kw) == arg, kw
    for kw in (dict(dlogp=C + 2), dict(ctrl=C + 4), dict(dh=D + 8), dict(dw=D + 8), dict(dhs=68), dict(dws=68)):
        assert grad(_head(zs), **kw) == align, kw
    assert zs.zero_kernel_launches() == 0


def _norm(zs, **kw):
    v = dict(x=A, gamma=B, beta=B, rows=4, width=100, x_stride=100, type=zs.ZS_BF16, param_type=zs.ZS_F32, eps=1e-5)
    v.update(kw)
    return zs.Norm(*[v[n] for n, _ in zs.Norm._fields_])


def test_norm_refusals(zs):
    L, arg, align = zs.lib(), zs.ZS_ERR_ARG, zs.ZS_ERR_ALIGN

    def fwd(n, y=C, ys=100, saved=None):
        return L.zero_layer_norm_async(None if n is None else ctypes.byref(n), y, ys, saved, None)

    def bwd(n, dy=C, dys=100, saved=C, dx=D, dxs=100, dg=D, db=D, work=A, size=BIG):
        return L.zero_layer_norm_grad_async(None if n is None else ctypes.byref(n), dy, dys, saved, dx, dxs, dg, db, work, size, None)

    for call in (fwd, bwd):
        assert call(None) == arg
        for kw in (dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=(1 << 24) + 1), dict(type=3), dict(type=-1),
                   dict(param_type=3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
                   dict(x_stride=99), dict(x_stride=-100)):
            assert call(_norm(zs, **kw)) == arg, kw
        for kw in (dict(x=A + 1), dict(gamma=B + 2), dict(beta=B + 1), dict(x=A + 2, type=zs.ZS_F32)):
            assert call(_norm(zs, **kw)) == align, kw
        assert call(_norm(zs), saved=C + 2) == align
    assert fwd(_norm(zs), y=None) == arg and fwd(_norm(zs), ys=99) == arg and fwd(_norm(zs), y=C + 1) == align
    assert fwd(_norm(zs, rows=0, x=None), y=None) == zs.ZS_OK
    for kw in (dict(dy=None), dict(saved=None), dict(dx=None, dg=None, db=None), dict(dys=99), dict(dxs=99), dict(work=None),
               dict(size=L.zero_layer_norm_work_bytes(4, 100) - 1)):
        assert bwd(_norm(zs), **kw) == arg, kw
    for kw in (dict(dy=C + 1), dict(dx=D + 1), dict(dg=D + 2), dict(db=D + 2), dict(work=A + 8)):
        assert bwd(_norm(zs), **kw) == align, kw
    assert bwd(_norm(zs, rows=0, x=None), dy=None, saved=None, dg=None, db=None) == zs.ZS_OK
    assert zs.zero_kernel_launches() == 0


def _embed(zs, **kw):
    v = dict(table=A, ids=B, tokens=4, vocab=100, width=50, table_stride=50, type=zs.ZS_BF16, reserved=0, scale=1.0)
    v.update(kw)
    return zs.Embed(*[v[n] for n, _ in zs.Embed._fields_])


def test_embed_refusals(zs):
    L, arg, align = zs.lib(), zs.ZS_ERR_ARG, zs.ZS_ERR_ALIGN

    def fwd(e, out=C, stride=50):
        return L.zero_embed_async(None if e is None else ctypes.byref(e), out, stride, None)

    def bwd(e, dout=C, ds=50, dt=D, dts=50, kind=None, add=0, work=A, size=BIG):
        return L.zero_embed_grad_async(None if e is None else ctypes.byref(e), dout, ds, dt, dts,
                                       zs.ZS_BF16 if kind is None else kind, add, work, size, None)

    for call in (fwd, bwd):
        assert call(None) == arg
        for kw in (dict(tokens=-1), dict(tokens=(1 << 28) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(width=0),
                   dict(width=(1 << 24) + 1), dict(type=3), dict(reserved=1), dict(scale=float("nan")), dict(scale=float("inf")),
                   dict(scale=1e31), dict(ids=None)):
            assert call(_embed(zs, **kw)) == arg, kw
        assert call(_embed(zs, ids=B + 4)) == align
    assert fwd(_embed(zs, table=None)) == arg and fwd(_embed(zs, table_stride=49)) == arg
    assert fwd(_embed(zs), out=None) == arg and fwd(_embed(zs), stride=49) == arg
    assert fwd(_embed(zs, table=A + 1)) == align and fwd(_embed(zs), out=C + 1) == align
    assert fwd(_embed(zs, tokens=0, ids=None, table=None), out=None) == zs.ZS_OK
    for kw in (dict(dout=None), dict(ds=49), dict(dt=None), dict(dts=49), dict(kind=zs.ZS_F16), dict(kind=3), dict(add=2),
               dict(work=None), dict(size=L.zero_embed_work_bytes(4, 50) - 1)):
        assert bwd(_embed(zs), **kw) == arg, kw
    for kw in (dict(dout=C + 1), dict(dt=D + 1), dict(dt=D + 2, kind=zs.ZS_F32), dict(work=A + 8)):
        assert bwd(_embed(zs), **kw) == align, kw
    assert zs.zero_kernel_launches() == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(zs):
    h, w, y, o = torch.zeros(2, 8).half(), torch.zeros(5, 8).half(), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    with pytest.raises(TypeError, match="CUDA"):
        zs.zero_head_logp_async(h, w, y, o, o)
    with pytest.raises(TypeError, match="CUDA"):
        zs.zero_layer_norm_async(o[None], None, None, o[None])
    with pytest.raises(TypeError, match="CUDA"):
        zs.zero_embed_async(w, y, h)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        zs.zero_embed_grad_async(y, h.double(), w, o)
