"""Host-side checks of the loss and tensor-list entry points that need no GPU:
struct layouts, and every refusal happens before anything is enqueued."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B, C, D = 0x100000, 0x200000, 0x300000, 0x400000


def test_struct_layouts_and_constants(zs):
    assert ctypes.sizeof(zs.Logits) == 48 and zs.Logits.inv_temperature.offset == 40
    assert ctypes.sizeof(zs.Policy) == 40
    assert ctypes.sizeof(zs.Preference) == 32 and zs.Preference.kind.offset == 24
    assert ctypes.sizeof(zs.Tensor) == 96 and zs.Tensor.n.offset == 56 and zs.Tensor.grad_type.offset == 80
    text = open(os.path.join(ROOT, "include", "zero_shard.h")).read()
    for name in ("ZS_F32", "ZS_F16", "ZS_BF16", "ZS_STATE_F32", "ZS_STATE_U8", "ZS_WORK_BYTES", "ZS_MAX_TENSORS",
                 "ZS_POLICY_TOTALS", "ZS_PREFERENCE_TOTALS", "ZS_PREFERENCE_SIGMOID", "ZS_PREFERENCE_HINGE",
                 "ZS_PREFERENCE_SQUARED"):
        assert re.search(rf"#define {name} {getattr(zs, name)}\b", text), name


def _logits(zs, **kw):
    v = dict(data=A, rows=4, vocab=100, row_stride=100, type=zs.ZS_BF16, reserved=0, inv_temperature=1.0)
    v.update(kw)
    return zs.Logits(*[v[k] for k in ("data", "rows", "vocab", "row_stride", "type", "reserved", "inv_temperature")])


BAD_LOGITS = [dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 30) + 1, row_stride=1 << 31), dict(row_stride=99),
              dict(type=3), dict(type=-1), dict(reserved=1), dict(inv_temperature=0.0),
              dict(inv_temperature=-1.0), dict(inv_temperature=float("nan")), dict(inv_temperature=float("inf")),
              dict(data=None)]


def test_logits_refusals(zs):
    L, arg, align = zs.lib(), zs.ZS_ERR_ARG, zs.ZS_ERR_ALIGN

    def logp(x, labels=B, out=C, ent=None, saved=None):
        return L.zero_token_logp_async(None if x is None else ctypes.byref(x), labels, out, ent, saved, None)

    def grad(x, labels=B, saved=C, dlogp=C, ent=None, dent=None, ctrl=None, out=D, stride=100):
        return L.zero_token_logp_grad_async(None if x is None else ctypes.byref(x), labels, saved, dlogp, ent, dent,
                                            ctrl, out, stride, None)

    def policy(x, labels=B, old=C, adv=C, hp=None, out=D, stride=100, totals=C, work=D, lp=C, ctrl=None, w=None):
        hp = zs.policy() if hp is None else hp
        return L.zero_policy_loss_async(None if x is None else ctypes.byref(x), labels, old, adv, None, w,
                                        None if hp is False else ctypes.byref(hp), ctrl, lp, None, None, out, stride,
                                        totals, work, None)

    for kw in BAD_LOGITS:
        for call in (logp, grad, policy):
            assert call(_logits(zs, **kw)) == arg, (call, kw)
    for call in (logp, grad, policy):
        assert call(None) == arg
        assert call(_logits(zs, data=A + 1)) == align
        assert call(_logits(zs, data=A + 2, type=zs.ZS_F32)) == align
        assert call(_logits(zs), labels=None) == arg
        assert call(_logits(zs), labels=B + 4) == align
    assert logp(_logits(zs), out=None) == arg and logp(_logits(zs), out=C + 2) == align
    assert logp(_logits(zs), ent=C + 1) == align and logp(_logits(zs), saved=C + 3) == align
    assert logp(_logits(zs, rows=0, data=None), labels=None, out=None) == zs.ZS_OK
    for kw in (dict(saved=None), dict(dlogp=None), dict(out=None), dict(stride=99), dict(ent=C), dict(dent=C)):
        assert grad(_logits(zs), **kw) == arg, kw
    for kw in (dict(saved=C + 2), dict(ctrl=C + 4), dict(out=D + 1)):
        assert grad(_logits(zs), **kw) == align, kw
    for kw in (dict(old=None), dict(adv=None), dict(lp=None), dict(totals=None), dict(work=None), dict(stride=50),
               dict(hp=False), dict(hp=zs.policy(clip_low=-0.1)), dict(hp=zs.policy(clip_low=1.1)),
               dict(hp=zs.policy(clip_high=-0.1)), dict(hp=zs.policy(clip_high=float("nan"))),
               dict(hp=zs.policy(dual_clip=0.5)), dict(hp=zs.policy(dual_clip=1.0)),
               dict(hp=zs.policy(kl_coef=float("inf"))), dict(hp=zs.policy(entropy_coef=float("nan")))):
        assert policy(_logits(zs), **kw) == arg, kw
    for kw in (dict(work=D + 4), dict(old=C + 2), dict(w=C + 1), dict(ctrl=C + 4), dict(out=D + 1)):
        assert policy(_logits(zs), **kw) == align, kw
    assert zs.zero_kernel_launches() == 0


def test_preference_refusals(zs):
    L, arg, align = zs.lib(), zs.ZS_ERR_ARG, zs.ZS_ERR_ALIGN

    def call(logp=A, n=10, cu=B, pairs=1, hp=None, loss=C, reward=C, totals=C, work=D, w=None, dlogp=None, ref=None):
        hp = zs.preference(0.1) if hp is None else hp
        return L.zero_preference_loss_async(logp, ref, None, n, cu, w, pairs,
                                            None if hp is False else ctypes.byref(hp), loss, reward, dlogp, totals,
                                            work, None)

    for kw in (dict(n=-1), dict(pairs=-1), dict(logp=None), dict(cu=None), dict(loss=None), dict(reward=None),
               dict(totals=None), dict(work=None), dict(hp=False), dict(hp=zs.preference(0.0)),
               dict(hp=zs.preference(float("nan"))), dict(hp=zs.preference(float("inf"))),
               dict(hp=zs.preference(0.1, kind=3)), dict(hp=zs.preference(0.1, kind=-1)),
               dict(hp=zs.preference(0.1, label_smoothing=0.6)), dict(hp=zs.preference(0.1, label_smoothing=-0.1)),
               dict(hp=zs.preference(0.1, "hinge", label_smoothing=0.1)),
               dict(hp=zs.preference(0.1, margin=float("nan")))):
        assert call(**kw) == arg, kw
    odd = zs.preference(0.1)
    odd.average = 2
    assert call(hp=odd) == arg
    for kw in (dict(cu=B + 4), dict(work=D + 4), dict(logp=A + 2), dict(w=C + 1), dict(dlogp=C + 2), dict(ref=C + 2),
               dict(totals=C + 2)):
        assert call(**kw) == align, kw
    assert zs.zero_kernel_launches() == 0


def _tensor(zs, **kw):
    t = zs.Tensor(A, B, C, D, None, None, None, 100, 1.0, 1.0, zs.ZS_BF16, zs.ZS_BF16, zs.ZS_STATE_F32, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def test_tensor_list_refusals(zs):
    L, arg, align = zs.lib(), zs.ZS_ERR_ARG, zs.ZS_ERR_ALIGN
    hp = zs.adam(1e-3)

    def norm(t, n=1, ctrl=A, out=B, work=C):
        arr = None if t is None else (zs.Tensor * 1)(t)
        return L.zero_tensors_sqnorm_async(arr, n, ctrl, out, work, None)

    def step(t, n=1, h=hp, max_norm=0.0, sq=None, ctrl=A):
        arr = None if t is None else (zs.Tensor * 1)(t)
        return L.zero_tensors_adamw_async(arr, n, None if h is None else ctypes.byref(h), max_norm, sq, ctrl, None)

    for call in (norm, step):
        assert call(None) == arg and call(_tensor(zs), n=0) == arg and call(_tensor(zs), n=-1) == arg
        assert call(_tensor(zs), n=zs.ZS_MAX_TENSORS + 1) == arg
        for kw in (dict(n=-1), dict(grad_type=3), dict(grad=None), dict(reserved=1), dict(n=1 << 42)):
            assert call(_tensor(zs, **kw)) == arg, kw
        assert call(_tensor(zs, grad=A + 1)) == align
        assert call(_tensor(zs, grad=A + 2, grad_type=zs.ZS_F32)) == align
        assert call(_tensor(zs), ctrl=None) == arg and call(_tensor(zs), ctrl=A + 4) == align
    for kw in (dict(out=None), dict(work=None)):
        assert norm(_tensor(zs), **kw) == arg, kw
    for kw in (dict(out=B + 4), dict(work=C + 4)):
        assert norm(_tensor(zs), **kw) == align, kw
    for kw in (dict(master=None), dict(m=None), dict(v=None), dict(state=2), dict(state=zs.ZS_STATE_U8),
               dict(param=A, param_type=zs.ZS_F32), dict(lr_mult=float("nan")), dict(decay_mult=float("inf"))):
        assert step(_tensor(zs, **kw)) == arg, kw
    for kw in (dict(master=B + 2), dict(m=C + 2), dict(v=D + 1), dict(param=A + 1),
               dict(state=zs.ZS_STATE_U8, m_scale=A + 2, v_scale=A)):
        assert step(_tensor(zs, **kw)) == align, kw
    assert step(_tensor(zs), h=None) == arg and step(_tensor(zs), h=zs.adam(1e-3, beta1=1.0)) == arg
    assert step(_tensor(zs), max_norm=1.0) == arg and step(_tensor(zs), max_norm=float("nan")) == arg
    assert step(_tensor(zs), max_norm=1.0, sq=B + 4) == align
    assert L.zero_adam8_dequantize(A, B, -1, 0, C, None) == arg
    assert L.zero_adam8_dequantize(A, B, 5, 2, C, None) == arg
    assert L.zero_adam8_dequantize(None, B, 5, 0, C, None) == arg
    assert L.zero_adam8_dequantize(A, B + 1, 5, 0, C, None) == align
    assert L.zero_adam8_dequantize(None, None, 0, 0, None, None) == zs.ZS_OK
    assert zs.zero_kernel_launches() == 0


def test_binding_refuses_host_tensors_and_wrong_types(zs):
    x, y, o = torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    with pytest.raises(TypeError, match="CUDA"):
        zs.zero_token_logp_async(x, y, o)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        zs.zero_token_logp_async(x.double(), y, o)
    with pytest.raises(TypeError, match="CUDA"):
        zs.TensorView(grad=o, master=o, m=o, v=o)
    with pytest.raises(TypeError, match="grad"):
        zs.TensorView(grad=y, master=o, m=o, v=o)
    with pytest.raises(ValueError, match="go with uint8"):
        zs.TensorView(grad=o, master=o, m=o, v=o, m_scale=o, v_scale=o)
    with pytest.raises(ValueError, match="elements"):
        zs.TensorView(grad=torch.zeros(3), master=o, m=o, v=o)
    with pytest.raises(TypeError, match="param"):
        zs.TensorView(grad=o, master=o, m=o, v=o, param=o)
    with pytest.raises(ValueError, match="2 n_pairs"):
        zs.zero_preference_loss_async(o, torch.zeros(2, dtype=torch.int64), zs.preference(0.1), o, o, o, o)
    with pytest.raises(TypeError, match="mask"):
        zs.zero_preference_loss_async(o, torch.zeros(3, dtype=torch.int64), zs.preference(0.1), o, o, o, o, mask=o)
