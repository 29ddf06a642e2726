"""What the operators around the layer refuse (norm, 8-bit data and experts,
balance loss), on the host and before any device work: no GPU needed."""
import ctypes

import pytest
import torch

from mixture_experts_layer_55_b200 import MoELayer
from mixture_experts_layer_55_b200 import _binding as B
from mixture_experts_layer_55_b200 import build as build_mod

FAKE = 0x10000  # an aligned address the library never dereferences here


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def _cfg(**kw):
    base = dict(T=64, D=128, F=256, E=8, K=2, dtype="bf16")
    base.update(kw)
    return B.MoeConfig.make(**base)


def _norm(lib, T=4, D=64, dtype=B.MOE_BF16, x=FAKE, residual=None, gamma=FAKE, eps=1e-6, s=None, n=FAKE, rstd=None,
          q=None, qs=None):
    return lib.moe_rmsnorm(T, D, dtype, x, residual, gamma, eps, s, n, rstd, q, qs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), B.MOE_ERR_SHAPE),
    (dict(D=0), B.MOE_ERR_SHAPE),
    (dict(T=2**31), B.MOE_ERR_SHAPE),
    (dict(D=60), B.MOE_ERR_ALIGN),
    (dict(D=40, q=FAKE, qs=FAKE), B.MOE_ERR_ALIGN),     # 8-bit blocks of 32
    (dict(D=65544), B.MOE_ERR_UNSUPPORTED),
    (dict(dtype=2), B.MOE_ERR_ARG),
    (dict(x=None), B.MOE_ERR_ARG),
    (dict(gamma=None), B.MOE_ERR_ARG),
    (dict(n=None), B.MOE_ERR_ARG),                       # no output at all
    (dict(q=FAKE), B.MOE_ERR_ARG),                       # q without its scales
    (dict(s=FAKE), B.MOE_ERR_ARG),                       # a sum without a residual
    (dict(residual=FAKE, s=FAKE, n=FAKE), B.MOE_ERR_ARG),  # s and n in one buffer
    (dict(eps=-1.0), B.MOE_ERR_ARG),
    (dict(eps=float("nan")), B.MOE_ERR_ARG),
    (dict(x=FAKE + 8), B.MOE_ERR_ALIGN),
    (dict(residual=FAKE + 8), B.MOE_ERR_ALIGN),
    (dict(rstd=FAKE + 2), B.MOE_ERR_ALIGN),
])
def test_rmsnorm_refusals(lib, kw, code):
    assert _norm(lib, **kw) == code


def test_rmsnorm_backward_refusals(lib):
    def call(T=4, D=64, dtype=B.MOE_F32, dn=FAKE, ds=None, s=FAKE, gamma=FAKE, rstd=FAKE, dx=FAKE, dg=FAKE, ws=FAKE,
             nb=1 << 30):
        return lib.moe_rmsnorm_backward(T, D, dtype, dn, ds, s, gamma, rstd, dx, dg, ws, nb, None)
    for name in ("dn", "s", "gamma", "rstd", "dx", "dg"):
        assert call(**{name: None}) == B.MOE_ERR_ARG
    assert call(T=0) == B.MOE_ERR_SHAPE
    assert call(D=20) == B.MOE_ERR_ALIGN
    assert call(D=65544) == B.MOE_ERR_UNSUPPORTED
    assert call(ds=FAKE + 4) == B.MOE_ERR_ALIGN
    assert call(ws=None) == B.MOE_ERR_WORKSPACE
    assert call(nb=B.rmsnorm_backward_workspace_size(4, 64) - 1) == B.MOE_ERR_WORKSPACE
    assert call(ws=FAKE + 16) == B.MOE_ERR_ALIGN
    with pytest.raises(B.MoEError):
        B.rmsnorm_backward_workspace_size(4, 20)


def test_mx8_refusals(lib):
    for fn in (lib.moe_mx8_quantize, lib.moe_mx8_dequantize):
        assert fn(4, 48, B.MOE_BF16, FAKE, FAKE, FAKE, None) == B.MOE_ERR_ALIGN
        assert fn(0, 64, B.MOE_BF16, FAKE, FAKE, FAKE, None) == B.MOE_ERR_SHAPE
        assert fn(4, 64, 3, FAKE, FAKE, FAKE, None) == B.MOE_ERR_ARG
        assert fn(4, 64, B.MOE_BF16, None, FAKE, FAKE, None) == B.MOE_ERR_ARG
        assert fn(4, 64, B.MOE_BF16, FAKE, FAKE, None, None) == B.MOE_ERR_ARG
        assert fn(4, 64, B.MOE_BF16, FAKE + 8, FAKE, FAKE, None) == B.MOE_ERR_ALIGN
    prep = lib.moe_mx8_prepare_weight
    assert prep(0, 32, 8, B.MOE_BF16, FAKE, FAKE, FAKE, None) == B.MOE_ERR_SHAPE
    assert prep(2, 40, 8, B.MOE_BF16, FAKE, FAKE, FAKE, None) == B.MOE_ERR_ALIGN
    assert prep(2, 32, 12, B.MOE_BF16, FAKE, FAKE, FAKE, None) == B.MOE_ERR_ALIGN
    assert prep(2, 32, 8, B.MOE_BF16, FAKE, None, FAKE, None) == B.MOE_ERR_ARG
    assert prep(70000, 32, 8, B.MOE_BF16, FAKE, FAKE, FAKE, None) == B.MOE_ERR_UNSUPPORTED


def _weights(**kw):
    v = dict.fromkeys(("gate", "gate_scales", "up", "up_scales", "down", "down_scales"), FAKE)
    v.update(kw)
    return B.Mx8Weights(**v)


def test_expert_ffn_mx8_refusals(lib):
    c = _cfg()

    def call(cfg=c, xq=FAKE, xs=FAKE, off=FAKE, perm=FAKE, w=FAKE, wt=_weights(), hq=FAKE, hs=FAKE, y=FAKE, ws=FAKE,
             nb=1 << 30):
        return lib.moe_expert_ffn_mx8(ctypes.byref(cfg), xq, xs, off, perm, w, ctypes.byref(wt) if wt else None, hq,
                                      hs, y, ws, nb, None)
    for name in ("xq", "xs", "off", "hq", "hs", "y", "perm", "w", "wt"):
        assert call(**{name: None}) == B.MOE_ERR_ARG, name
    for name in ("gate", "gate_scales", "up", "up_scales", "down", "down_scales"):
        assert call(wt=_weights(**{name: None})) == B.MOE_ERR_ARG
        assert call(wt=_weights(**{name: FAKE + 4})) == B.MOE_ERR_ALIGN
    assert call(cfg=_cfg(dtype="f32")) == B.MOE_ERR_UNSUPPORTED
    assert call(cfg=_cfg(D=136)) == B.MOE_ERR_ALIGN
    assert call(cfg=_cfg(F=72)) == B.MOE_ERR_ALIGN
    assert call(cfg=_cfg(K=9, E=16)) == B.MOE_ERR_ARG
    assert call(xs=FAKE + 4) == B.MOE_ERR_ALIGN
    assert call(hq=FAKE + 16) == B.MOE_ERR_ALIGN  # these two on 32 bytes
    assert call(y=FAKE + 16) == B.MOE_ERR_ALIGN
    assert call(ws=None) == B.MOE_ERR_WORKSPACE
    assert call(nb=B.mx8_workspace_size(c) - 1) == B.MOE_ERR_WORKSPACE
    assert call(ws=FAKE + 64) == B.MOE_ERR_ALIGN


def test_forward_mx8_refusals(lib):
    c = _cfg()

    def call(cfg=c, x=FAKE, xq=FAKE, xs=FAKE, wr=FAKE, wt=_weights(), y_add=None, y=FAKE, ws=FAKE, nb=1 << 40):
        return lib.moe_forward_mx8(ctypes.byref(cfg), x, xq, xs, wr, None, None, None, None,
                                   ctypes.byref(wt) if wt else None, y_add, y, None, None, None, None, None, ws, nb,
                                   None)
    for name in ("x", "wr", "y", "wt", "xq", "xs"):  # xq and xs: both or neither
        assert call(**{name: None}) == B.MOE_ERR_ARG, name
    assert call(cfg=_cfg(F_shared=64)) == B.MOE_ERR_UNSUPPORTED
    assert call(cfg=_cfg(dtype="f32")) == B.MOE_ERR_UNSUPPORTED
    assert call(cfg=_cfg(D=136)) == B.MOE_ERR_ALIGN
    assert call(y_add=FAKE + 8) == B.MOE_ERR_ALIGN
    assert call(nb=B.forward_mx8_workspace_size(c) - 1) == B.MOE_ERR_WORKSPACE


def test_balance_refusals(lib):
    c = _cfg()

    def call(cfg=c, S=2, logits=FAKE, ids=FAKE, starts=FAKE, mask=None, cb=0.1, cz=0.1, counts=FAKE, losses=FAKE,
             seq=FAKE, dl=None, ws=FAKE, nb=1 << 30):
        return lib.moe_balance_loss(ctypes.byref(cfg), S, logits, ids, starts, mask, cb, cz, counts, losses, seq, dl,
                                    ws, nb, None)
    for name in ("logits", "ids", "starts", "counts", "losses", "seq"):
        assert call(**{name: None}) == B.MOE_ERR_ARG, name
    assert call(S=0) == B.MOE_ERR_SHAPE
    assert call(S=2**28) == B.MOE_ERR_SHAPE          # S * E beyond int32
    assert call(cb=float("inf")) == B.MOE_ERR_ARG
    assert call(cz=float("nan")) == B.MOE_ERR_ARG
    assert call(dl=FAKE + 4) == B.MOE_ERR_ALIGN
    assert call(ws=None) == B.MOE_ERR_WORKSPACE
    assert call(nb=B.balance_workspace_size(c, 2) - 1) == B.MOE_ERR_WORKSPACE
    assert call(cfg=_cfg(K=9, E=16)) == B.MOE_ERR_ARG


def test_train_state_router_offsets(lib):
    c = _cfg()
    lo, io = B.train_state_router(c)
    assert lo % 256 == 0 and io % 256 == 0 and 0 < io < lo < B.train_state_size(c)
    assert lo + 4 * c.T * c.E <= B.train_state_size(c)


def test_binding_checks_tensors(lib):
    """Tensors of the wrong place, type, size or layout are refused by name."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    g = torch.ones(64)
    with pytest.raises(ValueError, match="CUDA device"):
        B.moe_rmsnorm(x, g, torch.empty_like(x))
    with pytest.raises(ValueError, match="gamma"):
        B.moe_rmsnorm(x, g.bfloat16(), torch.empty_like(x))
    with pytest.raises(ValueError, match="gamma"):
        B.moe_rmsnorm(x, torch.ones(32), torch.empty_like(x))
    with pytest.raises(ValueError, match="n has"):
        B.moe_rmsnorm(x, g, torch.empty(3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="n has dtype"):
        B.moe_rmsnorm(x, g, torch.empty(4, 64))
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_rmsnorm(torch.zeros(64, 4, dtype=torch.bfloat16).t(), g, torch.empty_like(x))
    with pytest.raises(ValueError, match="x must be"):
        B.moe_rmsnorm(x.half(), g, x)
    with pytest.raises(ValueError, match="w must be"):
        B.moe_mx8_prepare_weight(x, x, x)
    c = _cfg(T=4)
    with pytest.raises(ValueError, match="logits"):
        B.moe_balance_loss(c, torch.zeros(4, 7), torch.zeros(4, 2, dtype=torch.int32),
                           torch.zeros(2, dtype=torch.int32), torch.zeros(1, 8, dtype=torch.int32), torch.zeros(2),
                           torch.zeros(1), torch.zeros(256, dtype=torch.uint8))


def test_binding_refuses_missing_workspace_and_wrong_gradient(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="workspace"):
        B.moe_rmsnorm_backward(x, x, torch.ones(64), torch.ones(4), x, torch.ones(64), None)
    c = _cfg(T=4)
    for bad in (torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 7)):
        with pytest.raises(ValueError, match="dlogits_add"):
            B.moe_backward(c, *([None] * 13), dlogits_add=bad)


def test_calls_go_to_the_tensors_device(monkeypatch):
    """Tensors on a device that is not the current one: the call is made with that
    device current and on its current stream, and the current device comes back."""
    log, current = [], [0]

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.old

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)

    def fn(*args):
        log.append((current[0], args))
        return B.MOE_OK
    B._run("x", 0, fn, (1, 2), None)
    B._run("x", 3, fn, (1, 2), None)
    B._run("x", 3, fn, (1, 2), 77)
    assert log == [(0, (1, 2, 1000)), (3, (1, 2, 1003)), (3, (1, 2, 77))] and current == [0]
    with pytest.raises(B.MoEError):
        B._run("x", 0, lambda *a: B.MOE_ERR_ARG, (), None)


def test_layer_refuses(lib):
    """8-bit experts with a shared expert, an unknown kind of experts."""
    w = [torch.zeros(2, 64, 64, dtype=torch.bfloat16) for _ in range(3)]
    r = torch.zeros(64, 2)
    with pytest.raises(ValueError, match="experts"):
        MoELayer(4, r, *w, K=1, experts="int4")
    with pytest.raises(ValueError, match="shared"):
        MoELayer(4, r, *w, K=1, experts="mx8", shared=tuple(torch.zeros(64, 64, dtype=torch.bfloat16) for _ in range(3)))
    layer = MoELayer(4, r, *w, K=1)
    with pytest.raises(ValueError, match="norm_weight"):
        layer.forward_block(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        layer.backward_block(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        layer.balance_loss(torch.zeros(2, dtype=torch.int32))
