"""The operators around the layer without a GPU: what they refuse beyond
test_block_cpu, and what their sources must not do."""
import os
import re

import pytest
import torch

from mixture_experts_layer_55_b200 import MoELayer
from mixture_experts_layer_55_b200 import _binding as B
from mixture_experts_layer_55_b200 import build as build_mod

CSRC = os.path.join(os.path.dirname(B.__file__), "csrc")


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def test_rows_scales_are_not_read_through_the_read_only_path():
    """The down product is resident while the gate/up product writes its rows' scales:
    the read-only path, for data that nothing writes while a kernel runs, is left
    to the weights' scales."""
    with open(os.path.join(CSRC, "ffn_mx8.cu")) as f:
        text = f.read()
    calls = re.findall(r"= load_scales(<\w+>)?\((\w+),", text)
    assert len(calls) == 6
    for how, what in calls:
        assert how == ("<false>" if what in ("pa", "px") else "<true>"), what
    assert [line.strip() for line in text.splitlines() if "__ldg(" in line] == [
        "return WEIGHT ? __ldg(reinterpret_cast<const V*>(p)) : *reinterpret_cast<const V*>(p);"]


def _parts(T, D, F, E, K):
    """(parts, rows) of the down product's contracted axis, from the rule: rows of few
    tokens an expert, tiles that leave SMs idle, two groups of 512 a part at least."""
    R = T * K
    if R > 24 * E:
        return 1, R
    tiles = min(R, E + R // 32) * -(-D // 256)
    return max(1, min(148 // tiles, 8, -(-F // 512) // 2)), R


@pytest.mark.parametrize("D,F,E,K", [(4096, 14336, 8, 2), (256, 4096, 8, 2), (256, 8192, 1, 1), (96, 8192, 4, 1),
                                     (2048, 1408, 64, 6), (7168, 2048, 256, 8), (32, 16384, 2, 2), (512, 2080, 40, 1)])
def test_mx8_workspace_of_a_larger_batch_serves_a_smaller_one(lib, D, F, E, K):
    last = 0
    for T in list(range(1, 300)) + [512, 1000, 3000, 10000, 70000]:
        size = B.mx8_workspace_size(B.MoeConfig.make(T, D, F, E, K, "bf16"))
        n, R = _parts(T, D, F, E, K)
        need = 256 + -(-2 * E * 128 // 256) * 256 + (n * R * D * 4 if n > 1 else 0)
        assert size >= max(last, need), T
        last = size


def test_dlogits_add_is_checked_like_every_tensor(lib):
    """A host tensor, a transposed one or one on another device than the state never
    reaches a kernel as an address."""
    c = B.MoeConfig.make(4, 64, 64, 8, 2, "bf16")
    state = torch.zeros(16, dtype=torch.uint8)
    for args in (dict(), dict(state=state)):
        rest = dict.fromkeys(("x", "w_router", "w_gate", "w_up", "w_down", "state", "dy", "dx", "dw_router", "dw_gate",
                              "dw_up", "dw_down", "workspace"))
        rest.update(args)
        with pytest.raises(ValueError, match="CUDA device"):
            B.moe_backward(c, **rest, dlogits_add=torch.zeros(4, 8))
        with pytest.raises(ValueError, match="contiguous"):
            B.moe_backward(c, **rest, dlogits_add=torch.zeros(8, 4).t())
        with pytest.raises(ValueError, match="dlogits_add must be a tensor"):
            B.moe_backward(c, **rest, dlogits_add=[0.0] * 32)


def _layer(T=4, D=64, F=64, E=2, **kw):
    w = [torch.zeros(E, D, F, dtype=torch.bfloat16) for _ in range(2)] + [torch.zeros(E, F, D, dtype=torch.bfloat16)]
    return MoELayer(T, torch.zeros(D, E), *w, K=1, norm_weight=torch.ones(D), **kw)


def test_block_refuses_what_is_not_a_whole_batch(lib):
    """A batch of fewer rows, another type or layout would be read or written out of
    range by the layer's kernels: each is refused by name, before any device work."""
    layer = _layer()
    good = torch.zeros(4, 64, dtype=torch.bfloat16)
    bad = {"elements": torch.zeros(3, 64, dtype=torch.bfloat16), "dtype": torch.zeros(4, 64),
           "contiguous": torch.zeros(64, 4, dtype=torch.bfloat16).t(), "must be a tensor": [1.0]}
    for call, names in ((layer.forward_block, ("x", "residual", "y")), (layer.forward_block_train, ("x", "residual", "y"))):
        for name in names:
            for what, t in bad.items():
                args = {"x": good, name: t}
                with pytest.raises(ValueError, match=f"{call.__name__}: {name} .*{what}"):
                    call(**args)
        with pytest.raises(ValueError, match="logit_noise has 7 elements"):
            call(good, logit_noise=torch.zeros(7))
        with pytest.raises(ValueError, match="CUDA device"):
            call(good)
    # with 8-bit experts: by the call that takes them
    w = (torch.zeros(1, dtype=torch.uint8),) * 6
    for x, y, what in ((good[:3], good, "x has 192"), (good, good[:3], "y has 192"), (good.float(), good, "x has dtype")):
        with pytest.raises(ValueError, match=f"moe_forward_mx8: {what}"):
            B.moe_forward_mx8(layer.cfg, x, layer.w_router, w, y, layer.workspace)
    layer._block = (good, torch.ones(4))
    for name in ("dy", "ds"):
        for what, t in bad.items():
            with pytest.raises(ValueError, match=f"backward_block: {name} .*{what}"):
                layer.backward_block(**{"dy": good, name: t})


def test_block_refuses_outputs_over_what_it_still_needs(lib):
    """Without a residual x is the sum that the call returns and the backward reads: y
    in its place is refused; so is a ds in the buffer that the layer's dx goes to."""
    layer = _layer()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (layer.forward_block, layer.forward_block_train):
        with pytest.raises(ValueError, match="y must not be x"):
            call(x, y=x)
        with pytest.raises(ValueError, match="y must not be x"):
            call(x, y=x.view(-1).view(4, 64))
        with pytest.raises(ValueError, match="CUDA device"):  # over x or the residual beside a sum of its own: no
            call(x, residual=torch.zeros_like(x), y=x)        # refusal but that of host tensors
    layer._block = (x, torch.ones(4))
    dx = torch.zeros_like(x)
    with pytest.raises(ValueError, match="ds must not be"):
        layer.backward_block(torch.zeros_like(x), ds=dx, grads={"dx": dx})


def test_arguments_that_are_no_tensors_are_refused_by_name(lib):
    c = B.MoeConfig.make(4, 64, 64, 8, 2, "bf16")
    x, i = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int32)
    for ws in (None, [0], 4096):
        with pytest.raises(ValueError, match="workspace must be a tensor"):
            B.moe_rmsnorm_backward(x, x, torch.ones(64), torch.ones(4), x, torch.ones(64), ws)
    for starts in (None, [0, 4], torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="seq_starts must be"):
            B.moe_balance_loss(c, torch.zeros(4, 8), i, starts, i, x, x, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="weights"):
        B.moe_expert_ffn_mx8(c, x, x, i, None, None, None, x, x, x, torch.zeros(64, dtype=torch.uint8))
    layer = _layer()
    layer._train_x = x
    with pytest.raises(ValueError, match="seq_starts must be"):
        layer.balance_loss([0, 4])


def test_block_runs_on_the_layers_device(lib, monkeypatch):
    """A layer on a device that is not the current one: every call of its block paths is
    made with the layer's device current (the norm and the layer on one stream)."""
    layer = _layer()
    current, log = [0], []

    class Device:
        def __init__(self, d):
            self.d = d.index

        def __enter__(self):
            self.old, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.old

    class Where:
        type, index = "cuda", 3
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(layer, "device", Where())
    monkeypatch.setattr(layer, "_check_rows", lambda *a, **k: None)
    layer.state = layer.bwd_workspace = layer.norm_workspace = torch.zeros(8, dtype=torch.uint8)
    # the norm goes to its tensors' device by itself
    monkeypatch.setattr(B, "moe_rmsnorm", lambda *a, **k: None)
    monkeypatch.setattr(B, "moe_rmsnorm_backward", lambda *a, **k: None)
    for name in ("moe_forward", "moe_forward_train", "moe_backward", "moe_forward_mx8", "moe_router_prepare"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **k: log.append((_n, current[0])))
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    grads = dict.fromkeys(("dw_router", "dw_gate", "dw_up", "dw_down"), x)
    layer.forward_block(x)
    layer.forward_block_train(x, x.clone())
    layer.backward_block(x.clone(), grads=dict(grads, dx=torch.zeros_like(x), dgamma=torch.zeros(64)))
    layer.mx8 = (x,) * 6
    layer.forward_block(x)
    layer.forward(x)
    names = [n for n, _ in log if n != "moe_router_prepare"]
    assert names == ["moe_forward", "moe_forward_train", "moe_backward", "moe_forward_mx8", "moe_forward_mx8"]
    assert {d for _, d in log} == {3} and current == [0]


def test_block_as_the_first_call_of_a_process(lib, monkeypatch):
    """The tensors of a first call are told from other objects like any later call's."""
    monkeypatch.setattr(B, "_TYPES", None)
    monkeypatch.setattr(B, "_TENSOR", ())
    with pytest.raises(ValueError, match="CUDA device"):
        _layer().forward_block(torch.zeros(4, 64, dtype=torch.bfloat16))


def test_balance_reads_other_blocks_results_behind_its_waits():
    """What the balance kernel's blocks write for each other is read by loads that the
    compiler may not move over a wait; the logits, written by nobody, by any."""
    with open(os.path.join(CSRC, "balance.cu")) as f:
        text = f.read()
    assert {re.sub(r"\s+", " ", line).strip() for line in text.splitlines() if "__ldcg(" in line} == {
        "MOE_DEVICE int4 bal_get4(const float* p) { return __ldcg(reinterpret_cast<const int4*>(p)); }",
        "MOE_DEVICE float bal_get(const float* p) { return __ldcg(p); }"}
    loads = re.findall(r'asm volatile\("ld\.relaxed\.gpu[^;]*;"[^;]*;', text)
    assert len(loads) == 4 and all('"memory"' in x for x in loads)
