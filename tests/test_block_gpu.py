"""The operators around the layer on the GPU (norm and its backward, 8-bit data
and experts, balance loss), each against a plain 64-bit implementation, and the
layer's paths that run them together.

Tolerances.  A rounding to a type is off by at most half a step, eps / 2 of the
value (bf16 2^-8, fp32 2^-24; e4m3 2^-4, or half of its least step, 2^-10 of the
block's scale).  A chain of n fp32 additions is off by at most n 2^-24 of the sum
of the magnitudes; the row sums here are at most 128 deep in one thread and
across its block, so 2^-17; the tensor cores' sums are held to 2^-23 per added
product, n being the contracted length.
"""
import math

import pytest
import torch

import mixture_experts_layer_55_b200 as M
from mixture_experts_layer_55_b200 import MoELayer
from mixture_experts_layer_55_b200 import _binding as B

pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}
SUM = 2.0**-17
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _within(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    over = err > tol
    assert not bool(over.any()), f"{what}: {int(over.sum())} off, worst {float((err - tol).max()):.3e} over the tolerance"


def _scale_exponent(amax):
    """Least e with amax <= 448 2^e (64 bits); -127 for a block of zeros."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448)).clamp(-127, 127)
    e = torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _quantize_ref(v):
    b = v.double().unflatten(-1, (-1, 32))
    e = _scale_exponent(b.abs().amax(-1))
    q = (b / torch.exp2(e)[..., None]).float().to(torch.float8_e4m3fn).flatten(-2)
    return q, (e + 127).to(torch.uint8)


def _value(q, s):
    f = q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    return (f * torch.exp2(s.double() - 127)[..., None]).flatten(-2)


# ---------------------------------------------------------------------- norm --

NORM = [(1, 8, "bf16", False, False), (1, 32, "f32", True, True), (5, 72, "bf16", True, False),
        (3, 256, "bf16", True, True), (129, 1000, "f32", True, False), (7, 1024, "f32", False, True),
        (2, 7168, "bf16", True, True), (33, 8200, "f32", True, False), (3, 16640, "bf16", True, True),
        (2, 40000, "f32", False, False), (1, 65536, "bf16", True, True), (700, 4096, "bf16", True, True),
        (1500, 64, "bf16", False, True)]


@pytest.mark.parametrize("T,D,dt,residual,bits8", NORM)
def test_rmsnorm(T, D, dt, residual, bits8):
    dtype = DT[dt]
    g = _gen(T * 100003 + D)
    x = _randn(g, T, D) * torch.exp(2 * _randn(g, T, 1))
    x = x.to(dtype)
    res = _randn(g, T, D, dtype=dtype) if residual else None
    gamma = 1 + 0.3 * _randn(g, D)
    n, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    s = torch.empty_like(x) if residual else None
    q = torch.empty(T, D, dtype=torch.float8_e4m3fn, device="cuda") if bits8 else None
    qs = torch.empty(T, D // 32, dtype=torch.uint8, device="cuda") if bits8 else None
    M.moe_rmsnorm(x, gamma, n, residual=res, s=s, rstd=rstd, q=q, q_scales=qs, eps=1e-5)
    summed = x if res is None else (x.float() + res.float()).to(dtype)
    if residual:
        assert torch.equal(s, summed)
    ref_r = (summed.double().square().mean(1) + 1e-5).rsqrt()
    _within(rstd, ref_r, SUM * ref_r, "rstd")
    ref = summed.double() * ref_r[:, None] * gamma.double()
    _within(n, ref, (ROUND[dtype] + SUM) * ref.abs() + 1e-38, "n")
    if bits8:  # the 8-bit rows are those of the n that was stored, bit for bit
        rq, rs = _quantize_ref(n)
        assert torch.equal(qs, rs)
        assert torch.equal(_value(q, qs), _value(rq, rs))
        q2, qs2 = torch.empty_like(q), torch.empty_like(qs)
        M.moe_rmsnorm(x, gamma, None, residual=res, q=q2, q_scales=qs2, eps=1e-5)  # without n and s
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(qs2, qs)
    # in place: the sum over the residual, the norm over x
    x2, r2 = x.clone(), res.clone() if residual else None
    M.moe_rmsnorm(x2, gamma, x2, residual=r2, s=r2, eps=1e-5)
    assert torch.equal(x2, n) and (not residual or torch.equal(r2, s))


# many rows a team, all widths' forms; the last rows ragged
MANY = [(20003, 64, "bf16"), (20001, 96, "f32"), (9001, 512, "f32"), (9001, 512, "bf16"), (5003, 1000, "bf16"),
        (6001, 1024, "f32"), (4003, 2048, "bf16"), (2501, 4096, "f32"), (1801, 7168, "bf16"), (1201, 8192, "f32"),
        (900, 12288, "bf16"), (700, 16384, "f32")]


@pytest.mark.parametrize("T,D,dt", MANY)
def test_rmsnorm_many_rows(T, D, dt):
    """Forward (with a residual and, where D allows, the 8-bit output) and backward of
    more rows than there are teams, and nothing written around the outputs."""
    dtype, pad = DT[dt], 4096
    g = _gen(T + D)

    def out(n, t):
        b = torch.full((n + 2 * pad,), 77, dtype=torch.uint8, device="cuda") if t == torch.uint8 else \
            torch.full((n + 2 * pad,), 77.0, dtype=t, device="cuda")
        bufs.append(b)
        return b[pad:-pad]
    bufs = []
    x, res = _randn(g, T, D, dtype=dtype), _randn(g, T, D, dtype=dtype)
    gamma = 1 + 0.3 * _randn(g, D)
    n, s, rstd = out(T * D, dtype).view(T, D), out(T * D, dtype).view(T, D), out(T, torch.float32)
    q, qs = (out(T * D, torch.uint8), out(T * D // 32, torch.uint8)) if D % 32 == 0 else (None, None)
    M.moe_rmsnorm(x, gamma, n, residual=res, s=s, rstd=rstd, q=q, q_scales=qs, eps=1e-5)
    assert torch.equal(s, (x.float() + res.float()).to(dtype))
    for a in range(0, T, 2048):
        at = slice(a, a + 2048)
        s64 = s[at].double()
        r = (s64.square().mean(1) + 1e-5).rsqrt()
        _within(rstd[at], r, SUM * r, "rstd")
        ref = s64 * r[:, None] * gamma.double()
        _within(n[at], ref, (ROUND[dtype] + SUM) * ref.abs() + 1e-38, "n")
        if q is not None:
            rq, rs = _quantize_ref(n[at])
            assert torch.equal(qs.view(T, -1)[at], rs)
            assert torch.equal(_value(q.view(T, D)[at], qs.view(T, -1)[at]), _value(rq, rs))
    dn, ds = _randn(g, T, D, dtype=dtype), _randn(g, T, D, dtype=dtype)
    dx, dg = out(T * D, dtype).view(T, D), out(D, torch.float32)
    ws = torch.zeros(M.rmsnorm_backward_workspace_size(T, D), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_backward(dn, s, gamma, rstd, dx, dg, ws, ds=ds)
    dgr, dgm = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for a in range(0, T, 2048):
        at = slice(a, a + 2048)
        r, dn64 = rstd[at].double()[:, None], dn[at].double()
        xh, gg = s[at].double() * r, dn64 * gamma.double()
        mean, mag = (gg * xh).mean(1, keepdim=True), (gg * xh).abs().mean(1, keepdim=True)
        ref = r * (gg - xh * mean) + ds[at].double()
        parts = r * (gg.abs() + xh.abs() * mag) + ds[at].double().abs()
        _within(dx[at], ref, ROUND[dtype] * ref.abs() + SUM * parts, "dx")
        dgr += (dn64 * xh).sum(0)
        dgm += (dn64 * xh).abs().sum(0)
    _within(dg, dgr, SUM * dgm, "dgamma")
    for b in bufs:
        assert bool((b[:pad] == 77).all()) and bool((b[-pad:] == 77).all())


@pytest.mark.parametrize("scale,eps", [(1e-18, 0.0), (1e-12, 0.0), (1e15, 0.0), (1e18, 1e-6), (1.0, 1e4), (1e-30, 0.0),
                                       (1e-25, 1e-12), (1e30, 1e-6), (2e38, 1e-6)])
def test_rmsnorm_scales(scale, eps):
    """Rows of very small and very large values (whose squares leave fp32), a large
    eps, and weights beyond the range the correction is carried in."""
    g = _gen(77)
    x = (scale * (0.5 + torch.rand(40, 512, generator=g, device="cuda"))).float()
    gamma = 1 + 0.3 * _randn(g, 512)
    gamma[5], gamma[200] = 1e32, -1e33
    n, rstd = torch.empty_like(x), torch.empty(40, device="cuda")
    M.moe_rmsnorm(x, gamma, n, rstd=rstd, eps=eps)
    r = (x.double().square().mean(1) + eps).rsqrt()
    _within(rstd, r, SUM * r, "rstd")
    ref = x.double() * r[:, None] * gamma.double()
    _within(n, ref, (ROUND[torch.float32] + SUM) * ref.abs() + 1e-38, "n")


def test_rmsnorm_rows_that_are_not_numbers():
    """An infinity or NaN stays in its row and shows in its 8-bit block; a row of
    zeros is zeros."""
    g = _gen(3)
    x = _randn(g, 6, 256, dtype=torch.bfloat16)
    clean = x.clone()
    x[1, 70] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 0
    gamma = torch.ones(256, device="cuda")

    def run(v):
        n, q = torch.empty_like(v), torch.empty(6, 256, dtype=torch.uint8, device="cuda")
        qs = torch.empty(6, 8, dtype=torch.uint8, device="cuda")
        M.moe_rmsnorm(v, gamma, n, q=q, q_scales=qs)
        return n, q, qs
    n, q, qs = run(x)
    n0, q0, qs0 = run(clean)
    for r in (0, 4, 5):
        assert torch.equal(n[r], n0[r]) and torch.equal(q[r], q0[r]) and torch.equal(qs[r], qs0[r])
    assert bool(n[1].isnan().all()) and bool((qs[1] == 255).all()) and bool((q[1] == 0x7F).all())
    assert bool(n[2, 5].isnan()) and int(qs[2, 0]) == 255 and bool((q[2, :32] == 0x7F).all())
    assert bool((n[2, 32:] == 0).all()) and bool((qs[2, 1:] == 0).all())
    assert bool((n[3] == 0).all()) and bool((q[3] == 0).all()) and bool((qs[3] == 0).all())


@pytest.mark.parametrize("T,D,dt,with_ds", [
    (1, 8, "f32", False), (1, 64, "bf16", True), (3, 72, "bf16", False), (301, 1000, "f32", True),
    (1300, 256, "f32", False), (4099, 96, "bf16", True), (900, 4096, "bf16", True), (5, 16640, "f32", True),
    (3, 40000, "bf16", True), (2, 65536, "f32", False), (1200, 2048, "bf16", False)])
def test_rmsnorm_backward(T, D, dt, with_ds):
    dtype = DT[dt]
    g = _gen(T + 7 * D)
    s, dn = _randn(g, T, D, dtype=dtype), _randn(g, T, D, dtype=dtype)
    ds = _randn(g, T, D, dtype=dtype) if with_ds else None
    gamma = 1 + 0.3 * _randn(g, D)
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dg = torch.empty_like(s), torch.empty(D, device="cuda")
    ws = torch.zeros(M.rmsnorm_backward_workspace_size(T, D), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_backward(dn, s, gamma, rstd, dx, dg, ws, ds=ds)
    r, s64, dn64 = rstd.double()[:, None], s.double(), dn.double()
    xh, gg = s64 * r, dn64 * gamma.double()
    mean, mag = (gg * xh).mean(1, keepdim=True), (gg * xh).abs().mean(1, keepdim=True)
    ref = r * (gg - xh * mean) + (0 if ds is None else ds.double())
    parts = r * (gg.abs() + xh.abs() * mag) + (0 if ds is None else ds.double().abs())
    _within(dx, ref, ROUND[dtype] * ref.abs() + SUM * parts, "dx")
    _within(dg, (dn64 * xh).sum(0), SUM * (dn64 * xh).abs().sum(0), "dgamma")
    # over dn in place, and again: the same bits
    dn2, dg2 = dn.clone(), torch.empty_like(dg)
    M.moe_rmsnorm_backward(dn2, s, gamma, rstd, dn2, dg2, ws, ds=ds)
    assert torch.equal(dn2, dx) and torch.equal(dg2, dg)


def test_rmsnorm_gradient_against_differences():
    """<dx, v> and <dgamma, w> against central differences of the 64-bit forward
    (error h^2 times third derivatives of order one: 1e-8 at h = 1e-4)."""
    g = _gen(11)
    T, D = 9, 104
    s, dn, v = (_randn(g, T, D) for _ in range(3))
    ds = _randn(g, T, D)
    gamma, w = 1 + 0.3 * _randn(g, D), _randn(g, D)

    def loss(sv, gv):
        n = sv * (sv.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gv
        return float((n * dn.double()).sum() + (sv * ds.double()).sum())
    n, rstd = torch.empty_like(s), torch.empty(T, device="cuda")
    M.moe_rmsnorm(s, gamma, n, rstd=rstd)
    dx, dg = torch.empty_like(s), torch.empty(D, device="cuda")
    ws = torch.zeros(M.rmsnorm_backward_workspace_size(T, D), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_backward(dn, s, gamma, rstd, dx, dg, ws, ds=ds)
    h, s64, g64 = 1e-4, s.double(), gamma.double()
    want = (loss(s64 + h * v.double(), g64) - loss(s64 - h * v.double(), g64)) / (2 * h)
    got = float((dx.double() * v.double()).sum())
    assert abs(got - want) <= SUM * float((dx.double() * v.double()).abs().sum()) * 4 + 1e-5
    want = (loss(s64, g64 + h * w.double()) - loss(s64, g64 - h * w.double())) / (2 * h)
    got = float((dg.double() * w.double()).sum())
    assert abs(got - want) <= SUM * float((dg.double() * w.double()).abs().sum()) * 4 + 1e-5


# ---------------------------------------------------------------- 8-bit data --

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (257, 1024), (70, 7168)])
def test_mx8_quantize(rows, cols, dt):
    g = _gen(rows + cols)
    x = (_randn(g, rows, cols) * torch.exp(8 * _randn(g, rows, 1))).to(DT[dt])
    x[0, :32] = 0
    x[-1, -1] = 1.75 * 2.0**20  # a maximum on the border of a scale
    q, s = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    M.moe_mx8_quantize(x, q, s)
    rq, rs = _quantize_ref(x)
    assert torch.equal(s, rs)
    assert torch.equal(_value(q, s), _value(rq, rs))
    out = torch.empty_like(x)
    M.moe_mx8_dequantize(q, s, out)
    assert torch.equal(out.double(), _value(q, s).to(DT[dt]).double())


def test_mx8_extremes():
    """The least and largest values, infinities and NaN; every byte read back."""
    x = torch.zeros(8, 32, device="cuda")
    x[0, 0] = 2.0**-149
    x[1, 3] = torch.finfo(torch.float32).max
    x[2, 31] = float("inf")
    x[3, 1] = float("nan")
    x[4, 0] = -float("inf")
    x[5, 0], x[5, 1] = 448.0, 2.0**-9
    x[6, 0] = -1.7500001 * 2.0**8
    q, s = torch.empty(8, 32, dtype=torch.uint8, device="cuda"), torch.empty(8, 1, dtype=torch.uint8, device="cuda")
    M.moe_mx8_quantize(x, q, s)
    assert s.flatten().tolist() == [0, 247 if x[1, 3] > 1.75 * 2.0**127 else 246, 255, 255, 255, 127, 128, 0]
    v = _value(q, s)
    assert bool(v[2:5].isnan().all()) and bool((q[2:5] == 0x7F).all())
    assert v[5, 0] == 448 and v[5, 1] == 2.0**-9 and v[6, 0] == -448
    assert abs(float(v[1, 3]) / float(x[1, 3]) - 1) <= 2.0**-4
    byte = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(5).reshape(-1, 32).contiguous()
    sc = torch.tensor([0, 1, 127, 200, 255], device="cuda", dtype=torch.uint8).repeat_interleave(8).reshape(-1, 1).contiguous()
    out = torch.empty(40, 32, device="cuda")
    M.moe_mx8_dequantize(byte, sc, out)
    ref = _value(byte, sc)
    ref[32:] = float("nan")
    assert torch.equal(out.double().nan_to_num(nan=1e30), ref.float().double().nan_to_num(nan=1e30))


@pytest.mark.parametrize("E,K,N,dt", [(1, 32, 8, "f32"), (3, 96, 136, "bf16"), (2, 512, 264, "f32")])
def test_mx8_prepare_weight(E, K, N, dt):
    w = 0.02 * _randn(_gen(K), E, K, N)
    w = w.to(DT[dt])
    q = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    M.moe_mx8_prepare_weight(w, q, s)
    rq, rs = _quantize_ref(w.transpose(1, 2).contiguous())
    assert torch.equal(s, rs) and torch.equal(_value(q, s), _value(rq, rs))


# ------------------------------------------------------------------- balance --

def _balance_ref(logits, ids, starts, mask, score, cb, cz):
    T, E = logits.shape
    K, S = ids.shape[1], len(starts) - 1
    on = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    at = torch.arange(T, device="cuda")
    rows = [at[a:b][on[a:b]] for a, b in zip(starts[:-1], starts[1:])]
    used, total = sum(len(r) > 0 for r in rows), sum(len(r) for r in rows)
    counts = torch.zeros(S, E, dtype=torch.int64, device="cuda")
    seq, d, z = torch.zeros(S, dtype=torch.float64, device="cuda"), torch.zeros(T, E, dtype=torch.float64, device="cuda"), 0.0
    for i, r in enumerate(rows):
        if not len(r):
            continue
        l = logits[r].double().requires_grad_(True)
        counts[i] = torch.bincount(ids[r].flatten().long(), minlength=E)
        p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
        p = p / p.sum(1, keepdim=True)
        bal = E * (counts[i].double() / (len(r) * K) * p.mean(0)).sum()
        zi = torch.logsumexp(l, 1).square().sum() / total
        (d[r],) = torch.autograd.grad(cb * bal / used + cz * zi, l)
        seq[i] = bal.detach()
        z += float(zi.detach())
    return counts, seq, d, z, float(seq.sum() / max(1, used))


def _balance(logits, ids, starts, mask=None, score="softmax", cb=0.01, cz=0.001, grad=True, ws=None):
    T, E = logits.shape
    S = len(starts) - 1
    cfg = M.MoeConfig.make(T, 8, 8, E, ids.shape[1], "bf16", score_func=score)
    if ws is None:
        ws = torch.zeros(M.balance_workspace_size(cfg, S), dtype=torch.uint8, device="cuda")
    out = (torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda"),
           torch.empty(S, device="cuda"), torch.empty(T, E, device="cuda") if grad else None)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    M.moe_balance_loss(cfg, logits, ids, st, out[0], out[1], out[2], ws, token_mask=mask, dlogits=out[3],
                       c_balance=cb, c_z=cz)
    return out, ws


def _ids(g, T, E, K):
    return torch.rand(T, E, generator=g, device="cuda").topk(K, 1).indices.to(torch.int32).contiguous()


BALANCE = [(1, 2, 1, [0, 1], "none"), (1, 256, 8, [0, 1], "none"), (5, 3, 3, [0, 2, 2, 5], "none"),
           (64, 8, 2, [0, 64], "random"), (257, 17, 4, [3, 3, 90, 91, 91, 250], "random"),
           (1000, 64, 6, [0, 1000], "none"), (1000, 64, 6, list(range(0, 1001, 1)), "random"),
           (3000, 256, 8, [0, 700, 701, 2999], "random"), (300, 33, 1, [0] * 400 + [300], "none"),
           (40, 8, 2, [0, 40], "all"), (129, 100, 5, [5, 60, 129], "first"), (8192, 8, 2, [0, 2048, 4096, 6144, 8192], "none")]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", range(len(BALANCE)))
def test_balance_loss(case, score):
    T, E, K, starts, kind = BALANCE[case]
    g = _gen(case + 50)
    logits = 3 * _randn(g, T, E)
    ids = _ids(g, T, E, K)
    mask = None
    if kind == "random":
        mask = (torch.rand(T, generator=g, device="cuda") < 0.6).to(torch.uint8) * 3
    elif kind == "all":
        mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    elif kind == "first":
        mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
        mask[starts[0]] = 1
    if mask is not None:  # what does not count is not read into anything
        logits[mask == 0] = float("nan")
    (counts, losses, seq, d), ws = _balance(logits, ids, starts, mask, score)
    rc, rs, rd, rz, rb = _balance_ref(logits, ids, starts, mask, score, 0.01, 0.001)
    assert B.moe_get_device_status(ws) == 0
    assert torch.equal(counts.long(), rc)
    # the exponents' arguments carry |l - max| 2^-24 <= 25 2^-24, sums 2^-24 a term:
    # 2^-18 of a probability; a token's share of a loss is rounded by 2^-33
    tol = 2.0**-18
    _within(seq, rs, tol * rs + E * 2.0**-33, "seq_loss")
    assert abs(float(losses[1]) - rb) <= tol * rb + E * 2.0**-33
    assert abs(float(losses[0]) - rz) <= tol * rz
    # the gradient's two parts: cb E / (S' n) p (f - c), every factor at most 1
    n = torch.zeros(T, dtype=torch.float64, device="cuda")
    for a, b in zip(starts[:-1], starts[1:]):
        m = torch.ones(b - a, device="cuda") if mask is None else (mask[a:b] != 0).double()
        n[a:b] = 1 / m.sum().clamp(min=1)
    p = torch.softmax(logits.double(), 1).nan_to_num(0)
    lse = torch.logsumexp(logits.double(), 1).abs().nan_to_num(0)
    score_p = p if score == "softmax" else (torch.sigmoid(logits.double()) / torch.sigmoid(logits.double()).sum(1, keepdim=True)).nan_to_num(0)
    used, total = max(1, int((rs > 0).sum())), max(1, int((n > 0).sum()) if mask is None else int((mask != 0).sum()))
    bound = 2 * 0.01 * E / used * n[:, None] * score_p + 2 * 0.001 * lse[:, None] * p / total
    _within(d, rd, tol * bound + 1e-30, "dlogits")
    # again with the same workspace, without a gradient: the same bits
    (c2, l2, s2, _), _ = _balance(logits, ids, starts, mask, score, grad=False, ws=ws)
    assert torch.equal(c2, counts) and torch.equal(l2, losses) and torch.equal(s2, seq)


@pytest.mark.parametrize("T,E,K,S,masked", [(32771, 256, 8, 16, True), (30001, 130, 3, 7, False), (65537, 64, 6, 300, True),
                                            (140000, 8, 2, 3, True), (40003, 33, 2, 5, True), (70001, 17, 1, 9, False)])
def test_balance_loss_many_tokens(T, E, K, S, masked):
    """Batches whose blocks take several rounds of tokens each, the last one
    ragged: every gradient row, and nothing written around the outputs."""
    g = _gen(T)
    logits, ids = _randn(g, T, E), _ids(g, T, E, K)
    cuts = torch.sort(torch.randint(0, T + 1, (S,), generator=g, device="cuda")).values.tolist()
    starts = [0] + cuts
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8) if masked else None
    cfg = M.MoeConfig.make(T, 8, 8, E, K, "bf16")
    ws = torch.zeros(M.balance_workspace_size(cfg, S), dtype=torch.uint8, device="cuda")
    pad = 4096  # a multiple of 16 bytes around every output
    bufs = [torch.full((n + 2 * pad,), 77, dtype=dt, device="cuda") for n, dt in
            ((S * E, torch.int32), (2, torch.float32), (S, torch.float32), (T * E, torch.float32))]
    counts, losses, seq, d = (b[pad:-pad] for b in bufs)
    M.moe_balance_loss(cfg, logits, ids, torch.tensor(starts, dtype=torch.int32, device="cuda"), counts, losses, seq,
                       ws, token_mask=mask, dlogits=d, c_balance=0.01, c_z=0.001)
    assert B.moe_get_device_status(ws) == 0
    for b in bufs:
        assert bool((b[:pad] == 77).all()) and bool((b[-pad:] == 77).all())
    rc, rs, rd, rz, rb = _balance_ref(logits, ids, starts, mask, "softmax", 0.01, 0.001)
    assert torch.equal(counts.reshape(S, E).long(), rc)
    tol = 2.0**-18
    _within(seq, rs, tol * rs + E * 2.0**-33, "seq_loss")
    assert abs(float(losses[0]) - rz) <= tol * rz and abs(float(losses[1]) - rb) <= tol * rb + E * 2.0**-33
    # the gradient's two parts, as above
    on = torch.ones(T, dtype=torch.float64, device="cuda") if mask is None else (mask != 0).double()
    n, total = torch.zeros(T, dtype=torch.float64, device="cuda"), 0.0
    for a, b in zip(starts[:-1], starts[1:]):
        n[a:b] = 1 / on[a:b].sum().clamp(min=1)
        total += float(on[a:b].sum())
    l64 = logits.double()
    p, lse = torch.softmax(l64, 1), torch.logsumexp(l64, 1).abs()
    used = max(1, int((rs > 0).sum()))
    bound = 2 * 0.01 * E / used * n[:, None] * p + 2 * 0.001 * lse[:, None] * p / max(1.0, total)
    _within(d.reshape(T, E), rd, tol * bound + 1e-30, "dlogits")


def test_balance_gradient_against_differences():
    g = _gen(5)
    T, E, K, starts = 60, 12, 3, [0, 25, 25, 55]
    logits, ids, v = _randn(g, T, E), _ids(g, T, E, K), _randn(g, T, E).double()
    (_, _, _, d), _ = _balance(logits, ids, starts, cb=0.7, cz=0.3)

    def loss(l):
        _, _, _, z, b = _balance_ref(l, ids, starts, None, "softmax", 0.0, 0.0)
        return 0.7 * b + 0.3 * z
    h = 1e-4
    want = (loss(logits.double() + h * v) - loss(logits.double() - h * v)) / (2 * h)
    got = float((d.double() * v).sum())
    assert abs(got - want) <= 2.0**-17 * float((d.double() * v).abs().sum()) + 1e-6


def test_balance_faults_are_seen():
    """Malformed borders and ids raise the bounds flag; a counted NaN shows in its
    sequence's loss alone; masked infinities do not matter."""
    g = _gen(8)
    logits, ids = _randn(g, 32, 8), _ids(g, 32, 8, 2)
    for starts in ([0, 20, 10], [0, 33], [-1, 32]):
        _, ws = _balance(logits, ids, starts)
        assert B.moe_get_device_status(ws) == B.MOE_DEVFLAG_BOUNDS
        B.moe_clear_device_status(ws)
        _, ws = _balance(logits, ids, [0, 20, 32])
        assert B.moe_get_device_status(ws) == 0
    for bad in (-1, 8):
        i2 = ids.clone()
        i2[3, 1] = bad
        _, ws = _balance(logits, i2, [0, 32])
        assert B.moe_get_device_status(ws) == B.MOE_DEVFLAG_BOUNDS
    l2 = logits.clone()
    l2[5, 2] = float("nan")
    (counts, losses, seq, d), ws = _balance(l2, ids, [0, 10, 32])
    (c0, _, seq0, d0), _ = _balance(logits, ids, [0, 10, 32])
    assert math.isnan(seq[0]) and torch.equal(seq[1], seq0[1]) and bool(losses.isnan().all())
    assert bool(d[5].isnan().any()) and torch.equal(d[6:], d0[6:]) and torch.equal(counts, c0)
    # an expert that is masked off by -inf has probability 0
    l3 = logits.clone()
    l3[:, 7] = -float("inf")
    (_, losses, _, d), _ = _balance(l3, ids.clamp(max=6), [0, 32])
    assert bool(losses.isfinite().all()) and bool((d[:, 7] == 0).all()) and bool(d.isfinite().all())


# ------------------------------------------------------------- 8-bit experts --

def _experts_state(T, D, F, E, K, seed, counts=None, wscale=0.05):
    """Rows grouped by expert (counts: rows per expert, their sum T K), weights."""
    g = _gen(seed)
    R = T * K
    if counts is None:
        ids = _ids(g, T, E, K).flatten().long()
        counts = torch.bincount(ids, minlength=E).tolist()
    offsets = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")
    perm = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    def spread(*shape):  # every block at a scale of its own
        v = _randn(g, *shape).unflatten(-1, (-1, 32))
        k = torch.randint(-4, 5, (*v.shape[:-1], 1), generator=g, device="cuda")
        return (v * torch.exp2(k.float())).flatten(-2)
    xq, xs = _quantize_ref(spread(R, D))
    w = []
    for n, k in ((F, D), (F, D), (D, F)):
        w += list(_quantize_ref(wscale / 16 * spread(E, n, k)))
    return dict(cfg=M.MoeConfig.make(T, D, F, E, K, "bf16"), xq=xq, xs=xs, offsets=offsets, perm=perm,
                topk_w=torch.rand(T, K, generator=g, device="cuda"), w=tuple(w), counts=counts)


def _run_experts(st, weighted=True, sentinel=7.0):
    c = st["cfg"]
    R = c.T * c.K
    pad = 64  # rows before and behind each output that nothing may touch
    full = (torch.full((R + 2 * pad, c.F), 0x55, dtype=torch.uint8, device="cuda"),
            torch.full((R + 2 * pad, c.F // 32), 0x55, dtype=torch.uint8, device="cuda"),
            torch.full((R + 2 * pad, c.D), sentinel, dtype=torch.bfloat16, device="cuda"))
    hq, hs, y = (b[pad:-pad] for b in full)
    ws = torch.zeros(M.mx8_workspace_size(c), dtype=torch.uint8, device="cuda")
    M.moe_expert_ffn_mx8(c, st["xq"], st["xs"], st["offsets"], st["perm"] if weighted else None,
                         st["topk_w"] if weighted else None, st["w"], hq, hs, y, ws)
    for b, v in zip(full, (0x55, 0x55, sentinel)):
        assert bool((b[:pad] == v).all()) and bool((b[-pad:] == v).all())
    return hq, hs, y, ws


def _check_experts(st, hq, hs, y, weighted=True):
    """h against the 64-bit products of the 8-bit operands, y against the 64-bit
    products of the h that was stored."""
    c, off = st["cfg"], st["offsets"].tolist()
    w64 = [_value(st["w"][i], st["w"][i + 1]) for i in (0, 2, 4)]
    wt = st["topk_w"].flatten()[st["perm"].long()].double() if weighted else torch.ones(c.T * c.K, device="cuda", dtype=torch.float64)
    for e in range(c.E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = _value(st["xq"][a:b], st["xs"][a:b])
        gate, up = x @ w64[0][e].T, x @ w64[1][e].T
        eg, eu = (c.D * 2.0**-23 * (x.abs() @ w.abs().T) for w in (w64[0][e], w64[1][e]))
        h = gate * torch.sigmoid(gate) * up
        # |silu'| <= 1.1, |silu(g)| <= |g|; silu itself to 2^-20
        eh = 1.1 * eg * up.abs() + (gate.abs() + eg) * eu + 2.0**-20 * h.abs()
        got = _value(hq[a:b], hs[a:b])
        scale = torch.exp2(hs[a:b].double() - 127).repeat_interleave(32, 1)
        _within(got, h, 2.0**-4 * (h.abs() + eh) + 2.0**-10 * scale + eh, f"h of expert {e}")
        top, etop = h.abs().unflatten(1, (-1, 32)).amax(2), eh.unflatten(1, (-1, 32)).amax(2)
        sc = scale[:, ::32]
        assert bool((top - etop <= 448 * sc).all()) and bool(((top + etop > 224 * sc) | (hs[a:b] == 0)).all())
        want = wt[a:b, None] * (got @ w64[2][e].T)
        mag = wt[a:b, None] * (got.abs() @ w64[2][e].abs().T)
        _within(y[a:b], want, 2.0**-8 * want.abs() + (c.F + 2) * 2.0**-23 * mag + 1e-38, f"y of expert {e}")


EXPERTS = [(1, 32, 32, 1, 1, None), (1, 256, 512, 8, 2, None), (3, 96, 160, 2, 2, None), (5, 64, 32, 4, 1, [0, 5, 0, 0]),
           (40, 224, 288, 3, 2, [79, 0, 1]), (129, 256, 96, 1, 1, None), (300, 128, 64, 5, 2, [128, 129, 0, 127, 216]),
           (64, 512, 1408, 64, 6, None), (1000, 160, 416, 4, 2, [256, 257, 1, 1486]), (700, 1024, 544, 2, 1, [333, 367]),
           (4, 7168, 64, 256, 8, None), (2000, 2048, 256, 8, 2, None), (60, 224, 160, 8, 2, [70, 0, 33, 1, 16, 0, 0, 0]),
           (20, 1408, 2080, 4, 2, None), (96, 32, 544, 8, 2, [0, 32, 32, 64, 31, 33, 0, 0]),
           # several tiles a CTA in each form (pairs, single CTAs, few rows)
           (1500, 256, 2816, 8, 2, None), (200, 128, 4096, 8, 2, None), (150, 4096, 1536, 24, 3, None),
           # few tokens: the down product's contracted axis in parts (4, 5, 2, 8)
           (1, 256, 4096, 8, 2, None), (3, 224, 5600, 4, 2, None), (20, 512, 2080, 1, 1, None),
           (60, 96, 8192, 4, 1, [40, 0, 20, 0])]


@pytest.mark.parametrize("case", range(len(EXPERTS)))
def test_experts_mx8(case):
    T, D, F, E, K, counts = EXPERTS[case]
    st = _experts_state(T, D, F, E, K, case, counts)
    hq, hs, y, ws = _run_experts(st)
    assert B.moe_get_device_status(ws) == 0
    _check_experts(st, hq, hs, y)
    hq2, hs2, y2, _ = _run_experts(st)
    assert torch.equal(y, y2) and torch.equal(hq, hq2) and torch.equal(hs, hs2)


@pytest.mark.parametrize("T,E,F,counts", [(100, 3, 96, [70, 0, 50]), (40, 6, 96, [0, 33, 1, 0, 6, 0]),
                                          (400, 3, 96, [300, 0, 129]), (10, 3, 2048, [5, 0, 9])])
def test_experts_mx8_unit_weights_and_unused_rows(T, E, F, counts):
    """Weight 1 without perm; rows behind offsets[E] stay as they were."""
    st = _experts_state(T, 128, F, E, 2, 9, counts=counts)  # fewer than the 2 T rows there are
    used = sum(counts)
    hq, hs, y, ws = _run_experts(st, weighted=False)
    assert B.moe_get_device_status(ws) == 0
    _check_experts(st, hq, hs, y, weighted=False)
    assert bool((y[used:] == 7).all()) and bool((hq[used:] == 0x55).all()) and bool((hs[used:] == 0x55).all())
    none = _experts_state(T, 64, F, E, 2, 9, counts=[0] * E)
    hq, hs, y, ws = _run_experts(none)
    assert B.moe_get_device_status(ws) == 0 and bool((y == 7).all()) and bool((hq == 0x55).all())


# single CTAs, few rows, CTA pairs, few rows with the down product in parts
@pytest.mark.parametrize("T,E,F", [(50, 2, 128), (50, 8, 128), (300, 2, 128), (20, 8, 4096)])
def test_experts_mx8_faults_are_seen(T, E, F):
    """A NaN scale makes its row NaN and no other; malformed offsets compute nothing
    and raise the bounds flag, as does a perm entry out of range."""
    st = _experts_state(T, 256, F, E, 1, 4)
    _, _, y0, _ = _run_experts(st)
    st["xs"] = st["xs"].clone()
    st["xs"][17, 3] = 255
    _, hs, y, _ = _run_experts(st)
    assert bool(y[17].isnan().all()) and bool((hs[17] == 255).all())
    keep = [r for r in range(T) if r != 17]
    assert torch.equal(y[keep], y0[keep])
    st = _experts_state(T, 256, F, E, 1, 4)
    good = st["offsets"].tolist()
    for bad in (good[:-1] + [T + 1], good[:1] + [T - 1] + good[1:-1], [-5] + good[1:]):
        st2 = dict(st, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        _, _, y, ws = _run_experts(st2)
        assert B.moe_get_device_status(ws) == B.MOE_DEVFLAG_BOUNDS
        assert bool((y == 7).all())
    for bad in (-1, T):
        p = st["perm"].clone()
        p[7] = bad
        _, _, y, ws = _run_experts(dict(st, perm=p))
        assert B.moe_get_device_status(ws) == B.MOE_DEVFLAG_BOUNDS
        assert torch.equal(y[8:], y0[8:]) and bool((y[7] == 0).all())
    _, _, y, ws = _run_experts(st)
    assert B.moe_get_device_status(ws) == 0 and torch.equal(y, y0)


@pytest.mark.parametrize("T,E,F", [(200, 4, 192), (30, 8, 192), (400, 2, 192), (2, 8, 4096)])
def test_experts_mx8_on_another_stream_and_in_a_graph(T, E, F):
    st = _experts_state(T, 256, F, E, 2, 21)
    hq, hs, y0, _ = _run_experts(st)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = torch.zeros_like(y0)
    ws = torch.zeros(M.mx8_workspace_size(st["cfg"]), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def call(stream=None):
        M.moe_expert_ffn_mx8(st["cfg"], st["xq"], st["xs"], st["offsets"], st["perm"], st["topk_w"], st["w"], hq, hs,
                             y, ws, stream=stream)
    call(side)
    side.synchronize()
    assert torch.equal(y, y0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):  # new rows in the same buffers
        st["xq"].copy_(st["xq"].view(torch.uint8).flip(0).view(torch.float8_e4m3fn))
        st["xs"].copy_(st["xs"].flip(0))
        graph.replay()
        torch.cuda.synchronize()
        _check_experts(st, hq, hs, y)


# ------------------------------------------------------- the layer's own paths --

def _layer(T, D, F, E, K, seed, dtype=torch.bfloat16, **kw):
    g = _gen(seed)
    wr = 0.1 * _randn(g, D, E)
    w = [0.05 * _randn(g, E, D, F), 0.05 * _randn(g, E, D, F), 0.05 * _randn(g, E, F, D)]
    return MoELayer(T, wr, *(v.to(dtype) for v in w), K, norm_weight=1 + 0.2 * _randn(g, D), **kw)


@pytest.mark.parametrize("T,D,F,E,K,cf", [(1, 64, 96, 4, 2, 0.0), (37, 256, 160, 8, 2, 0.0), (600, 128, 256, 4, 2, 0.5),
                                          (2500, 512, 128, 16, 4, 1.0)])
def test_block_with_mx8_experts(T, D, F, E, K, cf):
    """norm -> routing -> 8-bit experts -> combine as one call, against the same
    operators called one by one (bit for bit), and against 64 bits without the
    rounding of h (2^-4 of each of its elements, or half its block's least step)."""
    layer = _layer(T, D, F, E, K, T, experts="mx8", capacity_factor=cf)
    g = _gen(T + 1)
    x, res = _randn(g, T, D, dtype=torch.bfloat16), _randn(g, T, D, dtype=torch.bfloat16)
    y, s = layer.forward_block(x, res)
    assert B.moe_get_device_status(layer.workspace) == 0
    n, q = torch.empty_like(x), torch.empty(T, D, dtype=torch.float8_e4m3fn, device="cuda")
    qs, s2 = torch.empty(T, D // 32, dtype=torch.uint8, device="cuda"), torch.empty_like(x)
    M.moe_rmsnorm(x, layer.norm_weight, n, residual=res, s=s2, q=q, q_scales=qs)
    assert torch.equal(s, s2)
    c = layer.cfg
    R = M.max_rows(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.empty(T, K, **i32), torch.empty(T, K, device="cuda")
    ws = torch.zeros(M.workspace_size(c), dtype=torch.uint8, device="cuda")
    M.moe_route(c, n, layer.w_router, ids, w, ws, w_router_terms=layer._terms())
    cnt, kept, off = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
    perm, row_of = torch.zeros(R, **i32), torch.empty(T, K, **i32)
    M.moe_dispatch(c, None, ids, cnt, kept, off, perm, row_of, None, ws)
    rows = perm.long() // K
    st = dict(cfg=c, offsets=off, perm=perm, topk_w=w, w=layer.mx8,
              xq=q.view(torch.uint8)[rows].view(torch.float8_e4m3fn), xs=qs[rows].contiguous())
    hq, hs = torch.zeros(R, F, dtype=torch.uint8, device="cuda"), torch.zeros(R, F // 32, dtype=torch.uint8, device="cuda")
    yp, mws = torch.zeros(R, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(M.mx8_workspace_size(c), dtype=torch.uint8, device="cuda")
    M.moe_expert_ffn_mx8(c, st["xq"], st["xs"], off, perm, w, layer.mx8, hq, hs, yp, mws)
    want = torch.empty_like(x)
    M.moe_combine(c, yp, row_of, want)
    assert torch.equal(y, want)
    # quantised in the call, and with y_add
    y2 = layer.forward(n)
    assert torch.equal(y2, want)
    y3 = torch.empty_like(x)
    M.moe_forward_mx8(c, n, layer.w_router, layer.mx8, y3, layer.workspace, xq=q, xs=qs, y_add=s,
                      w_router_terms=layer._terms())
    M.moe_combine(c, yp, row_of, want, y_add=s)
    assert torch.equal(y3, want)
    # 64 bits, expert by expert
    ref, tol = torch.zeros(T, D, device="cuda", dtype=torch.float64), torch.zeros(T, D, device="cuda", dtype=torch.float64)
    w64 = [_value(layer.mx8[i], layer.mx8[i + 1]) for i in (0, 2, 4)]
    o = off.tolist()
    for e in range(E):
        if o[e] == o[e + 1]:
            continue
        r = torch.arange(o[e], o[e + 1], device="cuda")
        xe, t = _value(st["xq"][r], st["xs"][r]), rows[r]
        wt = w.flatten()[perm[r].long()].double()[:, None]
        gate, up = xe @ w64[0][e].T, xe @ w64[1][e].T
        h = gate * torch.sigmoid(gate) * up
        top = h.abs().unflatten(1, (-1, 32)).amax(2).repeat_interleave(32, 1)
        ye = wt * (h @ w64[2][e].T)
        ref.index_add_(0, t, ye)
        # the scale is below top / 224; products to 2^-15 of their magnitudes' sum
        tol.index_add_(0, t, wt * ((2.0**-4 * h.abs() + 2.0**-10 * top / 224 + 2.0**-10 * h.abs()) @ w64[2][e].abs().T)
                       + 2.0**-8 * ye.abs())
    _within(y, ref, tol * 1.01 + 2.0**-8 * ref.abs() + 1e-6, "y")


def test_block_bf16_and_requantized_weights():
    T, D, F, E, K = 130, 128, 64, 4, 2
    layer = _layer(T, D, F, E, K, 3)
    g = _gen(1)
    x, res = _randn(g, T, D, dtype=torch.bfloat16), _randn(g, T, D, dtype=torch.bfloat16)
    y, s = layer.forward_block(x, res)
    n = torch.empty_like(x)
    M.moe_rmsnorm(x, layer.norm_weight, n, residual=res)
    assert torch.equal(y, layer.forward(n)) and torch.equal(s, (x.float() + res.float()).bfloat16())
    y1, s1 = layer.forward_block(x)  # no residual: the sum is x itself
    assert s1 is x
    m8 = _layer(T, D, F, E, K, 3, experts="mx8")
    a = m8.forward(n)
    m8.w_down.mul_(2)
    m8.quantize_experts()
    b = m8.forward(n)
    assert torch.equal(b, a * 2)  # scales one power of two up
    with pytest.raises(ValueError):
        m8.forward_train(n)
    graph = m8.capture(n, b)
    want = b.clone()
    b.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, want)


@pytest.mark.parametrize("dt,score", [("f32", "softmax"), ("bf16", "sigmoid")])
def test_block_training_step(dt, score):
    """forward_block_train, the balance loss over sequences, backward_block: the
    pieces called one by one give the same bits, and the balance gradient reaches
    the router weight and dx as 64 bits have it."""
    T, D, F, E, K = 200, 128, 64, 6, 2
    dtype = DT[dt]
    layer = _layer(T, D, F, E, K, 8, dtype=dtype, score_func=score)
    g = _gen(2)
    x, res, dy, ds = (_randn(g, T, D, dtype=dtype) for _ in range(4))
    starts = torch.tensor([0, 50, 50, 140, 190], dtype=torch.int32, device="cuda")
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    y, s = layer.forward_block_train(x, res)
    bal = layer.balance_loss(starts, mask, c_balance=2.0, c_z=0.5)
    grads = {k: v.clone() for k, v in layer.backward_block(dy, ds, c_z=0.001, dlogits_add=bal["dlogits"]).items()}
    n, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    M.moe_rmsnorm(x, layer.norm_weight, n, residual=res, rstd=rstd)
    # the logits it was routed on, and the loss over them
    lo, io = M.train_state_router(layer.cfg)
    logits = layer.state[lo:lo + 4 * T * E].view(torch.float32).reshape(T, E)
    ids = layer.state[io:io + 4 * T * K].view(torch.int32).reshape(T, K)
    rc, rs, rd, rz, rb = _balance_ref(logits, ids, starts.tolist(), mask, score, 2.0, 0.5)
    assert torch.equal(bal["counts"].long(), rc)
    _within(bal["seq_loss"], rs, 2.0**-17 * rs, "seq_loss")
    _within(bal["dlogits"], rd, 2.0**-15 * rd.abs().amax(), "dlogits")
    # one by one
    y2 = layer.forward_train(n)
    assert torch.equal(y, y2)
    plain = {k: v.clone() for k, v in layer.backward(dy, c_z=0.001).items()}
    aux = layer.backward(dy, c_z=0.001, dlogits_add=bal["dlogits"])
    for k in ("dw_router", "dw_gate", "dw_up", "dw_down"):
        assert torch.equal(aux[k], grads[k])
    # what dlogits_add does: dw_router gains n^T d, dx gains d W_r^T, the experts nothing
    d = bal["dlogits"].double()
    gain = n.double().T @ d
    _within(aux["dw_router"].double() - plain["dw_router"].double(), gain,
            2.0**-15 * (n.double().abs().T @ d.abs()) + 2.0**-15 * plain["dw_router"].double().abs(), "dw_router")
    gx = d @ layer.w_router.double().T
    _within(aux["dx"].double() - plain["dx"].double(), gx,
            2 * (ROUND[dtype] + 2.0**-17) * (plain["dx"].double().abs() + aux["dx"].double().abs() + gx.abs()) + 1e-6, "dx")
    assert torch.equal(aux["dw_gate"], plain["dw_gate"])
    dn = aux["dx"].clone()
    dx, dg = torch.empty_like(x), torch.empty(D, device="cuda")
    ws = torch.zeros(M.rmsnorm_backward_workspace_size(T, D), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_backward(dn, s, layer.norm_weight, rstd, dx, dg, ws, ds=ds)
    assert torch.equal(dx, grads["dx"]) and torch.equal(dg, grads["dgamma"])
    layer.forward_train(n)
    with pytest.raises(RuntimeError):
        layer.backward_block(dy)  # the last forward was not a block's


def test_training_step_in_a_graph():
    """A captured training step of the block (norm, layer, balance loss, backward)
    gives at replay what the eager step gives on the same inputs."""
    T, D, F, E, K = 96, 64, 64, 4, 2
    layer = _layer(T, D, F, E, K, 5)
    g = _gen(4)
    x, res, dy = (_randn(g, T, D, dtype=torch.bfloat16) for _ in range(3))
    starts = torch.tensor([0, 40, 96], dtype=torch.int32, device="cuda")
    grads = {}

    def step():
        layer.forward_block_train(x, res)
        bal = layer.balance_loss(starts, c_balance=0.1, c_z=0.01)
        return layer.backward_block(dy, dlogits_add=bal["dlogits"], grads=grads or None)
    grads.update(step())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(_randn(g, T, D, dtype=torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in grads.items()}
    step()
    for k, v in grads.items():
        assert torch.equal(v, got[k]), k


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams at the same time."""
    g = _gen(30)
    cases = []
    for seed in (1, 2):
        logits, ids = _randn(g, 5000, 32), _ids(g, 5000, 32, 4)
        (c, l, s, d), _ = _balance(logits, ids, [0, 2000, 5000])
        cases.append((logits, ids, c, l, s, d))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for st, (logits, ids, *_r) in zip(streams, cases):
        with torch.cuda.stream(st):
            got.append([_balance(logits, ids, [0, 2000, 5000])[0] for _ in range(5)])
    torch.cuda.synchronize()
    for (_, _, *want), runs in zip(cases, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, want))
