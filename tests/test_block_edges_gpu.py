"""Edges of the operators around the layer on the GPU: values at the ends of the
types' ranges, calls that other tests do not make.

A comparison holds where the error is at most a finite tolerance, or where both
sides are the same infinity: a NaN is off.  Tolerances as in test_block_gpu: a
rounding is off by at most half a step (bf16 2^-8, fp32 2^-24 of the value), a
row's sum by 2^-17.
"""
import pytest
import torch

import mixture_experts_layer_55_b200 as M
from mixture_experts_layer_55_b200 import _binding as B

pytestmark = pytest.mark.gpu

ROUND = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}
SUM = 2.0**-17
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def within(got, ref, tol, what=""):
    got, ref = got.double(), ref.double()
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).broadcast_to(got.shape)
    err = (got - ref).abs()
    ok = ((err <= tol) & tol.isfinite()) | (got == ref)
    assert bool(ok.all()), (f"{what}: {int((~ok).sum())} off, {int(got.isnan().sum())} NaN, worst "
                            f"{float((err - tol).nan_to_num(nan=float('inf')).max()):.3e} over the tolerance")


# ---------------------------------------------------------------------- norm --

# (rms of the rows, eps): squares below fp32's range with eps 0 and with eps of their
# own size, above it, at and below the least normal value, at the largest
RANGE = [(1e-18, 0.0), (1e-18, 1e-36), (1e-18, 1e-31), (1e-20, 7e-31), (1e-30, 0.0), (1e-16, 1e-40), (3e-39, 0.0),
         (1e-42, 0.0), (1e-42, 1e-44), (1e-12, 0.0), (1e19, 0.0), (1e30, 1e-6), (1.5e38, 0.0), (1.5e38, 1e30), (0.0, 1e-36)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(3, 64), (40, 512), (700, 4096), (2, 16640)])
@pytest.mark.parametrize("scale,eps", RANGE)
def test_rmsnorm_range(scale, eps, T, D, dt):
    """A row of finite values has a finite norm, whatever its size: every row of the
    range beside rows of ordinary size, which it does not touch."""
    dtype = DT[dt]
    if dt == "bf16" and scale > 0:
        scale = max(scale, 1e-39)  # bf16's least value is 2^-133
    g = _gen(T + D)
    x = (0.25 + torch.rand(T, D, generator=g, device="cuda"))
    x[:, ::3] *= -1
    x[::2] *= scale
    x = x.to(dtype)
    gamma = 1 + 0.3 * _randn(g, D)
    eps = float(torch.tensor(eps))  # as the call takes it, in fp32
    n, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    q, qs = torch.empty(T, D, dtype=torch.uint8, device="cuda"), torch.empty(T, D // 32, dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm(x, gamma, n, rstd=rstd, q=q, q_scales=qs, eps=eps)
    r = (x.double().square().mean(1) + eps).rsqrt()
    # rstd leaves fp32 above (an infinity), or falls below its normal values (a step of 2^-149)
    big = r > torch.finfo(torch.float32).max
    assert bool((rstd[big] == float("inf")).all())
    within(rstd[~big], r[~big], SUM * r[~big] + 2.0**-149, "rstd")
    ref = x.double() * r[:, None] * gamma.double()
    within(n, ref, (ROUND[dtype] + SUM) * ref.abs() + 1e-38, "n")
    assert bool((qs != 255).all())
    # the 8-bit rows: half an e4m3 step, 2^-4 of a value or half the least step of its block
    v = q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32)) * torch.exp2(qs.double() - 127)[..., None]
    step = torch.exp2(qs.double() - 127).repeat_interleave(32, 1)
    within(v.flatten(-2), n, 2.0**-4 * n.double().abs() + 2.0**-10 * step, "values")


# ------------------------------------------------------------------- balance --

def _balance(logits, ids, starts, score, cb, cz):
    T, E = logits.shape
    S = len(starts) - 1
    cfg = M.MoeConfig.make(T, 8, 8, E, ids.shape[1], "bf16", score_func=score)
    ws = torch.zeros(M.balance_workspace_size(cfg, S), dtype=torch.uint8, device="cuda")
    out = (torch.empty(S, E, dtype=torch.int32, device="cuda"), torch.empty(2, device="cuda"),
           torch.empty(S, device="cuda"), torch.empty(T, E, device="cuda"))
    M.moe_balance_loss(cfg, logits, ids, torch.tensor(starts, dtype=torch.int32, device="cuda"), out[0], out[1], out[2],
                       ws, dlogits=out[3], c_balance=cb, c_z=cz)
    assert B.moe_get_device_status(ws) == 0
    return out


def _balance_ref(logits, ids, starts, score, cb, cz):
    """(seq_loss, dlogits, magnitude of the gradient's terms) in 64 bits, from the
    formulas; every token counts."""
    T, E = logits.shape
    K, S = ids.shape[1], len(starts) - 1
    l = logits.double()
    soft, lse = torch.softmax(l, 1), torch.logsumexp(l, 1, keepdim=True)
    s = torch.sigmoid(l)
    p, dp = (soft, soft) if score == "softmax" else (s / s.sum(1, keepdim=True),) * 2
    if score != "softmax":
        dp = p * torch.sigmoid(-l)
    seq, d, mag = [], torch.zeros_like(l), torch.zeros_like(l)
    for a, b in zip(starts[:-1], starts[1:]):
        f = torch.bincount(ids[a:b].flatten().long(), minlength=E).double() / ((b - a) * K)
        c = (p[a:b] * f).sum(1, keepdim=True)
        seq.append(E * c.mean())
        k = cb * E / (S * (b - a))
        d[a:b], mag[a:b] = k * dp[a:b] * (f - c), abs(k) * dp[a:b] * (f + c)
    # lse is the sum of the largest logit and a logarithm, either sign each: its error
    # goes by 2^-24 of those two, which may cancel to a smaller lse
    top = l.amax(1, keepdim=True)
    d, mag = d + cz * 2 * lse / T * soft, mag + abs(cz) * 2 * (top.abs() + (lse - top)) / T * soft
    return torch.stack(seq), d, mag


# An element of the gradient is off by at most 2^-18 of its terms: two exponentials to
# 2^-22 and the rounding of their arguments, sums of 8 + 5 terms and some ten
# products and quotients at 2^-24 each.
GRAD = 2.0**-18


def _ids(g, T, E, K):
    return torch.rand(T, E, generator=g, device="cuda").topk(K, 1).indices.to(torch.int32).contiguous()


@pytest.mark.parametrize("E,K", [(8, 2), (17, 3), (64, 6), (256, 8)])
@pytest.mark.parametrize("level,spread", [(-4, 1), (-19.5, 1), (-20.5, 1), (-60, 1), (-88, 0.3), (-88, 12), (-120, 5), (-300, 1),
                                          (12, 2), (25, 3), (60, 1), (0, 25)])
def test_balance_sigmoid_levels(level, spread, E, K):
    """Sigmoid scores of logits far from zero: their shares of a token's sum are
    what they are however small all of them get, and the gradient of a saturated
    score is its own size, p (1 - sigmoid), not a difference of numbers near 1."""
    g = _gen(E + 7)
    T = 300
    logits = level + spread * (2 * torch.rand(T, E, generator=g, device="cuda") - 1)
    ids = _ids(g, T, E, K)
    starts = [0, 120, 300]
    counts, losses, seq, d = _balance(logits, ids, starts, "sigmoid", 0.01, 0.0)
    rs, rd, mag = _balance_ref(logits, ids, starts, "sigmoid", 0.01, 0.0)
    within(seq, rs, 2.0**-18 * rs, "seq_loss")
    within(d, rd, GRAD * mag + 1e-38, "dlogits")


@pytest.mark.parametrize("score,level", [("sigmoid", -4.0), ("sigmoid", -10.0), ("sigmoid", -60.0), ("softmax", -10.0)])
def test_balance_gradient_is_fp32s(score, level):
    """Root mean square of the gradient's error: some fifteen independent roundings
    of 2^-24 / sqrt(3) each are 2^-22.8 of its terms, an exponential's ulp beside
    them; held to twice 2^-22."""
    g = _gen(6)
    T, E, K = 2000, 64, 4
    logits, ids = level + _randn(g, T, E), _ids(g, T, E, K)
    *_, d = _balance(logits, ids, [0, T], score, 0.01, 0.0)
    _, rd, mag = _balance_ref(logits, ids, [0, T], score, 0.01, 0.0)
    rms = float(((d.double() - rd) / mag).square().mean().sqrt())
    assert rms <= 2.0**-21


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,gap", [(1, 20), (60, 15), (60, 22), (3000, 18), (70001, 14)])
def test_balance_loss_of_experts_against_their_scores(T, gap, score):
    """Ids that a selection bias turned against the scores: a token's share of the
    loss is a small number, and the loss keeps its digits.  A share is held in units
    of 2^-(63 - b), b the bits of T."""
    g = _gen(T)
    E, K = 16, 2
    logits = _randn(g, T, E) - 3
    logits[:, 4:8] -= gap
    ids = (4 + _ids(g, T, 4, K)).contiguous()
    starts = [0, T // 3, T] if T > 2 else [0, T]
    counts, losses, seq, d = _balance(logits, ids, starts, score, 0.01, 0.001)
    rs, rd, mag = _balance_ref(logits, ids, starts, score, 0.01, 0.001)
    within(seq, rs, 2.0**-18 * rs + E * 2.0**-(64 - T.bit_length()), "seq_loss")
    within(losses[1], rs.mean(), 2.0**-18 * rs.mean() + E * 2.0**-(64 - T.bit_length()), "balance")
    within(d, rd, GRAD * mag + 1e-38, "dlogits")


# ------------------------------------------------------------- 8-bit experts --

def _mx8(v):
    """v (.., n) as e4m3 blocks of 32 under power-of-two scales (any valid pair will do)."""
    b = v.unflatten(-1, (-1, 32))
    e = torch.ceil(torch.log2(b.abs().amax(-1).clamp(min=1e-30) / 448)).clamp(-126, 127)
    return (b / torch.exp2(e)[..., None]).to(torch.float8_e4m3fn).flatten(-2), (e + 127).to(torch.uint8)


# pairs, single CTAs, few rows, few rows with the down product in parts
@pytest.mark.parametrize("T,D,F,E,K", [(400, 256, 192, 2, 2), (100, 224, 160, 4, 2), (30, 256, 192, 8, 2), (2, 256, 4096, 8, 2)])
def test_experts_mx8_see_the_rows_of_their_own_call(T, D, F, E, K):
    """Calls in a row on the same buffers with other rows each time: every call's
    output is its own rows', bit for bit (the down product starts under the end of
    the product that writes what it reads)."""
    g = _gen(T)
    R = T * K
    counts = torch.bincount(_ids(g, T, E, K).flatten().long(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    w = []
    for n, k in ((F, D), (F, D), (D, F)):
        w += list(_mx8(0.05 * _randn(g, E, n, k)))
    rows = [_mx8(s * _randn(g, R, D)) for s in (1.0, 30.0, 0.01)]
    cfg = M.MoeConfig.make(T, D, F, E, K, "bf16")
    xq, xs = torch.empty_like(rows[0][0]), torch.empty_like(rows[0][1])
    hq, hs = torch.empty(R, F, dtype=torch.uint8, device="cuda"), torch.empty(R, F // 32, dtype=torch.uint8, device="cuda")
    y, ws = torch.empty(R, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(M.mx8_workspace_size(cfg), dtype=torch.uint8, device="cuda")

    def call(i):
        xq.view(torch.uint8).copy_(rows[i][0].view(torch.uint8))
        xs.copy_(rows[i][1])
        M.moe_expert_ffn_mx8(cfg, xq, xs, offsets, None, None, w, hq, hs, y, ws)
        return y.clone(), hs.clone()
    want = []
    for i in range(3):
        want.append(call(i))
        torch.cuda.synchronize()
    assert not torch.equal(want[0][1], want[1][1])
    got = [call(i % 3) for i in range(60)]
    for i, (yi, hi) in enumerate(got):
        assert torch.equal(yi, want[i % 3][0]) and torch.equal(hi, want[i % 3][1]), i
    assert B.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("T,E", [(400, 1), (60, 1), (20, 1)])  # pairs, single CTAs, few rows
def test_experts_mx8_silu_far_below_zero(T, E):
    """Gates from -87 on, where e^-g passes 2^126, beside values that make g e^g u a
    number of ordinary size: h is silu(g) u, to its own rounding of 2^-4 (or half its
    block's least step) and that of e^g, a denormal number (half a step, 2^-150)."""
    D, F = 32, 64
    gates = torch.linspace(-86.5, -95, T, device="cuda")
    x = torch.zeros(T, D, device="cuda")
    x[:, 0] = 1
    x[:, 1] = torch.floor(-gates)          # 1.0 x whole part and 1.0 x a fraction of it, both exact in 8 bits
    x[:, 1] = (x[:, 1] / 8).floor() * 8    # 80, 88
    x[:, 2] = ((-gates - x[:, 1]).clamp(0, 8) * 2).round() / 2
    xq, xs = _mx8(x)
    xv = (xq.double().unflatten(-1, (-1, 32)) * torch.exp2(xs.double() - 127)[..., None]).flatten(-2)
    gate, up, down = torch.zeros(E, F, D, device="cuda"), torch.zeros(E, F, D, device="cuda"), torch.zeros(E, D, F, device="cuda")
    gate[:, :, 1] = gate[:, :, 2] = -1
    up[:, :, 0] = 2.0**120 * (1 + torch.arange(F, device="cuda") % 7)
    w = [t for v in (gate, up, down) for t in _mx8(v)]
    cfg = M.MoeConfig.make(T, D, F, E, 1, "bf16")
    hq, hs = torch.empty(T, F, dtype=torch.uint8, device="cuda"), torch.empty(T, F // 32, dtype=torch.uint8, device="cuda")
    y, ws = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(M.mx8_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    M.moe_expert_ffn_mx8(cfg, xq, xs, offsets, None, None, w, hq, hs, y, ws)
    assert B.moe_get_device_status(ws) == 0
    g = xv @ gate[0].double().T
    assert float(g.min()) < -94 and float(g.max()) > -88
    h = g * torch.sigmoid(g) * (xv @ up[0].double().T)
    step = torch.exp2(hs.double() - 127).repeat_interleave(32, 1)
    got = hq.view(torch.float8_e4m3fn).double() * step
    # the fast exponential, 2 + 1.2 |g| units of 2^-23, and its own half step
    eh = h.abs() * ((4 + 1.2 * g.abs()) * 2.0**-23 + 2.0**-150 / torch.exp(g))
    within(got, h, 2.0**-4 * (h.abs() + eh) + 2.0**-10 * step + eh, "h")


def test_experts_mx8_one_workspace_for_every_batch():
    """The workspace of the largest batch through all of them, forms in turn: the bits
    of calls with workspaces of their own."""
    D, F, E, K = 256, 4096, 4, 2
    g = _gen(2)
    w = [t for n, k in ((F, D), (F, D), (D, F)) for t in _mx8(0.05 * _randn(g, E, n, k))]
    size = M.mx8_workspace_size(M.MoeConfig.make(600, D, F, E, K, "bf16"))
    shared = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    shared[size:] = 77
    for T in (600, 1, 20, 3, 100, 2, 47, 600):
        cfg, R = M.MoeConfig.make(T, D, F, E, K, "bf16"), T * K
        counts = torch.bincount(_ids(g, T, E, K).flatten().long(), minlength=E)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        xq, xs = _mx8(_randn(g, R, D))
        hq, hs = torch.empty(R, F, dtype=torch.uint8, device="cuda"), torch.empty(R, F // 32, dtype=torch.uint8, device="cuda")
        y = [torch.empty(R, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        own = torch.zeros(M.mx8_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        for out, ws in zip(y, (own, shared[:size])):
            M.moe_expert_ffn_mx8(cfg, xq, xs, offsets, None, None, w, hq, hs, out, ws)
            assert B.moe_get_device_status(ws) == 0
        assert torch.equal(*y)
    assert bool((shared[size:] == 77).all())


# ------------------------------------------------------- the layer's own paths --

def _layer(T, D, F, E, K, seed, dtype=torch.bfloat16, **kw):
    g = _gen(seed)
    wr = 0.1 * _randn(g, D, E)
    w = [0.05 * _randn(g, E, D, F), 0.05 * _randn(g, E, D, F), 0.05 * _randn(g, E, F, D)]
    return M.MoELayer(T, wr, *(v.to(dtype) for v in w), K, norm_weight=1 + 0.2 * _randn(g, D), **kw)


@pytest.mark.parametrize("experts", [None, "mx8"])
def test_block_outputs_over_its_inputs(experts):
    """y over x or over the residual where the sum has a buffer of its own: the same
    bits as into a fresh one."""
    T, D = 90, 128
    layer = _layer(T, D, 64, 4, 2, 1, experts=experts)
    g = _gen(3)
    x, res = _randn(g, T, D, dtype=torch.bfloat16), _randn(g, T, D, dtype=torch.bfloat16)
    y, s = layer.forward_block(x, res)
    for over in range(2):
        a = [x.clone(), res.clone()]
        y2, s2 = layer.forward_block(*a, y=a[over])
        assert y2 is a[over] and torch.equal(y2, y) and torch.equal(s2, s)
    with pytest.raises(ValueError):
        layer.forward_block(x, y=x)


def test_layer_balance_loss_shows_malformed_borders():
    """The flag of a batch with malformed borders can be asked for, call by call; the
    next call is clean."""
    T, D = 40, 64
    layer = _layer(T, D, 64, 4, 2, 5)
    layer.forward_block_train(_randn(_gen(1), T, D, dtype=torch.bfloat16))
    good = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    want = layer.balance_loss(good, c_balance=0.1)
    assert B.moe_get_device_status(want["workspace"]) == 0
    for starts in ([0, 30, 20], [0, 10, 41], [-1, 10, 40]):
        bad = layer.balance_loss(torch.tensor(starts, dtype=torch.int32, device="cuda"), c_balance=0.1)
        assert B.moe_get_device_status(bad["workspace"]) == B.MOE_DEVFLAG_BOUNDS
    again = layer.balance_loss(good, c_balance=0.1)
    assert B.moe_get_device_status(again["workspace"]) == 0
    for k in ("losses", "seq_loss", "counts", "dlogits"):
        assert torch.equal(again[k], want[k])


def test_norm_in_graphs_of_any_shape():
    """The norm, which is launched under the end of what stands before it, captured as
    a graph's first node, behind a copy and a fill, behind two branches, and on two
    branches at once: what it reads has been written at each replay."""
    g = _gen(9)
    T, D = 64, 512
    x, src, other = (_randn(g, T, D) for _ in range(3))
    gamma = torch.ones(D, device="cuda")
    n, n2 = torch.empty_like(x), torch.empty_like(x)
    for kind in ("first", "copy", "fill", "two branches before", "two branches"):
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            cur = torch.cuda.current_stream()
            if kind == "copy":
                x.copy_(src)
            elif kind == "fill":
                x.fill_(2.0)
            elif kind == "two branches before":
                side.wait_stream(cur)
                with torch.cuda.stream(side):
                    x.copy_(src)
                    x.mul_(2)
                other.copy_(src)
                cur.wait_stream(side)
            elif kind == "two branches":
                x.mul_(1.5)
                side.wait_stream(cur)
                with torch.cuda.stream(side):
                    M.moe_rmsnorm(x, gamma, n2)
            M.moe_rmsnorm(x, gamma, n)
            if kind == "two branches":
                cur.wait_stream(side)
        for _ in range(3):
            src.normal_(generator=g)
            graph.replay()
            torch.cuda.synchronize()
            ref = x.double() * (x.double().square().mean(1, keepdim=True) + 1e-6).rsqrt()
            within(n, ref, (2.0**-24 + SUM) * ref.abs(), kind)
            assert kind != "two branches" or torch.equal(n, n2)
