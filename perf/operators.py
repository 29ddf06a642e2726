"""Measured cases of the operators around the expert layer's products.

Three operators, each with its plain form (elementary torch operations) and the
calls a user makes of this framework:

  norm      residual addition and root-mean-square norm before the layer, with
            the optional 8-bit output the 8-bit experts read; and its backward
  balance   balance loss, z-loss and per-expert counts over the sequences of a
            ragged, padded batch, with the gradient of the routing logits
  experts   the grouped SwiGLU experts on 8-bit rows and weights

8-bit data is e4m3 in blocks of 32 along the contracted axis, each block with
one power-of-two scale 2^(byte - 127).
"""
import math

import torch

own = False

EPS = 1e-6
MASK_NONE, MASK_TAIL, MASK_RANDOM = "none", "tail", "random"


# ------------------------------------------------------------------ the cases --

def listed():
    return [
        # training, Mixtral-shaped batch: forward of the norm before the layer
        dict(name="norm_train", op="norm", T=8192, D=4096, dtype="bf16", residual=True, bits8=False),
        # the same batch, backward: input and weight gradients
        dict(name="norm_train_backward", op="norm_backward", T=8192, D=4096, dtype="bf16", residual=True),
        # a decode step of 128 sequences at d_model 7168, feeding the 8-bit experts
        dict(name="norm_8bit_decode", op="norm", T=128, D=7168, dtype="bf16", residual=True, bits8=True),
        # the small fp32 layer: latency
        dict(name="norm_fp32", op="norm", T=512, D=256, dtype="f32", residual=False, bits8=False),
        # a ragged batch at an odd width, fp32 backward without a second gradient
        dict(name="norm_odd_backward", op="norm_backward", T=1001, D=1000, dtype="f32", residual=False),
        # training batch of four full sequences, 8 experts
        dict(name="balance_full", op="balance", T=8192, E=8, K=2, S=4, score="softmax", mask=MASK_NONE),
        # fine-grained experts, sigmoid scores, 37 packed sequences with padding tokens
        dict(name="balance_packed", op="balance", T=16384, E=64, K=6, S=37, score="sigmoid", mask=MASK_TAIL),
        # the widest router and the longest batch
        dict(name="balance_wide", op="balance", T=32768, E=256, K=8, S=16, score="softmax", mask=MASK_RANDOM),
        # one token through the small layer: latency
        dict(name="experts_one_token", op="experts", T=1, D=256, F=512, E=8, K=2, skew=0.0),
        # a large batch of the Mixtral-shaped layer (prefill)
        dict(name="experts_prefill", op="experts", T=8192, D=4096, F=14336, E=8, K=2, skew=0.0),
        # fine-grained experts with a skewed load
        dict(name="experts_fine", op="experts", T=16384, D=2048, F=1408, E=64, K=6, skew=0.5),
        # a decode step over 256 experts: the weight stream
        dict(name="experts_decode", op="experts", T=128, D=7168, F=2048, E=256, K=8, skew=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "balance", "balance", "experts", "experts"])
    if op in ("norm", "norm_backward"):
        T = _log_int(rng, 1, 16384)
        bits8 = op == "norm" and rng.random() < 0.5
        D = _log_int(rng, 32, 8192, 32 if bits8 else 8)
        while T * D > 8192 * 4096:
            T = max(1, T // 2)
        c = dict(op=op, T=T, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.7)
        if op == "norm":
            c["bits8"] = bits8
        return c
    if op == "balance":
        T = _log_int(rng, 1, 32768)
        E = _log_int(rng, 2, 256)
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(8, E)), S=min(T, _log_int(rng, 1, 512)),
                    score=rng.choice(["softmax", "sigmoid"]),
                    mask=rng.choice([MASK_NONE, MASK_TAIL, MASK_RANDOM]))
    T = _log_int(rng, 1, 8192)
    E = _log_int(rng, 1, 128)
    D = _log_int(rng, 64, 7168, 32)
    F = _log_int(rng, 64, 7168, 32)
    while E * D * F > 1 << 29:
        E = max(1, E // 2)
    return dict(op=op, T=T, D=D, F=F, E=E, K=rng.randint(1, min(8, E)), skew=rng.choice([0.0, 0.5]))


# ----------------------------------------------------------------- the inputs --

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _block_exponent(amax):
    """The least exponent e with amax <= 448 * 2^e (448 = 1.75 * 2^8, the largest
    e4m3 value), for a tensor of block maxima; -127 for a block of zeros."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _quantize(v):
    """(e4m3 values, scale bytes) of v (.., n), n a multiple of 32, in v's precision."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    e = _block_exponent(b.abs().amax(-1))
    q = (b * torch.exp2(-e.to(v.dtype))[..., None]).to(torch.float8_e4m3fn)
    return q.reshape(v.shape), (e + 127).to(torch.uint8)


def _values(q, scales, dt=torch.float32):
    """The values that 8-bit data stands for."""
    b = q.to(dt).reshape(*scales.shape, 32)
    return (b * torch.exp2(scales.to(dt) - 127)[..., None]).reshape(q.shape)


def _prepare_norm(case, g):
    T, D, dt = case["T"], case["D"], _dtype(case)
    st = dict(case=case, gamma=1 + 0.1 * torch.randn(D, generator=g, device="cuda"))
    rows = torch.exp(0.5 * torch.randn(T, 1, generator=g, device="cuda"))  # rows of different sizes
    x = (rows * torch.randn(T, D, generator=g, device="cuda")).to(dt)
    if case["op"] == "norm":
        st["x"] = x
        st["residual"] = torch.randn(T, D, generator=g, device="cuda").to(dt) if case["residual"] else None
        st["s"] = torch.empty_like(x) if case["residual"] else None
        st["n"] = torch.empty_like(x)
        st["rstd"] = torch.empty(T, device="cuda")
        if case["bits8"]:
            st["q"] = torch.empty(T, D, dtype=torch.float8_e4m3fn, device="cuda")
            st["q_scales"] = torch.empty(T, D // 32, dtype=torch.uint8, device="cuda")
            st["values"] = torch.empty_like(x)
        return st
    st["s"] = x  # the forward's stored sum and reciprocal roots
    st["rstd"] = torch.cat([1 / torch.sqrt(c.double().square().mean(1) + EPS) for c in x.split(2048)]).float()
    st["dn"] = torch.randn(T, D, generator=g, device="cuda").to(dt)
    st["ds"] = torch.randn(T, D, generator=g, device="cuda").to(dt) if case["residual"] else None
    st["dx"], st["dgamma"] = torch.empty_like(x), torch.empty(D, device="cuda")
    return st


def _prepare_balance(case, g):
    T, E, K, S = case["T"], case["E"], case["K"], case["S"]
    popular = 0.5 * torch.randn(E, generator=g, device="cuda")  # an unbalanced router
    logits = torch.randn(T, E, generator=g, device="cuda") + popular
    ids = torch.topk(logits, K, dim=1).indices.to(torch.int32)
    # sequence borders: even where every token is full, else ragged with a few
    # tokens behind the last sequence
    if case["mask"] == MASK_NONE:
        starts = torch.arange(S + 1, device="cuda") * T // S
    else:
        # some of these sequences come out empty, as in a serving or packing queue
        cuts = torch.sort(torch.randint(0, T + 1, (S,), generator=g, device="cuda")).values
        starts = torch.cat([torch.zeros(1, dtype=cuts.dtype, device="cuda"), cuts])
    mask = None
    if case["mask"] == MASK_RANDOM:
        mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    elif case["mask"] == MASK_TAIL:  # the last eighth of every sequence is padding
        at = torch.arange(T, device="cuda")
        seq = torch.searchsorted(starts[1:].contiguous(), at, right=True).clamp(max=S - 1)
        mask = (at - starts[seq] < (starts[seq + 1] - starts[seq]) * 7 // 8 + 1).to(torch.uint8)
    return dict(case=case, logits=logits, ids=ids, starts=starts.to(torch.int32), mask=mask,
                counts=torch.empty(S, E, dtype=torch.int32, device="cuda"),
                losses=torch.empty(2, device="cuda"), seq_loss=torch.empty(S, device="cuda"),
                dlogits=torch.empty(T, E, device="cuda"))


def _weights(E, N, K, g):
    """(E, N, K) 8-bit weights of standard deviation 0.02 and their scales."""
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        w = 0.02 * torch.randn(min(step, E - e), N, K, generator=g, device="cuda")
        q[e:e + step], s[e:e + step] = _quantize(w)
    return q, s


def _prepare_experts(case, g):
    T, D, F, E, K = case["T"], case["D"], case["F"], case["E"], case["K"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits += case["skew"] * torch.randn(E, generator=g, device="cuda")
    top = torch.topk(logits, K, dim=1)
    weight = torch.softmax(top.values, 1).float().contiguous()
    order = torch.sort(top.indices.reshape(-1), stable=True)
    perm = order.indices
    counts = torch.bincount(order.values, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    xq, xs = _quantize(torch.randn(T, D, generator=g, device="cuda"))
    R = T * K
    st = dict(case=case, perm=perm.to(torch.int32), offsets=offsets.to(torch.int32), topk_w=weight,
              xq=xq.view(torch.uint8)[perm // K].view(torch.float8_e4m3fn), xs=xs[perm // K].contiguous(),
              hq=torch.empty(R, F, dtype=torch.float8_e4m3fn, device="cuda"),
              hs=torch.empty(R, F // 32, dtype=torch.uint8, device="cuda"),
              y=torch.empty(R, D, dtype=torch.bfloat16, device="cuda"),
              most=int(counts.max()))
    st["w"] = _weights(E, F, D, g) + _weights(E, F, D, g) + _weights(E, D, F, g)  # gate, up, down
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "balance":
        return _prepare_balance(case, g)
    if case["op"] == "experts":
        return _prepare_experts(case, g)
    return _prepare_norm(case, g)


# ------------------------------------------------------------ the plain forms --

def _plain_norm(st):
    dt = st["x"].dtype
    s = st["x"].float()
    if st["residual"] is not None:
        s = (s + st["residual"].float()).to(dt).float()  # the sum as it is stored
    rstd = 1 / torch.sqrt(s.square().mean(1) + EPS)
    n = (s * rstd[:, None] * st["gamma"]).to(dt)
    out = dict(n=n, rstd=rstd)
    if st["residual"] is not None:
        out["s"] = s.to(dt)
    if st["case"]["bits8"]:
        out["values"] = _values(*_quantize(n.float())).to(dt)
    return out


def _plain_norm_backward(st):
    s, rstd = st["s"].float(), st["rstd"][:, None]
    xhat, dn = s * rstd, st["dn"].float()
    g = dn * st["gamma"]
    dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["ds"] is not None:
        dx = dx + st["ds"].float()
    return dict(dx=dx.to(st["s"].dtype), dgamma=(dn * xhat).sum(0))


C_BALANCE, C_Z = 0.01, 0.001


def _balance(st, dt):
    """The balance operator's results in the precision dt."""
    c, K, E = st["case"], st["case"]["K"], st["case"]["E"]
    T, S = c["T"], c["S"]
    starts = st["starts"].long()
    at = torch.arange(T, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), at, right=True)
    on = (at < starts[-1]) & (seq < S)
    if st["mask"] is not None:
        on = on & (st["mask"] != 0)
    seq = seq.clamp(max=S - 1)
    tokens = torch.zeros(S, dtype=torch.int64, device=starts.device).index_add_(0, seq, on.long())
    counts = torch.zeros(S * E, dtype=torch.int64, device=starts.device).index_add_(
        0, (seq[:, None] * E + st["ids"].long()).reshape(-1), on.long()[:, None].expand(T, K).reshape(-1))
    counts = counts.reshape(S, E)
    used = (tokens > 0).sum().clamp(min=1).to(dt)
    total = tokens.sum().clamp(min=1).to(dt)
    n = tokens.clamp(min=1).to(dt)
    f = counts.to(dt) / (n[:, None] * K)
    l = torch.where(on[:, None], st["logits"], torch.zeros((), device=starts.device)).to(dt)
    top = l.amax(1, keepdim=True)
    ex = torch.exp(l - top)
    lse = (top + torch.log(ex.sum(1, keepdim=True)))[:, 0]
    soft = ex / ex.sum(1, keepdim=True)
    if c["score"] == "softmax":
        p, dp = soft, soft
    else:
        s = 1 / (1 + torch.exp(-l))
        p = s / s.sum(1, keepdim=True)
        dp = p * (1 - s)
    fs = f[seq]
    dot = (fs * p).sum(1)
    zero = torch.zeros((), dtype=torch.float64, device=starts.device)
    sums = torch.zeros(S, dtype=torch.float64, device=starts.device).index_add_(0, seq, torch.where(on, dot.double(), zero))
    seq_loss = E * sums / tokens.clamp(min=1)
    z = torch.where(on, lse.double().square(), zero).sum() / total.double()
    d = (C_BALANCE * E / used / n)[seq][:, None] * dp * (fs - dot[:, None])
    d = d + (2 * C_Z / total) * lse[:, None] * soft
    d = torch.where(on[:, None], d, torch.zeros((), dtype=dt, device=starts.device))
    return dict(counts=counts.to(torch.int32), seq_loss=seq_loss, dlogits=d,
                losses=torch.stack([z, seq_loss.sum() / used.double()]))


def _plain_balance(st):
    r = _balance(st, torch.float32)
    return {k: v.float() if v.is_floating_point() else v for k, v in r.items()}


def _plain_experts(st):
    c, offsets = st["case"], st["offsets"].long()
    R, E, M = st["perm"].numel(), c["E"], st["most"]
    gq, gs, uq, us, dq, ds = st["w"]
    at = offsets[:-1, None] + torch.arange(M, device=offsets.device)  # (E, M) rows, padded to the longest
    fits = at < offsets[1:, None]
    at = torch.where(fits, at, torch.zeros((), dtype=at.dtype, device=at.device))
    x = _values(st["xq"], st["xs"])[at]
    gate = torch.bmm(x, _values(gq, gs).transpose(1, 2))
    up = torch.bmm(x, _values(uq, us).transpose(1, 2))
    h = _values(*_quantize(gate / (1 + torch.exp(-gate)) * up))
    y = torch.bmm(h, _values(dq, ds).transpose(1, 2))
    w = st["topk_w"].reshape(-1)[st["perm"].long()]
    out = torch.empty(R, c["D"], device=y.device)
    out[at[fits]] = y[fits]
    return dict(y=(w[:, None] * out).to(torch.bfloat16))


# ------------------------------------------------------- the framework's calls --

def _own_norm(st):
    import mixture_experts_layer_55_b200 as M
    out = dict(n=st["n"], rstd=st["rstd"])
    if not st["case"]["bits8"]:
        M.moe_rmsnorm(st["x"], st["gamma"], st["n"], residual=st["residual"], s=st["s"], rstd=st["rstd"], eps=EPS)
    else:
        M.moe_rmsnorm(st["x"], st["gamma"], st["n"], residual=st["residual"], s=st["s"], rstd=st["rstd"],
                      q=st["q"], q_scales=st["q_scales"], eps=EPS)
        M.moe_mx8_dequantize(st["q"], st["q_scales"], st["values"])
        out["values"] = st["values"]
    if st["residual"] is not None:
        out["s"] = st["s"]
    return out


def _own_norm_backward(st):
    import mixture_experts_layer_55_b200 as M
    if "ws" not in st:
        st["ws"] = torch.zeros(M.rmsnorm_backward_workspace_size(*st["s"].shape), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_backward(st["dn"], st["s"], st["gamma"], st["rstd"], st["dx"], st["dgamma"], st["ws"], ds=st["ds"])
    return dict(dx=st["dx"], dgamma=st["dgamma"])


def _own_balance(st):
    import mixture_experts_layer_55_b200 as M
    c = st["case"]
    if "ws" not in st:
        st["cfg"] = M.MoeConfig.make(c["T"], 8, 8, c["E"], c["K"], "bf16", score_func=c["score"])
        st["ws"] = torch.zeros(M.balance_workspace_size(st["cfg"], c["S"]), dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(st["cfg"], st["logits"], st["ids"], st["starts"], st["counts"], st["losses"], st["seq_loss"],
                       st["ws"], token_mask=st["mask"], dlogits=st["dlogits"], c_balance=C_BALANCE, c_z=C_Z)
    return dict(counts=st["counts"], seq_loss=st["seq_loss"], dlogits=st["dlogits"], losses=st["losses"])


def _own_experts(st):
    import mixture_experts_layer_55_b200 as M
    c = st["case"]
    if "ws" not in st:
        st["cfg"] = M.MoeConfig.make(c["T"], c["D"], c["F"], c["E"], c["K"], "bf16")
        st["ws"] = torch.zeros(M.mx8_workspace_size(st["cfg"]), dtype=torch.uint8, device="cuda")
    M.moe_expert_ffn_mx8(st["cfg"], st["xq"], st["xs"], st["offsets"], st["perm"], st["topk_w"], st["w"],
                         st["hq"], st["hs"], st["y"], st["ws"])
    return dict(y=st["y"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(norm=_own_norm, norm_backward=_own_norm_backward, balance=_own_balance, experts=_own_experts)[op](state)
    return dict(norm=_plain_norm, norm_backward=_plain_norm_backward, balance=_plain_balance,
                experts=_plain_experts)[op](state)


# ---------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, s = case["T"] * case["D"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            b = n * s * (4 if case["residual"] else 2) + 4 * case["T"] + 4 * case["D"]  # x (+ residual, sum), n
            if case["bits8"]:
                b += n * (1 + 1 / 32) * 2 + n * s  # written, read back, its values
            return dict(bytes=b, flops=n * (8 if case["bits8"] else 5))
        return dict(bytes=n * s * (4 if case["residual"] else 3) + 4 * case["T"] + 8 * case["D"], flops=n * 9)
    T, E, K = case["T"], case["E"], case["K"]
    if op == "balance":
        return dict(bytes=T * E * 8 + T * K * 4 + (T if case["mask"] != MASK_NONE else 0) + case["S"] * (4 * E + 8),
                    flops=T * E * 12)
    D, F = case["D"], case["F"]
    R, active = T * K, min(E, T * K)
    weights = 3 * active * D * F * (1 + 1 / 32)
    return dict(bytes=weights + R * D * (1 + 1 / 32) + R * D * 2 + R * 8, flops=6 * R * D * F)


# --------------------------------------------------------------- in 64 bits --

def _round_block(v):
    """v (.., 32) in 64 bits rounded to e4m3 at its block's scale: a step of
    2^-3 of the value's binade, of 2^-9 below 2^-6, ties to even."""
    top = v.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448))
    for k in (-1, 0, 1):  # the least e whose range holds the maximum, whatever log2 rounded to
        e = torch.where((top <= 448 * torch.exp2(e - 1)) & (k < 1), e - 1, e)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(-127, 127)
    u = v / torch.exp2(e)
    binade = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
    binade = torch.where(torch.exp2(binade) > u.abs().clamp(min=2.0 ** -6), binade - 1, binade)
    step = torch.exp2(binade - 3)
    return torch.round(u / step) * step * torch.exp2(e)


def _exact_rounded(v):
    return _round_block(v.reshape(*v.shape[:-1], -1, 32)).reshape(v.shape)


def _exact_norm(st):
    dt, gamma = st["x"].dtype, st["gamma"].double()
    out = dict(n=[], rstd=[], s=[], values=[])
    for i in range(0, st["x"].shape[0], 2048):
        s = st["x"][i:i + 2048].double()
        if st["residual"] is not None:
            s = s + st["residual"][i:i + 2048].double()
            out["s"].append(s)
            s = s.to(dt).double()
        r = (s.square().mean(1) + EPS).rsqrt()
        n = s * r[:, None] * gamma
        out["n"].append(n)
        out["rstd"].append(r)
        if st["case"]["bits8"]:
            out["values"].append(_exact_rounded(n.to(dt).double()))
    return {k: torch.cat(v) for k, v in out.items() if v}


def _exact_norm_backward(st):
    gamma, dx, dgamma = st["gamma"].double(), [], 0
    for i in range(0, st["s"].shape[0], 2048):
        at = slice(i, i + 2048)
        s, r, dn = st["s"][at].double(), st["rstd"][at].double()[:, None], st["dn"][at].double()
        # n = s r gamma with r = (mean s^2 + eps)^(-1/2): dr/ds = -r^3 s / D
        d = r * gamma * dn - r.pow(3) * s * (dn * gamma * s).sum(1, keepdim=True) / s.shape[1]
        dx.append(d if st["ds"] is None else d + st["ds"][at].double())
        dgamma = dgamma + (dn * s * r).sum(0)
    return dict(dx=torch.cat(dx), dgamma=dgamma)


def _exact_balance(st):
    """Sequence by sequence, the gradient by the derivative of the sum itself."""
    c = st["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    starts = st["starts"].tolist()
    on = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"] != 0
    rows = [torch.nonzero(on[a:b])[:, 0] + a for a, b in zip(starts[:-1], starts[1:])]
    used, total = max(1, sum(len(r) > 0 for r in rows)), max(1, sum(len(r) for r in rows))
    counts = torch.zeros(S, E, dtype=torch.int64, device="cuda")
    seq_loss = torch.zeros(S, dtype=torch.float64, device="cuda")
    d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    z = torch.zeros((), dtype=torch.float64, device="cuda")
    for i, r in enumerate(rows):
        if not len(r):
            continue
        with torch.enable_grad():
            l = st["logits"][r].double().requires_grad_(True)
            counts[i] = torch.bincount(st["ids"][r].reshape(-1).long(), minlength=E)
            if c["score"] == "softmax":
                p = torch.softmax(l, 1)
            else:
                p = torch.sigmoid(l)
                p = p / p.sum(1, keepdim=True)
            bal = E * (counts[i].double() / (len(r) * K) * p.mean(0)).sum()
            zi = torch.logsumexp(l, 1).square().sum()
            (g,) = torch.autograd.grad(C_BALANCE * bal / used + C_Z * zi / total, l)
        d[r] = g
        seq_loss[i], z = bal.detach(), z + zi.detach()
    return dict(counts=None, seq_loss=seq_loss, dlogits=d, losses=torch.stack([z / total, seq_loss.sum() / used]))


def _exact_experts(st):
    c, offsets = st["case"], st["offsets"].tolist()
    y = torch.empty(st["perm"].numel(), c["D"], dtype=torch.float64, device="cuda")
    w = st["topk_w"].reshape(-1)[st["perm"].long()].double()

    def wide(q, s):
        v = q.to(torch.float64).unflatten(-1, (-1, 32))
        return torch.ldexp(v, s.to(torch.int32)[..., None] - 127).flatten(-2)

    gq, gs, uq, us, dq, ds = st["w"]
    for e in range(c["E"]):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        x = wide(st["xq"][a:b], st["xs"][a:b])
        gate, up = x @ wide(gq[e], gs[e]).T, x @ wide(uq[e], us[e]).T
        h = _exact_rounded(gate * torch.sigmoid(gate) * up)
        y[a:b] = w[a:b, None] * (h @ wide(dq[e], ds[e]).T)
    return dict(y=y)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(norm=_exact_norm, norm_backward=_exact_norm_backward, balance=_exact_balance,
                experts=_exact_experts)[case["op"]](st)
