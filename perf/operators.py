"""Cases of the sublayer operators: LayerNorm with weight and bias (forward, backward), the linear layer with bias,
activation and residual (forward, backward), and causal attention over packed sequences with grouped heads.

`run` computes a case in plain torch operations (32 bits, rounded once at the end) or, with `own` set, through
comm_overlap_gb300.torch_ops.  Matrices are bf16 as everywhere in this package; statistics, bias and norm gradients fp32.
"""
import math

import torch

own = False

D = 128  # head dimension
EPS = 1e-5


def listed():
    return [
        # one token of a decoding step; latency only
        dict(name="ln_fwd_token", op="ln_fwd", rows=1, h=4096),
        # the token chunk of the 4-layer stack workload
        dict(name="ln_fwd_stack", op="ln_fwd", rows=32768, h=4096),
        # a ragged micro-batch at another width, with the gradient of the residual path added
        dict(name="ln_bwd_ragged", op="ln_bwd", rows=1237, h=2560, res=True),
        # the stack workload's backward pass
        dict(name="ln_bwd_stack", op="ln_bwd", rows=32768, h=4096, res=True),
        # first MLP linear of one decoded token: the weight is read once, little else happens
        dict(name="linear_fwd_token", op="linear_fwd", m=1, k=4096, n=16384, act="gelu", bias=True, res=False, save=False),
        # first MLP linear of a short ragged prompt in training (pre-activation kept)
        dict(name="linear_fwd_ragged", op="linear_fwd", m=777, k=2560, n=10240, act="gelu", bias=True, res=False, save=True),
        # second MLP linear of a training step, added to the residual stream
        dict(name="linear_fwd_large", op="linear_fwd", m=16384, k=16384, n=4096, act="none", bias=True, res=True, save=False),
        # its gradients on a short ragged batch: no activation behind it
        dict(name="linear_bwd_ragged", op="linear_bwd", m=777, k=10240, n=2560, act="none", bias=True),
        # gradients of the first MLP linear in a training step
        dict(name="linear_bwd_large", op="linear_bwd", m=16384, k=4096, n=16384, act="gelu", bias=True),
        # eight prompts of different lengths, prefilled together from one fused projection
        dict(name="attn_prompts", op="attn", hq=32, hkv=8, n=8, qmin=1, qmax=4096, pmin=0, pmax=0, cap=0, total=11000),
        # one long prompt
        dict(name="attn_long", op="attn", hq=32, hkv=8, n=1, qmin=16384, qmax=16384, pmin=0, pmax=0, cap=0, total=16384),
        # one decoding step of 64 sequences over a cache with room for 8192 tokens each
        dict(name="attn_decode", op="attn", hq=32, hkv=8, n=64, qmin=1, qmax=1, pmin=64, pmax=8000, cap=8192, total=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return max(lo, 8 * (_log(rng, lo, hi) // 8))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "linear_fwd", "linear_bwd", "attn", "attn"])
    if op in ("ln_fwd", "ln_bwd"):
        h = _eights(rng, 256, 12288)
        rows = _log(rng, 1, min(32768, 32768 * 4096 // h))
        return dict(op=op, rows=rows, h=h) if op == "ln_fwd" else dict(op=op, rows=rows, h=h, res=rng.random() < 0.5)
    if op in ("linear_fwd", "linear_bwd"):
        k, n = _eights(rng, 256, 16384), _eights(rng, 256, 16384)
        m = _log(rng, 1 if op == "linear_fwd" else 128, min(16384, 16384 * 16384 * 4096 // (k * n)))
        act, bias = rng.choice(["none", "relu", "gelu"]), rng.random() < 0.7
        if op == "linear_bwd":
            return dict(op=op, m=m, k=k, n=n, act=act, bias=bias)
        res = rng.random() < 0.5
        return dict(op=op, m=m, k=k, n=n, act=act, bias=bias, res=res, save=not res and rng.random() < 0.5)
    hkv, g = rng.choice([(32, 1), (16, 2), (8, 4), (8, 5), (4, 7), (8, 8), (1, 16)])
    kind = rng.choice(["prompts", "decode", "chunks"])
    if kind == "prompts":  # prompts prefilled from a fused projection
        n = _log(rng, 1, 32)
        most = _log(rng, 32, 8192) if n < 8 else _log(rng, 32, 2048)
        return dict(op=op, hq=hkv * g, hkv=hkv, n=n, qmin=1, qmax=most, pmin=0, pmax=0, cap=0, total=0)
    if kind == "decode":  # one token for each sequence, over a padded cache
        n = _log(rng, 1, 64)
        cap = _log(rng, 128, 32768 if n <= 8 else 8192)
        return dict(op=op, hq=hkv * g, hkv=hkv, n=n, qmin=1, qmax=1, pmin=0, pmax=cap - 1, cap=cap, total=0)
    n = _log(rng, 1, 8)  # chunks of prompts, and single tokens among them, over the cache of what came before
    cap = _log(rng, 1024, 8192)
    return dict(op=op, hq=hkv * g, hkv=hkv, n=n, qmin=1, qmax=512, pmin=0, pmax=cap - 512, cap=cap, total=0)


def _lengths(case):
    """Query lengths and cached lengths of a case's sequences, ragged; the listed total where there is one.  Sizes
    belong to the case: they come from its own values, not from the inputs' seed."""
    key = "%d %d %d %d %d" % (case["hq"], case["n"], case["qmax"], case["pmax"], case["cap"])
    state = sum((i + 1) * ord(c) for i, c in enumerate(key)) or 1

    def unit():
        nonlocal state
        state = (state * 6364136223846793005 + 1442695040888963407) % 2**64
        return (state >> 11) / 2**53

    lo, hi = case["qmin"], case["qmax"]
    q = [lo + int((hi + 1 - lo) * unit()) for _ in range(case["n"])]
    if case["total"]:
        scale = case["total"] / sum(q)
        q = [min(hi, max(lo, int(x * scale))) for x in q]
        q[0] = max(lo, min(hi, q[0] + case["total"] - sum(q)))
    p = [case["pmin"] + int((case["pmax"] + 1 - case["pmin"]) * unit()) for _ in q]
    return q, p


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) % (2**62))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g).to(dtype)

    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        rows, h = case["rows"], case["h"]
        # a residual stream: rows of different size, some channels larger than the others
        x = (normal(rows, h, dtype=torch.float32) * (1 + 3 * (normal(h, dtype=torch.float32) > 2)) + 0.2).mul_(
            torch.exp(normal(rows, 1, std=0.3, dtype=torch.float32))).to(torch.bfloat16)
        s = dict(case=case, x=x, gamma=normal(h, std=0.1, mean=1.0), beta=normal(h, std=0.1))
        if op == "ln_bwd":
            var, mean = torch.var_mean(x.float(), dim=1, correction=0)
            s.update(gy=normal(rows, h), mean=mean, rstd=torch.rsqrt(var + EPS), gres=normal(rows, h) if case["res"] else None)
        return s
    if op in ("linear_fwd", "linear_bwd"):
        m, k, n = case["m"], case["k"], case["n"]
        s = dict(case=case, x=normal(m, k), w=normal(n, k, std=0.02), b=normal(n, std=0.1) if case["bias"] else None)
        if op == "linear_fwd":
            s["r"] = normal(m, n) if case["res"] else None
        else:
            s["gy"] = normal(m, n)
            s["z"] = normal(m, n, std=0.02 * math.sqrt(k)) if case["act"] != "none" else None
        return s
    q, p = _lengths(case)
    hq, hkv, cap = case["hq"], case["hkv"], case["cap"]
    at = [0]
    for length in q:
        at.append(at[-1] + length)
    if cap:  # queries of this step over a cache: row i * cap is the first token of sequence i
        qs = normal(at[-1], hq, D)
        ks, vs = normal(case["n"] * cap, hkv, D), normal(case["n"] * cap, hkv, D)
        starts, lens = [i * cap for i in range(case["n"])], [a + b for a, b in zip(q, p)]
    else:  # one fused projection of whole prompts
        qkv = normal(at[-1], hq + 2 * hkv, D)
        qs, ks, vs = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        starts, lens = at[:-1], q
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(case=case, q=qs, k=ks, v=vs, cu_q=torch.tensor(at, **i32), k_start=torch.tensor(starts, **i32),
                k_len=torch.tensor(lens, **i32), qlens=q, klens=lens, qat=at, kat=starts)


def _act(name, z):
    return torch.relu(z) if name == "relu" else 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5))) if name == "gelu" else z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _attend(q, k, v, qlen, klen):
    """Batched plain attention: q [n, tq, hkv, g, D], k and v [n, tk, hkv, D] in 32 bits; query i of a sequence sees the
    keys up to klen - qlen + i."""
    n, tq, hkv, g, _ = q.shape
    tk = k.shape[1]
    qt = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, g * tq, D)
    s = torch.matmul(qt, k.permute(0, 2, 3, 1)).view(n, hkv, g, tq, tk).mul_(1 / math.sqrt(D))
    last = (klen - qlen).view(n, 1, 1) + torch.arange(tq, device=q.device).view(1, tq, 1)
    s.masked_fill_((torch.arange(tk, device=q.device).view(1, 1, tk) > last).view(n, 1, 1, tq, tk), -math.inf)
    top = s.amax(dim=-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, g * tq, tk), v.permute(0, 2, 1, 3)).view(n, hkv, g, tq, D).div_(total)
    lse = (top + total.log()).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(n, tq, hkv * g, D), lse.permute(0, 3, 1, 2).reshape(n, tq, hkv * g)


def _plain_attention(s):
    hq, hkv = s["case"]["hq"], s["case"]["hkv"]
    qlens, klens, qat, kat = s["qlens"], s["klens"], s["qat"], s["kat"]
    n, tq, tk = len(qlens), max(qlens), max(klens)
    qlen, klen = s["cu_q"].diff(), s["k_len"]
    if tq == 1:  # one query each: all sequences at once, over the longest
        rows = (s["k_start"].long().view(n, 1) + torch.arange(tk, device="cuda")).clamp_(max=s["k"].shape[0] - 1)
        o, lse = _attend(s["q"].float().view(n, 1, hkv, hq // hkv, D), s["k"][rows].float(), s["v"][rows].float(), qlen, klen)
        return o.view(n, hq, D).to(torch.bfloat16), lse.view(n, hq)
    o = torch.empty((qat[-1], hq, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((qat[-1], hq), dtype=torch.float32, device="cuda")
    for i in range(n):  # ragged: one sequence after the other
        a, b, c, d = qat[i], qat[i + 1], kat[i], kat[i] + klens[i]
        oi, li = _attend(s["q"][a:b].float().view(1, b - a, hkv, hq // hkv, D), s["k"][c:d].float().unsqueeze(0),
                         s["v"][c:d].float().unsqueeze(0), qlen[i:i + 1], klen[i:i + 1])
        o[a:b], lse[a:b] = oi[0], li[0]
    return o, lse


def _run_own(s):
    from comm_overlap_gb300 import torch_ops as ops
    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        return ops.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS)
    if op == "ln_bwd":
        return ops.layer_norm_bwd(s["gy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["gres"])
    if op == "linear_fwd":
        y, z = ops.linear_fwd(s["x"], s["w"], s["b"], case["act"], s["r"], save=case["save"])
        return (y, z) if case["save"] else (y,)
    if op == "linear_bwd":
        gx, gw, gb = ops.linear_bwd(s["gy"], s["x"], s["w"], s["z"], case["act"], bias_grad=case["bias"])
        return (gx, gw, gb) if case["bias"] else (gx, gw)
    return ops.packed_attention(s["q"], s["k"], s["v"], s["cu_q"], s["k_start"], s["k_len"], return_lse=True)


def run(state):
    if own:
        return _run_own(state)
    s, case = state, state["case"]
    op, bf = case["op"], torch.bfloat16
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(dim=1, keepdim=True)
        x = x - mean
        rstd = torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS)
        return (x * rstd * s["gamma"].float() + s["beta"].float()).to(bf), mean.view(-1), rstd.view(-1)
    if op == "ln_bwd":
        gy, rstd = s["gy"].float(), s["rstd"].view(-1, 1)
        xhat = (s["x"].float() - s["mean"].view(-1, 1)) * rstd
        gn = gy * s["gamma"].float()
        gx = rstd * (gn - gn.mean(dim=1, keepdim=True) - xhat * (gn * xhat).mean(dim=1, keepdim=True))
        if s["gres"] is not None:
            gx = gx + s["gres"].float()
        return gx.to(bf), (gy * xhat).sum(dim=0), gy.sum(dim=0)
    if op == "linear_fwd":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z += s["b"].float()
        y = _act(case["act"], z)
        if s["r"] is not None:
            y = y + s["r"].float()
        return (y.to(bf), z.to(bf)) if case["save"] else (y.to(bf),)
    if op == "linear_bwd":
        gz = s["gy"].float()
        if s["z"] is not None:
            gz = gz * _act_grad(case["act"], s["z"].float())
        gx, gw = (gz @ s["w"].float()).to(bf), (gz.t() @ s["x"].float()).to(bf)
        return (gx, gw, gz.sum(dim=0)) if case["bias"] else (gx, gw)
    return _plain_attention(s)


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        rows, h = case["rows"], case["h"]
        if op == "ln_fwd":
            return dict(bytes=4 * rows * h + 4 * h + 8 * rows, flops=8 * rows * h)
        return dict(bytes=(8 if case["res"] else 6) * rows * h + 10 * h + 8 * rows, flops=14 * rows * h)
    if op in ("linear_fwd", "linear_bwd"):
        m, k, n = case["m"], case["k"], case["n"]
        if op == "linear_fwd":
            return dict(bytes=2 * (m * k + n * k + m * n * (1 + case["res"] + case["save"]) + n * case["bias"]), flops=2 * m * n * k)
        return dict(bytes=2 * (2 * m * k + 2 * n * k + m * n * (1 + (case["act"] != "none"))) + 4 * n * case["bias"], flops=4 * m * n * k)
    q, p = _lengths(case)
    hq, hkv = case["hq"], case["hkv"]
    pairs = sum(b * a + a * (a + 1) // 2 for a, b in zip(q, p))
    keys = sum(q) if not case["cap"] else sum(q) + sum(p)
    return dict(bytes=2 * D * (2 * hq * sum(q) + 2 * hkv * keys) + 4 * hq * sum(q), flops=4 * D * hq * pairs)


def exact(case, seed):
    """The operators' definitions in 64 bits, on what `prepare` makes of the seed."""
    s = prepare(case, seed)
    op = case["op"]

    def f64(t):
        return t.to(torch.float64)

    if op == "ln_fwd":
        x = f64(s["x"])
        var, mean = torch.var_mean(x, dim=1, correction=0)
        y = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        return y * f64(s["gamma"]) + f64(s["beta"]), mean, (var + EPS) ** -0.5
    if op == "ln_bwd":
        # gx is J^T (gy gamma), J = rstd (I - 1/h - xhat xhat^T / h)
        h = case["h"]
        xhat = (f64(s["x"]) - f64(s["mean"])[:, None]) * f64(s["rstd"])[:, None]
        u = f64(s["gy"]) * f64(s["gamma"])
        gx = u - u.sum(1, keepdim=True) / h - xhat * torch.einsum("rc,rc->r", u, xhat)[:, None] / h
        gx *= f64(s["rstd"])[:, None]
        if s["gres"] is not None:
            gx += f64(s["gres"])
        return gx, torch.einsum("rc,rc->c", f64(s["gy"]), xhat), torch.einsum("rc->c", f64(s["gy"]))
    if op == "linear_fwd":
        z = torch.einsum("mk,nk->mn", f64(s["x"]), f64(s["w"]))
        if s["b"] is not None:
            z = z + f64(s["b"])[None, :]
        y = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "gelu": lambda t: t * torch.special.ndtr(t)}[case["act"]](z)
        if s["r"] is not None:
            y = y + f64(s["r"])
        return (y, z) if case["save"] else (y,)
    if op == "linear_bwd":
        gz = f64(s["gy"])
        if case["act"] == "relu":
            gz = torch.where(s["z"] > 0, gz, torch.zeros_like(gz))
        elif case["act"] == "gelu":
            z = f64(s["z"])
            gz = gz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        gx, gw = torch.einsum("mn,nk->mk", gz, f64(s["w"])), torch.einsum("mn,mk->nk", gz, f64(s["x"]))
        return (gx, gw, torch.einsum("mn->n", gz)) if case["bias"] else (gx, gw)
    hq, g = case["hq"], case["hq"] // case["hkv"]
    o = torch.empty((s["qat"][-1], hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["qat"][-1], hq), dtype=torch.float64, device="cuda")
    for i, (ql, kl) in enumerate(zip(s["qlens"], s["klens"])):
        a, c = s["qat"][i], s["kat"][i]
        hidden = torch.ones((ql, kl), dtype=torch.bool, device="cuda").triu(kl - ql + 1)
        for head in range(hq):
            k, v = (f64(t[c:c + kl, head // g]) for t in (s["k"], s["v"]))
            scores = (f64(s["q"][a:a + ql, head]) @ k.t() / math.sqrt(D)).masked_fill_(hidden, -math.inf)
            lse[a:a + ql, head] = torch.logsumexp(scores, dim=1)
            o[a:a + ql, head] = torch.softmax(scores, dim=1) @ v
    return o, lse
