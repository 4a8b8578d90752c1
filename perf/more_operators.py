"""Cases of the operators between the fused projection and the attention, and of the quantised cache: norms of queries and
keys with the position rotation (forward, backward), writing keys and values into the cache in 8 bits and reading them
back, and attention of single tokens over that cache.

`run` computes a case in plain torch operations (32 bits, angles in 64, rounded once at the end) or, with `own` set,
through comm_overlap_gb300.torch_ops.  The cache holds E4M3 codes with one power of two for each token and key head.
"""
import math

import torch

own = False

D = 128  # head dimension
EPS = 1e-6
BIAS = 127  # of the cache's exponents
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # queries and keys of one token of a decoding step; latency only
        dict(name="rotary_fwd_token", op="rotary_fwd", tokens=1, hq=32, hkv=8, rot=128, layout="half", norm=True, factor=8.0, far=100000),
        # the tokens of a training step or a long prompt
        dict(name="rotary_fwd_large", op="rotary_fwd", tokens=16384, hq=32, hkv=8, rot=128, layout="half", norm=True, factor=1.0, far=16384),
        # gradients of a short ragged batch, half of each head rotated, no norm
        dict(name="rotary_bwd_ragged", op="rotary_bwd", tokens=1237, hq=40, hkv=8, rot=64, layout="interleaved", norm=False, factor=1.0, far=4096),
        # gradients of a training step
        dict(name="rotary_bwd_large", op="rotary_bwd", tokens=16384, hq=32, hkv=8, rot=128, layout="half", norm=True, factor=1.0, far=16384),
        # one decoding step of 64 sequences: q rotated, k and v into the cache; what was written is read back
        dict(name="cache_step", op="cache", tokens=64, read=0, cap=8192, hq=32, hkv=8, rot=128, layout="half", norm=True, factor=8.0, far=100000),
        # a ragged chunk of a prompt, and the cached context of its sequence read back for the attention
        dict(name="cache_chunk", op="cache", tokens=777, read=9001, cap=32768, hq=28, hkv=4, rot=64, layout="interleaved", norm=False, factor=1.0, far=9001),
        # a long prompt written, a long context read
        dict(name="cache_large", op="cache", tokens=16384, read=131072, cap=262144, hq=32, hkv=8, rot=128, layout="half", norm=True, factor=8.0, far=131072),
        # one token of one sequence with a short context; latency only
        dict(name="attn_token", op="attn", n=1, t=1, hq=32, hkv=8, lmin=701, lmax=701, cap=1024, prefix=0),
        # one decoding step of 64 sequences over a cache with room for 8192 tokens each
        dict(name="attn_step", op="attn", n=64, t=1, hq=32, hkv=8, lmin=64, lmax=8000, cap=8192, prefix=0),
        # five drafted tokens for each of 16 sequences, checked together
        dict(name="attn_drafts", op="attn", n=16, t=5, hq=28, hkv=4, lmin=5, lmax=3001, cap=4096, prefix=0),
        # one sequence with a very long context
        dict(name="attn_long", op="attn", n=1, t=1, hq=32, hkv=8, lmin=262001, lmax=262001, cap=262144, prefix=0),
        # 48 answers that share a long prompt, each with a short text of its own
        dict(name="attn_prefix", op="attn", n=48, t=1, hq=32, hkv=8, lmin=1, lmax=500, cap=512, prefix=16001),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_bwd", "cache", "attn", "attn", "attn"])
    hkv, g = rng.choice([(32, 1), (16, 2), (8, 4), (8, 5), (4, 7), (8, 8), (1, 16)])
    hq = hkv * g
    rotation = dict(rot=rng.choice([16, 32, 64, 96, 128, 128]), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5,
                    factor=rng.choice([1.0, 1.0, 4.0, 8.0]))
    if op in ("rotary_fwd", "rotary_bwd"):
        tokens = _log(rng, 1, 16384 * 40 // (hq + hkv))
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, far=_log(rng, 16, 1000000), **rotation)
    if op == "cache":
        tokens = _log(rng, 1, 16384 * 8 // max(8, hkv, hq // 4))
        read = 0 if rng.random() < 0.4 else _log(rng, 1, 131072 * 8 // max(8, hkv))
        return dict(op=op, tokens=tokens, read=read, cap=tokens + read + _log(rng, 1, 100000), hq=hq, hkv=hkv, far=_log(rng, 16, 1000000), **rotation)
    kind = rng.choice(["step", "step", "drafts", "prefix"])
    n = _log(rng, 1, 64)
    most = 64 * 4096 * 8 // (n * max(8, hkv))  # cached rows of a sequence
    if kind == "step":  # one token a sequence
        cap = _log(rng, 16, min(most, 262144))
        return dict(op=op, n=n, t=1, hq=hq, hkv=hkv, lmin=rng.choice([0, 1, cap]), lmax=cap, cap=cap, prefix=0)
    if kind == "drafts":  # a few tokens a sequence; some see nothing
        cap = _log(rng, 16, min(most, 32768))
        return dict(op=op, n=n, t=rng.randint(2, 16), hq=hq, hkv=hkv, lmin=rng.choice([0, 16]), lmax=cap, cap=cap, prefix=0)
    cap = _log(rng, 16, min(most, 1024))
    return dict(op=op, n=n, t=rng.choice([1, 1, 4]), hq=hq, hkv=hkv, lmin=0, lmax=cap, cap=cap, prefix=_log(rng, 1, 16384))


def _lengths(case):
    """Cached lengths of a case's sequences, ragged.  They belong to the case: they come from its own values, not from
    the inputs' seed."""
    state = 1 + case["n"] + 101 * case["lmax"] + 10007 * case["hq"] + 1000003 * case["t"]
    lens = []
    for _ in range(case["n"]):
        state = (state * 6364136223846793005 + 1442695040888963407) % 2**64
        lens.append(case["lmin"] + int((case["lmax"] + 1 - case["lmin"]) * ((state >> 11) / 2**53)))
    return lens


def _frequencies(case):
    """Radians a position of the pairs: 500000^(-2i/rot); with a factor, those that turn less than once over 8192
    positions are slowed down by it, those that turn over four times stay, and a ramp lies between."""
    f = 500000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) * 2 / case["rot"])
    keep = ((8192 * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
    return f * (keep + (1 - keep) / case["factor"])


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0


def _power(e):
    """2^e, exactly, for whole numbers between -126 and 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 codes of x [..., D] (fp32) and the powers of two that they are multiples of: the least e with
    amax <= 448 * 2^e, between -51 and 51 (0 for a head of zeros)."""
    amax = x.abs().amax(dim=-1)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, (e - 9 + (m > 0.875)).clamp(-51, 51), torch.zeros_like(e))
    return (x * _power(-e).unsqueeze(-1)).to(FP8), e


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) % (2**62))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g).to(dtype)

    def whole(lo, hi, count):
        return torch.randint(lo, hi, (count,), generator=g, device="cuda", dtype=torch.int32)

    hq, hkv = case["hq"], case["hkv"]
    s = dict(case=case)
    if case["op"] == "attn":
        lens, n, t, cap, prefix = _lengths(case), case["n"], case["t"], case["cap"], case["prefix"]
        rows = n * cap + prefix
        s["q"] = normal(n, t, hq, D)
        i32 = dict(dtype=torch.int32, device="cuda")
        s.update(k_start=torch.arange(n, **i32) * cap, k_len=torch.tensor(lens, **i32))
        s["prefix"] = torch.tensor([n * cap, prefix], **i32) if prefix else None
        for name in ("k", "v"):  # heads of different size, a few channels of the keys larger than the others
            big = 1 + 3 * (normal(D, dtype=torch.float32) > 1.5) if name == "k" else 1
            codes, e = _quantise((normal(rows, hkv, D) * big).float() * torch.exp2(whole(-2, 3, hkv).float()).view(hkv, 1))
            s[name + "8"], s[name + "_exp"] = codes, (e + BIAS).to(torch.uint8).t().contiguous()
            del codes, e
        return s
    tokens = case["tokens"]
    s["qkv"] = normal(tokens, hq + 2 * hkv, D) * torch.exp2(whole(-2, 3, hq + 2 * hkv).float()).view(-1, 1).to(torch.bfloat16)
    s["positions"] = whole(0, case["far"], tokens)
    s["frequencies"] = _frequencies(case).cuda()
    s["wq"], s["wk"] = (normal(D, std=0.2, mean=1.0), normal(D, std=0.2, mean=1.0)) if case["norm"] else (None, None)
    if case["op"] == "rotary_bwd":
        s["gq"], s["gk"] = normal(tokens, hq, D), normal(tokens, hkv, D)
    if case["op"] == "cache":
        cap = case["cap"]
        for name in ("k", "v"):
            codes = whole(0, 254, cap * hkv * D)
            s[name + "8"] = (codes + (codes >= 127)).to(torch.uint8).view(FP8).view(cap, hkv, D)  # all but the two NaN
            del codes
            s[name + "_exp"] = (whole(-6, 6, cap * hkv) + BIAS).to(torch.uint8).view(hkv, cap)
        places = torch.randperm(cap, generator=g, device="cuda").to(torch.int32)
        s["rows"] = places[:tokens].contiguous()
        s["back"] = s["rows"] if not case["read"] else torch.cat([s["rows"], places[tokens:tokens + case["read"]]])
    return s


def _angles(s, dtype):
    return s["positions"].to(torch.float64).view(-1, 1) * s["frequencies"], torch.tensor(_amplitude(s["case"]), dtype=dtype, device="cuda")


def _turn(case, x, cos, sin):
    """x [tokens, heads, D] with its first rot elements rotated in pairs; cos, sin [tokens, rot / 2]."""
    r = case["rot"]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., r:]], dim=-1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2), x[..., r:]], dim=-1)


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w.float() if w is not None else x


def _plain_rotary(s):
    hq, hkv = s["case"]["hq"], s["case"]["hkv"]
    angle, size = _angles(s, torch.float32)
    cos, sin = torch.cos(angle).float() * size, torch.sin(angle).float() * size
    q, k = s["qkv"][:, :hq].float(), s["qkv"][:, hq:hq + hkv].float()
    return _turn(s["case"], _norm(q, s["wq"]), cos, sin), _turn(s["case"], _norm(k, s["wk"]), cos, sin)


def _plain_gradient(s, x, gy, w, cos, sin):
    u = _turn(s["case"], gy.float(), cos, -sin)
    if w is None:
        return u.to(torch.bfloat16), None
    x = x.float()
    rstd = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    n, uw = x * rstd, u * w.float()
    return (rstd * (uw - n * (uw * n).mean(dim=-1, keepdim=True))).to(torch.bfloat16), (u * n).sum(dim=(0, 1))


def _values(codes, exps, rows, dtype):
    """What the cache stands for at `rows` [...]: [..., heads, D]."""
    size = _power(exps[:, rows].movedim(0, -1).to(torch.int32) - BIAS)
    return codes.view(torch.uint8)[rows].view(FP8).to(dtype) * size.unsqueeze(-1)


def _plain_cache(s):
    case, rows, hq, hkv = s["case"], s["rows"].long(), s["case"]["hq"], s["case"]["hkv"]
    q, k = _plain_rotary(s)
    for name, x in (("k", k), ("v", s["qkv"][:, hq + hkv:].float())):
        codes, e = _quantise(x)
        s[name + "8"].view(torch.uint8)[rows] = codes.view(torch.uint8)
        s[name + "_exp"][:, rows] = (e + BIAS).to(torch.uint8).t()
    back = s["back"].long()
    k, v = (_values(s[name + "8"], s[name + "_exp"], back, torch.float32).to(torch.bfloat16) for name in ("k", "v"))
    return q.to(torch.bfloat16), k, v


def _plain_attention(s):
    """All sequences at once, padded to the longest; a shared prefix stands before each one's own keys."""
    case = s["case"]
    n, t, hq, hkv, prefix = case["n"], case["t"], case["hq"], case["hkv"], case["prefix"]
    own_keys = max(1, max(_lengths(case)))
    at = torch.arange(own_keys, device="cuda")
    q = s["q"].float().view(n, t, hkv, hq // hkv, D).permute(2, 0, 3, 1, 4)  # hkv, n, g, t, D
    g = hq // hkv

    def keys(name, rows):
        return _values(s[name + "8"], s[name + "_exp"], rows, torch.float32)

    rows = s["k_start"].long().view(n, 1) + at.clamp(max=case["cap"] - 1)
    last = (s["k_len"] - t).view(n, 1, 1, 1) + torch.arange(t, device="cuda").view(1, 1, t, 1)
    hidden = at.view(1, 1, 1, own_keys) > last
    scores = torch.matmul(q.reshape(hkv, n, g * t, D), keys("k", rows).permute(2, 0, 3, 1)).view(hkv, n, g, t, own_keys)
    scores.mul_(1 / math.sqrt(D)).masked_fill_(hidden, -math.inf)
    if prefix:
        shared = n * case["cap"] + torch.arange(prefix, device="cuda")
        before = torch.matmul(q.reshape(hkv, n * g * t, D), keys("k", shared).permute(1, 2, 0)).view(hkv, n, g, t, prefix)
        scores = torch.cat([before.mul_(1 / math.sqrt(D)), scores], dim=-1)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - top.clamp(min=-3e38))  # a query that sees nothing: zeros
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p[..., prefix:].reshape(hkv, n, g * t, own_keys), keys("v", rows).permute(2, 0, 1, 3)).view(hkv, n, g, t, D)
    if prefix:
        o = o + torch.matmul(p[..., :prefix].reshape(hkv, n * g * t, prefix), keys("v", shared).permute(1, 0, 2)).view(o.shape)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    return o.permute(1, 3, 0, 2, 4).reshape(n, t, hq, D).to(torch.bfloat16), lse.permute(1, 3, 0, 2).reshape(n, t, hq)


def _run_own(s):
    from comm_overlap_gb300 import torch_ops as ops
    case = s["case"]
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "attn":
        cache = ops.QuantizedCache(s["k8"], s["v8"], s["k_exp"], s["v_exp"])
        return ops.cached_attention(s["q"], cache, s["k_start"], s["k_len"], s["prefix"], return_lse=True)
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]
    how = dict(q_weight=s["wq"], k_weight=s["wk"], layout=case["layout"], eps=EPS, amplitude=_amplitude(case))
    if case["op"] == "rotary_fwd":
        return ops.qk_rotary_fwd(q, k, s["positions"], s["frequencies"], **how)
    if case["op"] == "rotary_bwd":
        grads = ops.qk_rotary_bwd(s["gq"], s["gk"], q, k, s["positions"], s["frequencies"], **how)
        return grads if case["norm"] else grads[:2]
    cache = ops.QuantizedCache(s["k8"], s["v8"], s["k_exp"], s["v_exp"])
    turned = ops.cache_write(cache, s["rows"], k, v, q, s["positions"], s["frequencies"], **how)
    return (turned, *ops.cache_read(cache, s["back"]))


def run(state):
    if own:
        return _run_own(state)
    s, case = state, state["case"]
    if case["op"] == "attn":
        return _plain_attention(s)
    if case["op"] == "cache":
        return _plain_cache(s)
    if case["op"] == "rotary_fwd":
        q, k = _plain_rotary(s)
        return q.to(torch.bfloat16), k.to(torch.bfloat16)
    hq, hkv = case["hq"], case["hkv"]
    angle, size = _angles(s, torch.float32)
    cos, sin = torch.cos(angle).float() * size, torch.sin(angle).float() * size
    gq, gwq = _plain_gradient(s, s["qkv"][:, :hq], s["gq"], s["wq"], cos, sin)
    gk, gwk = _plain_gradient(s, s["qkv"][:, hq:hq + hkv], s["gk"], s["wk"], cos, sin)
    return (gq, gk, gwq, gwk) if case["norm"] else (gq, gk)


def work(case):
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "attn":
        lens, t = _lengths(case), case["t"]
        keys, queries = sum(lens) + case["prefix"], case["n"] * t * hq
        pairs = sum(max(0, x - i) for x in lens for i in range(t)) + case["n"] * t * case["prefix"]
        return dict(bytes=2 * hkv * (D + 1) * keys + (4 * D + 4) * queries, flops=4 * D * hq * pairs)
    values = case["tokens"] * (hq + hkv) * D
    if case["op"] == "rotary_fwd":
        return dict(bytes=4 * values + 4 * case["tokens"], flops=(8 if case["norm"] else 3) * values)
    if case["op"] == "rotary_bwd":
        return dict(bytes=(6 if case["norm"] else 4) * values + 4 * case["tokens"], flops=(14 if case["norm"] else 3) * values)
    written, back = case["tokens"] * hkv, (case["tokens"] + case["read"]) * hkv
    return dict(bytes=4 * case["tokens"] * hq * D + 2 * written * (3 * D + 1) + 2 * back * (3 * D + 1), flops=8 * values + 4 * back * D)


def exact(case, seed):
    """The operators' definitions in 64 bits, on what `prepare` makes of the seed."""
    s = prepare(case, seed)
    hq, hkv, g = case["hq"], case["hkv"], case["hq"] // case["hkv"]
    f64 = torch.float64

    if case["op"] == "attn":
        n, t, prefix = case["n"], case["t"], case["prefix"]
        if sum(_lengths(case)) * hkv > 3e7:
            return None
        o = torch.zeros((n, t, hq, D), dtype=f64, device="cuda")
        lse = torch.full((n, t, hq), -math.inf, dtype=f64, device="cuda")
        scale = {name: _power(s[name + "_exp"].to(torch.int32) - BIAS).to(f64) for name in ("k", "v")}
        for i, length in enumerate(_lengths(case)):
            a = i * case["cap"]
            for h in range(hkv):
                def rows(name):
                    x = torch.cat([s[name + "8"][n * case["cap"]:, h], s[name + "8"][a:a + length, h]]).to(f64)
                    return x * torch.cat([scale[name][h, n * case["cap"]:], scale[name][h, a:a + length]]).unsqueeze(1)
                k, v = rows("k"), rows("v")
                for j in range(t):
                    seen = prefix + max(0, length - t + j + 1)
                    if seen == 0:
                        continue
                    z = torch.einsum("gd,kd->gk", s["q"][i, j, h * g:(h + 1) * g].to(f64), k[:seen]) / math.sqrt(D)
                    lse[i, j, h * g:(h + 1) * g] = torch.logsumexp(z, dim=1)
                    o[i, j, h * g:(h + 1) * g] = torch.softmax(z, dim=1) @ v[:seen]
        return o, lse

    # the rotation as a complex product, the norm as division by a root
    unit = torch.polar(torch.full_like(_angles(s, f64)[0], _amplitude(case)), _angles(s, f64)[0]).unsqueeze(1)
    r = case["rot"]

    def turned(x, by):
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == "half" else torch.view_as_complex(x[..., :r].unflatten(-1, (-1, 2)).contiguous())
        z = z * by
        front = torch.cat([z.real, z.imag], dim=-1) if case["layout"] == "half" else torch.view_as_real(z).flatten(-2)
        return torch.cat([front, x[..., r:]], dim=-1)

    def root(x):
        return torch.sqrt(torch.einsum("thd,thd->th", x, x) / D + EPS).unsqueeze(-1)

    q, k = s["qkv"][:, :hq].to(f64), s["qkv"][:, hq:hq + hkv].to(f64)
    if case["op"] == "rotary_bwd":
        out, sums = [], []
        for x, gy, w in ((q, s["gq"], s["wq"]), (k, s["gk"], s["wk"])):
            u = turned(gy.to(f64), unit.conj())
            if w is not None:  # J = (I - n n^T / D) / root
                n = x / root(x)
                sums.append(torch.einsum("thd,thd->d", u, n))
                u = u * w.to(f64)
                u = (u - n * torch.einsum("thd,thd->th", u, n).unsqueeze(-1) / D) / root(x)
            out.append(u)
        return (*out, *sums)
    if case["norm"]:
        q, k = q / root(q) * s["wq"].to(f64), k / root(k) * s["wk"].to(f64)
    q, k = turned(q, unit), turned(k, unit)
    if case["op"] == "rotary_fwd":
        return q, k
    # the nearest multiples of the E4M3 steps, ties to even
    held = []
    for name, x in (("k", k), ("v", s["qkv"][:, hq + hkv:].to(f64))):
        size = x.abs().amax(dim=-1, keepdim=True)
        e = torch.where(size > 0, torch.ceil(torch.log2(size / 448)), torch.zeros_like(size)).clamp(-51, 51)
        y = x * _power(-e).to(f64)
        step = _power(torch.frexp(y.abs().clamp(min=2.0**-6))[1] - 4).to(f64)
        values = s[name + "8"].to(f64) * _power(s[name + "_exp"].to(torch.int32) - BIAS).to(f64).t().unsqueeze(-1)
        values[s["rows"].long()] = torch.round(y / step) * step * _power(e).to(f64)
        held.append(values[s["back"].long()])
    return (q, *held)
