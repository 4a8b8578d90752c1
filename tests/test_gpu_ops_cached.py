"""Attention of the last tokens of sequences over the 8-bit cache, with and without shared rows, against softmax(scale q K^T) V
in 64 bits on the values that the cache stands for.

What the kernel rounds, for a row with keys j: q, as two terms, is off by at most 2^-21 of its largest value, an element, which is
2^-21 max |q| sum |k|; the score's 2 x 128 products are summed in fp32 by 8 instructions, each off by at most 5 U32 of its terms'
sizes (at most 1 + 2^-3 times sum |q k|), joined and scaled (4 roundings), and so is the logarithm t = s log2 e + b, and t - m: delta =
scale (2^-21 max |q| sum |k| + 50 U32 sum |q k|) + 6 U32 |t|; the exponential adds 2^-22, the weight's two terms 2^-8 of it, or 2^-18 of the
row's largest weight (the second term's smallest step is 2^-9, half of that counts a sixteenth, the largest weight is at least 2^4).  Sums
over n keys: an instruction for 32 of them for each term, 5 U32 of their sizes each time, and the
denominator at most n / 4 + 64 roundings: n + 64 covers both.  So O is off by at most sum_j p_j |v_j| (2^-8 + 2 delta + 2^-21 + 2 (n + 64) U32)
(delta, the exponential and the sums once for the numerator and once for the denominator, which the weight's rounding does not
enter) and 2^-18 sum_j |v8_j| / l."""
import math

import pytest
import torch

from cache_helpers import D, power, random_cache, values
from ops_helpers import U32, close, device_ok, randn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def ops():
    from comm_overlap_gb300 import torch_ops
    return torch_ops


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reference(q, cache, starts, lens, prefix=None, scale=None):
    """(o, slop of o, lse, slop of lse) for q [n, t, heads, 128]."""
    n, t, hq, _ = q.shape
    hkv = cache.k.shape[1]
    g = hq // hkv
    scale = D ** -0.5 if scale is None else scale
    o, so = torch.zeros(n, t, hq, D, dtype=torch.float64, device="cuda"), torch.zeros(n, t, hq, D, dtype=torch.float64, device="cuda")
    lse, sl = torch.full((n, t, hq), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(n, t, hq, dtype=torch.float64, device="cuda")
    first, shared = prefix if prefix else (0, 0)
    for s in range(n):
        rows = list(range(first, first + shared)) + list(range(starts[s], starts[s] + lens[s]))
        if not rows:
            continue
        k, v = values(cache, "k", rows), values(cache, "v", rows)
        b = cache.v_exp[:, torch.tensor(rows, device="cuda")].double().t() - 127
        for i in range(t):
            seen = shared + max(0, lens[s] - t + i + 1)
            if seen == 0:
                continue
            qi = q[s, i].double().view(hkv, g, D)
            z = torch.einsum("hgd,khd->hgk", qi, k[:seen]) * scale
            size = torch.einsum("hgd,khd->hgk", qi.abs(), k[:seen].abs()) * scale
            lse[s, i] = torch.logsumexp(z, -1).view(-1)
            p = torch.softmax(z, -1)
            o[s, i] = torch.einsum("hgk,khd->hgd", p, v[:seen]).view(hq, D)
            bias = b[:seen].t()[:, None]
            tt = z / math.log(2) + bias
            coarse = 2.0 ** -21 * qi.abs().amax(-1)[..., None] * k[:seen].abs().sum(-1).t()[:, None] * scale
            delta = (coarse + U32 * (50 * size + 6 * tt.abs())).amax(-1, keepdim=True)
            each = 2.0 ** -8 + 2 * delta + 2.0 ** -21 + 2 * (seen + 64) * U32
            m = tt.amax(-1, keepdim=True)
            den = torch.exp2(tt - bias - m).sum(-1, keepdim=True)
            v8 = v[:seen].abs() / torch.exp2(b[:seen])[..., None]
            so[s, i] = (torch.einsum("hgk,khd->hgd", p * each, v[:seen].abs()) + 2.0 ** -18 * v8.sum(0)[:, None] / den).view(hq, D)
            sl[s, i] = (delta[..., 0] + 2.0 ** -21 + (seen + 64) * U32).view(-1) + 8 * U32 * (lse[s, i].abs() + 60)
    return o, so, lse, sl


def check(ops, q, cache, starts, lens, prefix=None, scale=None):
    o, lse = ops.cached_attention(q, cache, ints(*starts), ints(*lens), ints(*prefix) if prefix else None, scale, return_lse=True)
    q4 = q.view(len(lens), -1, *q.shape[-2:])
    ro, so, rl, sl = reference(q4, cache, starts, lens, prefix, scale)
    close(o.view(q4.shape), ro, so, what="o")
    lse = lse.view(rl.shape)
    none = rl == -math.inf
    assert (lse[none] == -math.inf).all() and not o.view(q4.shape)[none].any()
    assert ((lse.double() - rl).abs()[~none] <= sl[~none]).all(), ((lse.double() - rl).abs() / sl)[~none].max()
    device_ok()
    return o, lse


HEADS = [(1, 1), (8, 1), (4, 4), (32, 8), (28, 4), (16, 1), (40, 2), (130, 1)]
LENGTHS = [[1], [0], [31], [32], [33], [700], [0, 1, 2, 64, 0, 95, 96, 97, 0]]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_single_tokens(ops, hq, hkv, lens):
    cache = random_cache(1200, hkv, seed=hq)
    starts = [(7 + 131 * i) % 450 for i in range(len(lens))]  # any row, also rows of other sequences
    check(ops, randn(len(lens), hq, D, seed=1), cache, starts, lens)


@pytest.mark.parametrize("lens", [[0], [1], [3], [37], [500, 2, 64, 33, 5]], ids=str)
@pytest.mark.parametrize("t", [2, 5, 16, 33])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 2), (14, 2), (16, 1)])
def test_a_few_tokens(ops, hq, hkv, t, lens):
    cache = random_cache(900, hkv, seed=t)
    starts = [3 + 70 * i for i in range(len(lens))]
    check(ops, randn(len(lens), t, hq, D, seed=2), cache, starts, lens)


@pytest.mark.parametrize("prefix", [(0, 0), (5, 1), (11, 32), (300, 333)], ids=str)
@pytest.mark.parametrize("n,t,hq,hkv", [(1, 1, 4, 4), (3, 1, 32, 8), (9, 2, 14, 2), (33, 1, 16, 1), (70, 1, 8, 2)])
def test_shared_rows(ops, n, t, hq, hkv, prefix):
    cache = random_cache(1000, hkv, seed=n)
    lens = [(37 * i * i + i) % 130 for i in range(n)]
    starts = [(i * 13) % 700 for i in range(n)]
    check(ops, randn(n, t, hq, D, seed=3), cache, starts, lens, prefix)


def test_many_sequences(ops):
    """More sequences than a block's threads, most of them short or empty, tiles few and many."""
    n = 1500
    g = torch.Generator().manual_seed(0)
    lens = [int(x) if i % 3 else 0 for i, x in enumerate(torch.randint(0, 70, (n,), generator=g))]
    lens[700], lens[-1] = 1900, 450
    cache = random_cache(2500, 2, seed=9)
    starts = [int(x) for x in torch.randint(0, 500, (n,), generator=g)]
    check(ops, randn(n, 4, D, seed=4), cache, starts, lens)
    check(ops, randn(n, 4, D, seed=4), cache, starts, [0] * n)
    lens = [0] * n
    lens[1001] = 77
    check(ops, randn(n, 4, D, seed=4), cache, starts, lens, (100, 50))


@pytest.mark.parametrize("scale", [1e-3, 0.088, 3.0, 1000.0])
def test_scores_of_any_size(ops, scale):
    """From nearly uniform weights to one key that takes all; queries of very different size."""
    cache = random_cache(600, 2, seed=5, spread=8)
    q = randn(3, 8, D, seed=5) * torch.exp2(torch.arange(-12, 12, device="cuda").view(3, 8) * 0.5).to(BF)[..., None]
    o, lse = ops.cached_attention(q, cache, ints(0, 5, 100), ints(600, 400, 1), scale=scale, return_lse=True)
    ro, so, rl, sl = reference(q[:, None], cache, [0, 5, 100], [600, 400, 1], scale=scale)
    close(o[:, None], ro, so + 2 ** -133)
    assert ((lse[:, None].double() - rl).abs() <= sl).all()


def test_rows_growing_and_falling(ops):
    """Scores that rise with the position move the running maximum in every tile; values of very different size."""
    hkv, rows = 1, 1000
    cache = random_cache(rows, hkv, seed=6)
    q = torch.ones(2, 4, D, dtype=BF, device="cuda")
    ramp = torch.linspace(-3, 3, rows, device="cuda")
    k = (ramp[:, None, None] * torch.ones(rows, 1, D, device="cuda") + 0.1 * randn(rows, 1, D, seed=2).float()).to(BF)
    v = (randn(rows, 1, D, seed=3).float() * torch.exp2(torch.arange(rows, device="cuda") % 41 - 20.0)[:, None, None]).to(BF)
    ops.cache_write(cache, torch.arange(rows, dtype=torch.int32, device="cuda"), k, v)
    check(ops, q, cache, [0, 0], [rows, 37])
    ops.cache_write(cache, torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda"), k, v)
    check(ops, q, cache, [0, 0], [rows, 37])
    # the last value tiny beside the others, with all of the weight; and the other way round
    ops.cache_write(cache, ints(999, 0), k[[999, 0]], torch.cat([v[:1] * 0 + 2.0 ** -40, v[:1] * 0 + 2.0 ** 40]))
    check(ops, q, cache, [0, 0], [rows, 37])


def test_extreme_exponents(ops):
    """All values near the ends of the cache's range of powers of two."""
    for e in (-51, 51):
        cache = random_cache(300, 2, seed=7)
        cache.v_exp[0].fill_(127 + e)
        cache.k_exp[0].fill_(127 - 20)
        cache.k.view(torch.uint8)[:, 0] &= 0xBF  # exponents below 2: scores of moderate size
        o, lse = ops.cached_attention(randn(2, 4, D, seed=1), cache, ints(0, 9), ints(300, 40), return_lse=True)
        ro, so, rl, sl = reference(randn(2, 4, D, seed=1)[:, None], cache, [0, 9], [300, 40])
        close(o[:, None], ro, so)
        assert ((lse[:, None].double() - rl).abs() <= sl).all()
    zero = ops.QuantizedCache.empty(50, 1)
    o, lse = ops.cached_attention(randn(1, 4, D), zero, ints(0), ints(50), return_lse=True)
    assert not o.any() and ((lse - math.log(50)).abs() < 1e-5).all()


@pytest.mark.parametrize("t", [1, 4])
def test_what_a_query_does_not_see_has_no_effect(ops, t):
    """NaN codes, and exponents of any value, around the sequences and past what a query sees."""
    hkv, hq, rows = 2, 8, 400
    starts, lens, prefix = [10, 101, 333], [33, 70, t + 1], (210, 45)
    clean = random_cache(rows, hkv, seed=8)
    dirty = random_cache(rows, hkv, seed=8)
    outside = torch.ones(rows, dtype=torch.bool, device="cuda")
    for a, x in list(zip(starts, lens)) + [prefix]:
        outside[a:a + x] = False
    for x in dirty[:2]:
        x.view(torch.uint8)[outside] = 0x7F
    for x in dirty[2:]:
        x[:, outside] = 255
    q = randn(3, t, hq, D, seed=9)
    for p in (None, ints(*prefix)):
        a = ops.cached_attention(q, clean, ints(*starts), ints(*lens), p, return_lse=True)
        b = ops.cached_attention(q, dirty, ints(*starts), ints(*lens), p, return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if t == 1:
        return
    # the last key's NaN, in K and in some of V: the last query alone; the key before: the last two
    for back in (1, 2):
        for name in ("k", "v"):
            dirty = random_cache(rows, hkv, seed=8)
            codes = (dirty.k if name == "k" else dirty.v).view(torch.uint8)
            for a, x in zip(starts, lens):
                codes[a + x - back, 1, 5 if name == "v" else slice(None)] = 0xFF
            for p in (None, ints(*prefix)):
                a = ops.cached_attention(q, clean, ints(*starts), ints(*lens), p)
                b = ops.cached_attention(q, dirty, ints(*starts), ints(*lens), p)
                assert torch.equal(a[:, :t - back], b[:, :t - back])
                assert torch.equal(a[:, :, :4], b[:, :, :4])  # the other key head
                hit = b[:, t - back:, 4:]
                assert hit.isnan().all() if name == "k" else (hit[..., 5].isnan().all() and hit.isnan().sum() == hit[..., 5].numel())


def test_nan_and_infinite_queries_stay_in_their_rows(ops):
    cache = random_cache(100, 2, seed=1)
    q = randn(2, 3, 8, D, seed=1)
    clean = ops.cached_attention(q, cache, ints(0, 20), ints(80, 80))
    q[0, 1, 2, 3], q[1, 0, 7, 9] = float("nan"), float("inf")
    o = ops.cached_attention(q, cache, ints(0, 20), ints(80, 80))
    assert o[0, 1, 2].isnan().all() and o[1, 0, 7].isnan().all()
    o[0, 1, 2], o[1, 0, 7] = clean[0, 1, 2], clean[1, 0, 7]
    assert torch.equal(o, clean)


def test_lengths_that_leave_the_cache(ops):
    from comm_overlap_gb300 import domino as dm
    cache = random_cache(100, 2, seed=1)
    q = randn(4, 4, D, seed=1)
    for starts, lens in (([0, 50, 0, 0], [100, 51, 5, 0]), ([0, -1, 0, 0], [100, 5, 5, 0]), ([0, 3, 0, 0], [100, -5, 5, 0]),
                         ([0, 2**31 - 1, 0, 0], [100, 2**31 - 1, 5, 0])):
        o, lse = ops.cached_attention(q, cache, ints(*starts), ints(*lens), return_lse=True)
        with pytest.raises(dm.DominoError, match="INVALID_ARG"):
            ops.device_status()
        assert not o[1].any() and (lse[1] == -math.inf).all()
        lens[1], starts[1] = 0, 0
        assert torch.equal(o, ops.cached_attention(q, cache, ints(*starts), ints(*lens)))
        ops.device_status()
    o = ops.cached_attention(q, cache, ints(0, 0, 0, 0), ints(10, 20, 0, 1), ints(90, 11))
    with pytest.raises(dm.DominoError, match="INVALID_ARG"):
        ops.device_status()
    close(o, ops.cached_attention(q, cache, ints(0, 0, 0, 0), ints(10, 20, 0, 1)).double(), 2.0 ** -8 * o.double().abs())


def test_strides_given_outputs_and_empty_calls(ops):
    cache = random_cache(200, 2, seed=3)
    qkv = randn(5, 8, D, seed=2)
    q = qkv[:, :4]
    starts, lens = ints(0, 10, 20, 30, 40), ints(100, 0, 3, 64, 33)
    want = ops.cached_attention(q.contiguous(), cache, starts, lens)
    wide = torch.full((5, 7, D), 3.0, dtype=BF, device="cuda")
    got = ops.cached_attention(q, cache, starts, lens, out=wide[:, 1:5])
    assert torch.equal(got, want) and (wide[:, 0] == 3).all() and (wide[:, 5:] == 3).all()
    assert torch.equal(ops.cached_attention(q[:, None], cache, starts, lens)[:, 0], want)
    strided = torch.stack([starts, lens], dim=1)
    assert torch.equal(ops.cached_attention(q, cache, strided[:, 0], strided[:, 1]), want)
    assert ops.cached_attention(q[:0], cache, starts[:0], lens[:0]).shape == (0, 4, D)
    assert ops.cached_attention(q[:, None][:, :0], cache, starts, lens).shape == (5, 0, 4, D)
    none = ops.QuantizedCache.empty(0, 2)
    o, lse = ops.cached_attention(q, none, ints(0, 0, 0, 0, 0), ints(0, 0, 0, 0, 0), return_lse=True)
    assert not o.any() and (lse == -math.inf).all()
    with pytest.raises(ValueError, match="out"):
        ops.cached_attention(q, cache, starts, lens, out=torch.empty(4, 5, D, dtype=BF, device="cuda").transpose(0, 1))
    # exponents with a stride, codes of one layer of a larger cache
    exps = torch.zeros(2, 2, 300, dtype=torch.uint8, device="cuda")
    exps[0, :, 7:207], exps[1, :, 7:207] = cache.k_exp, cache.v_exp
    assert torch.equal(ops.cached_attention(q, (cache.k, cache.v, exps[0, :, 7:207], exps[1, :, 7:207]), starts, lens), want)


def test_offsets_beyond_32_bits(ops):
    """4.4 GB of codes each: the last rows' offsets pass 2^32."""
    rows, hkv = (1 << 32) // (8 * D) + 1000, 8
    cache = ops.QuantizedCache.empty(rows, hkv)
    k, v = randn(900, hkv, D, seed=1), randn(900, hkv, D, seed=2)
    last = torch.arange(rows - 900, rows, dtype=torch.int32, device="cuda")
    ops.cache_write(cache, last, k, v)
    small = ops.QuantizedCache.empty(900, hkv)
    ops.cache_write(small, torch.arange(900, dtype=torch.int32, device="cuda"), k, v)
    q = randn(2, 16, D, seed=3)
    a = ops.cached_attention(q, cache, ints(rows - 900, rows - 33), ints(900, 33))
    b = ops.cached_attention(q, small, ints(0, 867), ints(900, 33))
    assert torch.equal(a, b)
    assert torch.equal(ops.cache_read(cache, last)[0], ops.cache_read(small, ints(*range(900)))[0])
    device_ok()


def test_same_bits_again_and_on_another_stream(ops):
    cache = random_cache(4000, 4, seed=2)
    q = randn(6, 3, 28, D, seed=1)
    starts, lens = ints(0, 100, 200, 300, 400, 500), ints(3000, 17, 0, 900, 2222, 3)
    first = ops.cached_attention(q, cache, starts, lens, ints(3500, 500), return_lse=True)
    for _ in range(5):
        again = ops.cached_attention(q, cache, starts, lens, ints(3500, 500), return_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = ops.cached_attention(q, cache, starts, lens, ints(3500, 500), return_lse=True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert power(torch.tensor([3])).item() == 8
