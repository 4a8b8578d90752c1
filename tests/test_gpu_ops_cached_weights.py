"""Attention over the 8-bit cache where the softmax's weights differ widely: one key that holds most of them before a long rest, and
rows whose value is zero.

The bound is one of an attention whose weights are rounded, each for itself: with p the weights in 64 bits, O is off by its own rounding
to bf16, 2^-8 |O|, and by sum_j p_j |v_j| times

* 2^-9 + 2^-11, the rounding of a weight to three terms of three bits from fp16's eleven,
* 2 delta, delta = scale (2^-21 max |q| sum |k| + 50 U32 sum |q k|) + 6 U32 (|t| + 60), the scores' arithmetic (2 x 128 products by 8
  instructions, each off by at most 5 U32 of its terms' sizes, which are at most 9/8 of sum |q k|), once in O and once in the denominator,
* 2^-21, the exponential, in both,
* 2 (n / 4 + 64) U32, the sums: for each term an instruction for 32 keys, off by at most 5 U32 of its terms' sizes, 1 + 2^-3 + 2^-5 of the
  whole; the denominator's n / 128 a thread, then 128,

and by n 1.125 2^-31 of the largest p_j max|v_j|: weights below 2^-13 are off by half the third term's smallest step, 2^-17 / 32, and by half
of fp16's, 2^-25, where the row's largest is at least 2^9.  (n 2^-31 <= 2^-13 here.)"""
import math

import pytest
import torch

from cache_helpers import D, values
from ops_helpers import U32, device_ok, randn

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


def signs(seed):
    """A direction of norm sqrt(128): a query along it has scores of unit variance with normal keys."""
    return torch.where(randn(D, seed=seed) > 0, 1.0, -1.0)


def queries(n, t, hq, u):
    return (u + 0.1 * randn(n, t, hq, D, seed=4).float()).to(BF)


def filled(ops, k, v):
    """A cache with k and v [rows, heads, 128] written to its rows."""
    cache = ops.QuantizedCache.empty(k.shape[0], k.shape[1])
    ops.cache_write(cache, torch.arange(k.shape[0], dtype=torch.int32, device="cuda"), k.to(BF), v.to(BF))
    return cache


def check(ops, q, cache, first, n, prefix=None):
    """Every sequence of q [sequences, t, heads, 128] has the same n keys from row `first` (behind those of `prefix`): o, lse and the
    softmax's weights in 64 bits by head."""
    count, t, hq, _ = q.shape
    hkv = cache.k.shape[1]
    g = hq // hkv
    ones = torch.full((count,), 1, dtype=torch.int32, device="cuda")
    o, lse = ops.cached_attention(q, cache, first * ones, n * ones, ints(*prefix) if prefix else None, return_lse=True)
    device_ok()
    a, b = prefix if prefix else (0, 0)
    rows = list(range(a, a + b)) + list(range(first, first + n))
    weights = []
    for h in range(hkv):
        k, v = (values(cache, x, rows)[:, h] for x in "kv")
        bias = cache.v_exp[h][torch.tensor(rows, device="cuda")].double() - 127
        qh = q[:, :, h * g:(h + 1) * g].double().reshape(-1, D)  # sequences, t, group
        z = qh @ k.t() * D ** -0.5
        hidden = torch.arange(len(rows), device="cuda") >= (b + n - t + 1 + torch.arange(t, device="cuda")).repeat(count).repeat_interleave(g)[:, None]
        z.masked_fill_(hidden, -math.inf)
        p = torch.softmax(z, -1)
        size = (qh.abs() @ k.abs().t()).amax(-1) * D ** -0.5
        coarse = 2.0 ** -21 * qh.abs().amax(-1) * k.abs().sum(-1).amax() * D ** -0.5
        tt = (z.masked_fill(hidden, 0) / math.log(2) + bias).abs().amax(-1)
        delta = coarse + U32 * (50 * size + 6 * (tt + 60))
        each = 2.0 ** -9 + 2.0 ** -11 + 2 * delta + 2.0 ** -21 + 2 * (len(rows) / 4 + 64) * U32
        ref, spread = p @ v, p @ v.abs()
        slop = each[:, None] * spread + len(rows) * 1.125 * 2.0 ** -31 * (p * v.abs().amax(-1)).amax(-1, keepdim=True)
        got = o[:, :, h * g:(h + 1) * g].double().reshape(-1, D)
        err = (got - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 1.01 * slop).all(), f"off by {float((err - 2.0 ** -8 * ref.abs()).max()):.3g} at a size of " \
            f"{float(ref.abs().max()):.3g}, norms' ratio {float(err.norm() / ref.norm()):.3g}"
        assert err.norm() <= 2.0 ** -8 * ref.norm() + 1.01 * slop.norm()
        want = torch.logsumexp(z, -1)
        off = (lse[:, :, h * g:(h + 1) * g].double().reshape(-1) - want).abs()
        assert (off <= delta + 2.0 ** -21 + (len(rows) / 4 + 64) * U32 + 8 * U32 * (want.abs() + 120)).all(), float(off.max())
        weights.append(p)
    return weights


# (sequences, tokens, query heads, key heads): blocks of 8, 16 and 32 rows, and more sequences than there are ranges of blocks, so that a
# range holds whole ones
SHAPES = [(160, 1, 4, 2), (320, 1, 16, 1), (320, 2, 16, 1), (310, 3, 6, 1)]
KEYS = [(8192, share, place) for share in (0.5, 0.9, 0.99) for place in ("first", "middle", "last")]
KEYS += [(131072, share, place) for share in (0.9, 0.99) for place in ("first", "last")]


@pytest.mark.parametrize("n,share,place", KEYS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_key_before_a_long_rest(ops, shape, n, share, place):
    """Values with a mean, so that what the rest weighs does not cancel out."""
    count, t, hq, hkv = shape
    if n > 10000 and hkv == 2:
        count = 40
    u = signs(1)
    k, v = randn(n, hkv, D, seed=2).float(), randn(n, hkv, D, seed=3).float() + 0.5
    at = dict(first=0, middle=n // 2, last=n - t)[place]
    k[at] = u * (math.log(n * math.exp(0.5) * share / (1 - share)) / math.sqrt(D))
    for p in check(ops, queries(count, t, hq, u), filled(ops, k, v), 0, n):
        assert abs(float(p[:, at].mean()) - share) < 0.15


@pytest.mark.parametrize("gap", [12.0, 13.0])
def test_one_key_before_262143(ops, gap):
    u, n = signs(1), 262144
    k, v = randn(n, 1, D, seed=2).float(), randn(n, 1, D, seed=3).float() + 0.5
    k[0] = u * (gap / math.sqrt(D))
    check(ops, queries(310, 1, 2, u), filled(ops, k, v), 0, n)
    check(ops, queries(1, 1, 2, u), filled(ops, k, v), 0, n)


@pytest.mark.parametrize("share", [0.5, 0.95])
@pytest.mark.parametrize("shape", [(1, 1, 4, 2), (8, 1, 32, 8), (48, 1, 32, 8), (20, 5, 28, 4)], ids=str)
def test_one_key_of_the_shared_rows(ops, shape, share):
    count, t, hq, hkv = shape
    u, n, own = signs(1), 16001, 200
    k, v = randn(n + own, hkv, D, seed=2).float(), randn(n + own, hkv, D, seed=3).float() + 0.5
    k[3] = u * (math.log(n * math.exp(0.5) * share / (1 - share)) / math.sqrt(D))
    check(ops, queries(count, t, hq, u), filled(ops, k, v), n, own, (0, n))


@pytest.mark.parametrize("gap", [0.0, 3.0, 5.0, 8.0, 30.0])
@pytest.mark.parametrize("size", [1.0, 0.05, 1e-4])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_a_row_without_value(ops, place, size, gap):
    """A key whose value is zero, so many nats above the others, takes from the others' weight and adds nothing, whatever their size."""
    n, u = 1000, signs(1)
    for count, t, hq, hkv in ((2, 1, 4, 2), (1, 2, 16, 2), (40, 3, 32, 8)):
        k, v = randn(n, hkv, D, seed=2).float(), (randn(n, hkv, D, seed=3).float() + 0.5) * size
        at = dict(first=0, middle=n // 2, last=n - 1)[place]
        k[at], v[at] = u * (gap / math.sqrt(D)), 0
        check(ops, queries(count, t, hq, u), filled(ops, k, v), 0, n)


def test_a_row_without_value_in_a_long_range(ops):
    for n, gap in ((8192, 8.0), (8192, 9.0), (100000, 12.0)):
        u = signs(1)
        k, v = randn(n, 1, D, seed=2).float(), randn(n, 1, D, seed=3).float() + 0.5
        k[0], v[0] = u * (gap / math.sqrt(D)), 0
        check(ops, queries(310, 1, 4, u), filled(ops, k, v), 0, n)


@pytest.mark.parametrize("shape", [(1, 1, 4, 2), (3, 2, 16, 2), (48, 1, 32, 8)], ids=str)
def test_rows_left_empty(ops, shape):
    """Rows of the cache that nothing was written to, among small values; also in front of others and shared."""
    count, t, hq, hkv = shape
    n, u = 3001, signs(1)
    k, v = randn(n, hkv, D, seed=2).float(), (randn(n, hkv, D, seed=3).float() + 0.5) * 1e-3
    empty = torch.rand(n, generator=torch.Generator().manual_seed(5)) < 0.3
    empty[:200] = True
    k[empty], v[empty] = 0, 0
    check(ops, queries(count, t, hq, u), filled(ops, k, v), 0, n)
    check(ops, queries(count, t, hq, u), filled(ops, k, v), 2000, 1001, (0, 2000))
    v[:] = 0
    check(ops, queries(count, t, hq, u), filled(ops, k, v), 0, n)


def test_a_row_of_zeros_and_nan(ops):
    """A value of zeros and a NaN is NaN there, and elsewhere as one of zeros."""
    n, u = 1000, signs(1)
    for count, t, hq, hkv in ((2, 1, 4, 2), (40, 3, 32, 8)):
        k, v = randn(n, hkv, D, seed=2).float(), (randn(n, hkv, D, seed=3).float() + 0.5) * 0.01
        k[100], v[100] = u * (5 / math.sqrt(D)), 0
        q, one = queries(count, t, hq, u), torch.ones(count, dtype=torch.int32, device="cuda")
        want = ops.cached_attention(q, filled(ops, k, v), 0 * one, n * one)
        v[100, :, 7] = float("inf")
        got = ops.cached_attention(q, filled(ops, k, v), 0 * one, n * one)
        assert got[..., 7].isnan().all()
        got[..., 7] = want[..., 7]
        assert torch.equal(got, want)
    device_ok()
