"""Rotary positions, the 8-bit cache and attention over it, on the GPU, against
the fp64 oracle.

Tolerances (eps = torch.finfo(dtype).eps, a rounding is off by eps / 2):
  rope    an output is off by eps/2 of itself and by 6e-7 of its pair's length:
          sincospif's 2 ulp of each (2^-23 sqrt 2 in all), the angle's float
          (pi 2^-25) and three roundings of products and sums (3 * 2^-24).
  codes   u / 2^e is computed with 7 additions and 2 products, so it is off by
          9 * 2^-24 * sum|x| / sqrt h / 2^e <= 9 * 2^-24 * ||u|| / 2^e
          <= 9 * 2^-24 * sqrt(128) * 127 < 8e-4 steps: a code may differ from
          the oracle's, by one, only within 1e-3 of a border.
  read    u = code * 2^e is exact; the transform's 7 additions and one product
          are off by 8 * 2^-24 ||u|| at most, then eps/2 of the value.
  attn    for each row, the oracle's bound (roundings of queries and weights to
          fp16) plus eps/2 of the row's norm (+ 8 * 2^-24 of it for the turn).
"""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import rpbh as orpbh

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def oq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from calibration_free_rotated_b200 import build
    build.build()
    from calibration_free_rotated_b200 import orbitquant
    return orbitquant


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cum(v):
    return [0] + list(np.cumsum(v))


def rotation(oq, d, block, seed=0):
    if not block:
        return None, None
    perm, signs = orpbh.draw_permutation_and_signs(seed, d)
    return oq.Rpbh(seed, d, block), (perm, signs, block)


def rows(rng, shape, dt, loud=True):
    x = rng.standard_normal(shape)
    if loud:
        x = x * np.exp(0.4 * rng.standard_normal(shape[-2:])) * (1 + 7 * (rng.random(shape[-2:]) < 0.03))
    return torch.from_numpy(x).to(DT[dt]).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------ rope
ROPES = [  # T, heads, d, axis_dims, layout, dtype
    (1, 1, 64, (64,), "interleaved", "bf16"),
    (1, 40, 128, (128,), "halves", "bf16"),
    (17, 3, 128, (16, 56, 56), "interleaved", "fp16"),
    (130, 24, 128, (44, 42, 42), "interleaved", "bf16"),
    (33, 5, 128, (32, 32), "halves", "fp32"),          # a part of the head turns
    (33, 5, 72, (30, 4), "interleaved", "bf16"),       # the turned part ends inside a vector
    (33, 5, 72, (30, 4), "interleaved", "fp32"),
    (9, 2, 40, (6,), "interleaved", "fp16"),
    (5, 2, 24, (16,), "halves", "bf16"),               # one vector stands alone at the end
    (7, 1, 512, (512,), "halves", "fp32"),
    (7, 1, 512, (128, 128, 128, 128), "interleaved", "fp32"),
    (3000, 2, 8, (4, 4), "interleaved", "fp32"),
]


@pytest.mark.parametrize("T,heads,d,dims,layout,dt", ROPES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(oq, T, heads, d, dims, layout, dt, inverse):
    rng = np.random.default_rng(T + d)
    r = oq.Rope(dims, layout=layout)
    fused = torch.from_numpy(rng.standard_normal((T, heads + 2, d))).to(DT[dt]).cuda()
    x = fused[:, 1:1 + heads]
    pos = rng.integers(-5, 2_000_000_000, (T, len(dims)))
    pos[: T // 2] %= 70
    freq = [10000.0 ** (-2 * k / n) for n in dims for k in range(n // 2)]
    axis = [a for a, n in enumerate(dims) for _ in range(n // 2)]
    want = oc.rope(f64(x), pos, freq, axis, layout == "halves", inverse)
    got = f64(oq.rope_apply(r, x, ints(pos), inverse=inverse))
    n = sum(dims) // 2
    length = np.zeros(want.shape)
    i = np.arange(n)
    a, b = (i, i + n) if layout == "halves" else (2 * i, 2 * i + 1)
    length[..., a] = length[..., b] = np.hypot(want[..., a], want[..., b])
    # the angle's products in the oracle are rounded too: pos * freq to 2^-53 of itself
    drift = np.zeros(want.shape)
    phi = np.abs(pos[:, axis] * np.array(freq))[:, None] * 2.0 ** -51
    drift[..., a] = drift[..., b] = phi
    assert np.all(np.abs(got - want) <= torch.finfo(DT[dt]).eps / 2 * 1.001 * np.abs(want) + (6e-7 + drift) * length)
    assert np.array_equal(got[..., 2 * n:], f64(x)[..., 2 * n:])  # carried over
    keep = fused.clone()
    oq.rope_apply(r, x, ints(pos), out=x, inverse=inverse)  # in place
    assert np.array_equal(f64(x), got)
    assert torch.equal(fused[:, 0], keep[:, 0]) and torch.equal(fused[:, 1 + heads:], keep[:, 1 + heads:])


def test_rope_ladders_and_infinities(oq):
    rng = np.random.default_rng(5)
    x = rows(rng, (6, 2, 64), "fp32")
    pos = rng.integers(0, 1000, (6, 3))
    shared = [10000.0 ** (-2 * p / 48) for p in range(24)]
    axis = [0] * 8 + [1] * 8 + [2] * 8
    want = oc.rope(f64(x), pos, shared, axis, True)
    got = oq.rope_apply(oq.Rope((16, 16, 16), layout="halves", ladder="shared"), x, ints(pos))
    again = oq.rope_apply(oq.Rope(freqs=shared, axes=axis, layout="halves"), x, ints(pos))
    assert torch.equal(got, again)
    assert np.abs(f64(got) - want).max() <= 1e-6 * np.abs(want).max() * 2
    # what is carried over keeps its bits, whatever stands in it
    for dt in ("bf16", "fp32"):
        y = rows(rng, (3, 1, 40), dt)
        y[:, :, 6:] = float("inf")
        y[1, 0, 7:20] = float("nan")
        for layout, dims in (("interleaved", (6,)), ("halves", (16,))):
            z = oq.rope_apply(oq.Rope(dims, layout=layout), y, ints(np.ones((3, 1))))
            assert torch.equal(z.view(torch.int8)[..., sum(dims) * y.element_size():],
                               y.view(torch.int8)[..., sum(dims) * y.element_size():])


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_rope_gradient(oq, layout):
    """dX = the inverse turn of dY: against a difference quotient of the forward
    pass (linear, so exact up to rounding) and as the transpose."""
    rng = np.random.default_rng(11)
    r = oq.Rope((16, 24, 24), layout=layout)
    pos = ints(rng.integers(0, 5000, (9, 3)))
    x, dy, dx = (rows(rng, (9, 3, 64), "fp32", loud=False) for _ in range(3))
    grad = oq.rope_apply(r, dy, pos, inverse=True)
    up, down = oq.rope_apply(r, x + dx, pos), oq.rope_apply(r, x - dx, pos)
    lhs = float(((up - down).double() / 2 * dy.double()).sum())
    rhs = float((dx.double() * grad.double()).sum())
    size = float(dx.double().norm() * dy.double().norm())
    assert abs(lhs - rhs) <= 4e-6 * size
    back = oq.rope_apply(r, oq.rope_apply(r, x, pos), pos, inverse=True)
    assert float((back - x).abs().max()) <= 4e-6 * float(x.abs().max())


# ----------------------------------------------------------------------- cache
class Batch:
    """Sequences with pages of their own in a shuffled pool."""

    def __init__(self, rng, new, past, page, spare=2, extra_width=1):
        self.new, self.past, self.page = new, past, page
        self.total = [a + b for a, b in zip(new, past)]
        self.width = max(max(-(-t // page) for t in self.total), 1) + extra_width
        need = sum(-(-t // page) for t in self.total)
        pool = list(rng.permutation(need + spare))
        self.n_pages = need + spare
        self.table = np.full((len(new), self.width), -7, dtype=np.int64)  # what is not needed is not read
        for b, t in enumerate(self.total):
            for s in range(-(-t // page)):
                self.table[b, s] = pool.pop()
        self.T = sum(new)
        self.cu = cum(new)


def snapshot(cache):
    e = np.round(np.log2(np.maximum(f64(cache.k_scale), 2.0 ** -60))).astype(int)
    ev = np.round(np.log2(np.maximum(f64(cache.v_scale), 2.0 ** -60))).astype(int)
    return cache.k.cpu().numpy().astype(int), e, cache.v.cpu().numpy().astype(int), ev


def check_write(oq, cache, bt, k, v, r, rot):
    kc, ke, vc, ve = snapshot(cache)
    oq.cache_write(cache, k, v, ints(bt.cu), ints(bt.past), ints(bt.table), rpbh=r)
    oq.device_status()
    gk, gke, gv, gve = snapshot(cache)
    for codes, exps, got, gexp, x in ((kc, ke, gk, gke, k), (vc, ve, gv, gve, v)):
        near = oc.write(codes, exps, f64(x), bt.cu, bt.past, bt.table, rot)
        assert np.array_equal(exps, gexp)
        diff = np.abs(got - codes)
        assert diff.max() <= 1
        free = np.zeros(codes.shape, bool)  # written, and near a border
        P = bt.page
        for b in range(len(bt.new)):
            for i in range(bt.new[b]):
                p = bt.past[b] + i
                free[bt.table[b, p // P], :, p % P] = near[bt.cu[b] + i] < 1e-3
        assert not np.any(diff.astype(bool) & ~free)
        assert diff.sum() <= 0.002 * max(1000, near.size)


WRITES = [  # new, past, heads, d, page, block, dtype
    ([1], [0], 1, 64, 16, 64, "bf16"),
    ([1, 1, 1], [0, 15, 16], 2, 128, 16, 128, "bf16"),
    ([5, 0, 33, 1], [3, 9, 63, 127], 3, 128, 64, 64, "fp16"),
    ([200], [0], 2, 64, 32, 32, "bf16"),
    ([130, 7], [100, 0], 1, 128, 128, 128, "bf16"),
    ([130, 7], [1, 60], 2, 64, 128, 0, "fp16"),
    ([64, 16, 17], [0, 16, 47], 2, 64, 16, 0, "bf16"),
]


@pytest.mark.parametrize("new,past,heads,d,page,block,dt", WRITES)
def test_write_and_read(oq, new, past, heads, d, page, block, dt):
    rng = np.random.default_rng(sum(new) + d + page)
    r, rot = rotation(oq, d, block)
    bt = Batch(rng, new, past, page)
    cache = oq.KVCache(bt.n_pages, heads, d, page)
    cache.k.copy_(torch.from_numpy(rng.integers(-127, 128, cache.k.shape)))  # pages' last users
    cache.v.copy_(torch.from_numpy(rng.integers(-127, 128, cache.k.shape)))
    cache.k_scale.fill_(2.0 ** 9)
    cache.v_scale.fill_(2.0 ** 9)
    old = Batch.__new__(Batch)
    old.__dict__.update(bt.__dict__)
    old.new, old.past, old.T, old.cu = bt.past, [0] * len(new), sum(past), cum(bt.past)
    if old.T:
        check_write(oq, cache, old, rows(rng, (old.T, heads, d), dt), rows(rng, (old.T, heads, d), dt), r, rot)
    # the new rows are larger: the pages' scales grow and the older codes are halved
    fused = rows(rng, (bt.T + 2, 2 * heads + 1, d), dt)
    fused *= 11
    k, v = fused[:bt.T, 1:1 + heads], fused[:bt.T, 1 + heads:]
    check_write(oq, cache, bt, k, v, r, rot)
    # the same call again changes nothing
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    oq.cache_write(cache, k, v, ints(bt.cu), ints(bt.past), ints(bt.table), rpbh=r)
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)))

    # read back: all of it, and a part from the middle, rows behind the last sequence left alone
    for first, count in (([0] * len(new), bt.total), ([t // 3 for t in bt.total], [t - t // 3 for t in bt.total])):
        cu = cum(count)
        ko, vo = (torch.full((cu[-1] + 3, heads, d), 7.0, dtype=DT[dt], device="cuda") for _ in range(2))
        oq.cache_read(cache, ints(cu), ints(first), ints(bt.table), rpbh=r, k=ko, v=vo)
        oq.device_status()
        for codes, scale, got in ((cache.k, cache.k_scale, ko), (cache.v, cache.v_scale, vo)):
            assert torch.all(got[cu[-1]:] == 7.0)
            for b in range(len(new)):
                u = oc.gather(codes.cpu().numpy(), f64(scale), bt.table[b], bt.total[b])[first[b]:]
                x = oc.turn_back(u, rot)
                tol = torch.finfo(DT[dt]).eps / 2 * 1.001 * np.abs(x) + 8 * 2.0 ** -24 * np.linalg.norm(u, axis=-1)[..., None]
                if rot is None and dt == "bf16":
                    tol = 0 * x  # 7 bits times a power of two: exact
                assert np.all(np.abs(f64(got[cu[b]:cu[b + 1]]) - x) <= tol)


def test_portions_stay_within_a_step(oq):
    """Tokens written one by one, each louder than the last, against the values
    themselves: no more than one step of the scale that stands."""
    rng = np.random.default_rng(3)
    d, heads, page = 64, 2, 16
    r, rot = rotation(oq, d, 64)
    cache = oq.KVCache(2, heads, d, page)
    x = rows(rng, (16, heads, d), "bf16", loud=False)
    x *= (1.3 ** torch.arange(16, device="cuda"))[:, None, None].to(x.dtype)
    table = ints([[1]])
    for t in range(16):
        oq.cache_write(cache, x[t:t + 1], x[t:t + 1], ints([0, 1]), ints([t]), table, rpbh=r)
    u = oc.turn(f64(x), rot)
    got = oc.gather(cache.k.cpu().numpy(), f64(cache.k_scale), [1], 16)
    step = f64(cache.k_scale)[1][None, :, None]
    assert np.all(np.abs(got - u) <= step * 1.001)
    assert np.abs(got - u).max() > 0.5 * step.min()  # the halvings did happen


def test_write_extremes(oq):
    d = 64
    cache = oq.KVCache(6, 1, d, 16)
    x = torch.zeros((6, 1, d), dtype=torch.bfloat16, device="cuda")
    x[1] = 3e38          # saturates
    x[2, 0, 0] = float("inf")
    x[3, 0, 0] = float("nan")
    x[3, 0, 1] = 127.0
    x[4] = 2.0 ** -60    # below the smallest step
    x[5, 0, :3] = torch.tensor([127.0, 0.5, 1.5])  # the largest value of a scale; ties go to even
    oq.cache_write(cache, x, x, ints(range(7)), ints([0] * 6), ints([[b] for b in range(6)]))
    oq.device_status()
    k, s = cache.k[:, 0, 0].cpu().numpy(), f64(cache.k_scale)[:, 0]
    assert not k[0].any() and s[0] == 2.0 ** -40
    assert np.all(k[1] == 127) and s[1] == 2.0 ** 40
    assert k[2, 0] == 127 and not k[2, 1:].any()
    assert k[3, 0] == 0 and k[3, 1] == 127 and s[3] == 1.0
    assert not k[4].any() and s[4] == 2.0 ** -40
    assert list(k[5, :3]) == [127, 0, 2] and s[5] == 1.0
    ko, _ = oq.cache_read(cache, ints(range(7)), ints([0] * 6), ints([[b] for b in range(6)]), T=6)
    assert torch.isfinite(ko.float()).all()


def test_bad_indices_are_left_out(oq):
    """Pages and lengths out of range: the others are served, the status says so."""
    rng = np.random.default_rng(8)
    d, heads, P = 64, 2, 16
    cache = oq.KVCache(4, heads, d, P)
    k = rows(rng, (8, heads, d), "bf16")
    cu = ints([0, 2, 4, 6, 8])
    good = ([[0, 1], [4, 1], [-1, 0], [2, 3]], [0, 0, 0, 15])
    for table, past in (good, ([[0, 1], [1, 1], [2, 0], [3, 3]], [0, -3, 31, 2 ** 31 - 1])):
        cache.k.zero_()
        oq.cache_write(cache, k, k, cu, ints(past), ints(table))
        with pytest.raises(oq.OQError) as e:
            oq.device_status()
        assert e.value.code == oq.OQ_ERR_ARG
        oq.device_status()  # cleared
        assert cache.k[0, :, :2].any() and not cache.k[0, :, 2:].any()
        out = torch.full((8, heads, d), 5.0, dtype=torch.bfloat16, device="cuda")
        vo = out.clone()
        oq.cache_read(cache, cu, ints(past), ints(table), k=out, v=vo)
        with pytest.raises(oq.OQError):
            oq.device_status()
        assert torch.all(out[2:4] == 5.0)
    assert not cache.k[1].any()  # only the bad sequences have it
    # decreasing and overlong offsets
    for bad in ([0, 2, 1, 3, 9], [-1, 2, 4, 6, 8], [2, 0, 0, 0, 100]):
        oq.cache_write(cache, k, k, ints(bad), ints([0] * 4), ints([[0], [1], [2], [3]]))
        with pytest.raises(oq.OQError):
            oq.device_status()
    # attention: a page out of range counts as empty, a sequence that does not fit is left alone
    cache = oq.KVCache(4, heads, d, P)
    oq.cache_write(cache, k, k, ints([0, 8]), ints([0]), ints([[2]]))
    q = rows(rng, (2, heads, d), "bf16")
    one = oq.cache_attention(cache, q[:1], ints([0, 1]), ints([8]), ints([[2]]))
    oq.device_status()
    out = torch.full((2, heads, d), 5.0, dtype=torch.bfloat16, device="cuda")
    oq.cache_attention(cache, q, ints([0, 1, 2]), ints([24, 99]), ints([[2, 9], [2, 2]]), out=out)
    with pytest.raises(oq.OQError):
        oq.device_status()
    assert torch.all(out[1] == 5.0)
    two = oq.cache_attention(cache, q[:1], ints([0, 1]), ints([16]), ints([[2]]))
    oq.device_status()
    assert torch.equal(out[:1], two) and one.shape == two.shape


# ------------------------------------------------------------------- attention
def filled(oq, rng, bt, heads, d, r, dt="bf16", loud=True):
    cache = oq.KVCache(bt.n_pages, heads, d, bt.page)
    n = sum(bt.total)
    if n:
        oq.cache_write(cache, rows(rng, (n, heads, d), dt, loud), rows(rng, (n, heads, d), dt, loud),
                       ints(cum(bt.total)), ints([0] * len(bt.total)), ints(bt.table), rpbh=r)
    return cache


def check_attention(oq, cache, bt, q, r, rot, causal, scale=None, empty_page=None):
    n_rows = q.shape[0]
    out = torch.full((n_rows, q.shape[1], q.shape[2]), 9.0, dtype=q.dtype, device="cuda")
    oq.cache_attention(cache, q, ints(bt.cu), ints(bt.total), ints(bt.table), rpbh=r, causal=causal, scale=scale, out=out)
    oq.device_status()
    assert torch.all(out[bt.cu[-1]:] == 9.0)
    eps = torch.finfo(q.dtype).eps
    codes = [c.cpu().numpy() for c in (cache.k, cache.v)]
    scales = [f64(s) for s in (cache.k_scale, cache.v_scale)]
    for b in range(len(bt.new)):
        k, v = (oc.gather(c, s, bt.table[b], bt.total[b]) for c, s in zip(codes, scales))
        empty = None
        if empty_page is not None:
            empty = np.array([[scales[0][bt.table[b][t // bt.page], h] == 0 for h in range(cache.heads)]
                              for t in range(bt.total[b])], dtype=bool).reshape(bt.total[b], cache.heads)
        want, bound = oc.attention(f64(q[bt.cu[b]:bt.cu[b + 1]]), k, v, causal,
                                   q.shape[2] ** -0.5 if scale is None else scale, rot, empty)
        got = f64(out[bt.cu[b]:bt.cu[b + 1]])
        # a value at or above the type's largest number plus half its last step (fp16: 65520) rounds to
        # infinity: right wherever the exact value is that large within the row's bound
        most = torch.finfo(q.dtype).max
        over = np.isinf(got) & (np.sign(got) * want + bound[..., None] >= most * (1 + eps / 4))
        got = np.where(over, want, got)
        err = np.linalg.norm(got - want, axis=-1)
        limit = bound + (eps / 2 + 8 * 2.0 ** -24) * 1.01 * np.linalg.norm(want, axis=-1)
        assert np.all(err <= limit), (b, (err / np.maximum(limit, 1e-300)).max())
    return out


ATTN = [  # new, past, heads, group, d, page, block, dtype, causal
    ([1], [0], 1, 1, 64, 16, 64, "bf16", True),
    ([1], [16], 2, 4, 128, 16, 128, "bf16", True),
    ([1, 1, 1, 1], [517, 0, 63, 64], 2, 8, 128, 64, 128, "bf16", True),
    ([1] * 7, [3, 900, 31, 32, 33, 2000, 1], 3, 5, 64, 32, 32, "fp16", True),
    ([1, 1], [1300, 700], 1, 16, 128, 128, 0, "bf16", True),
    ([1], [5000], 1, 1, 128, 64, 128, "bf16", False),
    ([4, 0, 2, 7], [100, 10, 1, 0], 2, 2, 64, 16, 64, "bf16", True),
    ([5, 3], [64, 200], 1, 3, 128, 32, 64, "fp16", False),
    ([37, 1, 90], [0, 300, 45], 2, 2, 64, 64, 64, "fp16", True),
    ([129, 40], [70, 0], 2, 1, 128, 16, 128, "bf16", True),
    ([129, 40], [70, 11], 1, 4, 128, 64, 0, "bf16", False),
    ([300], [0], 1, 2, 64, 128, 64, "bf16", True),
    ([33], [0], 2, 1, 128, 16, 128, "fp16", True),
    ([17, 0, 150, 2], [0, 20, 900, 1500], 2, 3, 128, 64, 64, "fp16", True),
    ([200, 9], [130, 64], 1, 5, 64, 32, 0, "fp16", False),
    ([64], [2000], 3, 2, 64, 128, 64, "bf16", False),
    ([128, 128], [0, 128], 1, 1, 128, 32, 128, "bf16", True),
]


@pytest.mark.parametrize("new,past,heads,group,d,page,block,dt,causal", ATTN)
def test_attention(oq, new, past, heads, group, d, page, block, dt, causal):
    rng = np.random.default_rng(sum(new) + sum(past) + d)
    r, rot = rotation(oq, d, block)
    bt = Batch(rng, new, past, page)
    cache = filled(oq, rng, bt, heads, d, r, dt)
    fused = rows(rng, (bt.T + 3, heads * group + 2, d), dt, loud=False) * 2
    check_attention(oq, cache, bt, fused[:, 1:1 + heads * group], r, rot, causal)


@pytest.mark.parametrize("new", [[1, 2], [40, 20]])
def test_attention_scales_far_apart(oq, new):
    """Pages whose values differ by many powers of two, and the score's own range."""
    rng = np.random.default_rng(21)
    r, rot = rotation(oq, 64, 64)
    bt = Batch(rng, new, [200, 90], 16)
    cache = filled(oq, rng, bt, 1, 64, r)
    cache.v_scale *= torch.exp2(torch.from_numpy(rng.integers(-12, 13, (bt.n_pages, 1))).cuda()).float()
    cache.k_scale *= torch.exp2(torch.from_numpy(rng.integers(-3, 2, (bt.n_pages, 1))).cuda()).float()
    for scale in (None, 0.0, -0.3, 2.0):
        check_attention(oq, cache, bt, rows(rng, (sum(new), 2, 64), "fp16", loud=False), r, rot, True, scale)
    q = rows(rng, (sum(new), 2, 64), "bf16", loud=False)
    for f in (1e-30, 1e25):  # a query's own power of two
        check_attention(oq, cache, bt, q * f, r, rot, True, 0.1 / f)


def test_attention_rows_without_keys(oq):
    rng = np.random.default_rng(22)
    bt = Batch(rng, [100, 30, 20], [0, 0, 4], 16)  # many rows
    bt.total = [70, 0, 6]
    cache = filled(oq, rng, bt, 2, 64, None)
    q = rows(rng, (150, 4, 64), "bf16")
    out = check_attention(oq, cache, bt, q, None, None, True)
    assert not out[:30].any() and out[30:100].any() and not out[100:130].any()
    cache.k_scale[bt.table[0, 1]] = 0
    cache.k_scale[bt.table[2, 0]] = 0
    out = check_attention(oq, cache, bt, q, None, None, True, empty_page=True)
    assert out[30:100].any() and not out[100:].any()
    bt = Batch(rng, [5, 3, 2], [0, 0, 4], 16)
    bt.total = [2, 0, 6]  # fewer tokens than queries; none at all
    cache = filled(oq, rng, bt, 2, 64, None)
    q = rows(rng, (10, 4, 64), "bf16")
    out = check_attention(oq, cache, bt, q, None, None, True)
    assert not out[:3].any() and out[3:5].any() and not out[5:8].any()
    out = check_attention(oq, cache, bt, q, None, None, False)
    assert out[:5].any() and not out[5:8].any()
    # pages that hold nothing (a key scale of 0)
    bt = Batch(rng, [1, 1], [100, 20], 16)
    cache = filled(oq, rng, bt, 2, 64, None)
    cache.k_scale[bt.table[0, 2]] = 0
    cache.k_scale[bt.table[1, :2]] = 0
    out = check_attention(oq, cache, bt, q[:2], None, None, True, empty_page=True)
    assert out[0].any() and not out[1].any()


@pytest.mark.parametrize("n", [3, 70])
def test_attention_nan_query_stays_in_its_row(oq, n):
    rng = np.random.default_rng(23)
    r, rot = rotation(oq, 128, 128)
    bt = Batch(rng, [n], [700], 64)
    cache = filled(oq, rng, bt, 1, 128, r)
    q = rows(rng, (n, 2, 128), "bf16")
    clean = oq.cache_attention(cache, q, ints(bt.cu), ints(bt.total), ints(bt.table), rpbh=r)
    q[1, 1, 5] = float("nan")
    out = oq.cache_attention(cache, q, ints(bt.cu), ints(bt.total), ints(bt.table), rpbh=r)
    assert torch.isnan(out[1, 1]).all()
    out[1, 1] = clean[1, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("new,past", [([1, 6], [21, 77]), ([2, 60], [20, 23])])
def test_attention_ignores_what_it_may_not_see(oq, new, past):
    """Codes behind the last token, other pages and their scales change nothing."""
    rng = np.random.default_rng(24)
    r, rot = rotation(oq, 64, 64)
    bt = Batch(rng, new, past, 32)
    cache = filled(oq, rng, bt, 2, 64, r)
    q = rows(rng, (sum(new), 4, 64), "bf16")
    args = (ints(bt.cu), ints(bt.total), ints(bt.table))
    clean = oq.cache_attention(cache, q, *args, rpbh=r)
    used = {int(bt.table[b, s]) for b in range(2) for s in range(-(-bt.total[b] // 32))}
    for p in range(bt.n_pages):
        if p not in used:
            cache.k[p], cache.v[p] = -127, 127
            cache.k_scale[p], cache.v_scale[p] = float("nan"), float("inf")
    cache.k[bt.table[0, 0], :, 22:], cache.v[bt.table[0, 0], :, 22:] = 127, -128
    cache.v[bt.table[1, 2], :, 83 - 64:] = -128
    assert torch.equal(clean, oq.cache_attention(cache, q, *args, rpbh=r))


def test_shared_pages_and_a_batch_beyond_one_block(oq):
    """Many sequences over one shared prefix; the sequences outnumber a CTA's threads."""
    rng = np.random.default_rng(25)
    r, rot = rotation(oq, 64, 64)
    B, P = 300, 16
    lens = [int(n) for n in rng.integers(0, 65, B)]
    cache = oq.KVCache(4, 1, 64, P)
    x = rows(rng, (64, 1, 64), "bf16")
    oq.cache_write(cache, x, x, ints([0, 64]), ints([0]), ints([[2, 0, 3, 1]]), rpbh=r)
    q = rows(rng, (B, 2, 64), "bf16")
    table = ints([[2, 0, 3, 1]] * B)
    out = oq.cache_attention(cache, q, ints(range(B + 1)), ints(lens), table, rpbh=r)
    k = oc.gather(cache.k.cpu().numpy(), f64(cache.k_scale), [2, 0, 3, 1], 64)
    v = oc.gather(cache.v.cpu().numpy(), f64(cache.v_scale), [2, 0, 3, 1], 64)
    for b in range(0, B, 13):
        want, bound = oc.attention(f64(q[b:b + 1]), k[:lens[b]], v[:lens[b]], False, 0.125, rot)
        err = np.linalg.norm(f64(out[b:b + 1]) - want, axis=-1)
        assert np.all(err <= bound + (2.0 ** -8 + 2.0 ** -20) * np.linalg.norm(want, axis=-1))
    # writing and reading with as many sequences
    cache = oq.KVCache(B, 1, 64, P)
    new = [int(n) for n in rng.integers(0, 5, B)]
    y = rows(rng, (sum(new), 1, 64), "bf16")
    tb = ints(rng.permutation(B)[:, None])
    oq.cache_write(cache, y, y, ints(cum(new)), ints([0] * B), tb, rpbh=r)
    ko, vo = oq.cache_read(cache, ints(cum(new)), ints([0] * B), tb, T=sum(new), rpbh=r)
    oq.device_status()
    assert torch.equal(ko, vo)
    assert float((ko.double() - y.double()).norm() / y.double().norm()) < 0.03


SPLITS = [  # new, past, heads, group, d, page, block, dtype, causal
    # several short row tiles of a sequence
    ([12, 30, 0, 5], [0, 700, 3, 64], 2, 2, 128, 64, 64, "fp16", True),
    ([48], [2500], 2, 1, 64, 16, 64, "bf16", True),
    ([3, 3], [1000, 0], 1, 16, 128, 32, 128, "bf16", True),
    ([1, 1], [33, 800], 2, 40, 64, 64, 0, "bf16", True),
    ([17, 40, 1], [90, 0, 2200], 1, 1, 128, 128, 128, "bf16", False),
    # items cut between many CTAs, and many items for each of them
    ([60], [9000], 1, 1, 128, 64, 128, "bf16", True),
    ([70], [4100], 1, 1, 64, 16, 64, "fp16", False),
    ([260, 1, 0, 520], [1000, 7, 0, 0], 3, 1, 128, 16, 128, "bf16", True),
    ([257, 255, 256], [31, 64, 0], 8, 1, 64, 64, 64, "bf16", True),
    ([30, 90] * 25, [40, 0] * 25, 3, 2, 64, 16, 64, "fp16", True),
    # items that are all alike, a few for each CTA (one, two), none of them cut
    ([257, 0, 257], [0, 0, 0], 30, 1, 64, 64, 64, "bf16", False),
    ([300], [0], 75, 1, 64, 64, 64, "bf16", False),
    ([129], [127], 37, 2, 128, 32, 128, "fp16", False),
]


@pytest.mark.parametrize("new,past,heads,group,d,page,block,dt,causal", SPLITS)
def test_attention_work_split(oq, new, past, heads, group, d, page, block, dt, causal):
    rng = np.random.default_rng(sum(new) + sum(past) + d)
    r, rot = rotation(oq, d, block)
    bt = Batch(rng, new, past, page)
    cache = filled(oq, rng, bt, heads, d, r, dt)
    q = rows(rng, (bt.T, heads * group, d), dt, loud=False) * 2
    out = check_attention(oq, cache, bt, q, r, rot, causal)
    # once more, into every other head and token of a larger tensor: the same bits, and nothing beside them
    wide = torch.full((2 * bt.T, 2 * heads * group, d), 3.0, dtype=q.dtype, device="cuda")
    oq.cache_attention(cache, q, ints(bt.cu), ints(bt.total), ints(bt.table), rpbh=r, causal=causal, out=wide[::2, 1::2])
    assert torch.equal(wide[::2, 1::2][:bt.cu[-1]], out[:bt.cu[-1]])
    assert torch.all(wide[1::2] == 3.0) and torch.all(wide[:, ::2] == 3.0)


# ----------------------------------------------------------- streams, graphs, devices
def test_streams_and_graphs(oq):
    """The operators on a stream of their own and in two captured graphs that share a workspace."""
    rng = np.random.default_rng(31)
    r, _ = rotation(oq, 128, 128)
    rope = oq.Rope((16, 56, 56))
    bt = Batch(rng, [1, 3], [300, 40], 64)
    q, k, v = (rows(rng, (4, n, 128), "bf16") for n in (8, 2, 2))
    pos = ints(rng.integers(0, 100, (4, 3)))
    cu, past, total, table = ints(bt.cu), ints(bt.past), ints(bt.total), ints(bt.table)
    ws = torch.empty((oq.cache_attention_workspace_bytes(oq.KVCache(1, 2, 128), 4, 2, 8),), dtype=torch.uint8,
                     device="cuda")
    base = filled(oq, rng, bt, 2, 128, r)

    def step(cache, out, stream=None):
        oq.cache_write(cache, oq.rope_apply(rope, k, pos, stream=stream), v, cu, past, table, rpbh=r, stream=stream)
        oq.cache_attention(cache, oq.rope_apply(rope, q, pos, stream=stream), cu, total, table, rpbh=r, out=out,
                           workspace=ws, stream=stream)

    def fresh():
        return oq.KVCache.wrap(*(t.clone() for t in (base.k, base.v, base.k_scale, base.v_scale)))

    want, cache = torch.empty_like(q), fresh()
    step(cache, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, other = torch.empty_like(q), fresh()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(other, got)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(cache.k, other.k)
    got.zero_()
    third = fresh()
    torch.cuda.synchronize()
    kr, qr = oq.rope_apply(rope, k, pos), oq.rope_apply(rope, q, pos)
    torch.cuda.synchronize()
    oq.cache_write(third, kr, v, cu, past, table, rpbh=r, stream=side)
    oq.cache_attention(third, qr, cu, total, table, rpbh=r, out=got, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    caches, outs, graphs = [fresh(), fresh()], [torch.zeros_like(q) for _ in range(2)], []
    for c, o in zip(caches, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c, o)
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    oq.device_status()


@pytest.mark.parametrize("n", [1, 20, 200])
def test_two_calls_at_once(oq, n):
    """Two streams with a workspace each, over one cache, many calls in flight."""
    rng = np.random.default_rng(34)
    r, _ = rotation(oq, 64, 64)
    bt = Batch(rng, [n, n], [700, 90], 16)
    cache = filled(oq, rng, bt, 2, 64, r)
    cu, total, table = ints(bt.cu), ints(bt.total), ints(bt.table)
    q = [rows(rng, (bt.T, 4, 64), "bf16") for _ in range(2)]
    want = [oq.cache_attention(cache, x, cu, total, table, rpbh=r) for x in q]
    need = oq.cache_attention_workspace_bytes(cache, bt.T, 2, 4)
    ws = [torch.empty((need,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [[torch.zeros_like(q[0]) for _ in range(20)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for j in range(2):
            oq.cache_attention(cache, q[j], cu, total, table, rpbh=r, out=outs[j][i], workspace=ws[j], stream=streams[j])
    torch.cuda.synchronize()
    oq.device_status()
    for j in range(2):
        for o in outs[j]:
            assert torch.equal(o, want[j])


def test_memory_made_for_another_stream_is_its_own(oq):
    """Without `out` and `workspace`, what a call on a given stream makes comes from that stream's memory."""
    rng = np.random.default_rng(36)
    bt = Batch(rng, [3, 1], [50, 700], 16)
    cache = filled(oq, rng, bt, 2, 64, None)
    q, rope, pos = rows(rng, (4, 4, 64), "bf16"), oq.Rope((64,)), ints([[0], [1], [2], [3]])
    cu, total, table = ints(bt.cu), ints(bt.total), ints(bt.table)
    want = oq.cache_attention(cache, oq.rope_apply(rope, q, pos), cu, total, table)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    turned = oq.rope_apply(rope, q, pos, stream=side)
    got = oq.cache_attention(cache, turned, cu, total, table, stream=side)
    k, _ = oq.cache_read(cache, cu, ints([0, 0]), table, T=4, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    blocks = [(s["address"], s["address"] + s["total_size"]) for s in torch.cuda.memory_snapshot()
              if s["stream"] == side.cuda_stream]
    for t in (turned, got, k):
        assert any(a <= t.data_ptr() < b for a, b in blocks)
    need = oq.cache_attention_workspace_bytes(cache, 4, 2, 4)
    assert sum(b - a for a, b in blocks) >= need


_CHILD = r"""
import sys
import torch
sys.path.insert(0, sys.argv[1])
from calibration_free_rotated_b200 import orbitquant as oq
torch.manual_seed(5)
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
r, rope, outs = oq.Rpbh(0, 128, 128), oq.Rope((16, 56, 56)), []
x = torch.randn(90, 6, 128, device="cuda").bfloat16()
pos = ints([[i, i // 7, i % 7] for i in range(90)])
for rep in range(3):  # back to back: each launch follows one that it reads from or that used the workspace
    cache = oq.KVCache(8, 2, 128, 32)
    table = ints([[1, 2, 3, 6], [4, 0, 5, 7]])
    for new, past in (([60, 30], [0, 0]), ([1, 1], [60, 30]), ([1, 2], [61, 31])):
        T, cu = sum(new), ints([0, new[0], sum(new)])
        kv = oq.rope_apply(rope, x[:T, :2], pos[:T])
        q = oq.rope_apply(rope, x[:T, 2:], pos[:T])
        oq.cache_write(cache, kv, x[:T, 1:3], cu, ints(past), table, rpbh=r)
        outs.append(oq.cache_attention(cache, q, cu, ints([a + b for a, b in zip(new, past)]), table, rpbh=r))
    outs += oq.cache_read(cache, ints([0, 62, 95]), ints([0, 0]), table, T=95, rpbh=r)
    outs += [cache.k, cache.v, cache.k_scale, cache.v_scale]
torch.cuda.synchronize()
oq.device_status()
n = len(outs) // 3
assert all(torch.equal(a, b) for i in (1, 2) for a, b in zip(outs[:n], outs[i * n:]))
torch.save([t.cpu() for t in outs[:n]], sys.argv[2])
"""


def test_the_same_with_and_without_programmatic_launches(oq, tmp_path):
    """The chained launches change no result (OQ_NO_PDL is read once per process: child processes)."""
    root, got = os.path.dirname(os.path.dirname(os.path.abspath(__file__))), []
    for off in ("0", "1"):
        path = str(tmp_path / off)
        run = subprocess.run([sys.executable, "-c", _CHILD, root, path], env={**os.environ, "OQ_NO_PDL": off},
                             capture_output=True, text=True, timeout=600)
        assert run.returncode == 0, run.stderr[-2000:]
        got.append(torch.load(path))
    assert len(got[0]) == len(got[1]) and all(torch.equal(a, b) for a, b in zip(*got))


def test_no_library_allocations(oq):
    rng = np.random.default_rng(32)
    r, _ = rotation(oq, 64, 64)
    rope = oq.Rope((64,))
    bt = Batch(rng, [2], [9], 16)
    cache = filled(oq, rng, bt, 1, 64, r)
    x = rows(rng, (2, 1, 64), "bf16")
    n = oq.device_allocations()
    oq.cache_write(cache, oq.rope_apply(rope, x, ints([[1], [2]])), x, ints(bt.cu), ints(bt.past), ints(bt.table), rpbh=r)
    oq.cache_attention(cache, x, ints(bt.cu), ints(bt.total), ints(bt.table), rpbh=r)
    oq.cache_read(cache, ints(bt.cu), ints([0]), ints(bt.table), T=2, rpbh=r)
    assert oq.device_allocations() == n


def test_a_block_from_its_projection_on(oq):
    """The operators together as a transformer block uses them, two steps of a
    stream: fused QKV by the codebook linear, rotary positions in place on the
    queries and keys, cache write, attention, output projection.  Held to fp64
    attention on what the cache holds, and to attention on the unquantized
    keys and values within the 8-bit cache's own loss."""
    rng = np.random.default_rng(33)
    d_model, H, d = 256, 4, 64
    rm, rh = oq.Rpbh(0, d_model, 64), oq.Rpbh(3, d, 64)
    perm, signs = orpbh.draw_permutation_and_signs(3, d)
    cb = oq.Codebook(d_model, 4)
    w = [oq.quantize_weight(rm, cb, (0.06 * torch.randn(n, d_model, device="cuda")).bfloat16()) for n in (3 * d_model, d_model)]
    rope = oq.Rope((16, 24, 24))
    cache = oq.KVCache(5, H, d, 16)
    table = ints([[4, 2, 0], [1, 3, 3]])
    seen_k, seen_v = [np.zeros((0, H, d))] * 2, [np.zeros((0, H, d))] * 2
    for new, past in (([20, 11], [0, 0]), ([1, 4], [20, 11])):
        T, cu = sum(new), cum(new)
        x = torch.randn(T, d_model, device="cuda").bfloat16()
        pos = ints([[b, i, i % 7] for b, n in enumerate(new) for i in range(n)])
        _, qkv = oq.linear(rm, cb, cb, x, *w[0], want_f32=False, want_bf16=True)
        qkv = qkv.view(T, 3 * H, d)
        oq.rope_apply(rope, qkv[:, :2 * H], pos, out=qkv[:, :2 * H])
        q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:]
        oq.cache_write(cache, k, v, ints(cu), ints(past), table, rpbh=rh)
        total = [a + b for a, b in zip(new, past)]
        o = oq.cache_attention(cache, q, ints(cu), ints(total), table, rpbh=rh)
        y, _ = oq.linear(rm, cb, cb, o.view(T, d_model), *w[1])
        oq.device_status()
        assert y.shape == (T, d_model) and torch.isfinite(y).all()
        for b in range(2):
            sl = slice(cu[b], cu[b + 1])
            seen_k[b] = np.concatenate([seen_k[b], f64(k[sl])])
            seen_v[b] = np.concatenate([seen_v[b], f64(v[sl])])
            kq, vq = (oc.gather(c.cpu().numpy(), f64(s), table[b].tolist(), total[b])
                      for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            want, bound = oc.attention(f64(q[sl]), kq, vq, True, d ** -0.5, (perm, signs, 64))
            err = np.linalg.norm(f64(o[sl]) - want, axis=-1)
            assert np.all(err <= bound + (2.0 ** -8 + 2.0 ** -20) * np.linalg.norm(want, axis=-1))
            full, _ = oc.attention(f64(q[sl]), seen_k[b], seen_v[b], True, d ** -0.5, None)
            assert np.linalg.norm(f64(o[sl]) - full) <= 0.05 * np.linalg.norm(full)


# ------------------------------------------------- one key far above thousands of others
LOUD = [  # rows, keys, d, page, dtype: row tiles of 8 and 16 rows, and of 256; long and short caches
    (1, 4097, 64, 64, "fp16"), (1, 4097, 128, 16, "bf16"), (7, 900, 64, 32, "bf16"), (1, 60000, 64, 128, "fp16"),
    (16, 4097, 128, 64, "fp16"), (40, 2100, 64, 16, "bf16"),
    (64, 4097, 64, 64, "fp16"), (300, 2049, 128, 32, "bf16"), (129, 1025, 128, 128, "fp16"),
]


@pytest.mark.parametrize("gap", [12.0, 16.0, 17.5, 20.0])
@pytest.mark.parametrize("n,keys,d,page,dt", LOUD)
def test_attention_keys_far_below_the_loudest(oq, n, keys, d, page, dt, gap):
    """The first key takes nearly all of the softmax and its value is 0, as a stream's first tokens
    do: the output is what thousands of keys up to 20 nats lower leave.  Queries of equal magnitudes
    are exact in fp16, so are the scores' integer sums; a weight is off by 2^-12 of itself (fp16),
    and by 2^-16 for the exponent's fp32 roundings (scores below 64: 3 * 2^-24 * 64 ln 2) and
    2^-22 of ex2; below 2^-14 it is off by up to 2^-25, where the largest stands at 2^12 or (more
    than 48 rows) as high as leaves the weakest 16 of 64 keys at 2^-10, no higher than 2^12."""
    rng = np.random.default_rng(keys + d)
    unit = 0.5 / (12.0 * d ** 0.5)  # nats a code's step: the others' scores spread by 0.5
    sign = rng.choice([-1.0, 1.0], d)
    codes = rng.integers(-20, 21, (keys, d)).astype(np.int8)
    codes[0] = np.rint(sign * gap / (unit * d))
    assert np.abs(codes).max() <= 127
    values = rng.integers(30, 128, (keys, d)).astype(np.int8)
    values[0] = 0
    pages = -(-keys // page)
    order = rng.permutation(pages)
    pad = lambda x: np.concatenate([x, np.zeros((pages * page - keys, d), np.int8)]).reshape(pages, 1, page, d)  # noqa: E731
    cache = oq.KVCache(pages, 1, d, page)
    for to, x in ((cache.k, codes), (cache.v, values)):
        to[torch.from_numpy(order).cuda()] = torch.from_numpy(pad(x)).cuda()
    cache.k_scale.fill_(2.0 ** -5)
    cache.v_scale.fill_(2.0 ** -3)
    part = 1.0 - rng.integers(0, 5, n) / 16  # a row's share of the gap
    q = sign[None, None] * part[:, None, None]
    q16 = torch.from_numpy(q).to(DT[dt]).cuda()
    assert np.array_equal(f64(q16), q)
    out = f64(oq.cache_attention(cache, q16, ints([0, n]), ints([keys]), ints(order[None]), causal=False, scale=32 * unit))
    oq.device_status()
    s = (q[:, 0] @ codes.T.astype(float)) * unit
    p = np.exp(s - s.max(1, keepdims=True))
    gap2 = (s[:, :64].max(1) - s[:, :64].reshape(n, 4, 16).max(2).min(1)) / np.log(2)
    low = 2.0 ** -(25 + (12 if n <= 48 else np.clip(gap2 - 10, 0, 12)[:, None]))  # beside the largest weight of 1
    total, v = p.sum(1, keepdims=True), values.astype(float) / 8
    want = (p / total) @ v
    # each weight's own error, in the same direction for all, and the sum's
    wrong = (np.minimum(p, (2.0 ** -12 + 2.0 ** -16) * p + low) / total) @ v + 2.0 ** -16 * want
    err, size = np.linalg.norm(out[:, 0] - want, axis=1), np.linalg.norm(want, axis=1)
    limit = np.linalg.norm(wrong, axis=1) + torch.finfo(DT[dt]).eps / 2 * 1.01 * size
    if dt == "fp16":  # outputs below the type's normal numbers
        limit += 2.0 ** -25 * d ** 0.5
    assert np.all(limit[part == 1] < 0.02 * size[part == 1])  # the limit does say something
    assert np.all(err <= limit), (err / limit).max()


@pytest.mark.parametrize("n,dt", [(1, "bf16"), (12, "fp16"), (12, "bf16"), (60, "fp16"), (200, "bf16")])
def test_attention_over_a_loud_first_token(oq, n, dt):
    """The same through the rotation and the cache's write: a first token about 18 nats above 2000 others,
    which it shares pages' scales with, its value near 0; held to the oracle's bound, itself a few per
    cent of the output (the query's rounding in a score of 18 nats, in the worst case)."""
    rng = np.random.default_rng(41)
    r, rot = rotation(oq, 64, 64)
    keys = 2000
    bt = Batch(rng, [n], [keys - n], 32)
    base = rng.standard_normal(64)
    base *= 8 / np.linalg.norm(base)
    k, v = 0.5 * rng.standard_normal((keys, 1, 64)), 1 + rng.standard_normal((keys, 1, 64))
    k[0, 0], v[0, 0] = 18 / 8 * base, 0.01 * v[0, 0]
    cache = oq.KVCache(bt.n_pages, 1, 64, 32)
    dev = lambda x: torch.from_numpy(x).to(DT[dt]).cuda()  # noqa: E731
    oq.cache_write(cache, dev(k), dev(v), ints([0, keys]), ints([0]), ints(bt.table), rpbh=r)
    q = dev(base[None, None] + 0.1 * rng.standard_normal((n, 1, 64)))
    out = f64(oq.cache_attention(cache, q, ints([0, n]), ints([keys]), ints(bt.table), rpbh=r, causal=False))
    oq.device_status()
    kc, vc = (oc.gather(c.cpu().numpy(), f64(s), bt.table[0], keys)
              for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    step = f64(cache.v_scale)[bt.table[0][np.arange(keys) // 32]]
    s64 = 0.125 * oc.turn(f64(q), rot)[:, 0] @ kc[:64, 0].T / np.log(2)
    shift = 12 if n <= 48 else float(np.clip(s64.max(1) - s64.reshape(n, 4, 16).max(2).min(1) - 10, 0, 12).min())
    want, bound = oc.attention(f64(q), kc, vc, False, 0.125, rot, shift=shift, step=step)
    size = np.linalg.norm(want, axis=-1)
    limit = bound + torch.finfo(DT[dt]).eps / 2 * 1.01 * size + (2.0 ** -25 * 8 if dt == "fp16" else 0)
    assert np.all(limit < 0.05 * size)
    assert np.all(np.linalg.norm(out - want, axis=-1) <= limit)


def test_read_leaves_out_sequences_that_do_not_fit(oq):
    """Offsets that fall or leave 0..T: the read serves the sequences before, leaves the others' rows
    as they were and reports them, as the write does."""
    rng = np.random.default_rng(51)
    d, heads, P, B, T = 64, 2, 16, 200, 600
    new = [3] * B
    cache = oq.KVCache(B, heads, d, P)
    x = rows(rng, (T, heads, d), "bf16")
    table = ints(rng.permutation(B)[:, None])
    oq.cache_write(cache, x, x, ints(cum(new)), ints([0] * B), table)
    for at in ([0, 1, 2], [31, 32, 33], [127, 128, 129, 198], [5, 150]):
        good = cum(new)
        whole, _ = oq.cache_read(cache, ints(good), ints([0] * B), table, T=T)
        oq.device_status()
        for kind in ("falls", "falls far", "ends behind T", "begins before 0"):
            cu, served = list(good), np.ones(T, bool)
            if kind == "falls":
                b = at[0]
                cu[b + 1] = cu[b] - 1
                served[good[b]:] = False
            elif kind == "falls far":
                b = at[-1]
                cu[b + 1] = 0
                served[good[b]:] = False
            elif kind == "ends behind T":  # the last sequences, all beyond the tensor
                b = at[-1]
                cu[b + 1:] = [T + 1 + i for i in range(B - b)]
                served[good[b]:] = False
            else:
                b = at[0]
                cu[:b + 1] = [-5] * (b + 1)
                served[:good[b + 1]] = False
            out = [torch.full((T, heads, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            oq.cache_read(cache, ints(cu), ints([0] * B), table, k=out[0], v=out[1])
            with pytest.raises(oq.OQError) as e:
                oq.device_status()
            assert e.value.code == oq.OQ_ERR_ARG
            oq.device_status()
            for o in out:
                keep = torch.from_numpy(served).cuda()
                assert torch.equal(o[keep], whole[keep]), (kind, at)
                assert torch.all(o[~keep] == 7.0), (kind, at)
    # the offsets of the write's test: nothing of sequences 1 to 3
    out = torch.full((8, heads, d), 5.0, dtype=torch.bfloat16, device="cuda")
    oq.cache_read(cache, ints([0, 2, 1, 3, 9]), ints([0] * 4), ints([[0], [1], [2], [3]]), k=out, v=out.clone())
    with pytest.raises(oq.OQError):
        oq.device_status()
    assert not torch.any(out[:2] == 5.0) and torch.all(out[2:] == 5.0)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("d,block", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (64, 0)])
def test_write_keeps_what_is_not_finite_in_its_block(oq, d, block, dt):
    """A NaN or an infinity reaches the coordinates of its own block of the rotation: those that come out
    as NaN are stored as 0, as infinities saturate; the row's other blocks are written as u = Pi x says."""
    rng = np.random.default_rng(61)
    r, rot = rotation(oq, d, block)
    perm = rot[0] if rot else np.arange(d)
    heads, n = 2, 10
    x = rng.standard_normal((n, heads, d))
    at = [perm[0], perm[d // 2 + 1], perm[d - 1]]  # in the first block, in the middle, in the last
    x[0, :, at[0]], x[1, :, at[1]], x[2, :, at[2]] = np.nan, np.nan, np.nan
    x[3, :, at[0]], x[4, :, at[2]] = np.inf, -np.inf
    x[5, :, perm[0]], x[5, :, perm[1]] = np.inf, np.inf  # meet with either sign
    x[6, 0, at[1]], x[6, 1, at[0]] = np.nan, -np.inf     # other heads, other places
    x[7, :, at[0]], x[7, :, at[2]] = np.inf, np.nan
    x[8] = np.nan
    x16 = torch.from_numpy(x).to(DT[dt]).cuda()
    cache = oq.KVCache(n, heads, d, 16)
    cache.k.fill_(77)
    cache.v.fill_(77)
    # a page for every row; keys as they are, values in the reversed order
    oq.cache_write(cache, x16, x16.flip(0).contiguous(), ints(range(n + 1)), ints([0] * n), ints([[b] for b in range(n)]), rpbh=r)
    oq.device_status()
    with np.errstate(invalid="ignore"):
        u = oc.turn(f64(x16), rot)
    near = np.abs(u[9]) if rot is None else u[9]
    assert np.isfinite(near).all()
    for codes, scale, rows_u in ((cache.k, cache.k_scale, u), (cache.v, cache.v_scale, u[::-1])):
        got, s = codes.cpu().numpy()[:, :, 0].astype(int), f64(scale)
        for b in range(n):
            for h in range(heads):
                w = np.where(np.isnan(rows_u[b, h]), 0, rows_u[b, h])
                e = oc.step_exponent(np.abs(w).max())
                assert s[b, h] == 2.0 ** e
                t = np.clip(w / 2.0 ** e, -127, 127)
                off = np.abs(got[b, h] - np.rint(t))
                assert off.max() <= 1 and np.all((off == 0) | (np.abs(t - np.floor(t) - 0.5) < 1e-3)), (b, h)


@pytest.mark.parametrize("new,past,heads,d,dt,block", [
    ([130, 60], [300, 20], 2, 128, "bf16", 128),  # turned; two items with two tiles, two with one
    ([200], [3000], 1, 64, "fp16", 0),            # not turned; items cut between CTAs, a join behind them
    ([100], [0], 3, 128, "fp16", 64),             # one stage of values
])
def test_chunk_attention_wait_runs_out_and_context_survives(oq, new, past, heads, d, dt, block):
    """The keys are never handed over, so the waits run out: the kernel reports it, frees what it holds
    and leaves, and the next launch gives what it gave before.  Nothing traps or hangs."""
    rng = np.random.default_rng(71)
    r, _ = rotation(oq, d, block)
    bt = Batch(rng, new, past, 64)
    cache = filled(oq, rng, bt, heads, d, r, dt)
    q = rows(rng, (bt.T, heads, d), dt)
    args = (q, ints(bt.cu), ints(bt.total), ints(bt.table))
    want = oq.cache_attention(cache, *args, rpbh=r)
    step = oq.cache_attention(cache, q[:1], ints([0, 1]), ints([20]), args[3][:1], rpbh=r)
    oq.device_status()
    assert oq.lib().oq_test_stall_next(7) == oq.OQ_OK
    # few rows go to another kernel, which does not consume it
    assert torch.equal(step, oq.cache_attention(cache, q[:1], ints([0, 1]), ints([20]), args[3][:1], rpbh=r))
    oq.device_status()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    oq.cache_attention(cache, *args, rpbh=r)
    end.record()
    torch.cuda.synchronize()
    with pytest.raises(oq.OQError) as e:
        oq.device_status()
    assert e.value.code == oq.OQ_ERR_TIMEOUT
    assert 900 < begin.elapsed_time(end) < 5000  # one wait's limit, not one for each step
    for _ in range(3):
        assert torch.equal(want, oq.cache_attention(cache, *args, rpbh=r))
    oq.device_status()


@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_rope_small_angles(oq, layout):
    """The sine of a small angle is right in itself, not only beside the cosine: 2^-24 for the angle's
    float, 2 * 2^-23 for sincospif, and the fixed point's |pos| * 2^-65 turns."""
    freq = [10.0 ** -(k / 2) for k in range(2, 18)]  # 0.1 down to 3e-9 radians a position
    r = oq.Rope(freqs=freq, axes=[0] * 16, layout=layout)
    pos = np.array([[1], [2], [-1], [-3], [17], [1000], [-70000], [0]])
    x = torch.zeros((8, 1, 32), device="cuda")
    i = np.arange(16)
    a, b = (i, i + 16) if layout == "halves" else (2 * i, 2 * i + 1)
    x[..., a] = 1.0
    for inverse in (False, True):
        y = f64(oq.rope_apply(r, x, ints(pos), inverse=inverse))[:, 0]
        phi = pos * np.array(freq) * (-1 if inverse else 1)
        slip = np.abs(pos) * 2.0 ** -65 * 2 * np.pi + np.abs(phi) * 2.0 ** -52
        assert np.all(np.abs(y[:, b] - np.sin(phi)) <= (2.0 ** -22 + 2.0 ** -24) * 1.01 * np.abs(np.sin(phi))
                      + slip + 2.0 ** -24 * np.abs(phi) * np.abs(np.cos(phi)))
        assert np.all(np.abs(y[:, a] - np.cos(phi)) <= 2.0 ** -21)


def test_offsets_beyond_32_bits(oq):
    """Pages behind 2^32 bytes of codes, rows of a tensor 2^31 elements apart: the same bits as near ones."""
    rng = np.random.default_rng(81)
    heads, d, page = 8, 128, 128
    n_pages = 2 ** 32 // (heads * page * d) + 8
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    codes = [torch.empty((n_pages, heads, page, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.empty((n_pages, heads), dtype=torch.float32, device="cuda") for _ in range(2)]
    cache = oq.KVCache.wrap(*codes, *scales)
    r, _ = rotation(oq, d, 128)
    k, v, q = (rows(rng, (300, n, d), "bf16") for n in (heads, heads, 2 * heads))
    outs = []
    for first in (0, n_pages - 3):
        table = ints([[first + 2, first, first + 1]])
        oq.cache_write(cache, k, v, ints([0, 300]), ints([0]), table, rpbh=r)
        got = list(oq.cache_read(cache, ints([0, 300]), ints([0]), table, T=300, rpbh=r))
        for n in (1, 9, 300):  # the three sizes of row tiles
            got.append(oq.cache_attention(cache, q[:n], ints([0, n]), ints([300]), table, rpbh=r))
        outs.append(got)
    oq.device_status()
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and outs[0][0].any() and outs[0][4].any()
    # a token's row every 2^27 elements of the same memory
    far = codes[0].view(-1).view(torch.bfloat16).as_strided((17, 3, 64), (2 ** 27 - 64, 64, 1))
    assert far.stride(0) * 16 >= 2 ** 31 - 2 ** 11
    x = rows(rng, (17, 3, 64), "bf16")
    far.copy_(x)
    rope, pos = oq.Rope((16, 24, 24)), ints(rng.integers(0, 100, (17, 3)))
    want = oq.rope_apply(rope, x, pos)
    assert torch.equal(oq.rope_apply(rope, far, pos), want)
    oq.rope_apply(rope, far, pos, out=far)
    assert torch.equal(far, want)


@pytest.mark.parametrize("causal", [False, True])
def test_many_chunks_beyond_one_block(oq, causal):
    """More sequences than the chunk kernel's CTA has threads, each with many rows; some empty."""
    rng = np.random.default_rng(82)
    r, rot = rotation(oq, 64, 64)
    B = 450
    new = [0 if b % 11 == 3 else int(rng.integers(50, 140)) for b in range(B)]
    past = [int(n) for n in rng.integers(0, 40, B)]
    assert sum(new) / B > 48
    bt = Batch(rng, new, past, 16)
    cache = filled(oq, rng, bt, 1, 64, r)
    q = rows(rng, (bt.T, 1, 64), "bf16", loud=False)
    out = oq.cache_attention(cache, q, ints(bt.cu), ints(bt.total), ints(bt.table), rpbh=r, causal=causal)
    oq.device_status()
    kc, vc = cache.k.cpu().numpy(), cache.v.cpu().numpy()
    for b in [0, 1, 3, 200, 415, 416, 417, B - 1]:
        k, v = (oc.gather(c, f64(s), bt.table[b], bt.total[b]) for c, s in ((kc, cache.k_scale), (vc, cache.v_scale)))
        sl = slice(bt.cu[b], bt.cu[b + 1])
        want, bound = oc.attention(f64(q[sl]), k, v, causal, 0.125, rot)
        err = np.linalg.norm(f64(out[sl]) - want, axis=-1)
        assert np.all(err <= bound + (2.0 ** -9 * 2 + 2.0 ** -20) * np.linalg.norm(want, axis=-1))
