"""The cache operators on the CPU: handles, argument checks, the oracle's own
properties.  No kernel is launched here."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import rpbh as orpbh


@pytest.fixture(scope="module")
def oq():
    from calibration_free_rotated_b200 import build
    build.build()
    from calibration_free_rotated_b200 import orbitquant
    return orbitquant


BASE = 1 << 20  # an aligned address that nothing reads: every call below is refused first


def struct(oq, **kw):
    f = dict(k=BASE, v=BASE, k_scale=BASE, v_scale=BASE, n_pages=4, heads=2, page=16, d=64)
    f.update(kw)
    return ctypes.byref(oq._CacheStruct(**f))


def code(oq, rc, word=""):
    assert word in oq.lib().oq_last_error().decode(), oq.lib().oq_last_error()
    return rc


@pytest.mark.parametrize("kw,want", [
    (dict(n_pages=0), "ARG"), (dict(heads=0), "ARG"), (dict(k=0), "ARG"), (dict(v_scale=0), "ARG"),
    (dict(page=24), "UNSUPPORTED"), (dict(page=256), "UNSUPPORTED"), (dict(d=96), "UNSUPPORTED"),
    (dict(n_pages=1 << 28), "UNSUPPORTED"), (dict(heads=70000), "UNSUPPORTED"), (dict(k=BASE + 8), "ALIGN"),
    (dict(k_scale=BASE + 4), "ALIGN"),
])
def test_cache_geometry_is_checked(oq, kw, want):
    L, err = oq.lib(), getattr(oq, "OQ_ERR_" + want)
    c = struct(oq, **kw)
    assert L.oq_cache_write(c, None, BASE, 64, 64, BASE, 64, 64, 0, 1, BASE, BASE, 1, BASE, 1, None) == err
    assert L.oq_cache_read(c, None, BASE, BASE, 0, 1, BASE, BASE, 1, BASE, 1, None) == err
    assert L.oq_cache_attention(c, None, BASE, 64, 64, BASE, 64, 64, 0, 2, 1, BASE, BASE, 1, BASE, 1, 1, 1.0, BASE,
                                1 << 40, None) == err
    assert L.oq_last_error()


def test_write_read_arguments(oq):
    L, c = oq.lib(), struct(oq)

    def write(cache=c, r=None, K=BASE, kt=64, kh=64, V=BASE, vt=64, vh=64, dtype=0, T=1, cu=BASE, past=BASE, B=1,
              table=BASE, width=1):
        return L.oq_cache_write(cache, r, K, kt, kh, V, vt, vh, dtype, T, cu, past, B, table, width, None)

    assert write(cache=None) == oq.OQ_ERR_ARG
    assert write(T=-1) == oq.OQ_ERR_ARG and write(B=-1) == oq.OQ_ERR_ARG
    assert write(T=0) == oq.OQ_OK and write(B=0) == oq.OQ_OK  # nothing to do: nothing is launched
    assert write(K=None) == oq.OQ_ERR_ARG and write(V=None) == oq.OQ_ERR_ARG
    assert write(cu=None) == oq.OQ_ERR_ARG and write(past=None) == oq.OQ_ERR_ARG and write(table=None) == oq.OQ_ERR_ARG
    assert write(width=0) == oq.OQ_ERR_ARG and write(width=1 << 27) == oq.OQ_ERR_UNSUPPORTED
    assert write(dtype=2) == oq.OQ_ERR_UNSUPPORTED and write(dtype=9) == oq.OQ_ERR_ARG
    assert write(K=BASE + 2) == oq.OQ_ERR_ALIGN and write(kt=60) == oq.OQ_ERR_ALIGN
    assert write(vh=4) == oq.OQ_ERR_ALIGN and write(cu=BASE + 2) == oq.OQ_ERR_ALIGN
    wide, small = oq.Rpbh(0, 128, 64), oq.Rpbh(0, 64, 16)
    assert write(r=wide.handle) == oq.OQ_ERR_ARG
    assert write(r=small.handle) == oq.OQ_ERR_UNSUPPORTED
    assert write(r=oq.Rpbh(0, 64, 32, rounds=2).handle) == oq.OQ_ERR_UNSUPPORTED
    assert L.oq_cache_read(c, wide.handle, BASE, BASE, 0, 1, BASE, BASE, 1, BASE, 1, None) == oq.OQ_ERR_ARG
    assert L.oq_cache_read(c, None, None, BASE, 0, 1, BASE, BASE, 1, BASE, 1, None) == oq.OQ_ERR_ARG
    assert L.oq_cache_read(c, None, BASE, BASE + 8, 0, 1, BASE, BASE, 1, BASE, 1, None) == oq.OQ_ERR_ALIGN
    assert L.oq_cache_read(c, None, BASE, BASE, 0, 0, BASE, BASE, 1, BASE, 1, None) == oq.OQ_OK


def test_attention_arguments(oq):
    L, c = oq.lib(), struct(oq)
    need = L.oq_cache_attention_workspace_bytes(c, 1, 1, 4)

    def attn(Q=BASE, O=2 * BASE, qt=256, heads=4, T=1, B=1, scale=1.0, ws=BASE, size=need, dtype=0):
        return L.oq_cache_attention(c, None, Q, qt, 64, O, 256, 64, dtype, heads, T, BASE, BASE, B, BASE, 1, 1, scale,
                                    ws, size, None)

    assert need > 0
    assert attn(heads=3) == oq.OQ_ERR_ARG and attn(heads=0) == oq.OQ_ERR_ARG
    assert attn(Q=None) == oq.OQ_ERR_ARG and attn(O=None) == oq.OQ_ERR_ARG and attn(O=BASE) == oq.OQ_ERR_ARG
    assert attn(scale=float("nan")) == oq.OQ_ERR_ARG and attn(scale=float("inf")) == oq.OQ_ERR_ARG
    assert attn(ws=None) == oq.OQ_ERR_ARG and attn(size=need - 1) == oq.OQ_ERR_ARG
    assert attn(ws=BASE + 4) == oq.OQ_ERR_ALIGN and attn(qt=257) == oq.OQ_ERR_ALIGN
    assert attn(dtype=2) == oq.OQ_ERR_UNSUPPORTED
    assert attn(T=1 << 30, size=1 << 50) == oq.OQ_ERR_UNSUPPORTED
    assert attn(T=0) == oq.OQ_OK and attn(B=0) == oq.OQ_OK


def test_rope_arguments(oq):
    L = oq.lib()
    h = ctypes.c_void_p()

    def make(n, freq, axis, axes, layout=0):
        return L.oq_make_rope(n, (ctypes.c_double * max(1, len(freq)))(*freq),
                              (ctypes.c_uint8 * max(1, len(axis)))(*axis), axes, layout, ctypes.byref(h))

    assert make(0, [], [], 1) == oq.OQ_ERR_ARG and make(257, [1.0] * 257, [0] * 257, 1) == oq.OQ_ERR_ARG
    assert make(1, [1.0], [1], 1) == oq.OQ_ERR_ARG and make(1, [1.0], [0], 9) == oq.OQ_ERR_ARG
    assert make(1, [float("inf")], [0], 1) == oq.OQ_ERR_ARG and make(1, [1.0], [0], 1, 2) == oq.OQ_ERR_ARG
    assert L.oq_make_rope(1, None, None, 1, 0, ctypes.byref(h)) == oq.OQ_ERR_ARG
    r, odd = oq.Rope((16, 24, 24)), oq.Rope((12,), layout="halves")
    n, a, lay = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    assert L.oq_rope_info(r.handle, ctypes.byref(n), ctypes.byref(a), ctypes.byref(lay)) == 0
    assert (n.value, a.value, lay.value) == (32, 3, 0)

    def apply(rope=r, X=BASE, xt=64, Y=2 * BASE, yt=64, dtype=0, T=1, heads=1, d=64, pos=BASE):
        return L.oq_rope_apply(rope.handle if rope else None, X, xt, 64, Y, yt, 64, dtype, T, heads, d, pos, 0, None)

    assert apply(rope=None) == oq.OQ_ERR_ARG and apply(d=56) == oq.OQ_ERR_ARG and apply(dtype=3) == oq.OQ_ERR_ARG
    assert apply(d=68) == oq.OQ_ERR_UNSUPPORTED and apply(d=520) == oq.OQ_ERR_UNSUPPORTED
    assert apply(rope=odd) == oq.OQ_ERR_UNSUPPORTED  # six pairs in halves
    assert apply(X=None) == oq.OQ_ERR_ARG and apply(Y=None) == oq.OQ_ERR_ARG and apply(pos=None) == oq.OQ_ERR_ARG
    assert apply(X=BASE + 8) == oq.OQ_ERR_ALIGN and apply(xt=68) == oq.OQ_ERR_ALIGN and apply(pos=BASE + 1) == oq.OQ_ERR_ALIGN
    assert apply(Y=BASE, yt=128) == oq.OQ_ERR_ARG  # in place with other strides
    assert apply(T=-1) == oq.OQ_ERR_ARG and apply(T=0) == oq.OQ_OK and apply(heads=0) == oq.OQ_OK
    for bad in (dict(axis_dims=(3,)), dict(axis_dims=()), dict(), dict(axis_dims=(4,), layout="x"),
                dict(axis_dims=(4,), ladder="x"), dict(freqs=[1.0]), dict(freqs=[1.0], axes=[0, 1])):
        with pytest.raises(ValueError):
            oq.Rope(**bad)


def test_sizes_at_the_end_of_32_bits(oq):
    """What the kernels' 32-bit places could not hold is refused before a launch."""
    L, c, most, many = oq.lib(), struct(oq), 0x7FFF0000, 0x7FFFFFFF
    r = oq.Rope((16, 24, 24))

    def apply(T, heads):
        return L.oq_rope_apply(r.handle, BASE, 64, 64, 2 * BASE, 64, 64, 0, T, heads, 64, BASE, 0, None)

    assert apply(most + 1, 1) == oq.OQ_ERR_UNSUPPORTED and apply(many, 1) == oq.OQ_ERR_UNSUPPORTED
    assert apply(1, 65536) == oq.OQ_ERR_UNSUPPORTED and apply(1, many) == oq.OQ_ERR_UNSUPPORTED
    for T, width in ((many, 1), (most + 1, 1), (1, most // 16 + 1), (1, many)):
        assert L.oq_cache_write(c, None, BASE, 64, 64, BASE, 64, 64, 0, T, BASE, BASE, 1, BASE, width,
                                None) == oq.OQ_ERR_UNSUPPORTED
        assert L.oq_cache_read(c, None, BASE, BASE, 0, T, BASE, BASE, 1, BASE, width, None) == oq.OQ_ERR_UNSUPPORTED
        assert L.oq_cache_attention(c, None, BASE, 256, 64, 2 * BASE, 256, 64, 0, 4, T, BASE, BASE, 1, BASE, width, 1,
                                    1.0, BASE, 1 << 60, None) == oq.OQ_ERR_UNSUPPORTED


def test_binding_checks_tensors(oq):
    """Shapes, types and devices that the library cannot see from pointers."""
    c = oq.KVCache(2, 1, 64, 16, device="cpu")
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    cu, at, table = i(0, 2), i(0), i(0).view(1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        oq.cache_write(c, x, x, cu, at, table)
    for k, v in ((x[:, :, :32], x), (x, x[:1]), (x, x.half()), (x.view(2, 64), x), (x.transpose(0, 2), x)):
        with pytest.raises(ValueError):
            oq.cache_write(c, k, v, cu, at, table)
    for bad in (dict(cu=cu.long()), dict(cu=i(0, 1, 2)), dict(at=at.long()), dict(table=i(0)), dict(table=table.long())):
        a = dict(cu=cu, at=at, table=table)
        a.update(bad)
        with pytest.raises(ValueError):
            oq.cache_write(c, x, x, a["cu"], a["at"], a["table"])
        with pytest.raises(ValueError):
            oq.cache_attention(c, x, a["cu"], a["at"], a["table"])
        with pytest.raises(ValueError):
            oq.cache_read(c, a["cu"], a["at"], a["table"], T=2)
    with pytest.raises(ValueError):
        oq.cache_read(c, cu, at, table)
    with pytest.raises(ValueError):
        oq.rope_apply(oq.Rope((64,)), x, i(0, 1))
    with pytest.raises(ValueError):
        oq.rope_apply(oq.Rope((64,)), x, i(0, 1).view(2, 1), out=x.float())
    for bad in ((c.k[:, :, :8], c.v, c.k_scale, c.v_scale), (c.k.half(), c.v, c.k_scale, c.v_scale),
                (c.k, c.v, c.k_scale.double(), c.v_scale), (c.k, c.v, c.k_scale.T, c.v_scale)):
        with pytest.raises(ValueError):
            oq.KVCache.wrap(*bad)


def test_oracle_turn_and_steps():
    rng = np.random.default_rng(0)
    perm, signs = orpbh.draw_permutation_and_signs(5, 64)
    x = rng.standard_normal((7, 64))
    u = oc.turn(x, (perm, signs, 32))
    assert np.abs(oc.turn_back(u, (perm, signs, 32)) - x).max() < 1e-13
    assert np.allclose(np.linalg.norm(u, axis=1), np.linalg.norm(x, axis=1))
    for e in (-40, -3, 0, 7, 39):
        assert oc.step_exponent(127 * 2.0 ** e) == e
        assert oc.step_exponent(np.nextafter(127 * 2.0 ** e, np.inf)) == e + 1
    assert oc.step_exponent(0.0) == -40 and oc.step_exponent(np.inf) == 40


def test_oracle_attention_and_rope():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 2, 8)), rng.standard_normal((3, 1, 8)), rng.standard_normal((3, 1, 8))
    out, _ = oc.attention(q, k, v, True, 0.5, None)
    for i, h in ((0, 0), (1, 1)):
        w = np.exp(0.5 * k[:2 + i, 0] @ q[i, h])
        assert np.allclose(out[i, h], (w / w.sum()) @ v[:2 + i, 0])
    x = rng.standard_normal((3, 2, 8))
    pos = np.array([[0, 0], [1, 5], [70, -3]])
    for halves in (False, True):
        y = oc.rope(x, pos, [1.0, 0.1, 0.5], [0, 1, 1], halves)
        assert np.allclose(oc.rope(y, pos, [1.0, 0.1, 0.5], [0, 1, 1], halves, inverse=True), x)
        assert np.array_equal(y[..., 6:], x[..., 6:]) and np.array_equal(y[0], x[0])


@pytest.mark.parametrize("gap,shift", [(9.0, 0), (12.0, 0), (12.0, 12), (16.0, 12), (17.5, 12), (18.0, 12)])
def test_oracle_attention_bound_finds_lost_keys(gap, shift):
    """One key far above thousands of others, its value 0: a sum without the others, or with their weights
    rounded as they are beside a largest weight of 1, lies outside the bound; beside 2^shift, inside."""
    rng = np.random.default_rng(2)
    d, n = 64, 3000
    q = rng.choice([-1.0, 1.0], (1, 1, d))
    codes, values = rng.integers(-20, 21, (n, 1, d)).astype(float), rng.integers(30, 128, (n, 1, d)).astype(float)
    unit = 0.5 / (12.0 * d ** 0.5)
    codes[0] = np.rint(q[0] * gap / (unit * d))
    values[0] = 0
    want, bound = oc.attention(q, codes, values, False, unit, None, shift=shift, step=np.ones((n, 1)))
    size = np.linalg.norm(want)
    assert bound[0, 0] < 0.1 * size  # the bound does say something
    s = unit * codes[:, 0] @ q[0, 0]
    p = np.exp(s - s.max())

    def off(weights):
        return np.linalg.norm(weights @ values[:, 0] / p.sum() - want[0, 0])

    assert off(p * (p == 1)) > 5 * bound[0, 0]
    half = lambda c: (p * 2.0 ** c).astype(np.float16).astype(float) / 2.0 ** c  # noqa: E731
    assert off(half(shift)) <= bound[0, 0]
    if gap > 17:
        assert off(half(0)) > 5 * bound[0, 0]


def test_oracle_attention_bound_holds_for_scales_far_apart():
    """Weights times their page's scale, rounded in fp16 beside the largest: always inside lost_weights' bound."""
    rng = np.random.default_rng(3)
    for _ in range(50):
        n, d = int(rng.integers(1, 400)), 64
        ev = np.repeat(rng.integers(-12, 13, -(-n // 16)), 16)[:n]
        codes = rng.integers(-127, 128, (n, d)).astype(float) * (rng.random((n, 1)) < 0.9)
        s = rng.standard_normal(n) * rng.choice([1.0, 5.0, 12.0])
        p = np.exp(s - s.max())
        p /= p.sum()
        w = p * 2.0 ** ev
        c = int(rng.integers(0, 13))
        w16 = (w / w.max() * 2.0 ** c).astype(np.float16).astype(float) / 2.0 ** c * w.max()
        small = w16 * 2.0 ** c / w.max() < 2.0 ** -14
        err = np.abs((small * (w16 - w)) @ codes)
        vv = codes * 2.0 ** ev[:, None]
        tight = oc.lost_weights(p, vv, c, 2.0 ** ev)
        assert np.all(err <= tight * (1 + 1e-9) + 1e-300)
        if np.abs(codes).any(1).all():  # (keys without a value tell nothing of their scale)
            assert np.all(tight <= oc.lost_weights(p, vv, c) * (1 + 1e-9) + 1e-300)


def test_most_query_heads(oq):
    """Query heads beyond 65535 are refused, also where one token's rows would fit: the units of causal
    rows are counted with 2 * group * 128 in 32 bits."""
    L, c = oq.lib(), struct(oq, heads=1)

    def attn(heads, T=1, causal=1):
        return L.oq_cache_attention(c, None, BASE, 64 * heads, 64, 2 * BASE, 64 * heads, 64, 0, heads, T, BASE, BASE, 1,
                                    BASE, 1, causal, 1.0, BASE, 0, None)

    for heads in (65536, 1 << 20, 1 << 24, 1 << 25, (1 << 31) - 1):
        for causal in (0, 1):
            assert code(oq, attn(heads, causal=causal), "heads") == oq.OQ_ERR_UNSUPPORTED
    assert code(oq, attn(65535), "workspace") == oq.OQ_ERR_ARG  # as far as the next check
    assert code(oq, attn(65536, T=0), "heads") == oq.OQ_ERR_UNSUPPORTED


def test_units_of_causal_rows_fit_64_bits():
    """The kernels' count of the key tiles before row tile q, floor(q (2 g past + RT (q + 1)) / (2 g TILE)),
    restated step by step: equal to the exact quotient over the sizes that are accepted, no step past 63
    bits (the product itself passes 64 at 65535 heads on one, 2^15 new tokens behind 2^30)."""
    most, rng = 0x7FFF0000, np.random.default_rng(4)
    assert 2 ** 31 // 8 * (2 * 65535 * 2 ** 30) > 2 ** 64
    for _ in range(20000):
        tile, rt = int(rng.choice([64, 128])), int(rng.choice([8, 16, 256]))
        g = int(2 ** rng.uniform(0, 16))
        n = int(2 ** rng.uniform(0, np.log2(most // g)))
        past, q = int(2 ** rng.uniform(0, 31)) % (most - n + 1), int(rng.integers(0, (n * g + rt - 1) // rt + 1))
        first = q * past
        rest = first % tile * 2 * g + rt * q * (q + 1)
        assert first < 2 ** 63 and rest < 2 ** 63 and 2 * g * tile < 2 ** 32
        assert first // tile + rest // (2 * g * tile) == q * (2 * g * past + rt * (q + 1)) // (2 * g * tile)


def test_a_cache_follows_its_tensors(oq):
    """A tensor that takes another's place is the one that the calls use (the first one's memory may be
    handed on), and is checked as the first one was."""
    c = oq.KVCache(3, 2, 64, 16, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale"):
        new = getattr(c, name).clone()
        setattr(c, name, new)
        assert getattr(c, name) is new and getattr(c._struct, name) == new.data_ptr()
        assert ctypes.cast(c._ref, ctypes.POINTER(oq._CacheStruct)).contents.d == 64
        with pytest.raises(ValueError):
            setattr(c, name, new[:2])
        with pytest.raises(ValueError):
            setattr(c, name, new.to(torch.float64))
        assert getattr(c, name) is new and getattr(c._struct, name) == new.data_ptr()
    c.k_scale *= 2  # in place: the same memory
    assert c._struct.k_scale == c.k_scale.data_ptr()
