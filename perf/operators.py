"""What is measured of the cache operators: rotary positions, the 8-bit cache, attention over it.

Three operators of the serving side of a quantized attention block, each with a
plain form (elementary torch operations) and the library's call:

  rope   rotary positions over several axes (time, height, width)
  cache  keys and values quantized as they are written into a paged 8-bit
         cache (power-of-two scale for each page and head, after the
         library's block-Hadamard rotation), and read back
  attn   attention of new tokens over that cache

Everything a case fixes (lengths, heads, types) follows from the case; the
values and the order of the pages follow from the seed.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E_MIN, E_MAX = -40, 40  # exponents a cache scale may take


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # One decoding step of a batch: 64 rows, text-style positions far into a stream.
        dict(name="rope_step", op="rope", T=64, heads=40, extra=8, d=128, axes="128", layout="halves", dtype="bf16",
             inverse=False, grid="far"),
        # Queries and keys of the fused QKV projection of an image transformer: 512 text + 64 x 64 latent tokens.
        dict(name="rope_image", op="rope", T=4608, heads=48, extra=24, d=128, axes="16,56,56", layout="interleaved",
             dtype="bf16", inverse=False, grid="image"),
        # Video: 21 x 30 x 52 latent tokens, 12 + 12 heads; the transposed rotation (the gradient's direction).
        dict(name="rope_video", op="rope", T=32760, heads=24, extra=12, d=128, axes="44,42,42", layout="interleaved",
             dtype="fp16", inverse=True, grid="video"),
        # One token for each of 64 sequences of different lengths, appended to pages that are partly full.
        dict(name="cache_step", op="cache", B=64, new_lo=1, new_hi=1, past_lo=1, past_hi=8000, heads=8, d=128, page=64,
             block=128, dtype="bf16"),
        # A chunk: every token of an image written at once.
        dict(name="cache_chunk", op="cache", B=1, new_lo=4608, new_hi=4608, past_lo=0, past_hi=0, heads=24, d=128,
             page=64, block=128, dtype="bf16"),
        # Sequences of very different lengths read back whole, narrow heads.
        dict(name="read_ragged", op="read", B=24, new_lo=3, new_hi=4001, past_lo=0, past_hi=0, heads=8, d=64, page=32,
             block=64, dtype="fp16"),
        # The smallest call: one new token over a short cache.
        dict(name="attn_step_short", op="attn", B=1, new_lo=1, new_hi=1, past_lo=517, past_hi=517, heads=8, group=4,
             d=128, page=64, block=128, causal=True, dtype="bf16"),
        # Serving: 64 sequences of 100 to 8200 tokens, one new token each, four query heads share a key head.
        dict(name="attn_step_batch", op="attn", B=64, new_lo=1, new_hi=1, past_lo=100, past_hi=8200, heads=8, group=4,
             d=128, page=64, block=128, causal=True, dtype="bf16"),
        # One long stream.
        dict(name="attn_step_long", op="attn", B=1, new_lo=1, new_hi=1, past_lo=131071, past_hi=131071, heads=8,
             group=4, d=128, page=128, block=128, causal=True, dtype="bf16"),
        # Chunks of different lengths behind different pasts, narrow heads, causal.
        dict(name="attn_chunk_ragged", op="attn", B=8, new_lo=1, new_hi=511, past_lo=0, past_hi=3600, heads=4, group=4,
             d=64, page=16, block=64, causal=True, dtype="fp16"),
        # An image transformer's joint attention: all 4608 tokens over all, 24 heads.
        dict(name="attn_image", op="attn", B=1, new_lo=4608, new_hi=4608, past_lo=0, past_hi=0, heads=24, group=1,
             d=128, page=64, block=128, causal=False, dtype="bf16"),
        # Streaming video: one new latent frame (30 x 52 tokens) over 21 cached frames, 12 heads.
        dict(name="attn_frame", op="attn", B=1, new_lo=1560, new_hi=1560, past_lo=31200, past_hi=31200, heads=12,
             group=1, d=128, page=64, block=128, causal=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "read", "attn", "attn", "attn"])
    d = rng.choice([64, 128])
    if op == "rope":
        heads = _log(rng, 1, 48)
        axes = rng.choice(["44,42,42", "16,56,56", "128", "64,64", "64,32,32", "96"] if d == 128
                          else ["16,24,24", "64", "32,32", "32", "8,28,28"])
        return dict(op="rope", T=_log(rng, 1, max(2, 786240 // heads)), heads=heads, extra=rng.randint(0, 12), d=d,
                    axes=axes, layout=rng.choice(["interleaved", "halves"]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    inverse=rng.random() < 0.4, grid=rng.choice(["far", "video"]))
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([0, 32, 64, d])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("cache", "read"):
        heads = rng.choice([1, 2, 3, 4, 8, 12, 24])
        B = _log(rng, 1, 128)
        most = max(1, min(8192, 110592 // (heads * B)))
        hi = _log(rng, 1, most)
        lo = rng.randint(1, hi)
        past = _log(rng, 1, 4000) if op == "cache" else 0
        return dict(op=op, B=B, new_lo=lo, new_hi=hi, past_lo=rng.randint(0, past), past_hi=past, heads=heads, d=d,
                    page=page, block=block, dtype=dtype)
    heads = rng.choice([1, 2, 4, 8, 12, 24])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16]) if heads <= 8 else rng.choice([1, 2])
    B = _log(rng, 1, 64)
    if rng.random() < 0.6:  # single tokens (or a few, checked together)
        hi = rng.choice([1, 1, 1, 2, 4, 7])
    else:
        hi = _log(rng, 8, 4608)
    # the plain form's padded scores stay below the largest listed case's
    most = max(16, min(131072, 600_000_000 // (B * heads * group * hi), 100_000_000 // (B * heads)))
    past_hi = _log(rng, 16, most)
    return dict(op="attn", B=B, new_lo=rng.randint(1, hi), new_hi=hi, past_lo=rng.randint(0, past_hi),
                past_hi=past_hi, heads=heads, group=group, d=d, page=page, block=block, causal=rng.random() < 0.7,
                dtype=dtype)


def _spread(lo, hi, n):
    """n lengths over [lo, hi] (both taken for n > 1), in no order."""
    if n == 1:
        return [hi]
    got = [lo + int(round((hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]
    got[n // 2] = hi
    return got


def _lengths(case):
    B = case["B"]
    new = _spread(case["new_lo"], case["new_hi"], B)
    past = _spread(case["past_lo"], case["past_hi"], B)[::-1]
    return new, past


# --------------------------------------------------------------------------- inputs
def _axes(case):
    return [int(a) for a in case["axes"].split(",")]


def _draws(seed, d):
    """SplitMix64 draws of a rotation: Fisher-Yates permutation, then signs."""
    mask, st = (1 << 64) - 1, seed

    def nxt():
        nonlocal st
        st = (st + 0x9E3779B97F4A7C15) & mask
        z = st
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        return z ^ (z >> 31)

    perm = list(range(d))
    for i in range(d - 1, 0, -1):
        j = nxt() % (i + 1)
        perm[i], perm[j] = perm[j], perm[i]
    signs = [-1.0 if nxt() >> 63 else 1.0 for _ in range(d)]
    return perm, signs


def _hadamard(h):
    m = np.ones((1, 1))
    while m.shape[0] < h:
        m = np.block([[m, m], [m, -m]])
    return m / math.sqrt(h)


def _rotation(d, block):
    """The d x d rotation matrix (rows: rotated coordinates), or None for no rotation."""
    if not block:
        return None
    perm, signs = _draws(0, d)
    pi = np.zeros((d, d))
    pi[np.arange(d), perm] = signs
    return torch.from_numpy(np.kron(np.eye(d // block), _hadamard(block)) @ pi).cuda()


def _handles(case):
    """What a program keeps of the library: the module and the rotation's handle."""
    if not own:
        return None, None
    from calibration_free_rotated_b200 import orbitquant as oq
    if case["op"] == "rope":
        return oq, oq.Rope(_axes(case), layout=case["layout"])
    return oq, (oq.Rpbh(0, case["d"], case["block"]) if case["block"] else None)


def _rows(gen, shape, dtype):
    """Keys or values: some channels carry larger values, as projections' outputs do."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.exp(0.4 * torch.randn(shape[-2:], generator=gen, device="cuda"))
    loud = (torch.rand(shape[-2:], generator=gen, device="cuda") < 0.02).float()
    return (x * gain * (1 + 7 * loud)).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cumulate(v):
    return _ints([0] + list(np.cumsum(v)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, d = DTYPES[case["dtype"]], case["d"]
    s = dict(case=case)
    s["oq"], s["handle"] = _handles(case)
    if case["op"] == "rope":
        T, axes = case["T"], _axes(case)
        fused = torch.randn((T, case["heads"] + case["extra"], d), generator=gen, device="cuda").to(dt)
        s["x"] = fused[:, :case["heads"]]
        s["out"] = torch.empty((T, case["heads"], d), dtype=dt, device="cuda")
        i = torch.arange(T, device="cuda")
        start = int(torch.randint(0, 1000, (1,), generator=gen, device="cuda"))
        if case["grid"] == "far":  # rows of different sequences, up to a million tokens in
            pos = torch.randint(0, 1_000_000, (T, len(axes)), generator=gen, device="cuda")
        elif case["grid"] == "image":  # 512 text tokens at the origin, then 64 x 64
            j = (i - 512).clamp(min=0)
            pos = torch.stack([torch.full_like(i, 0), j // 64, j % 64], 1)
        else:  # 30 x 52 frames from some time on
            pos = torch.stack([start + i // 1560, (i // 52) % 30, i % 52], 1)[:, :len(axes)]
        s["pos"] = pos.to(torch.int32).contiguous()
        freq, axis = [], []
        for a, n in enumerate(axes):
            freq += [10000.0 ** (-2.0 * k / n) for k in range(n // 2)]
            axis += [a] * (n // 2)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["axis"] = torch.tensor(axis, device="cuda")
        return s

    new, past = _lengths(case)
    B, H, P, T = case["B"], case["heads"], case["page"], sum(new)
    total = [a + b for a, b in zip(new, past)]
    width = max(-(-t // P) for t in total)
    need = sum(-(-t // P) for t in total)
    n_pages = need + 3
    # each sequence's pages, drawn from a shuffled pool; entries behind its last page are not used
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    at = 0
    for b, t in enumerate(total):
        n = -(-t // P)
        table[b, :n] = order[at:at + n]
        at += n
    s["table"], s["cu"], s["past"], s["total"] = table, _cumulate(new), _ints(past), _ints(total)
    s["n_new"], s["n_total"], s["T"], s["width"] = max(new), max(total), T, width
    s["R"] = _rotation(d, case["block"])
    s["k"] = torch.zeros((n_pages, H, P, d), dtype=torch.int8, device="cuda")
    s["v"] = torch.zeros((n_pages, H, P, d), dtype=torch.int8, device="cuda")
    s["ks"] = torch.full((n_pages, H), 2.0 ** E_MIN, device="cuda")
    s["vs"] = torch.full((n_pages, H), 2.0 ** E_MIN, device="cuda")
    # the cache as it stands before the call
    before = past if case["op"] == "cache" else total
    if sum(before):
        _write(s, _rows(gen, (sum(before), H, d), dt), _rows(gen, (sum(before), H, d), dt), _cumulate(before),
               _ints([0] * B))
    if s["oq"] is not None:
        s["cache"] = s["oq"].KVCache.wrap(s["k"], s["v"], s["ks"], s["vs"])
    if case["op"] == "cache":
        # what is read back: the new tokens and the pages' older ones beside them
        first = [p // P * P for p in past]
        s["first"], s["cu_read"] = _ints(first), _cumulate([t - f for t, f in zip(total, first)])
        s["T_read"] = sum(total) - sum(first)
        s["new_k"], s["new_v"] = _rows(gen, (T, H, d), dt), _rows(gen, (T, H, d), dt)
    elif case["op"] == "read":
        s["first"], s["cu_read"], s["T_read"] = _ints([0] * B), s["cu"], T
    else:
        s["q"] = (1.5 * torch.randn((T, H * case["group"], d), generator=gen, device="cuda")).to(dt)
        s["out"] = torch.empty_like(s["q"])
        if s["oq"] is not None:
            s["ws"] = torch.empty((s["oq"].cache_attention_workspace_bytes(s["cache"], T, B, H * case["group"]),),
                                  dtype=torch.uint8, device="cuda")
    if case["op"] in ("cache", "read"):
        s["out_k"] = torch.empty((s["T_read"], H, d), dtype=dt, device="cuda")
        s["out_v"] = torch.empty((s["T_read"], H, d), dtype=dt, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms
def _rope(s):
    case = s["case"]
    x = s["x"].float()
    n = s["freq"].numel()
    ang = s["pos"].double()[:, s["axis"]] * s["freq"]  # 64 bits: far positions
    if case["inverse"]:
        ang = -ang
    c, sn = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    out = x.clone()
    if case["layout"] == "interleaved":
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        out[..., 0:2 * n:2] = a * c - b * sn
        out[..., 1:2 * n:2] = a * sn + b * c
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        out[..., :n] = a * c - b * sn
        out[..., n:2 * n] = a * sn + b * c
    return out.to(s["x"].dtype)


def _places(s, cu, first, T):
    """Page, place in the page and sequence of each of T rows, first[b] being the first row's position."""
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i.to(torch.int32), right=True)
    p = first[b].long() + i - cu[b].long()
    P = s["k"].shape[2]
    return s["table"][b, p // P].long(), p % P, b


def _write_half(s, codes, scale, x, cu, past):
    T, P = x.shape[0], codes.shape[2]
    page, off, _ = _places(s, cu, past, T)
    u = x.double()  # 64 bits: values next to a border between two codes
    if s["R"] is not None:
        u = u @ s["R"].T
    amax = torch.zeros(scale.shape, dtype=torch.float64, device="cuda")
    amax.scatter_reduce_(0, page[:, None].expand(-1, scale.shape[1]), u.abs().amax(-1), "amax")
    m, e = torch.frexp(amax / 127)
    e = torch.where(m > 0.5, e, e - 1)  # the least e with amax <= 127 * 2^e
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    # the page that each sequence's first new token falls into, where it holds older tokens
    held = past % P
    some = (held > 0) & (cu[1:] > cu[:-1])
    p0 = s["table"].gather(1, (past // P).clamp(max=s["table"].shape[1] - 1).long()[:, None])[:, 0].long()
    keep = p0[some]
    e_old = torch.frexp(scale[keep])[1] - 1
    e_new = torch.maximum(e[keep], e_old)
    old = codes[keep]
    rows = (torch.arange(P, device="cuda")[None] < held[some][:, None])[:, None, :, None]
    moved = torch.round(torch.ldexp(old.float(), (e_old - e_new)[:, :, None, None])).to(torch.int8)
    codes[keep] = torch.where(rows, moved, old)
    e[keep] = e_new
    scale[page] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[page]
    codes[page, :, off] = torch.round(torch.ldexp(u, -e[page][:, :, None])).clamp(-127, 127).to(torch.int8)


def _write(s, k, v, cu, past):
    _write_half(s, s["k"], s["ks"], k, cu, past)
    _write_half(s, s["v"], s["vs"], v, cu, past)


def _read_half(s, codes, scale):
    page, off, _ = _places(s, s["cu_read"], s["first"], s["T_read"])
    x = codes[page, :, off].float() * scale[page][:, :, None]
    return x if s["R"] is None else x @ s["R"].float()


def _attend(s):
    case, q = s["case"], s["q"].float()
    B, H, G, d, P = case["B"], case["heads"], case["group"], case["d"], case["page"]
    n, L = s["n_new"], s["n_total"]
    if s["R"] is not None:
        q = q @ s["R"].float().T
    i = torch.arange(n, device="cuda")
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    here = i[None] < new[:, None]
    qp = q[(s["cu"][:-1].long()[:, None] + i[None]).clamp(max=s["T"] - 1)]  # [B, n, H * G, d]
    qp = qp.view(B, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)
    k = (s["k"][s["table"].long()].float() * s["ks"][s["table"].long()][..., None, None])
    k = k.permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)[:, :, :L]
    w = (qp @ k.transpose(2, 3)).view(B, H, G, n, L) * (1.0 / math.sqrt(d))
    del k
    j = torch.arange(L, device="cuda")
    last = s["total"].long()[:, None] - (new[:, None] - 1 - i[None] if case["causal"] else 0) - 1  # [B, n] or [B, 1]
    seen = (j[None, None] <= last[:, :, None])[:, None, None]
    w.masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    norm = w.sum(-1, keepdim=True)
    v = (s["v"][s["table"].long()].float() * s["vs"][s["table"].long()][..., None, None])
    v = v.permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)[:, :, :L]
    o = (w.view(B, H, G * n, L) @ v).view(B, H, G, n, d) / torch.where(norm > 0, norm, 1.0)
    if s["R"] is not None:
        o = o @ s["R"].float()
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, H * G, d)[here].to(s["q"].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        oq, handle = s["oq"], s["handle"]
        if op == "rope":
            return oq.rope_apply(handle, s["x"], s["pos"], out=s["out"], inverse=case["inverse"])
        if op == "cache":
            oq.cache_write(s["cache"], s["new_k"], s["new_v"], s["cu"], s["past"], s["table"], rpbh=handle)
        if op in ("cache", "read"):
            k, v = oq.cache_read(s["cache"], s["cu_read"], s["first"], s["table"], rpbh=handle, k=s["out_k"],
                                 v=s["out_v"])
            return (k, v, s["ks"], s["vs"]) if op == "cache" else (k, v)
        return oq.cache_attention(s["cache"], s["q"], s["cu"], s["total"], s["table"], rpbh=handle,
                                  causal=case["causal"], out=s["out"], workspace=s["ws"])
    if op == "rope":
        return _rope(s)
    if op == "cache":
        _write(s, s["new_k"], s["new_v"], s["cu"], s["past"])
    if op in ("cache", "read"):
        dt = DTYPES[case["dtype"]]
        k, v = _read_half(s, s["k"], s["ks"]).to(dt), _read_half(s, s["v"], s["vs"]).to(dt)
        return (k, v, s["ks"], s["vs"]) if op == "cache" else (k, v)
    return _attend(s)


# --------------------------------------------------------------------------- work
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    d = case["d"]
    if case["op"] == "rope":
        n = case["T"] * case["heads"] * d
        return {"bytes": 2 * n * size + 4 * case["T"] * len(_axes(case)), "flops": 3 * n}
    new, past = _lengths(case)
    H, P = case["heads"], case["page"]
    turn = 2 * math.log2(case["block"]) if case["block"] else 0  # butterflies of one element, there and back
    if case["op"] in ("cache", "read"):
        T = sum(new)
        rows = sum(n + p - p // P * P for n, p in zip(new, past))
        written = T * H * d * (size + 1) if case["op"] == "cache" else 0
        return {"bytes": 2 * (written + rows * H * d * (size + 1)), "flops": 2 * rows * H * d * (2 + turn)}
    pairs = read = 0
    for n, p in zip(new, past):
        t = n + p
        pairs += sum(t - n + 1 + i for i in range(n)) if case["causal"] else n * t
        read += t
    Hq = H * case["group"]
    return {"bytes": 2 * read * H * d + 8 * H * sum(-(-(n + p) // P) for n, p in zip(new, past)) + 2 * sum(new) * Hq * d * size,
            "flops": 4 * pairs * Hq * d}


# --------------------------------------------------------------------------- definitions in 64 bits
def _turned(x, d, block, back=False):
    """Rows x (64 bits) through the rotation or its transpose, by its definition."""
    if not block:
        return x
    perm, signs = _draws(0, d)
    perm, signs = torch.tensor(perm, device="cuda"), torch.tensor(signs, dtype=torch.float64, device="cuda")
    idx = np.arange(block)
    h = torch.tensor([[(-1.0) ** bin(int(a) & int(b)).count("1") for b in idx] for a in idx], dtype=torch.float64,
                     device="cuda") / math.sqrt(block)
    shape = x.shape
    if back:
        y = (x.reshape(-1, d // block, block) @ h).reshape(-1, d) * signs
        out = torch.empty_like(y)
        out[:, perm] = y
        return out.reshape(shape)
    y = x.reshape(-1, d)[:, perm] * signs
    return (y.reshape(-1, d // block, block) @ h).reshape(shape)


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "rope":
        x, out, base = s["x"].double(), s["x"].double().clone(), 0
        half = sum(_axes(case)) // 2
        for a, n in enumerate(_axes(case)):
            k = torch.arange(n // 2, dtype=torch.float64, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(case["T"], n // 2).contiguous(),
                               s["pos"][:, a].double()[:, None] / (10000.0 ** (2 * k / n)))
            if case["inverse"]:
                turn = turn.conj()
            j = torch.arange(base, base + n // 2, device="cuda")
            re, im = (2 * j, 2 * j + 1) if case["layout"] == "interleaved" else (j, j + half)
            z = torch.complex(x[..., re], x[..., im]) * turn[:, None]
            out[..., re], out[..., im] = z.real, z.imag
            base += n // 2
        return out
    new, past = _lengths(case)
    B, P, H = case["B"], case["page"], case["heads"]
    table = s["table"].tolist()
    if case["op"] in ("cache", "read"):
        halves, scales = [], []
        for codes, scale, rows in ((s["k"], s["ks"], s.get("new_k")), (s["v"], s["vs"], s.get("new_v"))):
            scale, at, got = scale.double().clone(), 0, []
            for b in range(B):
                first = past[b] // P * P
                pages = torch.tensor(table[b][first // P:-(-(past[b] + new[b]) // P)], device="cuda")
                n = past[b] + new[b] - first
                whole = codes[pages].double()  # [pages, H, P, d]
                if rows is not None:
                    pad = torch.zeros((len(pages) * P, H, d), dtype=torch.float64, device="cuda")
                    pad[past[b] - first:n] = _turned(rows[at:at + new[b]].double(), d, case["block"])
                    pad = pad.view(-1, P, H, d).permute(0, 2, 1, 3)
                    steps = torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device="cuda")
                    e = (127 * steps < pad.abs().amax((2, 3))[..., None]).sum(-1).clamp(max=E_MAX - E_MIN)
                    was = torch.searchsorted(steps, scale[pages])
                    fresh = torch.arange(len(pages), device="cuda")[:, None] * P >= past[b] - first
                    e = torch.where(fresh, e, torch.maximum(e, was))
                    old = (torch.arange(len(pages) * P, device="cuda") < past[b] - first).view(-1, 1, P, 1)
                    kept = torch.round(whole * (steps[was] / steps[e])[..., None, None])
                    whole = torch.where(old, kept, torch.round(pad / steps[e][..., None, None]).clamp(-127, 127))
                    scale[pages] = steps[e]
                    at += new[b]
                vals = (whole * scale[pages][..., None, None]).permute(0, 2, 1, 3).reshape(-1, H, d)[:n]
                got.append(_turned(vals, d, case["block"], back=True))
            halves.append(torch.cat(got))
            scales.append(scale)
        return tuple(halves + scales) if case["op"] == "cache" else tuple(halves)
    outs, at, G = [], 0, case["group"]
    q = _turned(s["q"].double(), d, case["block"])
    for b in range(B):
        n, t = new[b], new[b] + past[b]
        pages = torch.tensor(table[b][:-(-t // P)], device="cuda")
        k, v = ((c[pages].double() * sc[pages].double()[..., None, None]).transpose(0, 1).reshape(H, -1, d)[:, :t]
                for c, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        o = torch.empty((n, H * G, d), dtype=torch.float64, device="cuda")
        bar = torch.arange(n, device="cuda")[:, None] + (t - n) if case["causal"] else torch.full((n, 1), t, device="cuda")
        hide = torch.arange(t, device="cuda")[None] > bar
        for h in range(H * G):
            w = (q[at:at + n, h] @ k[h // G].T) / math.sqrt(d)
            w[hide] = -math.inf
            o[:, h] = torch.softmax(w, -1) @ v[h // G]
        outs.append(o)
        at += n
    return _turned(torch.cat(outs), d, case["block"], back=True)
