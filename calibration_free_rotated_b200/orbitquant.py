"""Thin ctypes binding of liborbitquant.so (argument marshalling only).

Every step of the hot path runs in the library's CUDA kernels; this module
only turns torch tensors into device pointers and sizes, picks the current
torch stream, and turns non-zero status codes into exceptions.  There is no
fallback: if the shared library is missing, importing this module fails.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liborbitquant.so")

OQ_OK, OQ_ERR_ARG, OQ_ERR_UNSUPPORTED, OQ_ERR_ALIGN, OQ_ERR_CUDA, OQ_ERR_TIMEOUT, OQ_ERR_NOMEM = range(7)
EPILOGUES = {"none": 0, "gelu": 1}
ROTATIONS = {"rpbh": 0, "block_rht": 1, "full_rht": 2}  # OQ_ROT_*

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m calibration_free_rotated_b200.build` "
        "(there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

_c_int, _c_void_p, _c_size_t, _c_i64 = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong
_SIGS = {
    "oq_version": (_c_int, []),
    "oq_device_allocations": (ctypes.c_longlong, []),
    "oq_last_error": (ctypes.c_char_p, []),
    "oq_get_device_status": (_c_int, [_c_void_p]),
    "oq_make_rpbh": (_c_int, [ctypes.c_uint64, _c_int, _c_int, ctypes.POINTER(_c_void_p)]),
    "oq_make_rotation": (_c_int, [ctypes.c_uint64, _c_int, _c_int, _c_int, ctypes.POINTER(_c_void_p)]),
    "oq_rotation_kind": (_c_int, [_c_void_p, ctypes.POINTER(_c_int)]),
    "oq_make_composed_rpbh": (_c_int, [ctypes.c_uint64, _c_int, _c_int, _c_int, ctypes.POINTER(_c_void_p)]),
    "oq_rotation_rounds": (_c_int, [_c_void_p, ctypes.POINTER(_c_int)]),
    "oq_rpbh_export_round": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_void_p]),
    "oq_rpbh_info": (_c_int, [_c_void_p, ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "oq_rpbh_export": (_c_int, [_c_void_p, _c_void_p, _c_void_p]),
    "oq_free_rpbh": (None, [_c_void_p]),
    "oq_build_codebook": (_c_int, [_c_int, _c_int, ctypes.POINTER(_c_void_p)]),
    "oq_codebook_info": (_c_int, [_c_void_p, ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "oq_codebook_export": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.POINTER(_c_int),
                                    ctypes.POINTER(ctypes.c_double)]),
    "oq_free_codebook": (None, [_c_void_p]),
    "oq_quantize_act": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "oq_quantize_weight": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "oq_linear_codes": (_c_int, [_c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p,
                                 _c_int, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "oq_linear_workspace_bytes": (_c_size_t, [_c_int, _c_int, _c_int]),
    "oq_row_flatness": (_c_int, [_c_void_p, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "oq_linear": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_int,
                           _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "oq_linear_noalloc": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p,
                                   _c_int, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "oq_make_rope": (_c_int, [_c_int, _c_void_p, _c_void_p, _c_int, _c_int, ctypes.POINTER(_c_void_p)]),
    "oq_rope_info": (_c_int, [_c_void_p, ctypes.POINTER(_c_int), ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "oq_free_rope": (None, [_c_void_p]),
    "oq_rope_apply": (_c_int, [_c_void_p, _c_void_p, _c_i64, _c_i64, _c_void_p, _c_i64, _c_i64, _c_int, _c_int,
                               _c_int, _c_int, _c_void_p, _c_int, _c_void_p]),
    "oq_cache_write": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_i64, _c_i64, _c_void_p, _c_i64, _c_i64, _c_int,
                                _c_int, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p]),
    "oq_cache_read": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_void_p, _c_void_p,
                               _c_int, _c_void_p, _c_int, _c_void_p]),
    "oq_cache_attention_workspace_bytes": (_c_size_t, [_c_void_p, _c_int, _c_int, _c_int]),
    "oq_cache_attention": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_i64, _c_i64, _c_void_p, _c_i64, _c_i64,
                                    _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_int,
                                    ctypes.c_float, _c_void_p, _c_size_t, _c_void_p]),
    "oq_test_composed_tables": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p]),
}
NOALLOC_SCRATCH_BYTES = 32 << 20
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class OQError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"orbitquant error {code}: {message}")
        self.code = code


def _check(rc):
    if rc != OQ_OK:
        raise OQError(rc, _lib.oq_last_error().decode())


def lib():
    """The loaded ctypes library (for tests that call the C ABI directly)."""
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Rpbh:
    """Handle of the RPBH rotation for one (seed, d, block); `kind` selects a
    variant of the rotation ablation ("rpbh", "block_rht", "full_rht");
    `rounds` > 1 composes that many RPBH rounds (oq_make_composed_rpbh)."""

    def __init__(self, seed: int, d: int, block: int = 0, kind: str = "rpbh", rounds: int = 1):
        h = ctypes.c_void_p()
        if rounds == 1:
            _check(_lib.oq_make_rotation(seed, d, block, ROTATIONS[kind], ctypes.byref(h)))
        else:
            if kind != "rpbh":
                raise ValueError("composed rounds are RPBH rounds")
            _check(_lib.oq_make_composed_rpbh(seed, d, block, rounds, ctypes.byref(h)))
        self._h = h
        dd, bb, kk, rr = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _check(_lib.oq_rpbh_info(h, ctypes.byref(dd), ctypes.byref(bb)))
        _check(_lib.oq_rotation_kind(h, ctypes.byref(kk)))
        _check(_lib.oq_rotation_rounds(h, ctypes.byref(rr)))
        self.seed, self.d, self.block, self.rounds = seed, dd.value, bb.value, rr.value
        self.kind = {v: k for k, v in ROTATIONS.items()}[kk.value]

    @property
    def handle(self):
        return self._h

    def export(self):
        import numpy as np
        perm = np.empty(self.d, dtype=np.int32)
        signs = np.empty((self.d + 31) // 32, dtype=np.uint32)
        _check(_lib.oq_rpbh_export(self._h, perm.ctypes.data, signs.ctypes.data))
        return perm, signs

    def export_round(self, rnd: int):
        """(perm, sign words) of round `rnd` (1-based) of a composed rotation."""
        import numpy as np
        perm = np.empty(self.d, dtype=np.int32)
        signs = np.empty((self.d + 31) // 32, dtype=np.uint32)
        _check(_lib.oq_rpbh_export_round(self._h, rnd, perm.ctypes.data, signs.ctypes.data))
        return perm, signs

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.oq_free_rpbh(h)


class Codebook:
    """Handle of the Lloyd-Max codebook C^(d,b)."""

    def __init__(self, d: int, bits: int):
        h = ctypes.c_void_p()
        _check(_lib.oq_build_codebook(d, bits, ctypes.byref(h)))
        self._h = h
        self.d, self.bits = d, bits

    @property
    def handle(self):
        return self._h

    def export(self):
        import numpy as np
        L = 1 << self.bits
        c = np.empty(L, dtype=np.float64)
        b = np.empty(L - 1, dtype=np.float64)
        lut = np.empty(L, dtype=np.uint16)
        it = ctypes.c_int()
        dist = ctypes.c_double()
        _check(_lib.oq_codebook_export(self._h, c.ctypes.data, b.ctypes.data, lut.ctypes.data,
                                       ctypes.byref(it), ctypes.byref(dist)))
        return {"centroids": c, "boundaries": b, "lut_fp16": lut, "iterations": it.value,
                "distortion": dist.value}

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.oq_free_codebook(h)


def code_bytes(d: int, bits: int) -> int:
    return d * bits // 8


def quantize_act(rpbh: Rpbh, cb: Codebook, X: torch.Tensor, codes=None, norms=None, stream=None):
    """X: cuda bf16 [M, d] -> (codes uint8 [M, d*b/8], norms float32 [M])."""
    M = X.shape[0]
    if codes is None:
        codes = torch.empty((M, code_bytes(rpbh.d, cb.bits)), dtype=torch.uint8, device=X.device)
    if norms is None:
        norms = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(_lib.oq_quantize_act(rpbh.handle, cb.handle, _ptr(X), M, _ptr(codes), _ptr(norms), _stream(stream)))
    return codes, norms


def quantize_weight(rpbh: Rpbh, cb: Codebook, W: torch.Tensor, codes=None, norms=None, stream=None):
    """W: cuda bf16 [N, d] -> (codes uint8 [N, d*b/8], norms bf16 [N])."""
    N = W.shape[0]
    if codes is None:
        codes = torch.empty((N, code_bytes(rpbh.d, cb.bits)), dtype=torch.uint8, device=W.device)
    if norms is None:
        norms = torch.empty((N,), dtype=torch.bfloat16, device=W.device)
    _check(_lib.oq_quantize_weight(rpbh.handle, cb.handle, _ptr(W), N, _ptr(codes), _ptr(norms), _stream(stream)))
    return codes, norms


def linear_codes(d, cb_a: Codebook, cb_w: Codebook, a_codes, a_norm, w_codes, w_norm, bias=None, epilogue="none",
                 out_f32=None, out_bf16=None, want_f32=True, want_bf16=False, stream=None):
    M, N = a_codes.shape[0], w_codes.shape[0]
    dev = a_codes.device
    if out_f32 is None and want_f32:
        out_f32 = torch.empty((M, N), dtype=torch.float32, device=dev)
    if out_bf16 is None and want_bf16:
        out_bf16 = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _check(_lib.oq_linear_codes(d, cb_a.handle, cb_w.handle, _ptr(a_codes), _ptr(a_norm), M, _ptr(w_codes),
                                _ptr(w_norm), N, _ptr(bias), EPILOGUES[epilogue], _ptr(out_f32), _ptr(out_bf16),
                                _stream(stream)))
    return out_f32, out_bf16


def row_flatness(X, rho3=None, rhoinf=None, batch_max=None, want_rows=True, stream=None):
    """Flatness check of the rows of X (cuda bf16 [M, d]): per-row rho3 and
    rhoinf (float [M] each, unless want_rows is False) and their batch maxima
    (float [2])."""
    M, d = X.shape
    dev = X.device
    if want_rows:
        rho3 = torch.empty((M,), dtype=torch.float32, device=dev) if rho3 is None else rho3
        rhoinf = torch.empty((M,), dtype=torch.float32, device=dev) if rhoinf is None else rhoinf
    batch_max = torch.empty((2,), dtype=torch.float32, device=dev) if batch_max is None else batch_max
    _check(_lib.oq_row_flatness(_ptr(X), M, d, _ptr(rho3), _ptr(rhoinf), _ptr(batch_max), _stream(stream)))
    return rho3, rhoinf, batch_max


def workspace_bytes(M: int, d: int, bits_a: int) -> int:
    return int(_lib.oq_linear_workspace_bytes(M, d, bits_a))


def linear(rpbh: Rpbh, cb_a: Codebook, cb_w: Codebook, X, w_codes, w_norm, bias=None, epilogue="none",
           out_f32=None, out_bf16=None, want_f32=True, want_bf16=False, workspace=None, stream=None):
    """Full layer: act-quant of X (cuda bf16 [M, d]) then the codebook GEMM."""
    M, N = X.shape[0], w_codes.shape[0]
    dev = X.device
    if out_f32 is None and want_f32:
        out_f32 = torch.empty((M, N), dtype=torch.float32, device=dev)
    if out_bf16 is None and want_bf16:
        out_bf16 = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    need = workspace_bytes(M, rpbh.d, cb_a.bits)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    _check(_lib.oq_linear(rpbh.handle, cb_a.handle, cb_w.handle, _ptr(X), M, _ptr(w_codes), _ptr(w_norm), N,
                          _ptr(bias), EPILOGUES[epilogue], _ptr(out_f32), _ptr(out_bf16), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream(stream)))
    return out_f32, out_bf16


def device_status(stream=None):
    """Raises OQError if a kernel's bounded wait gave up since the last call."""
    _check(_lib.oq_get_device_status(_stream(stream)))


def device_allocations() -> int:
    """How many device allocations the library has made in this process."""
    return int(_lib.oq_device_allocations())


def linear_noalloc(rpbh: Rpbh, cb_a: Codebook, cb_w: Codebook, X, w_codes, w_norm, bias=None, epilogue="none",
                   out_f32=None, out_bf16=None, stream=None):
    """oq_linear_noalloc: the full layer with the library's static scratch
    instead of a workspace.  Outputs must be passed in (this call is for code
    that cannot allocate)."""
    M, N = X.shape[0], w_codes.shape[0]
    _check(_lib.oq_linear_noalloc(rpbh.handle, cb_a.handle, cb_w.handle, _ptr(X), M, _ptr(w_codes), _ptr(w_norm),
                                  N, _ptr(bias), EPILOGUES[epilogue], _ptr(out_f32), _ptr(out_bf16),
                                  _stream(stream)))
    return out_f32, out_bf16


# ---------------------------------------------------------------------------
# Rotary positions, the 8-bit cache, attention over it
# ---------------------------------------------------------------------------
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # OQ_BF16 ..
ROPE_LAYOUTS = {"interleaved": 0, "halves": 1}


class Rope:
    """Rotary positions over several axes (oq_make_rope).

    axis_dims: how many of a head's leading elements turn with each axis, in
    order (even numbers; FLUX heads of 128: (16, 56, 56), Wan's: (44, 42, 42);
    one axis: (128,)).  With ladder "axis" every axis has frequencies of its
    own, theta^(-2k / axis_dim) for its pair k; with "shared" the axes share one
    ladder over all pairs, theta^(-2p / sum(axis_dims)) for pair p.  layout
    "interleaved" pairs elements 2p and 2p + 1, "halves" p and p + pairs.  Any
    other frequencies: pass `freqs` and `axes` (one of each for every pair)
    instead."""

    def __init__(self, axis_dims=None, theta: float = 10000.0, layout: str = "interleaved", ladder: str = "axis",
                 freqs=None, axes=None):
        if (axis_dims is None) == (freqs is None) or (freqs is None) != (axes is None):
            raise ValueError("pass either axis_dims, or freqs and axes")
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"unknown layout {layout!r}")
        if axis_dims is not None:
            if ladder not in ("axis", "shared"):
                raise ValueError(f"unknown ladder {ladder!r}")
            dims = [int(n) for n in axis_dims]
            if not dims or any(n < 2 or n % 2 for n in dims):
                raise ValueError(f"axis_dims must be even and positive (got {dims})")
            freqs, axes, total = [], [], sum(dims)
            for a, n in enumerate(dims):
                for k in range(n // 2):
                    e = 2 * k / n if ladder == "axis" else 2 * len(freqs) / total
                    freqs.append(float(theta) ** -e)
                    axes.append(a)
            n_axes = len(dims)
        else:
            freqs, axes = [float(f) for f in freqs], [int(a) for a in axes]
            if not freqs or len(freqs) != len(axes) or not all(0 <= a < 256 for a in axes):
                raise ValueError("freqs and axes need one entry for each pair, axes in 0..255")
            n_axes = max(axes) + 1
        n = len(freqs)
        h = ctypes.c_void_p()
        _check(_lib.oq_make_rope(n, (ctypes.c_double * n)(*freqs), (ctypes.c_uint8 * n)(*axes), n_axes,
                                 ROPE_LAYOUTS[layout], ctypes.byref(h)))
        self._h = h
        self.pairs, self.n_axes, self.layout = n, n_axes, layout

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.oq_free_rope(h)


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("heads", ctypes.c_int),
                ("page", ctypes.c_int), ("d", ctypes.c_int)]


class KVCache:
    """Paged 8-bit cache of keys and values (oq_kvcache): codes k, v int8
    [n_pages, heads, page, d], scales k_scale, v_scale float32 [n_pages, heads]."""

    def __init__(self, n_pages: int, heads: int, d: int, page: int = 64, device="cuda"):
        codes = [torch.zeros((n_pages, heads, page, d), dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.zeros((n_pages, heads), dtype=torch.float32, device=device) for _ in range(2)]
        self._set(*codes, *scales)

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale):
        """A cache over tensors that stand already."""
        c = cls.__new__(cls)
        c._set(k, v, k_scale, v_scale)
        return c

    def _set(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != torch.int8 or v.dtype != torch.int8:
            raise ValueError("k and v must be int8 [n_pages, heads, page, d]")
        if tuple(k_scale.shape) != tuple(k.shape[:2]) or k_scale.shape != v_scale.shape or \
                k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise ValueError("k_scale and v_scale must be float32 [n_pages, heads]")
        for t in (k, v, k_scale, v_scale):
            if not t.is_contiguous() or t.device != k.device:
                raise ValueError("cache tensors must be contiguous and on one device")
        self._tensors = (k, v, k_scale, v_scale)
        self.n_pages, self.heads, self.page, self.d = k.shape
        self.device, self._index = k.device, k.get_device()
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                    self.n_pages, self.heads, self.page, self.d)
        self._ref = ctypes.byref(self._struct)

    # A tensor that is put in another's place is checked, and its address taken, like the first one.
    @property
    def k(self):
        return self._tensors[0]

    @k.setter
    def k(self, t):
        self._set(t, *self._tensors[1:])

    @property
    def v(self):
        return self._tensors[1]

    @v.setter
    def v(self, t):
        self._set(self._tensors[0], t, *self._tensors[2:])

    @property
    def k_scale(self):
        return self._tensors[2]

    @k_scale.setter
    def k_scale(self, t):
        self._set(*self._tensors[:2], t, self._tensors[3])

    @property
    def v_scale(self):
        return self._tensors[3]

    @v_scale.setter
    def v_scale(self, t):
        self._set(*self._tensors[:3], t)


# The calls below are paced by the host where the work is small, so each looks at its
# tensors in as few steps as Python has: devices as their numbers, one expression for
# the checks, and the words of an error only when one fails.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda i: torch.cuda.current_stream(i).cuda_stream)
_I32 = torch.int32


def _launch(fn, index, stream, *args):
    """fn(*args, stream) with the tensors' device (its number) current."""
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    if index != _current_device():
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc)


def _empty(shape, dtype, device, stream):
    """A tensor in the memory of the stream that will use it (None: the current one), so that
    it is not handed to another stream's work while this one's is under way."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(name, t, index, heads, d, T=None, dtype=None):
    """Strides (token, head) of rows [T, heads, d] on device `index` (heads, d, T,
    dtype: None for any)."""
    shape, strides = t.shape, t.stride()
    if (len(shape) == 3 and strides[2] == 1 and t.get_device() == index and (d is None or shape[2] == d)
            and (heads is None or shape[1] == heads) and (T is None or shape[0] == T)
            and (t.dtype in DTYPES if dtype is None else t.dtype is dtype)):
        return strides
    if len(shape) == 3 and shape[2] == 1 and strides[2] != 1:  # one element: any stride
        return _rows(name, t.as_strided(shape, (strides[0], strides[1], 1)), index, heads, d, T, dtype)
    raise ValueError(f"{name} must be [{'T' if T is None else T}, {heads or 'heads'}, {d or 'd'}] rows of "
                     f"{dtype or 'bf16, fp16 or fp32'}, each contiguous, on device {index} "
                     f"(got {t.dtype} {list(shape)}, strides {list(strides)}, on {t.device})")


def _batch(cache, cu, at_name, at, table):
    """Pointers of a batch's index tensors, and B and the table's width."""
    index, B, width = cache._index, at.shape, table.shape
    if (len(B) == 1 and len(width) == 2 and width[0] == B[0] and cu.shape == (B[0] + 1,)
            and cu.dtype is _I32 and at.dtype is _I32 and table.dtype is _I32
            and cu.get_device() == index and at.get_device() == index and table.get_device() == index
            and cu.is_contiguous() and at.is_contiguous() and table.is_contiguous()):
        return cu.data_ptr(), at.data_ptr(), B[0], table.data_ptr(), width[1]
    said = ", ".join(f"{n} {t.dtype} {list(t.shape)} on {t.device}"
                     for n, t in (("cu", cu), (at_name, at), ("table", table)))
    raise ValueError(f"cu [B + 1], {at_name} [B] and table [B, width] must be contiguous int32 on {cache.device} "
                     f"(got {said})")


def rope_apply(rope: Rope, x: torch.Tensor, pos: torch.Tensor, out=None, inverse: bool = False, stream=None):
    """x: cuda bf16 / fp16 / fp32 [T, heads, d] (rows contiguous, any strides of
    tokens and heads) turned by pos: int32 [T, axes].  out: written and returned
    (x itself: in place); a new tensor if None.  inverse: the transposed turn,
    which is also the gradient."""
    index = x.get_device()
    sx = _rows("x", x, index, None, None)
    T, heads, d = x.shape
    dtype = x.dtype
    if out is None:
        out = _empty((T, heads, d), dtype, x.device, stream)
    so = _rows("out", out, index, heads, d, T, dtype)
    if pos.dtype is not _I32 or pos.shape != (T, rope.n_axes) or pos.get_device() != index or not pos.is_contiguous():
        raise ValueError(f"pos must be contiguous int32 [{T}, {rope.n_axes}] on x's device "
                         f"(got {pos.dtype} {list(pos.shape)} on {pos.device})")
    _launch(_lib.oq_rope_apply, index, stream, rope._h, x.data_ptr(), sx[0], sx[1], out.data_ptr(), so[0], so[1],
            DTYPES[dtype], T, heads, d, pos.data_ptr(), inverse)
    return out


def cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, past: torch.Tensor,
                table: torch.Tensor, rpbh: Rpbh = None, stream=None):
    """Quantizes the rows k, v (cuda bf16 / fp16 [T, heads, d], rows cu[b] ..
    cu[b+1]-1 are sequence b's) into the cache behind the past[b] tokens that
    the sequence holds, in the pages of table: int32 [B, width]."""
    index, T, dtype = cache._index, k.shape[0], k.dtype
    sk = _rows("k", k, index, cache.heads, cache.d)
    sv = _rows("v", v, index, cache.heads, cache.d, T, dtype)
    cu_p, at_p, B, table_p, width = _batch(cache, cu, "past", past, table)
    _launch(_lib.oq_cache_write, index, stream, cache._ref, None if rpbh is None else rpbh._h, k.data_ptr(), sk[0], sk[1],
            v.data_ptr(), sv[0], sv[1], DTYPES[dtype], T, cu_p, at_p, B, table_p, width)


def cache_read(cache: KVCache, cu: torch.Tensor, first: torch.Tensor, table: torch.Tensor, T: int = None,
               rpbh: Rpbh = None, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """Reads tokens first[b] .. of every sequence b back into rows cu[b] ..
    cu[b+1]-1 of k and v ([T, heads, d] contiguous; made as `dtype` if not
    passed, with T rows; rows outside all sequences then hold anything)."""
    if k is None or v is None:
        if k is not None or v is not None or T is None:
            raise ValueError("pass k and v, or T")
        k, v = (_empty((T, cache.heads, cache.d), dtype, cache.device, stream) for _ in range(2))
    index, dtype = cache._index, k.dtype
    _rows("k", k, index, cache.heads, cache.d, T)
    _rows("v", v, index, cache.heads, cache.d, k.shape[0], dtype)
    if not k.is_contiguous() or not v.is_contiguous():
        raise ValueError("k and v must be contiguous")
    cu_p, at_p, B, table_p, width = _batch(cache, cu, "first", first, table)
    _launch(_lib.oq_cache_read, index, stream, cache._ref, None if rpbh is None else rpbh._h, k.data_ptr(), v.data_ptr(),
            DTYPES[dtype], k.shape[0], cu_p, at_p, B, table_p, width)
    return k, v


def cache_attention_workspace_bytes(cache: KVCache, T: int, B: int, heads: int) -> int:
    return int(_lib.oq_cache_attention_workspace_bytes(cache._ref, T, B, heads))


def cache_attention(cache: KVCache, q: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                    rpbh: Rpbh = None, scale: float = None, causal: bool = True, out=None, workspace=None,
                    stream=None):
    """Attention of the rows q (cuda bf16 / fp16 [T, heads, d], rows cu[b] ..
    cu[b+1]-1 are sequence b's newest tokens) over the lens[b] tokens that the
    sequence holds in the cache, these among them.  scale: 1/sqrt(d) if None.
    out: written and returned, rows outside all sequences as they were; a new
    tensor if None, whose rows outside all sequences hold anything.  Single
    tokens and long chunks are faster in two calls (oq_cache_attention)."""
    index, dtype = cache._index, q.dtype
    sq = _rows("q", q, index, None, cache.d)
    T, heads, d = q.shape
    if out is None:
        out = _empty((T, heads, d), dtype, cache.device, stream)
    so = _rows("out", out, index, heads, d, T, dtype)
    cu_p, at_p, B, table_p, width = _batch(cache, cu, "lens", lens, table)
    if workspace is None:
        need = _lib.oq_cache_attention_workspace_bytes(cache._ref, T, B, heads)
        workspace = _empty((need,), torch.uint8, cache.device, stream)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on q's device")
    _launch(_lib.oq_cache_attention, index, stream, cache._ref, None if rpbh is None else rpbh._h, q.data_ptr(), sq[0],
            sq[1], out.data_ptr(), so[0], so[1], DTYPES[dtype], heads, T, cu_p, at_p, B, table_p, width, causal,
            d ** -0.5 if scale is None else scale, workspace.data_ptr(), workspace.nbytes)
    return out
