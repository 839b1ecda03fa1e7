"""ctypes binding of libgqa.so: argument marshalling only.

Every function here takes torch CUDA tensors, checks dtype / shape / device /
contiguity on the host, and passes raw device pointers, sizes and the current
CUDA stream to the C ABI declared in include/gqa.h.  All arithmetic happens in
the library's CUDA kernels; there is no CPU or PyTorch fallback, and a missing
library or a CPU tensor raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import types
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgqa.so")
_lib = None
_fast = _fast_pointers = None          # csrc/fastargs.c, set by load()

GQA_OK = 0
GQA_DEV_CAPACITY = 0x1
GQA_DEV_TIMEOUT = 0x2
GQA_DEV_BAD_LEN = 0x4

# Every symbol include/gqa.h declares, with (restype, argtypes).
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class RopeParams(ctypes.Structure):
    _fields_ = [("qk_norm", ctypes.c_int), ("eps", ctypes.c_float),
                ("rope_base", ctypes.c_float), ("scaling", ctypes.c_int),
                ("factor", ctypes.c_float), ("original_max_pos", ctypes.c_int),
                ("yarn_alpha", ctypes.c_float), ("yarn_beta", ctypes.c_float)]


MAX_AXES = 4


class RopeInputs(ctypes.Structure):
    _fields_ = [("q_gain", ctypes.c_void_p), ("k_gain", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("n_axes", ctypes.c_int),
                ("pair_axis", ctypes.c_uint8 * 64)]


ROPE_KINDS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


class RopeScaling:
    """A RoPE context-extension variant (see gqa.h): kind 'linear', 'ntk' or
    'yarn', the extension factor s >= 1 and, for YaRN, the trained context
    length and the ramp bounds alpha < beta."""

    def __init__(self, kind: str, factor: float, original_max_pos: int = 0,
                 alpha: float = 1.0, beta: float = 32.0):
        if kind not in ROPE_KINDS:
            raise ValueError("unknown RoPE scaling %r" % kind)
        self.kind, self.factor = kind, float(factor)
        self.original_max_pos, self.alpha, self.beta = int(original_max_pos), float(alpha), float(beta)


class RopeAxes:
    """Which position axis each rotation pair turns by: ``sections[a]`` pairs in a
    row for axis a (time, height, width, ...), or, with ``pairs``, the axis of every
    pair 0 .. D/2 - 1 (interleaved layouts)."""

    def __init__(self, sections=None, pairs=None):
        if (sections is None) == (pairs is None):
            raise ValueError("RopeAxes takes either sections or pairs")
        if pairs is None:
            if any(int(n) < 1 for n in sections):
                raise ValueError("every section needs at least one pair")
            pairs = [a for a, n in enumerate(sections) for _ in range(int(n))]
        self.pairs = tuple(int(a) for a in pairs)
        if not self.pairs or len(self.pairs) > 64:
            raise ValueError("RopeAxes needs 1 to 64 pairs, got %d" % len(self.pairs))
        self.n_axes = max(self.pairs) + 1
        if min(self.pairs) < 0 or self.n_axes > MAX_AXES:
            raise ValueError("axes are 0 .. %d" % (MAX_AXES - 1))
        if set(self.pairs) != set(range(self.n_axes)):
            raise ValueError("every axis needs at least one pair")
        x = RopeInputs(n_axes=self.n_axes)
        x.pair_axis[:len(self.pairs)] = self.pairs
        self._inputs = bytes(x)        # what a call copies and puts its pointers into


class Q4Cache:
    """A KV cache held in 4 bits (layout in gqa.h): codes uint8 [B, Hkv, Lmax, D/2] and
    scales bf16 [B, Hkv, Lmax, D/32, 2] of K and of V.  :meth:`zeros` makes one."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        self.k_codes, self.k_scales = k_codes, k_scales
        self.v_codes, self.v_scales = v_codes, v_scales
        if _fast is None:
            load()
        self.shape = _fast.cache(k_codes, k_scales, v_codes, v_scales)
        if self.shape is None:             # say which of them does not fit
            for name, part in zip(("k_codes", "k_scales", "v_codes", "v_scales"), self._parts()):
                _need_tensor(part, name)
            if k_codes.dim() != 4 or k_codes.shape[3] not in (32, 48, 64):
                raise ValueError("k_codes must be [B, Hkv, Lmax, D/2] with D 64, 96 or 128, "
                                 "got %s" % (tuple(k_codes.shape),))
            self.shape = tuple(k_codes.shape[:3]) + (2 * k_codes.shape[3],)
            _pointers(k_codes.device, self._spec())
        self.device = k_codes.device

    @classmethod
    def zeros(cls, B, Hkv, Lmax, D, device="cuda"):
        codes = [torch.zeros(B, Hkv, Lmax, D // 2, dtype=torch.uint8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros(B, Hkv, Lmax, D // 32, 2, dtype=torch.bfloat16, device=device)
                  for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1])

    def _parts(self):
        return self.k_codes, self.k_scales, self.v_codes, self.v_scales

    def _spec(self):
        """The cache's part of a call's tensors, for _pointers."""
        B, Hkv, Lmax, D = self.shape
        codes, scales = (B, Hkv, Lmax, D // 2), (B, Hkv, Lmax, D // 32, 2)
        return ("k_codes", self.k_codes, torch.uint8, codes,
                "k_scales", self.k_scales, torch.bfloat16, scales,
                "v_codes", self.v_codes, torch.uint8, codes,
                "v_scales", self.v_scales, torch.bfloat16, scales)


SIGNATURES = {
    "gqa_rope_apply": (_i, [_vp, _vp, _i, _i, _i, _i, RopeParams, _vp]),
    "kv_cache_append": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i,
                             RopeParams, _vp, _vp]),
    "gqa_rope_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _i,
                             RopeParams, _vp, _vp]),
    "gqa_prefill": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "gqa_prefill_chunk": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f,
                               _vp, _vp]),
    "gqa_doc_start": (_i, [_vp, _vp, _i, _i, _vp, _vp]),
    "gqa_prefill_lse": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "gqa_attention_backward": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                    _i, _i, _f, _vp, _sz, _vp, _vp]),
    "gqa_backward_workspace_bytes": (_sz, [_i, _i, _i]),
    "gqa_prefill_docs": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "gqa_decode": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _f, _vp, _sz,
                        _vp, _vp]),
    "gqa_decode_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "gqa_decode_noalloc": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "gqa_norm_rope_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i,
                                  _i, _i, RopeParams, ctypes.POINTER(RopeInputs), _vp, _vp]),
    "gqa_norm_rope_append_backward": (_i, [_vp] * 11 + [_i] * 7 + [
        RopeParams, ctypes.POINTER(RopeInputs), _vp, _sz, _vp, _vp]),
    "gqa_norm_rope_backward_workspace_bytes": (_sz, [_i]),
    "gqa_norm_rope_append_q4": (_i, [_vp] * 10 + [_i, _vp, _i, _i, _i, _i, _i, _i, RopeParams,
                                                  ctypes.POINTER(RopeInputs), _vp, _vp]),
    "kv_cache_read_q4": (_i, [_vp] * 8 + [_i, _i, _i, _i, _i, _vp, _vp]),
    "gqa_decode_q4": (_i, [_vp] * 6 + [_i, _vp, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp, _vp]),
    "gqa_decode_q4_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "gqa_selftest_bounded_wait": (_i, [_vp, _i, _vp]),
    "gqa_status_string": (ctypes.c_char_p, [_i]),
    "gqa_version": (_i, []),
}


class GqaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (fn, status_string(status), status))


def load(path: str | None = None):
    """Load libgqa.so (raises if it is missing: there is no fallback)."""
    global _lib, _fast, _fast_pointers
    if _lib is None:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                "libgqa.so not found at %s; build it with `python -m rope_gqa_kv_b200.build`" % p)
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        fast = _native_checks(lib)
        _fast, _fast_pointers = fast, fast.pointers
        _lib = lib
    return _lib


def _native_checks(lib):
    """csrc/fastargs.c, or, where it is not built or this torch lacks the interface it
    reads tensors through, functions that leave every call to the checks in Python."""
    try:
        from . import _fastargs
        _fastargs.setup(torch.Tensor.__dlpack_c_exchange_api__, (
            (torch.bfloat16, 4, 16), (torch.int32, 0, 32), (torch.uint8, 1, 8),
            (torch.float32, 2, 32)))
        _fastargs.entries(tuple(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "gqa_norm_rope_append", "gqa_norm_rope_append_q4", "gqa_norm_rope_append_backward",
            "kv_cache_read_q4", "gqa_decode_q4")))
        return _fastargs
    except (ImportError, AttributeError, RuntimeError, TypeError, ValueError) as e:
        warnings.warn("arguments are checked in Python, some 10 us a call slower: %s" % e,
                      RuntimeWarning, stacklevel=3)
        def none(*args):
            return None
        return types.SimpleNamespace(append=none, backward=none, read_back=none, decode=none,
                                     cache=none, pointers=none)


def status_string(status: int) -> str:
    return load().gqa_status_string(status).decode()


def _check(fn: str, st: int):
    if st != GQA_OK:
        raise GqaError(fn, st)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got %s" % (name, ndim, tuple(t.shape)))


def _pointers(dev, spec):
    """Data pointers of a call's tensors (0 for None) and, last, dev's current stream.

    spec = (name, tensor, dtype, shape, name, tensor, ...): every tensor must be a
    contiguous CUDA tensor on dev of that dtype and shape (None: any shape of at least
    one element).  csrc/fastargs.c says whether they are; what it does not accept is
    looked at here, one by one, to be refused by name."""
    if dev.type != "cuda":
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % spec[0])
    if _fast_pointers is None:
        load()
    ptrs = _fast_pointers(dev.index, spec)
    if ptrs is not None:
        return ptrs
    ptrs = []
    for i in range(0, len(spec), 4):
        name, t, dtype, shape = spec[i:i + 4]
        if t is None:
            ptrs.append(0)
            continue
        _need(t, name, dtype)
        if shape is not None and t.shape != tuple(shape):
            raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if t.numel() < 1:
            raise ValueError("%s is empty" % name)
        if t.device != dev:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
        ptrs.append(t.data_ptr())
    ptrs.append(torch.cuda.current_stream(dev).cuda_stream)
    return ptrs


def _new(stream, make):
    """make(), allocated for use on `stream` (default: the current one)."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _launch(name, dev, stream, current, *args):
    """Calls the library on device `dev`, whichever is current, with the stream (by
    default the handle `current`, dev's current one) as the last argument."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError("the stream is on %s, the tensors are on %s" % (stream.device, dev))
        current = stream.cuda_stream
    fn = getattr(_lib, name)
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, current)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, current)
    if st != GQA_OK:
        raise GqaError(name, st)


def _current(t):
    """The current device for a whole call in C; -1 (no device's) where t is not on one."""
    return torch.cuda.current_device() if isinstance(t, torch.Tensor) and t.is_cuda else -1


def _stream_handle(stream, t):
    """The handle for a whole call in C: None for the current stream, or, for a stream of
    another device than tensor t's, what sends the call to the checks in Python."""
    if stream is None:
        return None
    same = isinstance(t, torch.Tensor) and stream.device == t.device
    return stream.cuda_stream if same else "another device"


def _need_tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)


def _pos_shape(pos, axes, B, T, D):
    """The shape that pos must have."""
    if axes is not None and len(axes.pairs) != D // 2:
        raise ValueError("axes cover %d rotation pairs, D = %d has %d" %
                         (len(axes.pairs), D, D // 2))
    _need_tensor(pos, "pos")
    n = 1 if axes is None else axes.n_axes
    if pos.dim() != 2:
        return (n, B, T)
    if T == 1 and (n > 1 or pos.shape[0] == 1):
        return (n, B)
    return (B, T) if n == 1 else (n, B, T)


def _rope_spec(B, T, D, q_gain, k_gain, pos, axes, qk_norm):
    """Gains and positions as the last three tensors of a call's spec."""
    if axes is not None and pos is None:
        raise ValueError("axes need pos, the positions on every axis")
    if not qk_norm and (q_gain is not None or k_gain is not None):
        raise ValueError("q_gain and k_gain need qk_norm=True")
    gain = (D,)
    return ("q_gain", q_gain, torch.bfloat16, gain, "k_gain", k_gain, torch.bfloat16, gain,
            "pos", pos, torch.int32,
            None if pos is None else _pos_shape(pos, axes, B, T, D))


_ONE_AXIS = bytes(RopeInputs(n_axes=1))


def _rope_inputs(q_gain, k_gain, pos, axes):
    """The gqa_rope_inputs of these pointers, or None where nothing of it is used."""
    if not (q_gain or k_gain or pos):
        return None
    x = RopeInputs.from_buffer_copy(_ONE_AXIS if axes is None else axes._inputs)
    x.q_gain, x.k_gain, x.pos = q_gain, k_gain, pos
    return x


@functools.lru_cache(maxsize=64)       # of plain numbers: nothing is kept by an object's identity
def _plain_params(qk_norm, eps, rope_base):
    return RopeParams(qk_norm, eps, rope_base)


@functools.lru_cache(maxsize=64)
def _plain_params_bytes(qk_norm, eps, rope_base):
    return bytes(_plain_params(qk_norm, eps, rope_base))


def _params_bytes(qk_norm, eps, rope_base, scaling):
    if scaling is None:
        return _plain_params_bytes(1 if qk_norm else 0, float(eps), float(rope_base))
    return bytes(_params(qk_norm, eps, rope_base, scaling))


def _params(qk_norm, eps, rope_base, scaling=None):
    if scaling is None:                # passed by value: calls share the structure
        return _plain_params(1 if qk_norm else 0, float(eps), float(rope_base))
    return RopeParams(1 if qk_norm else 0, float(eps), float(rope_base), ROPE_KINDS[scaling.kind],
                      scaling.factor, scaling.original_max_pos, scaling.alpha, scaling.beta)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def gqa_rope_apply(q, pos0=None, qk_norm=False, eps=1e-6, rope_base=10000.0, stream=None,
                   scaling=None):
    """In place: q [B, T, H, D] <- RoPE(RMSNorm?(q)) at positions pos0[b] + t."""
    _need(q, "q", torch.bfloat16, 4)
    if pos0 is not None:
        _need(pos0, "pos0", torch.int32, 1)
    B, T, H, D = q.shape
    _check("gqa_rope_apply", load().gqa_rope_apply(
        _ptr(q), _ptr(pos0), B, T, H, D, _params(qk_norm, eps, rope_base, scaling),
        _stream(stream)))
    return q


def kv_cache_append(k, v, k_cache, v_cache, pos0=None, max_pos0=-1, new_len=None,
                    qk_norm=False, eps=1e-6, rope_base=10000.0, status=None, stream=None,
                    scaling=None):
    """Write RoPE(RMSNorm?(k)) and v of the new tokens [B, T, Hkv, D] into the caches."""
    _need(k, "k", torch.bfloat16, 4)
    _need(v, "v", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    B, T, Hkv, D = k.shape
    if v.shape != k.shape or k_cache.shape != v_cache.shape or k_cache.shape[0] != B or \
            k_cache.shape[1] != Hkv or k_cache.shape[3] != D:
        raise ValueError("k/v/cache shapes disagree")
    for name, t in (("pos0", pos0), ("new_len", new_len), ("status", status)):
        if t is not None:
            _need(t, name, torch.int32)
    _check("kv_cache_append", load().kv_cache_append(
        _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos0), int(max_pos0),
        _ptr(new_len), B, T, Hkv, D, k_cache.shape[2], _params(qk_norm, eps, rope_base, scaling),
        _ptr(status), _stream(stream)))


def gqa_rope_append(q, k, v, k_cache, v_cache, pos0=None, max_pos0=-1, new_len=None,
                    qk_norm=False, eps=1e-6, rope_base=10000.0, status=None, stream=None,
                    scaling=None):
    """gqa_rope_apply on q and kv_cache_append of k, v in one launch."""
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16)
    _need(v, "v", torch.bfloat16)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    if q.dim() == 3:            # decode layout [B, H, D] == [B, 1, H, D]
        q4, k4 = q.unsqueeze(1), k.unsqueeze(1)
    else:
        q4, k4 = q, k
    B, T, Hq, D = q4.shape
    Hkv = k4.shape[2]
    if k4.shape != (B, T, Hkv, D) or v.numel() != k.numel() or k_cache.shape[0] != B or \
            k_cache.shape[1] != Hkv or k_cache.shape[3] != D or v_cache.shape != k_cache.shape:
        raise ValueError("q/k/v/cache shapes disagree")
    for name, t in (("pos0", pos0), ("new_len", new_len), ("status", status)):
        if t is not None:
            _need(t, name, torch.int32)
    _check("gqa_rope_append", load().gqa_rope_append(
        _ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(pos0), int(max_pos0),
        _ptr(new_len), B, T, Hq, Hkv, D, k_cache.shape[2], _params(qk_norm, eps, rope_base, scaling),
        _ptr(status), _stream(stream)))


def gqa_prefill(q, k_cache, v_cache, out=None, scale=0.0, status=None, stream=None):
    """Causal GQA attention of a prompt from position 0: q [B, T, Hq, D] -> out."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    B, T, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Lmax, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape disagrees with q")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_prefill", load().gqa_prefill(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), B, T, Hq, Hkv, D, Lmax,
        float(scale), _ptr(status), _stream(stream)))
    return out


def gqa_prefill_chunk(q, k_cache, v_cache, pos0, max_pos0, n_tok=None, out=None, scale=0.0,
                      status=None, stream=None):
    """Causal attention of T new tokens per sequence continuing a cached prefix:
    query t of sequence b sits at position pos0[b] + t.  q [B, T, Hq, D] -> out;
    rows t >= n_tok[b] of out are left as they were."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(pos0, "pos0", torch.int32, 1)
    B, T, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Lmax, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape disagrees with q")
    if pos0.shape != (B,):
        raise ValueError("pos0 must be [B]")
    if n_tok is not None:
        _need(n_tok, "n_tok", torch.int32, 1)
        if n_tok.shape != (B,):
            raise ValueError("n_tok must be [B]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_prefill_chunk", load().gqa_prefill_chunk(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(pos0), _ptr(n_tok),
        int(max_pos0), B, T, Hq, Hkv, D, Lmax, float(scale), _ptr(status), _stream(stream)))
    return out


def gqa_prefill_lse(q, k_cache, v_cache, out=None, lse=None, scale=0.0, status=None,
                    stream=None):
    """gqa_prefill that also returns each row's log-sum-exp: (out, lse) with
    lse float32 [B, Hq, round_up(T, 4)] (the padding columns are not written)."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    B, T, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Lmax, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape disagrees with q")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, (T + 3) // 4 * 4, dtype=torch.float32, device=q.device)
    _need(out, "out", torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    if lse.shape != (B, Hq, (T + 3) // 4 * 4):
        raise ValueError("lse must be [B, Hq, round_up(T, 4)]")
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_prefill_lse", load().gqa_prefill_lse(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), B, T, Hq, Hkv, D, Lmax,
        float(scale), _ptr(status), _stream(stream)))
    return out, lse


def gqa_backward_workspace_bytes(B, T, Hq):
    return int(load().gqa_backward_workspace_bytes(B, T, Hq))


def gqa_attention_backward(q, k, v, out, dout, lse, dq=None, dk=None, dv=None, scale=0.0,
                           workspace=None, status=None, stream=None):
    """Gradients (dq, dk, dv) of causal GQA attention.  q, out, dout [B, T, Hq, D];
    k, v [B, Hkv, Lmax, D] (cache layout, slots < T used); lse from gqa_prefill_lse."""
    for name, t in (("q", q), ("out", out), ("dout", dout)):
        _need(t, name, torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4)
    _need(v, "v", torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    B, T, Hq, D = q.shape
    Hkv, Lmax = k.shape[1], k.shape[2]
    if k.shape != (B, Hkv, Lmax, D) or v.shape != k.shape or out.shape != q.shape or \
            dout.shape != q.shape:
        raise ValueError("q/k/v/out/dout shapes disagree")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.zeros_like(k) if dk is None else dk
    dv = torch.zeros_like(v) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, torch.bfloat16, 4)
    if workspace is None:
        workspace = torch.empty(max(gqa_backward_workspace_bytes(B, T, Hq), 16), dtype=torch.uint8,
                                device=q.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_attention_backward", load().gqa_attention_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
        B, T, Hq, Hkv, D, Lmax, float(scale), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)))
    return dq, dk, dv


def gqa_doc_start(doc_id, out=None, status=None, stream=None):
    """First position of each token's document, from non-decreasing per-token
    document ids doc_id [B, T] (int32)."""
    _need(doc_id, "doc_id", torch.int32, 2)
    B, T = doc_id.shape
    if out is None:
        out = torch.empty_like(doc_id)
    _need(out, "out", torch.int32, 2)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_doc_start", load().gqa_doc_start(_ptr(doc_id), _ptr(out), B, T, _ptr(status),
                                                 _stream(stream)))
    return out


def gqa_prefill_docs(q, k_cache, v_cache, doc_start, out=None, scale=0.0, status=None,
                     stream=None):
    """Causal attention of a prompt of packed documents: query t sees keys
    doc_start[b, t] .. t.  q [B, T, Hq, D] -> out."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(doc_start, "doc_start", torch.int32, 2)
    B, T, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Lmax, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape disagrees with q")
    if doc_start.shape != (B, T):
        raise ValueError("doc_start must be [B, T]")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_prefill_docs", load().gqa_prefill_docs(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(doc_start), B, T, Hq, Hkv, D, Lmax,
        float(scale), _ptr(status), _stream(stream)))
    return out


def gqa_decode_workspace_bytes(B, Hq, D, max_len):
    return int(load().gqa_decode_workspace_bytes(B, Hq, D, max_len))


def decode_workspace(B, Hq, D, max_len, device):
    """Scratch for gqa_decode; one workspace serves any number of calls that do
    not run at the same time."""
    need = gqa_decode_workspace_bytes(B, Hq, D, max_len)
    return torch.empty(max(need, 16), dtype=torch.uint8, device=device)


def gqa_decode(q, k_cache, v_cache, lens, max_len, out=None, workspace=None, scale=0.0,
               status=None, stream=None):
    """One query token per sequence: q [B, Hq, D] against lens[b] cached keys."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(lens, "lens", torch.int32, 1)
    B, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Lmax, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape disagrees with q")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    need = gqa_decode_workspace_bytes(B, Hq, D, max_len)
    if workspace is None:
        workspace = decode_workspace(B, Hq, D, max_len, q.device)
    _need(workspace, "workspace", torch.uint8)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_decode", load().gqa_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lens), int(max_len), _ptr(out), B, Hq, Hkv,
        D, Lmax, float(scale), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)))
    return out


def gqa_decode_noalloc(q, k_cache, v_cache, lens, max_len, out=None, scale=0.0, status=None,
                       stream=None):
    """gqa_decode with its scratch in the library's fixed device array (no
    workspace argument); for callers that cannot allocate device memory."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(lens, "lens", torch.int32, 1)
    B, Hq, D = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape != (B, Hkv, Lmax, D) or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape disagrees with q")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if status is not None:
        _need(status, "status", torch.int32)
    _check("gqa_decode_noalloc", load().gqa_decode_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(lens), int(max_len), _ptr(out), B, Hq, Hkv,
        D, Lmax, float(scale), _ptr(status), _stream(stream)))
    return out


def _norm_rope_append(name, q, k, v, cache, cache_names, pos0, n_tok, max_pos0, new_len,
                      q_out, q_gain, k_gain, pos, axes, qk_norm, eps, rope_base, scaling, status,
                      stream):
    """cache: the four tensors of a Q4Cache, or K's and V's and two Nones."""
    if _fast is None:
        load()
    if q is not None and q_out is None:
        _need_tensor(q, "q")
        q_out = _new(stream, lambda: torch.empty_like(q))
    st = _fast.append(
        cache[2] is not None, _current(k), q, k, v, q_out, *cache, pos0, n_tok,
        new_len, status, q_gain, k_gain, pos, max_pos0,
        _params_bytes(qk_norm, eps, rope_base, scaling), None if axes is None else axes._inputs,
        0 if axes is None else len(axes.pairs), _stream_handle(stream, k))
    if st is not None:
        if st != GQA_OK:
            raise GqaError(name, st)
        return q_out
    cache_spec, cache_shape = cache_names()
    _need_tensor(k, "k")
    ks = k.shape
    if len(ks) == 4:
        B, T, Hkv, D = ks
    elif len(ks) == 3:                     # decode layout [B, H, D]
        B, Hkv, D = ks
        T = 1
    else:
        raise ValueError("k must be [B, T, Hkv, D] or [B, Hkv, D], got %s" % (tuple(ks),))
    if cache_shape[0] != B or cache_shape[1] != Hkv or cache_shape[3] != D:
        raise ValueError("the cache's shape %s disagrees with k" % (tuple(cache_shape),))
    Hq, qs = 0, None
    if q is not None:
        _need_tensor(q, "q")
        if q.dim() != len(ks):
            raise ValueError("q and k must have the same number of dims")
        Hq = q.shape[-2]
        qs = (B, T, Hq, D) if len(ks) == 4 else (B, Hq, D)
    elif q_out is not None:
        raise ValueError("q_out without q")
    bf, i32, each = torch.bfloat16, torch.int32, (B,)
    dev = k.device
    p = _pointers(dev, ("k", k, bf, ks, "v", v, bf, ks, "q", q, bf, qs, "q_out", q_out, bf, qs,
                        "pos0", pos0, i32, each, "n_tok", n_tok, i32, each,
                        "new_len", new_len, i32, each, "status", status, i32, None) +
                  _rope_spec(B, T, D, q_gain, k_gain, pos, axes, qk_norm) + cache_spec)
    _launch(name, dev, stream, p[-1], p[2], p[0], p[1], p[3], *p[11:-1], p[4], p[5],
            int(max_pos0), p[6], B, T, Hq, Hkv, D, cache_shape[2],
            _params(qk_norm, eps, rope_base, scaling), _rope_inputs(p[8], p[9], p[10], axes),
            p[7])
    return q_out


def gqa_norm_rope_append(q, k, v, k_cache, v_cache, pos0=None, n_tok=None, max_pos0=-1,
                         new_len=None, q_out=None, q_gain=None, k_gain=None, pos=None, axes=None,
                         qk_norm=True, eps=1e-6, rope_base=10000.0, scaling=None, status=None,
                         stream=None):
    """RMSNorm with learned gains (bf16 [D]), rotation by pos (int32 [n_axes, B, T], with
    axes a RopeAxes; default pos0[b] + t) and the append of k, v, in one launch.  q, k, v
    [B, T, H, D] or [B, H, D]; q may be None.  Tokens t >= n_tok[b] are left out.
    Returns q_out (a new tensor unless given; it may be q)."""
    def spec():
        _need_tensor(k_cache, "k_cache")
        cs = k_cache.shape
        if len(cs) != 4:
            raise ValueError("k_cache must be [B, Hkv, Lmax, D], got %s" % (tuple(cs),))
        if v_cache is None:
            raise TypeError("v_cache must be a torch.Tensor")
        return ("k_cache", k_cache, torch.bfloat16, cs, "v_cache", v_cache, torch.bfloat16, cs), cs

    return _norm_rope_append("gqa_norm_rope_append", q, k, v, (k_cache, v_cache, None, None), spec,
                             pos0, n_tok, max_pos0, new_len, q_out, q_gain, k_gain, pos, axes,
                             qk_norm, eps, rope_base, scaling, status, stream)


def gqa_norm_rope_append_q4(q, k, v, cache, pos0=None, n_tok=None, max_pos0=-1, new_len=None,
                            q_out=None, q_gain=None, k_gain=None, pos=None, axes=None,
                            qk_norm=True, eps=1e-6, rope_base=10000.0, scaling=None, status=None,
                            stream=None):
    """gqa_norm_rope_append into a 4-bit cache (a Q4Cache)."""
    _need_q4(cache)
    return _norm_rope_append("gqa_norm_rope_append_q4", q, k, v, cache._parts(),
                             lambda: (cache._spec(), cache.shape), pos0, n_tok, max_pos0, new_len,
                             q_out, q_gain, k_gain, pos, axes, qk_norm, eps, rope_base, scaling,
                             status, stream)


def _need_q4(cache):
    if not isinstance(cache, Q4Cache):
        raise TypeError("cache must be a Q4Cache, got %s" % type(cache).__name__)


def gqa_norm_rope_backward_workspace_bytes(D):
    return int(load().gqa_norm_rope_backward_workspace_bytes(D))


def norm_rope_backward_workspace(D, device):
    """Scratch for gqa_norm_rope_append_backward; one serves any number of calls that do
    not run at the same time (two captured graphs that may overlap need one each)."""
    need = gqa_norm_rope_backward_workspace_bytes(D)
    return torch.empty(max(need, 16), dtype=torch.uint8, device=device)


def gqa_norm_rope_append_backward(q, k, dq_out, dk_cache, dv_cache, pos0=None, max_pos0=-1,
                                  dq=None, dk=None, dv=None, q_gain=None, k_gain=None, pos=None,
                                  axes=None, qk_norm=True, eps=1e-6, rope_base=10000.0,
                                  scaling=None, workspace=None, status=None, stream=None):
    """Gradients (dq, dk, dv, dq_gain, dk_gain) of gqa_norm_rope_append: q, k its inputs,
    dq_out [B, T, Hq, D] and dk_cache, dv_cache [B, Hkv, Lmax, D] those of its outputs
    (slots pos0[b] .. pos0[b] + T - 1 are read).  dq_gain, dk_gain are float32 [D], or
    None without qk_norm."""
    name = "gqa_norm_rope_append_backward"
    _need_tensor(q, "q")
    _need_tensor(k, "k")
    dev = q.device
    if _fast is None:
        load()
    dq = _new(stream, lambda: torch.empty_like(q)) if dq is None else dq
    dk = _new(stream, lambda: torch.empty_like(k)) if dk is None else dk
    dv = _new(stream, lambda: torch.empty_like(k)) if dv is None else dv
    both = None
    if qk_norm and dev.type == "cuda":
        both = _new(stream, lambda: torch.empty(2, q.shape[-1], dtype=torch.float32, device=dev))
        if workspace is None:
            workspace = _new(stream, lambda: norm_rope_backward_workspace(q.shape[-1], dev))
    dg = (None, None) if both is None else both.unbind(0)
    st = _fast.backward(
        _current(q), q, k, dq_out, dk_cache, dv_cache, dq, dk, dv, both, pos0, workspace, status,
        q_gain, k_gain, pos, max_pos0,
        _params_bytes(qk_norm, eps, rope_base, scaling), None if axes is None else axes._inputs,
        0 if axes is None else len(axes.pairs), _stream_handle(stream, q))
    if st is not None:
        if st != GQA_OK:
            raise GqaError(name, st)
        return dq, dk, dv, dg[0], dg[1]
    for name, t in (("q", q), ("k", k), ("dk_cache", dk_cache)):
        _need_tensor(t, name)
        if t.dim() != 4:
            raise ValueError("%s must have 4 dims, got %s" % (name, tuple(t.shape)))
    qs = q.shape
    B, T, Hq, D = qs
    Hkv, Lmax = k.shape[2], dk_cache.shape[2]
    ks, cs = (B, T, Hkv, D), (B, Hkv, Lmax, D)
    if dq_out is None or dv_cache is None:
        raise TypeError("dq_out and dv_cache must be tensors")
    bf = torch.bfloat16
    rope = _rope_spec(B, T, D, q_gain, k_gain, pos, axes, qk_norm)
    ws_bytes = 0
    if workspace is not None:
        _need_tensor(workspace, "workspace")
        ws_bytes = workspace.numel()
    p = _pointers(dev, ("q", q, bf, qs, "k", k, bf, ks, "dq_out", dq_out, bf, qs,
                        "dk_cache", dk_cache, bf, cs, "dv_cache", dv_cache, bf, cs,
                        "dq", dq, bf, qs, "dk", dk, bf, ks, "dv", dv, bf, ks,
                        "dq_gain", dg[0], torch.float32, (D,),
                        "dk_gain", dg[1], torch.float32, (D,),
                        "pos0", pos0, torch.int32, (B,),
                        "workspace", workspace, torch.uint8, None,
                        "status", status, torch.int32, None) + rope)
    _launch("gqa_norm_rope_append_backward", dev, stream, p[-1], *p[:11], int(max_pos0), B, T, Hq,
            Hkv, D, Lmax, _params(qk_norm, eps, rope_base, scaling),
            _rope_inputs(p[13], p[14], p[15], axes), p[11], ws_bytes, p[12])
    return dq, dk, dv, dg[0], dg[1]


def kv_cache_read_q4(cache, k_out=None, v_out=None, first=None, count=None, status=None,
                     stream=None):
    """Slots first[b] .. of a Q4Cache as bf16 rows: count[b] of them (default: all Lout)
    into k_out, v_out [B, Hkv, Lout, D], by default new zeros as long as the cache.
    Returns (k_out, v_out)."""
    _need_q4(cache)
    B, Hkv, Lmax, D = cache.shape
    dev = cache.device
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        k_out, v_out = (_new(stream, lambda: torch.zeros(B, Hkv, Lmax, D, dtype=torch.bfloat16,
                                                         device=dev)) for _ in range(2))
    st = _fast.read_back(_current(k_out), cache.k_codes, cache.k_scales, cache.v_codes,
                    cache.v_scales, first, count, k_out, v_out, status,
                    _stream_handle(stream, k_out))
    if st is not None:
        if st != GQA_OK:
            raise GqaError("kv_cache_read_q4", st)
        return k_out, v_out
    _need_tensor(k_out, "k_out")
    if k_out.dim() != 4:
        raise ValueError("k_out must be [B, Hkv, Lout, D], got %s" % (tuple(k_out.shape),))
    Lout = k_out.shape[2]
    shape, bf, i32 = (B, Hkv, Lout, D), torch.bfloat16, torch.int32
    p = _pointers(dev, cache._spec() + ("first", first, i32, (B,), "count", count, i32, (B,),
                                        "k_out", k_out, bf, shape, "v_out", v_out, bf, shape,
                                        "status", status, i32, None))
    _launch("kv_cache_read_q4", dev, stream, p[-1], *p[:8], B, Hkv, D, Lmax, Lout, p[8])
    return k_out, v_out


def gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, max_len):
    return int(load().gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, max_len))


def decode_q4_workspace(B, Hq, Hkv, D, max_len, device):
    """Scratch for gqa_decode_q4; one workspace serves any number of calls that do not
    run at the same time."""
    need = gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, max_len)
    return torch.empty(max(need, 16), dtype=torch.uint8, device=device)


def gqa_decode_q4(q, cache, lens, max_len, out=None, workspace=None, scale=0.0, status=None,
                  stream=None):
    """One query token per sequence against a 4-bit cache: q [B, Hq, D], lens[b] cached
    tokens of a Q4Cache, the new one included."""
    _need_q4(cache)
    _need_tensor(q, "q")
    _need_tensor(lens, "lens")
    B, Hkv, Lmax, D = cache.shape
    dev = cache.device
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D], got %s" % (tuple(q.shape),))
    Hq = q.shape[1]
    shape = (B, Hq, D)
    if out is None:
        out = _new(stream, lambda: torch.empty_like(q))
    if workspace is None:
        workspace = _new(stream, lambda: decode_q4_workspace(B, Hq, Hkv, D, max_len, dev))
    st = _fast.decode(_current(q), cache.k_codes, cache.k_scales, cache.v_codes,
                      cache.v_scales, q, lens, max_len, out, float(scale), workspace, status,
                      _stream_handle(stream, q))
    if st is not None:
        if st != GQA_OK:
            raise GqaError("gqa_decode_q4", st)
        return out
    _need_tensor(workspace, "workspace")
    bf = torch.bfloat16
    p = _pointers(dev, ("q", q, bf, shape) + cache._spec() +
                  ("lens", lens, torch.int32, (B,), "out", out, bf, shape,
                   "workspace", workspace, torch.uint8, None,
                   "status", status, torch.int32, None))
    _launch("gqa_decode_q4", dev, stream, p[-1], *p[:6], int(max_len), p[6], B, Hq, Hkv, D, Lmax,
            float(scale), p[7], workspace.numel(), p[8])
    return out
