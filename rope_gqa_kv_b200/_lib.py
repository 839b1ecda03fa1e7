"""ctypes binding of libgqa.so: argument marshalling only.

Every function here takes torch CUDA tensors, checks dtype / shape / device /
contiguity on the host, and passes raw device pointers, sizes and the current
CUDA stream to the C ABI declared in include/gqa.h.  All arithmetic happens in
the library's CUDA kernels; there is no CPU or PyTorch fallback, and a missing
library or a CPU tensor raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgqa.so")
_lib = None

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
        self._array = (ctypes.c_uint8 * 64)(*self.pairs)


class Q4Cache:
    """A KV cache held in 4 bits (layout in gqa.h): codes uint8 [B, Hkv, Lmax, D/2] and
    scales bf16 [B, Hkv, Lmax, D/32, 2] of K and of V.  :meth:`zeros` makes one."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        _need(k_codes, "k_codes", torch.uint8, 4)
        B, Hkv, Lmax, half = k_codes.shape
        self.device, self.shape = k_codes.device, (B, Hkv, Lmax, 2 * half)
        if half not in (32, 48, 64):
            raise ValueError("k_codes must be [B, Hkv, Lmax, D/2] with D 64, 96 or 128")
        scales = (B, Hkv, Lmax, half // 16, 2)
        _exact(k_scales, "k_scales", torch.bfloat16, scales, self.device)
        _exact(v_codes, "v_codes", torch.uint8, k_codes.shape, self.device)
        _exact(v_scales, "v_scales", torch.bfloat16, scales, self.device)
        self.k_codes, self.k_scales = k_codes, k_scales
        self.v_codes, self.v_scales = v_codes, v_scales

    @classmethod
    def zeros(cls, B, Hkv, Lmax, D, device="cuda"):
        codes = [torch.zeros(B, Hkv, Lmax, D // 2, dtype=torch.uint8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros(B, Hkv, Lmax, D // 32, 2, dtype=torch.bfloat16, device=device)
                  for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1])

    def _ptrs(self):
        return _ptr(self.k_codes), _ptr(self.k_scales), _ptr(self.v_codes), _ptr(self.v_scales)


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
    global _lib
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
        _lib = lib
    return _lib


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


def _exact(t, name, dtype, shape, dev):
    """_need, plus the exact shape and the device of the call's first tensor."""
    _need(t, name, dtype)
    if t.shape != tuple(shape):
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))


def _optional(t, name, dtype, shape, dev):
    if t is not None:
        _exact(t, name, dtype, shape, dev)


def _status_word(status, dev):
    if status is not None:
        _need(status, "status", torch.int32)
        if status.numel() < 1 or status.device != dev:
            raise ValueError("status must be an int32 word on %s" % dev)


def _new(stream, make):
    """make(), allocated for use on `stream` (default: the current one)."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _launch(name, dev, stream, *args):
    """Calls the library on device `dev`, whichever is current, with the stream (the
    device's current one by default) as the last argument."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif stream.device != dev:
        raise ValueError("the stream is on %s, the tensors are on %s" % (stream.device, dev))
    fn = getattr(load(), name)
    if torch.cuda.current_device() == dev.index:
        _check(name, fn(*args, ctypes.c_void_p(stream.cuda_stream)))
    else:
        with torch.cuda.device(dev):
            _check(name, fn(*args, ctypes.c_void_p(stream.cuda_stream)))


def _rope_inputs(B, T, D, q_gain, k_gain, pos, axes, qk_norm, dev):
    """The gqa_rope_inputs of a call, or None where nothing of it is used."""
    if axes is not None and pos is None:
        raise ValueError("axes need pos, the positions on every axis")
    if q_gain is None and k_gain is None and pos is None:
        return None
    if (q_gain is not None or k_gain is not None) and not qk_norm:
        raise ValueError("q_gain and k_gain need qk_norm=True")
    _optional(q_gain, "q_gain", torch.bfloat16, (D,), dev)
    _optional(k_gain, "k_gain", torch.bfloat16, (D,), dev)
    x = RopeInputs(_ptr(q_gain), _ptr(k_gain), _ptr(pos))
    if pos is not None:
        n = 1 if axes is None else axes.n_axes
        if axes is not None and len(axes.pairs) != D // 2:
            raise ValueError("axes cover %d rotation pairs, D = %d has %d" %
                             (len(axes.pairs), D, D // 2))
        _need(pos, "pos", torch.int32)
        shapes = [(n, B, T)] + ([(n, B)] if T == 1 else []) + ([(B, T)] if n == 1 else [])
        if tuple(pos.shape) not in shapes:
            raise ValueError("pos must be [n_axes, B, T] = %s, got %s" %
                             ((n, B, T), tuple(pos.shape)))
        if pos.device != dev:
            raise ValueError("pos is on %s, expected %s" % (pos.device, dev))
        x.n_axes = n
        if axes is not None:
            x.pair_axis = axes._array
    return x


def _params(qk_norm, eps, rope_base, scaling=None):
    if scaling is None:
        return RopeParams(1 if qk_norm else 0, float(eps), float(rope_base))
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


def _append_shapes(q, k, v, cache_shape):
    """(B, T, Hq, Hkv, D, device) of an append's new tokens; q may be None, T may be
    left out of the shapes (the decode layout)."""
    _need(k, "k", torch.bfloat16)
    if k.dim() not in (3, 4):
        raise ValueError("k must be [B, T, Hkv, D] or [B, Hkv, D], got %s" % (tuple(k.shape),))
    B, Hkv, D = k.shape[0], k.shape[-2], k.shape[-1]
    T = k.shape[1] if k.dim() == 4 else 1
    _exact(v, "v", torch.bfloat16, k.shape, k.device)
    Hq = 0
    if q is not None:
        _need(q, "q", torch.bfloat16, k.dim())
        Hq = q.shape[-2]
        _exact(q, "q", torch.bfloat16, k.shape[:-2] + (Hq, D), k.device)
    if cache_shape[:2] != (B, Hkv) or cache_shape[3] != D:
        raise ValueError("the cache's shape %s disagrees with k" % (tuple(cache_shape),))
    return B, T, Hq, Hkv, D, k.device


def _norm_rope_append(name, q, k, v, caches, cache_shape, pos0, n_tok, max_pos0, new_len, q_out,
                      q_gain, k_gain, pos, axes, qk_norm, eps, rope_base, scaling, status, stream):
    B, T, Hq, Hkv, D, dev = _append_shapes(q, k, v, cache_shape)
    for what, t in (("pos0", pos0), ("n_tok", n_tok), ("new_len", new_len)):
        _optional(t, what, torch.int32, (B,), dev)
    _status_word(status, dev)
    x = _rope_inputs(B, T, D, q_gain, k_gain, pos, axes, qk_norm, dev)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    elif q_out is None:
        q_out = _new(stream, lambda: torch.empty_like(q))
    else:
        _exact(q_out, "q_out", torch.bfloat16, q.shape, dev)
    _launch(name, dev, stream, _ptr(q), _ptr(k), _ptr(v), _ptr(q_out), *caches, _ptr(pos0),
            _ptr(n_tok), int(max_pos0), _ptr(new_len), B, T, Hq, Hkv, D, cache_shape[2],
            _params(qk_norm, eps, rope_base, scaling), x, _ptr(status))
    return q_out


def gqa_norm_rope_append(q, k, v, k_cache, v_cache, pos0=None, n_tok=None, max_pos0=-1,
                         new_len=None, q_out=None, q_gain=None, k_gain=None, pos=None, axes=None,
                         qk_norm=True, eps=1e-6, rope_base=10000.0, scaling=None, status=None,
                         stream=None):
    """RMSNorm with learned gains (bf16 [D]), rotation by pos (int32 [n_axes, B, T], with
    axes a RopeAxes; default pos0[b] + t) and the append of k, v, in one launch.  q, k, v
    [B, T, H, D] or [B, H, D]; q may be None.  Tokens t >= n_tok[b] are left out.
    Returns q_out (a new tensor unless given; it may be q)."""
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _exact(v_cache, "v_cache", torch.bfloat16, k_cache.shape, k_cache.device)
    if isinstance(k, torch.Tensor) and k.device != k_cache.device:
        raise ValueError("k_cache is on %s, expected %s" % (k_cache.device, k.device))
    return _norm_rope_append("gqa_norm_rope_append", q, k, v, (_ptr(k_cache), _ptr(v_cache)),
                             k_cache.shape, pos0, n_tok, max_pos0, new_len, q_out, q_gain, k_gain,
                             pos, axes, qk_norm, eps, rope_base, scaling, status, stream)


def gqa_norm_rope_append_q4(q, k, v, cache, pos0=None, n_tok=None, max_pos0=-1, new_len=None,
                            q_out=None, q_gain=None, k_gain=None, pos=None, axes=None,
                            qk_norm=True, eps=1e-6, rope_base=10000.0, scaling=None, status=None,
                            stream=None):
    """gqa_norm_rope_append into a 4-bit cache (a Q4Cache)."""
    _need_q4(cache)
    if isinstance(k, torch.Tensor) and k.device != cache.device:
        raise ValueError("the cache is on %s, expected %s" % (cache.device, k.device))
    return _norm_rope_append("gqa_norm_rope_append_q4", q, k, v, cache._ptrs(), cache.shape, pos0,
                             n_tok, max_pos0, new_len, q_out, q_gain, k_gain, pos, axes, qk_norm,
                             eps, rope_base, scaling, status, stream)


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
    _need(q, "q", torch.bfloat16, 4)
    dev = q.device
    B, T, Hq, D = q.shape
    _need(k, "k", torch.bfloat16, 4)
    Hkv = k.shape[2]
    _exact(k, "k", torch.bfloat16, (B, T, Hkv, D), dev)
    _exact(dq_out, "dq_out", torch.bfloat16, q.shape, dev)
    _need(dk_cache, "dk_cache", torch.bfloat16, 4)
    Lmax = dk_cache.shape[2]
    _exact(dk_cache, "dk_cache", torch.bfloat16, (B, Hkv, Lmax, D), dev)
    _exact(dv_cache, "dv_cache", torch.bfloat16, (B, Hkv, Lmax, D), dev)
    _optional(pos0, "pos0", torch.int32, (B,), dev)
    _status_word(status, dev)
    x = _rope_inputs(B, T, D, q_gain, k_gain, pos, axes, qk_norm, dev)
    grads = [dq, dk, dv]
    for i, (what, like) in enumerate((("dq", q), ("dk", k), ("dv", k))):
        if grads[i] is None:
            grads[i] = _new(stream, lambda: torch.empty_like(like))
        else:
            _exact(grads[i], what, torch.bfloat16, like.shape, dev)
    dg, ws_bytes = (None, None), 0
    if qk_norm:
        dg = _new(stream, lambda: torch.empty(2, D, dtype=torch.float32, device=dev)).unbind(0)
        if workspace is None:
            workspace = _new(stream, lambda: norm_rope_backward_workspace(D, dev))
        _need(workspace, "workspace", torch.uint8)
        if workspace.device != dev:
            raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
        ws_bytes = workspace.numel()
    _launch("gqa_norm_rope_append_backward", dev, stream, _ptr(q), _ptr(k), _ptr(dq_out),
            _ptr(dk_cache), _ptr(dv_cache), _ptr(grads[0]), _ptr(grads[1]), _ptr(grads[2]),
            _ptr(dg[0]), _ptr(dg[1]), _ptr(pos0), int(max_pos0), B, T, Hq, Hkv, D, Lmax,
            _params(qk_norm, eps, rope_base, scaling), x, _ptr(workspace), ws_bytes,
            _ptr(status))
    return grads[0], grads[1], grads[2], dg[0], dg[1]


def kv_cache_read_q4(cache, k_out=None, v_out=None, first=None, count=None, status=None,
                     stream=None):
    """Slots first[b] .. of a Q4Cache as bf16 rows: count[b] of them (default: all Lout)
    into k_out, v_out [B, Hkv, Lout, D], by default new zeros as long as the cache.
    Returns (k_out, v_out)."""
    _need_q4(cache)
    B, Hkv, Lmax, D = cache.shape
    dev = cache.device
    for what, t in (("first", first), ("count", count)):
        _optional(t, what, torch.int32, (B,), dev)
    _status_word(status, dev)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        k_out, v_out = (_new(stream, lambda: torch.zeros(B, Hkv, Lmax, D, dtype=torch.bfloat16,
                                                         device=dev)) for _ in range(2))
    _need(k_out, "k_out", torch.bfloat16, 4)
    Lout = k_out.shape[2]
    _exact(k_out, "k_out", torch.bfloat16, (B, Hkv, Lout, D), dev)
    _exact(v_out, "v_out", torch.bfloat16, (B, Hkv, Lout, D), dev)
    _launch("kv_cache_read_q4", dev, stream, *cache._ptrs(), _ptr(first), _ptr(count),
            _ptr(k_out), _ptr(v_out), B, Hkv, D, Lmax, Lout, _ptr(status))
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
    B, Hkv, Lmax, D = cache.shape
    dev = cache.device
    _need(q, "q", torch.bfloat16, 3)
    Hq = q.shape[1]
    _exact(q, "q", torch.bfloat16, (B, Hq, D), dev)
    _exact(lens, "lens", torch.int32, (B,), dev)
    _status_word(status, dev)
    if out is None:
        out = _new(stream, lambda: torch.empty_like(q))
    _exact(out, "out", torch.bfloat16, q.shape, dev)
    if workspace is None:
        workspace = _new(stream, lambda: decode_q4_workspace(B, Hq, Hkv, D, max_len, dev))
    _need(workspace, "workspace", torch.uint8)
    if workspace.device != dev:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
    _launch("gqa_decode_q4", dev, stream, _ptr(q), *cache._ptrs(), _ptr(lens), int(max_len),
            _ptr(out), B, Hq, Hkv, D, Lmax, float(scale), _ptr(workspace), workspace.numel(),
            _ptr(status))
    return out
