"""The generation loop's decode step captured in CUDA graphs and replayed per token.

A decode step is three launches: the fused QK-norm / RoPE / append of the new
token (``gqa_rope_append``), then the split decode over the cache and its merge
(``gqa_decode``).  At small batch each runs for a few microseconds, so issuing
them one by one from the host costs more than running them; the KV-cache loop
of page "750美元从零训练3个LLM：一位开发者的实战复盘" (section "V3：扩容与推理优化":
a prompt followed by 100 generated tokens, each token attending to the cached
keys and values) is then launch-bound.  Here the step is captured once, with
every buffer fixed: the new token's q, k and v, the output, the decode
workspace and a status word.  The per-sequence cache lengths ping-pong between
two device vectors -- the append reads one as the new token's position and
writes the other (length + 1), which the decode then reads -- so two graphs,
one for each direction, cover every step, and no host value changes between
replays.  The decode's grid covers ``max_len`` cache slots (default: the whole
capacity); the CTAs past a sequence's current length exit at once.  With a 4-bit
cache, learned gains or several position axes the append is
``gqa_norm_rope_append`` or ``gqa_norm_rope_append_q4``, and a 4-bit cache is read
by ``gqa_decode_q4``.
"""
from __future__ import annotations

import torch

from . import _lib


class DecodeGraph:
    """Replays one decode step per call of :meth:`step`.

    Write the new token's projections into ``q`` [B, Hq, D], ``k`` and ``v``
    [B, Hkv, D] (bfloat16), call :meth:`step`, and read ``out`` [B, Hq, D].
    ``lens`` (int32 [B], on the cache's device) are the cached lengths before
    the first step; :attr:`lens` is the current length vector.  The caches are
    updated in place, exactly as by the eager calls.  Device errors are OR-ed
    into ``status``.

    ``k_cache`` may be a ``Q4Cache`` (``v_cache`` is then None).  ``q_gain`` and
    ``k_gain`` (bfloat16 [D]) are learned gains of the norm; they are read at every
    step.  With ``axes`` (a ``RopeAxes``), write the new token's position on every
    axis into ``pos`` (int32 [n_axes, B]) before each step; without, it is the
    cached length.

    ``max_len`` bounds the lengths that the steps reach (default: the capacity).
    The decode is cut into chunks by it, so a bound near the lengths is faster: 16
    sequences of 2000 tokens on a 4-bit cache of 32768 take 20.6 us a step with 2048
    and 28.7 without.
    """

    def __init__(self, k_cache, v_cache, lens, Hq, max_len=None, qk_norm=False, eps=1e-6,
                 rope_base=10000.0, scaling=None, scale=0.0, q_gain=None, k_gain=None,
                 axes=None):
        q4 = isinstance(k_cache, _lib.Q4Cache)
        if q4 and v_cache is not None:
            raise ValueError("a Q4Cache holds K and V: v_cache must be None")
        if not q4 and not (isinstance(k_cache, torch.Tensor) and k_cache.is_cuda):
            raise ValueError("k_cache must be a CUDA tensor (no CPU path exists)")
        B, Hkv, Lmax, D = k_cache.shape
        dev = k_cache.device
        self.max_len = Lmax if max_len is None else int(max_len)
        bf = torch.bfloat16
        self.q = torch.zeros(B, Hq, D, dtype=bf, device=dev)
        self.k = torch.zeros(B, Hkv, D, dtype=bf, device=dev)
        self.v = torch.zeros(B, Hkv, D, dtype=bf, device=dev)
        self.out = torch.zeros(B, Hq, D, dtype=bf, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._lens = [lens.to(device=dev, dtype=torch.int32).clone(),
                      lens.to(device=dev, dtype=torch.int32).clone()]
        self.pos = None if axes is None else torch.zeros(axes.n_axes, B, dtype=torch.int32,
                                                         device=dev)
        rope = dict(qk_norm=qk_norm, eps=eps, rope_base=rope_base, scaling=scaling)
        learned = dict(q_gain=q_gain, k_gain=k_gain, pos=self.pos, axes=axes)
        q_rot = torch.empty_like(self.q)        # the learned-norm appends leave q as it is
        # The graphs hold addresses only: what they read and write stays alive with them.
        self._held = (k_cache, v_cache, q_gain, k_gain, q_rot)
        if q4:
            self._workspace = _lib.decode_q4_workspace(B, Hq, Hkv, D, self.max_len, dev)
        else:
            self._workspace = _lib.decode_workspace(B, Hq, D, self.max_len, dev)

        def one_step(a, b):
            args = dict(pos0=self._lens[a], new_len=self._lens[b], status=self.status, **rope)
            tail = dict(out=self.out, workspace=self._workspace, scale=scale, status=self.status)
            if q4:
                _lib.gqa_norm_rope_append_q4(self.q, self.k, self.v, k_cache, q_out=q_rot,
                                             **learned, **args)
                _lib.gqa_decode_q4(q_rot, k_cache, self._lens[b], self.max_len, **tail)
                return
            if q_gain is None and k_gain is None and axes is None:
                _lib.gqa_rope_append(self.q, self.k, self.v, k_cache, v_cache, **args)
                _lib.gqa_decode(self.q, k_cache, v_cache, self._lens[b], self.max_len, **tail)
                return
            _lib.gqa_norm_rope_append(self.q, self.k, self.v, k_cache, v_cache, q_out=q_rot,
                                      **learned, **args)
            _lib.gqa_decode(q_rot, k_cache, v_cache, self._lens[b], self.max_len, **tail)

        # A capture takes what is launched on its stream, by default one of the device that
        # was current at the process's first capture: with the caches on another one the
        # launches would go by the graph.
        self._device = dev
        with torch.cuda.device(dev):
            # One eager step first, on a side stream, so that every first-use setup
            # (kernel attributes, the library load) happens outside the capture.  It
            # writes only the cache slot at each sequence's current length -- the
            # slot the first real step overwrites -- and the second length vector.
            side = torch.cuda.Stream(device=dev)
            side.wait_stream(torch.cuda.current_stream(dev))
            with torch.cuda.stream(side):
                one_step(0, 1)
            torch.cuda.current_stream(dev).wait_stream(side)
            torch.cuda.synchronize(dev)
            self.status.zero_()
            self._graphs = []
            for a, b in ((0, 1), (1, 0)):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    one_step(a, b)
                self._graphs.append(g)
        self._cur = 0           # index of the length vector that holds the current lengths

    @property
    def lens(self) -> torch.Tensor:
        return self._lens[self._cur]

    def step(self) -> torch.Tensor:
        """Append the token in q, k, v at the current lengths and decode it."""
        if torch.cuda.current_device() == self._device.index:
            self._graphs[self._cur].replay()
        else:
            with torch.cuda.device(self._device):
                self._graphs[self._cur].replay()
        self._cur ^= 1
        return self.out
