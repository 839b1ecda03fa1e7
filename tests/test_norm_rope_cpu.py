"""What needs no GPU of the learned-norm append and the 4-bit cache: the float64 forms
the GPU tests compare with, and every refusal of the C entries and of the binding."""
import ctypes
import math
import sys

import pytest
import torch

import rope_gqa_kv_b200 as gqa
from rope_gqa_kv_b200 import _lib
from rope_gqa_kv_b200 import build as gqa_build

import norm_rope_reference as ref


@pytest.fixture(scope="module")
def lib():
    gqa_build.build()
    return gqa.load()


# ---------------------------------------------------------------------------
# the float64 forms
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,axes", [(64, 1), (96, 3), (128, 4)])
def test_gradient_formula_against_autograd_and_differences(D, axes):
    g = torch.Generator().manual_seed(D)
    B, T, H = 2, 3, 2
    x = torch.randn(B, T, H, D, generator=g, dtype=ref.F64)
    gain = 1 + 0.3 * torch.randn(D, generator=g, dtype=ref.F64)
    dy = torch.randn(B, T, H, D, generator=g, dtype=ref.F64)
    pos = torch.randint(-50, 50, (axes, B, T), generator=g)
    P = ref.positions(None, B, T, pos, torch.arange(D // 2) % axes, D)
    dx, dg = ref.norm_rope_grad(x, dy, P, gain)
    xa, ga = x.clone().requires_grad_(True), gain.clone().requires_grad_(True)
    (ref.norm_rope(xa, P, ga) * dy).sum().backward()
    # float64, sums of D (dx) and B T H (d gain) terms of order one
    assert (dx - xa.grad).abs().max() < 1e-12 and (dg - ga.grad).abs().max() < 1e-12
    u, ug = torch.randn_like(x), torch.randn_like(gain)
    h = 1e-5                           # the difference is off by h^2 and by 1e-16 / h
    f = lambda t: (ref.norm_rope(x + t * u, P, gain + t * ug) * dy).sum()
    want = (dx * u).sum() + (dg * ug).sum()
    assert abs((f(h) - f(-h)) / (2 * h) - want) < 1e-7


@pytest.mark.parametrize("D", [64, 96, 128])
def test_row_layout_is_a_permutation_and_values_are_within_half_a_step(D):
    assert sorted(ref.byte_of_pair(D).tolist()) == list(range(D // 2))
    assert sorted(ref.group_index(D).flatten().tolist()) == list(range(D))
    x = torch.randn(200, D, generator=torch.Generator().manual_seed(D)).to(torch.bfloat16)
    codes, scales = ref.pack(x)
    step = scales[..., 0].double()[:, (torch.arange(D) % (D // 2)) // 16]
    assert ((ref.values(codes, scales) - x.double()).abs() <= step / 2).all()
    c, _, _, _ = ref.quantise(x)
    assert c.min() == 0 and c.max() == 15
    assert torch.equal(ref.unpack_codes(codes), c)


def test_quantiser_ties_constants_and_values_that_are_not_finite():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    x[0, 0], x[0, 1:15] = 15.0, torch.arange(1, 15) - 0.5      # n + 1/2 goes to n
    x[1] = -3.25
    x[2, 5], x[2, 20] = math.nan, 1.0
    x[3, 40] = math.inf                # coordinate 40 = 32 + 8: group 0
    c, s, m, _ = ref.quantise(x)
    assert c[0, :15].tolist() == [15] + list(range(14))
    assert s[1].tolist() == [0.0, 0.0] and m[1].tolist() == [-3.25, -3.25]
    assert math.isnan(m[2, 0]) and s[2, 0] == 0 and m[2, 1] == 0.0
    assert math.isnan(m[3, 0]) and m[3, 1] == 0.0


# ---------------------------------------------------------------------------
# refusals of the C entries (pointers that are never followed)
# ---------------------------------------------------------------------------
F = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)             # not 16-byte aligned
ODD4 = ctypes.c_void_p(0x10002)            # not 4-byte aligned
NEXT = ctypes.c_void_p(0x10004)            # one int32 on
NORM = _lib.RopeParams(1, 1e-6, 10000.0)
PLAIN = _lib.RopeParams(0, 1e-6, 10000.0)


def _append_args(q4, **over):
    d = dict(q=F, k=F, v=F, q_out=F, c0=F, c1=F, c2=F, c3=F, pos0=None, n_tok=None, max_pos0=0,
             new_len=None, B=1, T=16, Hq=4, Hkv=2, D=64, L=128, p=NORM, x=None)
    d.update(over)
    caches = [d["c0"], d["c1"]] + ([d["c2"], d["c3"]] if q4 else [])
    return [d["q"], d["k"], d["v"], d["q_out"]] + caches + [
        d[n] for n in ("pos0", "n_tok", "max_pos0", "new_len", "B", "T", "Hq", "Hkv", "D", "L",
                       "p", "x")] + [None, None]


def _inputs(**kw):
    x = _lib.RopeInputs(kw.get("q_gain"), kw.get("k_gain"), kw.get("pos"), kw.get("n_axes", 1))
    for i, a in enumerate(kw.get("pair_axis", ())):
        x.pair_axis[i] = a
    return x


APPEND_REFUSED = [
    (1, dict(k=None)), (1, dict(v=None)), (1, dict(q_out=None)), (1, dict(c0=None)),
    (1, dict(c1=ODD)), (1, dict(q=ODD)), (1, dict(k=ODD)), (1, dict(q_out=ODD)),
    (1, dict(pos0=ODD4)), (1, dict(n_tok=ODD4)), (1, dict(new_len=ODD4)),
    (1, dict(B=0)), (1, dict(T=0)), (1, dict(Hq=0)), (1, dict(Hkv=0)), (1, dict(Hq=3)),
    (1, dict(L=100)), (1, dict(L=0)), (2, dict(D=80)), (2, dict(D=0)),
    (3, dict(T=129)), (3, dict(max_pos0=113)), (3, dict(n_tok=F, max_pos0=129)),
    (1, dict(pos0=F, new_len=F)), (1, dict(n_tok=F, new_len=F)),
    (1, dict(pos0=F, new_len=NEXT, B=2)), (1, dict(n_tok=NEXT, new_len=F, B=2)),
    (1, dict(p=_lib.RopeParams(1, -1.0, 10000.0))), (1, dict(p=_lib.RopeParams(1, 1e-6, 1.0))),
    (1, dict(p=PLAIN, x=_inputs(q_gain=0x10000))), (1, dict(p=PLAIN, x=_inputs(k_gain=0x10000))),
    (1, dict(x=_inputs(q_gain=0x10008))), (1, dict(x=_inputs(pos=0x10002))),
    (1, dict(x=_inputs(pos=0x10000, n_axes=0))), (1, dict(x=_inputs(pos=0x10000, n_axes=5))),
    (1, dict(x=_inputs(pos=0x10000, n_axes=2, pair_axis=[0, 2]))),
    (1, dict(B=1 << 16, T=1 << 16, L=1 << 16)), (1, dict(Hq=1 << 30, Hkv=1 << 29)),
]


@pytest.mark.parametrize("want,over", APPEND_REFUSED)
def test_append_refusals(lib, want, over):
    assert lib.gqa_norm_rope_append(*_append_args(False, **over)) == want
    assert lib.gqa_norm_rope_append_q4(*_append_args(True, **over)) == want


def test_append_q4_refuses_each_missing_or_misaligned_cache_part(lib):
    for name in ("c0", "c1", "c2", "c3"):
        for bad in (None, ODD):
            assert lib.gqa_norm_rope_append_q4(*_append_args(True, **{name: bad})) == 1


@pytest.mark.parametrize("want,over", [
    (1, {i: None}) for i in range(8)] + [(1, {i: ODD}) for i in range(8)] + [
    (1, dict(gain=ODD4)), (1, dict(pos0=ODD4)), (1, dict(p=PLAIN)), (1, dict(Hq=3)),
    (2, dict(D=48)), (1, dict(L=130)), (3, dict(T=129)), (3, dict(max_pos0=113)),
    (6, dict(ws=None)), (6, dict(ws=ODD)), (6, dict(ws_bytes=100)),
    (1, dict(x=_inputs(pos=0x10000, n_axes=2, pair_axis=[3])))])
def test_append_backward_refusals(lib, want, over):
    d = dict(gain=F, pos0=None, max_pos0=0, B=1, T=16, Hq=4, Hkv=2, D=64, L=128, p=NORM, x=None,
             ws=F, ws_bytes=1 << 20)
    d.update(over)
    data = [d.get(i, F) for i in range(8)]
    args = data + [d["gain"], None] + [d[n] for n in ("pos0", "max_pos0", "B", "T", "Hq", "Hkv",
                                                      "D", "L", "p", "x", "ws", "ws_bytes")]
    assert lib.gqa_norm_rope_append_backward(*args, None, None) == want


@pytest.mark.parametrize("want,over", [
    (1, dict(k0=None)), (1, dict(k0=ODD)), (1, dict(out=ODD)), (1, dict(first=ODD4)),
    (1, dict(count=ODD4)), (1, dict(B=0)), (1, dict(B=70000)), (1, dict(Hkv=0)),
    (2, dict(D=32)), (1, dict(L=64)), (1, dict(Lout=0)), (3, dict(Lout=129))])
def test_read_refusals(lib, want, over):
    d = dict(k0=F, out=F, first=None, count=None, B=1, Hkv=2, D=64, L=128, Lout=100)
    d.update(over)
    assert lib.kv_cache_read_q4(d["k0"], F, F, F, d["first"], d["count"], F, d["out"], d["B"],
                                d["Hkv"], d["D"], d["L"], d["Lout"], None, None) == want


@pytest.mark.parametrize("want,over", [
    (1, dict(q=None)), (1, dict(q=ODD)), (1, dict(c=ODD)), (1, dict(lens=None)),
    (1, dict(lens=ODD4)), (1, dict(Hq=5)), (1, dict(B=70000)), (2, dict(D=72)),
    (1, dict(L=200)), (1, dict(n=0)), (3, dict(n=4097)), (6, dict(ws=None)),
    (6, dict(ws=None, n=1)), (6, dict(ws=None, n=300)), (6, dict(ws_bytes=15, n=300)),
    (6, dict(ws_bytes=16, n=5000, L=8192)), (6, dict(ws=ODD))])
def test_decode_q4_refusals(lib, want, over):
    d = dict(q=F, c=F, lens=F, n=4000, Hq=4, B=1, D=64, L=4096, ws=F, ws_bytes=1 << 24)
    d.update(over)
    assert lib.gqa_decode_q4(d["q"], d["c"], F, F, F, d["lens"], d["n"], F, d["B"], d["Hq"], 2,
                             d["D"], d["L"], 0.0, d["ws"], d["ws_bytes"], None, None) == want


def test_workspace_sizes(lib):
    assert lib.gqa_norm_rope_backward_workspace_bytes(80) == 0
    assert lib.gqa_norm_rope_backward_workspace_bytes(128) >= 2 * 128 * 4
    f = lib.gqa_decode_q4_workspace_bytes
    assert f(0, 4, 2, 64, 100) == 0 and f(1, 5, 2, 64, 100) == 0 and f(1, 4, 2, 80, 100) == 0
    assert f(1, 4, 2, 64, 0) == 0
    assert f(1, 4, 2, 64, 1) == 16             # one chunk: no partials
    assert f(1, 4, 2, 64, 1000) == 16          # few, short rows: merged on the chip
    # whatever the cut: one to max_len / 64 rows of D + 2 floats per query head
    row = 64 * 24 * 130 * 4
    assert 2 * row <= f(64, 24, 8, 128, 2049) <= 33 * row + 16
    # few rows: a chunk for each place, but one for each of the other sequences
    assert f(4, 24, 8, 128, 65536) == 4 * 24 * (148 * 3 // 8 - 3) * 130 * 4
    assert f(1, 1, 1, 64, 4160) == 65 * 66 * 4 + 8          # (m, l) up to a 16-byte boundary


@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (1, 8, 8), (4, 24, 8), (6, 24, 8), (8, 24, 8),
                                      (16, 16, 2), (33, 8, 8), (64, 24, 8), (100, 4, 1),
                                      (125, 8, 8), (600, 32, 4)])
def test_a_workspace_of_the_capacity_serves_every_shorter_call(lib, B, Hq, Hkv):
    """Allocated once for the longest call, used for all: the size never falls with max_len."""
    f = lambda n: lib.gqa_decode_q4_workspace_bytes(B, Hq, Hkv, 128, n)
    sizes = [f(n) for n in list(range(1, 6000)) + list(range(6000, 140000, 61))]
    assert sizes == sorted(sizes)


# ---------------------------------------------------------------------------
# refusals of the binding (host tensors; device ones are refused in the GPU tests)
# ---------------------------------------------------------------------------
def test_rope_axes_refuses_what_is_not_a_layout():
    ok = gqa.RopeAxes((16, 24, 24))
    assert ok.n_axes == 3 and len(ok.pairs) == 64 and ok.pairs[15:17] == (0, 1)
    assert gqa.RopeAxes(pairs=[0, 1] * 16).n_axes == 2
    for bad in (dict(), dict(sections=(1,), pairs=(0,)), dict(sections=(0, 32)),
                dict(sections=(60, 5)), dict(sections=()), dict(pairs=()),
                dict(pairs=[0, 4]), dict(pairs=[-1, 0]), dict(pairs=[0, 2]),
                dict(sections=(1, 1, 1, 1, 1))):
        with pytest.raises(ValueError):
            gqa.RopeAxes(**bad)


def test_host_tensors_are_refused():
    bf = torch.bfloat16
    x, kc = torch.zeros(1, 4, 2, 64, dtype=bf), torch.zeros(1, 2, 128, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        gqa.gqa_norm_rope_append(x, x, x, kc, kc.clone())
    with pytest.raises(ValueError, match="CUDA"):
        gqa.gqa_norm_rope_append_backward(x, x, x, kc, kc)
    with pytest.raises(ValueError, match="CUDA"):
        gqa.Q4Cache.zeros(1, 2, 128, 64, device="cpu")
    for call in (lambda: gqa.gqa_norm_rope_append_q4(x, x, x, kc),
                 lambda: gqa.kv_cache_read_q4(kc),
                 lambda: gqa.gqa_decode_q4(x[0], kc, None, 1)):
        with pytest.raises(TypeError, match="Q4Cache"):
            call()


def test_gains_need_the_norm_and_axes_need_positions():
    with pytest.raises(ValueError, match="qk_norm"):
        _lib._rope_spec(1, 1, 64, torch.ones(64), None, None, None, False)
    with pytest.raises(ValueError, match="pos"):
        _lib._rope_spec(1, 1, 64, None, None, None, gqa.RopeAxes((32,)), True)


def test_native_argument_checks_leave_host_tensors_to_the_slow_path(lib):
    from rope_gqa_kv_b200 import _fastargs
    t = torch.zeros(2, 3)
    assert _fastargs.pointers(0, ("t", t, torch.float32, (2, 3))) is None
    assert _fastargs.pointers(0, ("t", "text", torch.float32, (2, 3))) is None
    for bad in ((0,), (0, ("t", t)), ("x", ()), (0, ["t", t, None, None])):
        with pytest.raises(TypeError):
            _fastargs.pointers(*bad)


def test_parameters_follow_a_value_that_changes_in_place():
    """eps and rope_base may be anything float() takes; none is kept by its identity."""
    eps = torch.tensor(1e-6)
    first = _lib._params_bytes(True, eps, 1e4, None)
    eps.fill_(0.5)
    assert _lib._params_bytes(True, eps, 1e4, None) != first
    assert _lib._params(True, eps, 1e4).eps == 0.5


@pytest.mark.parametrize("over", [
    dict(T=1, x=_inputs(pos=0x10000)), dict(T=1, B=2, x=_inputs(pos=0x10004)),
    dict(T=1, B=2, x=_inputs(pos=0x10000 - 4)), dict(x=_inputs(pos=0x10000 - 60)),
    dict(T=1, B=4, x=_inputs(pos=0x10000 - 44, n_axes=3, pair_axis=[0, 1, 2]))])
def test_append_refuses_new_lengths_written_over_positions(lib, over):
    """new_len (B words at F) is written while other warps still read pos (n_axes B T)."""
    assert lib.gqa_norm_rope_append(*_append_args(False, **dict(over, new_len=F))) == 1
    assert lib.gqa_norm_rope_append_q4(*_append_args(True, **dict(over, new_len=F))) == 1


# ---------------------------------------------------------------------------
# without the native argument checks
# ---------------------------------------------------------------------------
def _not_built(monkeypatch):
    monkeypatch.delattr(gqa, "_fastargs", raising=False)
    monkeypatch.setitem(sys.modules, "rope_gqa_kv_b200._fastargs", None)


def _torch_without_the_table(monkeypatch):
    from rope_gqa_kv_b200 import _fastargs  # noqa: F401  (it imports; torch is what lacks it)
    monkeypatch.setattr(_lib, "torch", _TorchWithout())


class _TorchWithout:
    """torch, but for Tensor.__dlpack_c_exchange_api__."""
    Tensor = type("Tensor", (), {})

    def __getattr__(self, name):
        return getattr(torch, name)


def _another_version(monkeypatch):
    from rope_gqa_kv_b200 import _fastargs

    def setup(*args):
        raise RuntimeError("torch's DLPack exchange table is of another version")
    monkeypatch.setattr(_fastargs, "setup", setup)


@pytest.mark.parametrize("lacking", [_not_built, _torch_without_the_table, _another_version])
def test_every_entry_works_without_the_native_checks(lib, monkeypatch, lacking):
    """The library loads, and calls go through the checks in Python."""
    for name in ("_lib", "_fast", "_fast_pointers"):
        monkeypatch.setattr(_lib, name, None)
    with monkeypatch.context() as m:
        lacking(m)
        with pytest.warns(RuntimeWarning, match="checked in Python"):
            other = gqa.load()
    assert gqa.load() is other
    assert other.gqa_prefill(None, F, F, F, 1, 16, 4, 2, 64, 128, 0.0, None, None) == 1
    assert gqa.gqa_decode_workspace_bytes(1, 3, 64, 64) == 3 * 66 * 4
    for call in (_lib._fast.append, _lib._fast.backward, _lib._fast.read_back, _lib._fast.decode,
                 _lib._fast.cache, _lib._fast_pointers):
        assert call(0, None) is None
    with pytest.raises(ValueError, match="CUDA"):
        gqa.Q4Cache.zeros(1, 2, 128, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        _lib._pointers(torch.device("cuda", 0), ("t", torch.zeros(2), torch.float32, (2,)))


def test_native_checks_are_built_again_for_another_torch_and_may_fail(monkeypatch, tmp_path):
    lib_path, made_for = tmp_path / "_fastargs.so", tmp_path / "fastargs.txt"
    monkeypatch.setattr(gqa_build, "ARGS_LIB", str(lib_path))
    monkeypatch.setattr(gqa_build, "ARGS_FOR", str(made_for))
    gqa_build._build_args(False)
    first = lib_path.stat().st_mtime_ns
    gqa_build._build_args(False)
    assert lib_path.stat().st_mtime_ns == first
    made_for.write_text("python 3, torch 1\n")
    gqa_build._build_args(False)
    assert lib_path.stat().st_mtime_ns > first and torch.__version__ in made_for.read_text()
    monkeypatch.setattr(gqa_build.shutil, "which", lambda name: "/bin/false")
    gqa_build._build_args(False)               # nothing to do
    with pytest.warns(RuntimeWarning, match="checked in Python"):
        gqa_build._build_args(True)
    assert not lib_path.exists()               # the library goes on without it


@pytest.mark.skipif(torch.cuda.is_available(), reason="the call goes on to its launch")
@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - (1 << 21), (1 << 31) - 128])
def test_decode_q4_takes_the_longest_caches(lib, n):
    """A cache of 2^31 slots of one head of 64 fits the device: chunk counts do not pass 2^31
    on the way.  Without a device an accepted call fails at its launch (5)."""
    size = lib.gqa_decode_q4_workspace_bytes(1, 2, 1, 64, n)
    assert size >= 1184 * 2 * 66 * 4
    for ws_bytes, want in ((size, 5), (16, 6)):
        assert lib.gqa_decode_q4(F, F, F, F, F, F, n, F, 1, 2, 1, 64, (1 << 31) - 128, 0.0, F,
                                 ws_bytes, None, None) == want
