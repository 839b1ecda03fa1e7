"""GPU parity of the learned-norm append (gains, several position axes, ragged token
counts) and of its backward, against float64.

Tolerances.  A rotated element is computed in fp32 from exact bf16 inputs -- a norm, two
products and a sum, fp32 sines of angles reduced in float64: some tens of fp32 units of
the magnitude |a| + |b| of its pair -- and rounded once to bf16: half a step, 2^-8 of the
value.  A gradient element likewise, with the magnitudes of its two terms.
"""
from types import SimpleNamespace

import pytest
import torch

import rope_gqa_kv_b200 as gqa

import norm_rope_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FP32_UNITS = 64 * 2.0 ** -24       # see above: "some tens"


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


def _assert_rounded(got, want, mag, what):
    """|got - want| <= 2^-8 |want| + FP32_UNITS mag, got a bf16 tensor."""
    d = (got.detach().cpu().double() - want).abs()
    allow = 2.0 ** -8 * want.abs() * (1 + FP32_UNITS) + FP32_UNITS * mag + 2.0 ** -133
    assert (d <= allow).all(), "%s: %d of %d off, worst %.3g of the bound" % (
        what, int((d > allow).sum()), d.numel(), float((d / allow).max()))


def _pair_mag(x):
    """|a| + |b| of every element's pair."""
    a, b = x.abs().chunk(2, dim=-1)
    return torch.cat((a + b, a + b), dim=-1)


def _case(seed, B, T, Hq, Hkv, D, L, n_axes=1, gains=True, far=False):
    g = torch.Generator().manual_seed(seed)
    c = dict(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, L=L)
    c["q"] = (2 * torch.randn(B, T, Hq, D, generator=g)).to(BF)
    c["k"] = torch.randn(B, T, Hkv, D, generator=g).to(BF)
    c["v"] = torch.randn(B, T, Hkv, D, generator=g).to(BF)
    c["kc"] = torch.randn(B, Hkv, L, D, generator=g).to(BF)
    c["vc"] = torch.randn(B, Hkv, L, D, generator=g).to(BF)
    c["q_gain"] = (1 + 0.5 * torch.randn(D, generator=g)).to(BF) if gains else None
    c["k_gain"] = (1 + 0.5 * torch.randn(D, generator=g)).to(BF) if gains else None
    c["pos0"] = torch.randint(0, L - T + 1, (B,), generator=g).to(torch.int32)
    if n_axes:
        lo, hi = (-(2 ** 31), 2 ** 31 - 1) if far else (0, 300)
        c["pos"] = torch.randint(lo, hi, (n_axes, B, T), generator=g).to(torch.int32)
        c["pair_axis"] = torch.randint(0, n_axes, (D // 2,), generator=g)
        c["pair_axis"][:n_axes] = torch.arange(n_axes)
        c["axes"] = gqa.RopeAxes(pairs=c["pair_axis"].tolist())
    else:
        c["pos"] = c["pair_axis"] = c["axes"] = None
    return c


def _dev(t):
    return None if t is None else t.to(DEV)


def _rope_kw(c, qk_norm=True):
    return dict(q_gain=_dev(c["q_gain"]), k_gain=_dev(c["k_gain"]), pos=_dev(c["pos"]),
                axes=c["axes"], qk_norm=qk_norm)


def _want(c, name, qk_norm=True):
    P = ref.positions(c["pos0"], c["B"], c["T"], c["pos"], c["pair_axis"], c["D"])
    y = ref.norm_rope(c[name], P, c[name + "_gain"], qk_norm)
    return y, _pair_mag(y)


def _check_append(c, q_out, kc, vc, qk_norm=True, n_tok=None, q_before=None):
    want_q, mag_q = _want(c, "q", qk_norm)
    want_k, mag_k = _want(c, "k", qk_norm)
    n_tok = [c["T"]] * c["B"] if n_tok is None else n_tok
    for b in range(c["B"]):
        p, n = int(c["pos0"][b]), n_tok[b]
        _assert_rounded(q_out[b, :n], want_q[b, :n], mag_q[b, :n], "q[%d]" % b)
        _assert_rounded(kc[b, :, p:p + n].transpose(0, 1), want_k[b, :n], mag_k[b, :n],
                        "k_cache[%d]" % b)
        assert torch.equal(_bits(vc[b, :, p:p + n].transpose(0, 1)), _bits(c["v"][b, :n]))
        keep = torch.ones(c["L"], dtype=torch.bool)
        keep[p:p + n] = False
        for got, was in ((kc, c["kc"]), (vc, c["vc"])):
            assert torch.equal(_bits(got[b].cpu()[:, keep]), _bits(was[b][:, keep]))
        if q_before is not None:
            assert torch.equal(_bits(q_out[b, n:]), _bits(q_before[b, n:]))


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv,n_axes", [
    (1, 1, 1, 1, 1), (3, 37, 6, 2, 3), (2, 5, 7, 1, 4), (64, 1, 24, 8, 3), (5, 1, 3, 3, 0),
    (2, 131, 8, 8, 2), (1, 700, 5, 5, 3)])
def test_append_against_float64(cuda_lib, D, B, T, Hq, Hkv, n_axes):
    c = _case(D + T, B, T, Hq, Hkv, D, 768, n_axes)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new_len = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    q = _dev(c["q"])
    q_out = gqa.gqa_norm_rope_append(q, _dev(c["k"]), _dev(c["v"]), kc, vc, pos0=_dev(c["pos0"]),
                                     new_len=new_len, status=status, **_rope_kw(c))
    torch.cuda.synchronize()
    assert status.item() == 0
    assert torch.equal(_bits(q), _bits(c["q"]))
    assert new_len.tolist() == (c["pos0"] + T).tolist()
    _check_append(c, q_out, kc, vc)


@pytest.mark.parametrize("qk_norm,gains", [(False, False), (True, False), (True, True)])
def test_far_and_negative_positions(cuda_lib, qk_norm, gains):
    c = _case(9, 2, 6, 4, 2, 128, 128, 3, gains, far=True)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    q_out = gqa.gqa_norm_rope_append(_dev(c["q"]), _dev(c["k"]), _dev(c["v"]), kc, vc,
                                     pos0=_dev(c["pos0"]), **_rope_kw(c, qk_norm))
    # an angle of 2^31 radians is known to 2^31 2^-53 and its product with 1 / 2 pi and
    # back to three times that: 3e-7 of the pair
    want, mag = _want(c, "q", qk_norm)
    _assert_rounded(q_out, want, mag * 2, "q")
    want, mag = _want(c, "k", qk_norm)
    for b in range(2):
        p = int(c["pos0"][b])
        _assert_rounded(kc[b, :, p:p + 6].transpose(0, 1), want[b], mag[b] * 2, "k")


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("qk_norm", [False, True])
@pytest.mark.parametrize("scaling", [None, gqa.RopeScaling("yarn", 4.0, 2048),
                                     gqa.RopeScaling("ntk", 2.0)])
def test_without_gains_or_axes_it_is_gqa_rope_append(cuda_lib, D, qk_norm, scaling):
    """Equal bits, also with a gain of one, explicit positions and q in place."""
    c = _case(D, 3, 33, 6, 2, D, 256, 0, gains=False)
    base = [_dev(c[n]) for n in ("q", "k", "v", "kc", "vc")]
    kw = dict(pos0=_dev(c["pos0"]), qk_norm=qk_norm, scaling=scaling)
    gqa.gqa_rope_append(*base, **kw)
    a = [_dev(c[n]) for n in ("q", "k", "v", "kc", "vc")]
    out = gqa.gqa_norm_rope_append(*a, q_out=a[0], **kw)
    assert out is a[0]
    b = [_dev(c[n]) for n in ("q", "k", "v", "kc", "vc")]
    one = torch.ones(D, dtype=BF, device=DEV) if qk_norm else None
    pos = (c["pos0"].view(-1, 1) + torch.arange(33)).to(torch.int32).to(DEV)
    q_b = gqa.gqa_norm_rope_append(*b, q_gain=one, k_gain=one, pos=pos, **kw)
    torch.cuda.synchronize()
    for i in (0, 3, 4):
        assert torch.equal(_bits(a[i]), _bits(base[i]))
        assert torch.equal(_bits(q_b if i == 0 else b[i]), _bits(base[i]))


def test_token_counts_leave_the_rest_alone(cuda_lib):
    c = _case(3, 4, 21, 6, 2, 96, 128, 3)
    n_tok = [0, 21, 1, 13]
    c["pos0"] = torch.tensor([128, 107, 127, 5], dtype=torch.int32)     # up to the last slot
    c["k"][1:, 20:], c["q"][2, 5:] = float("nan"), float("inf")         # padding may hold anything
    c["k"][1] = torch.randn(21, 2, 96).to(BF)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    before = torch.randn(4, 21, 6, 96).to(BF)
    q_out = _dev(before)
    new_len = torch.zeros(4, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gqa.gqa_norm_rope_append(_dev(c["q"]), _dev(c["k"]), _dev(c["v"]), kc, vc,
                             pos0=_dev(c["pos0"]), n_tok=torch.tensor(n_tok, dtype=torch.int32,
                                                                      device=DEV),
                             max_pos0=128, new_len=new_len, q_out=q_out, status=status,
                             **_rope_kw(c))
    torch.cuda.synchronize()
    assert status.item() == 0 and new_len.tolist() == [128, 128, 128, 18]
    _check_append(c, q_out, kc, vc, n_tok=n_tok, q_before=before)


def test_bad_sequences_are_skipped_whole(cuda_lib):
    c = _case(4, 4, 9, 4, 2, 64, 128, 1)
    c["pos0"] = torch.tensor([-1, 120, 3, 10], dtype=torch.int32)       # 120 + 9 > 128
    n_tok = torch.tensor([9, 9, 10, 9], dtype=torch.int32, device=DEV)  # 10 > T
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    before = torch.randn(4, 9, 4, 64).to(BF)
    q_out = _dev(before)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gqa.gqa_norm_rope_append(_dev(c["q"]), _dev(c["k"]), _dev(c["v"]), kc, vc,
                             pos0=_dev(c["pos0"]), n_tok=n_tok, q_out=q_out, status=status,
                             **_rope_kw(c))
    torch.cuda.synchronize()
    assert status.item() == gqa.GQA_DEV_BAD_LEN | gqa.GQA_DEV_CAPACITY
    c["pos0"][:3] = 0
    _check_append(c, q_out, kc, vc, n_tok=[0, 0, 0, 9], q_before=before)


def test_keys_and_values_only_and_the_decode_layout(cuda_lib):
    c = _case(6, 3, 1, 4, 2, 128, 128, 3)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    kw = dict(pos0=_dev(c["pos0"]), **_rope_kw(c))
    assert gqa.gqa_norm_rope_append(None, _dev(c["k"]), _dev(c["v"]), kc, vc, **kw) is None
    kc2, vc2 = _dev(c["kc"]), _dev(c["vc"])
    kw["pos"] = kw["pos"][:, :, 0].contiguous()                         # [n_axes, B]
    q_out = gqa.gqa_norm_rope_append(_dev(c["q"][:, 0]), _dev(c["k"][:, 0]), _dev(c["v"][:, 0]),
                                     kc2, vc2, **kw)
    torch.cuda.synchronize()
    assert q_out.shape == (3, 4, 128)
    assert torch.equal(_bits(kc), _bits(kc2)) and torch.equal(_bits(vc), _bits(vc2))
    _check_append(c, q_out.unsqueeze(1), kc2, vc2)


def test_zero_rows_and_rows_below_eps(cuda_lib):
    c = _case(7, 1, 2, 2, 1, 64, 128, 0)
    c["q"][0, 0], c["k"][0, 1] = 0, 0
    c["q"][0, 1] = 1e-20               # mean of squares far below eps
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    q_out = gqa.gqa_norm_rope_append(_dev(c["q"]), _dev(c["k"]), _dev(c["v"]), kc, vc,
                                     pos0=_dev(c["pos0"]), **_rope_kw(c))
    _check_append(c, q_out, kc, vc)
    assert (q_out[0, 0] == 0).all()


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------
def _backward_case(seed, B, T, Hq, Hkv, D, L, n_axes):
    c = _case(seed, B, T, Hq, Hkv, D, L, n_axes)
    g = torch.Generator().manual_seed(seed + 1)
    c["dq_out"] = torch.randn(B, T, Hq, D, generator=g).to(BF)
    c["dkc"] = torch.randn(B, Hkv, L, D, generator=g).to(BF)
    c["dvc"] = torch.randn(B, Hkv, L, D, generator=g).to(BF)
    return c


def _slots(c, cache):
    return torch.stack([cache[b, :, int(p):int(p) + c["T"]].transpose(0, 1)
                        for b, p in enumerate(c["pos0"])])


def _run_backward(c, qk_norm=True, **kw):
    return gqa.gqa_norm_rope_append_backward(
        _dev(c["q"]), _dev(c["k"]), _dev(c["dq_out"]), _dev(c["dkc"]), _dev(c["dvc"]),
        pos0=_dev(c["pos0"]), **_rope_kw(c, qk_norm), **kw)


def _check_backward(c, got, qk_norm=True):
    P = ref.positions(c["pos0"], c["B"], c["T"], c["pos"], c["pair_axis"], c["D"])
    dys = dict(q=c["dq_out"], k=_slots(c, c["dkc"]))
    for i, name in enumerate("qk"):
        x, dy = c[name].double(), dys[name].double()
        dx, dg = ref.norm_rope_grad(x, dy, P, c[name + "_gain"], qk_norm)
        mag = _pair_mag(dy)
        if qk_norm:
            gain = torch.ones(c["D"]) if c[name + "_gain"] is None else c[name + "_gain"]
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            gm = gain.double().abs() * mag
            mag = r * gm + x.abs() * r ** 3 * (x.abs() * gm).mean(-1, keepdim=True)
            # sums of n products: a lane adds one per token and the rest is a tree
            n = c["B"] * c["T"] * c[name].shape[2]
            allow = (n + 64) * 2.0 ** -24 * (_pair_mag(dy) * x.abs() * r).sum(dim=(0, 1, 2))
            d = (got[3 + i].cpu().double() - dg).abs()
            assert (d <= allow + 1e-30).all(), (name, float((d / allow).max()))
        _assert_rounded(got[i], dx, mag, "d" + name)
    assert torch.equal(_bits(got[2]), _bits(_slots(c, c["dvc"])))


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv,n_axes", [
    (1, 1, 1, 1, 1), (3, 37, 6, 2, 3), (2, 5, 7, 1, 4), (9, 1, 24, 8, 0), (2, 131, 8, 8, 2),
    (1, 700, 5, 5, 3)])
def test_backward_against_float64(cuda_lib, D, B, T, Hq, Hkv, n_axes):
    c = _backward_case(D + T, B, T, Hq, Hkv, D, 768, n_axes)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _run_backward(c, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    _check_backward(c, got)
    again = _run_backward(c)
    assert all(torch.equal(a, b) for a, b in zip(got[3:], again[3:])), "gains: equal bits"


@pytest.mark.parametrize("gains", [(True, False), (False, True), (False, False)])
def test_backward_without_a_gain_or_the_norm(cuda_lib, gains):
    c = _backward_case(21, 2, 19, 6, 3, 96, 128, 2)
    for name, on in zip("qk", gains):
        if not on:
            c[name + "_gain"] = None
    _check_backward(c, _run_backward(c))
    c["q_gain"] = c["k_gain"] = None
    got = _run_backward(c, qk_norm=False)
    assert got[3] is None and got[4] is None
    _check_backward(c, got, qk_norm=False)


@pytest.mark.parametrize("D", [64, 96, 128])
def test_backward_without_eps(cuda_lib, D):
    """eps = 0 with head counts that leave some of a warp's places empty: the gains'
    gradients stay those of the vectors that are there."""
    c = _backward_case(24, 2, 13, 6, 3, D, 128, 1)
    with_eps = _run_backward(c)
    got = _run_backward(c, eps=0.0)
    # 1e-6 next to a mean square of about 1 moves r by 5e-7 of itself, four roundings' worth,
    # and the gains' sums by that and the bounds of _check_backward twice over
    for i, name in enumerate("qk"):
        x, dy = c[name].double(), (c["dq_out"] if i == 0 else _slots(c, c["dkc"])).double()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True))
        n = 2 * 13 * c[name].shape[2]
        allow = (2 * (n + 64) * 2.0 ** -24 + 1e-6 * float((r * r).max())) * (
            _pair_mag(dy) * x.abs() * r).sum(dim=(0, 1, 2))
        d = (got[3 + i].double() - with_eps[3 + i].double()).abs().cpu()
        assert (d <= allow).all(), (name, float((d / allow).max()))
        P = ref.positions(c["pos0"], 2, 13, c["pos"], c["pair_axis"], D)
        dx, _ = ref.norm_rope_grad(x, dy, P, c[name + "_gain"], True, eps=0.0)
        gm = c[name + "_gain"].double().abs() * _pair_mag(dy)
        mag = r * gm + x.abs() * r ** 3 * (x.abs() * gm).mean(-1, keepdim=True)
        _assert_rounded(got[i], dx, mag, "d" + name)


def test_backward_against_differences(cuda_lib):
    """sum(grad . u) against the central difference of the float64 forward along u.  The
    kernel's dx are rounded: the sum may be off by 2^-8 of sum |dx u| (and far less)."""
    c = _backward_case(22, 2, 11, 4, 2, 64, 128, 3)
    got = _run_backward(c)
    P = ref.positions(c["pos0"], 2, 11, c["pos"], c["pair_axis"], 64)
    dys = dict(q=c["dq_out"].double(), k=_slots(c, c["dkc"]).double())
    g = torch.Generator().manual_seed(5)
    for i, name in enumerate("qk"):
        x, gain = c[name].double(), c[name + "_gain"].double()
        u, ug = torch.randn(x.shape, generator=g).double(), torch.randn(64, generator=g).double()
        f = lambda t: (ref.norm_rope(x + t * u, P, gain + t * ug) * dys[name]).sum()
        h = 1e-4
        diff = (f(h) - f(-h)) / (2 * h)
        dx, dg = got[i].cpu().double(), got[3 + i].cpu().double()
        allow = 2.0 ** -8 * (dx * u).abs().sum() + 1e-4 * (dg * ug).abs().sum() + 1e-4
        assert abs((dx * u).sum() + (dg * ug).sum() - diff) <= allow


def test_backward_in_place_and_bad_sequences(cuda_lib):
    c = _backward_case(23, 3, 10, 4, 2, 128, 128, 1)
    want = _run_backward(c)
    dq = _dev(c["dq_out"])
    got = gqa.gqa_norm_rope_append_backward(_dev(c["q"]), _dev(c["k"]), dq, _dev(c["dkc"]),
                                            _dev(c["dvc"]), pos0=_dev(c["pos0"]), dq=dq,
                                            **_rope_kw(c))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # sequence 1 is out of range: left alone, and its share of the gains is missing
    bad = dict(c, pos0=torch.tensor([int(c["pos0"][0]), 119, int(c["pos0"][2])],
                                    dtype=torch.int32))
    keep = [torch.full_like(t, 7.0) for t in want[:3]]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _run_backward(bad, status=status, dq=keep[0], dk=keep[1], dv=keep[2])
    assert status.item() == gqa.GQA_DEV_CAPACITY
    for a, b in zip(got[:3], want[:3]):
        assert (a[1] == 7).all() and torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    two = {n: (v[[0, 2]] if isinstance(v, torch.Tensor) and v.shape[:1] == (3,) else v)
           for n, v in c.items()}
    two.update(B=2, pos=c["pos"][:, [0, 2]].contiguous())
    dg = _run_backward(two)[3:]
    for a, b in zip(got[3:], dg):
        assert (a - b).abs().max() <= 1e-4 * b.abs().max()      # the same sums in another order


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------
def test_side_stream_and_captured_graphs(cuda_lib):
    c = _backward_case(31, 3, 50, 6, 2, 96, 128, 3)
    want = _run_backward(c)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    ins = [_dev(c[n]) for n in ("q", "k", "v")]
    kw = dict(pos0=_dev(c["pos0"]), **_rope_kw(c))
    q_want = gqa.gqa_norm_rope_append(*ins, kc, vc, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kc2, vc2 = _dev(c["kc"]), _dev(c["vc"])
    torch.cuda.synchronize()
    q_side = gqa.gqa_norm_rope_append(*ins, kc2, vc2, stream=side, **kw)
    side.synchronize()
    assert torch.equal(q_side, q_want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    # forward and backward in two graphs with a workspace each, replayed on new inputs
    bwd = [_dev(c[n]) for n in ("q", "k", "dq_out", "dkc", "dvc")]
    outs, graphs = [], []
    for _ in range(2):
        ws = gqa.norm_rope_backward_workspace(96, DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q_g = gqa.gqa_norm_rope_append(*ins, kc2, vc2, **kw)
            outs.append((q_g,) + gqa.gqa_norm_rope_append_backward(*bwd, workspace=ws, **kw))
        graphs.append(g)
    for rep in range(2):
        for g, out in zip(graphs, outs):
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], q_want)
            assert all(torch.equal(a, b) for a, b in zip(out[1:], want))


def test_binding_refuses_what_does_not_fit(cuda_lib):
    c = _case(41, 2, 4, 4, 2, 64, 128, 2)
    q, k, v, kc, vc = (_dev(c[n]) for n in ("q", "k", "v", "kc", "vc"))
    kw = _rope_kw(c)
    good = dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, **kw)
    bad = [
        dict(q=q[:, :, :, :32].contiguous()), dict(v=v[:1]), dict(q=q.float()), dict(q=q[:, :2]),
        dict(k_cache=kc[:, :1].contiguous()), dict(v_cache=vc[:, :, :64].contiguous()),
        dict(q_gain=torch.ones(32, dtype=BF, device=DEV)), dict(k_gain=torch.ones(64, device=DEV)),
        dict(q_gain=torch.ones(64, dtype=BF)), dict(pos=kw["pos"][:1].contiguous()),
        dict(pos=kw["pos"].long()), dict(pos=kw["pos"].cpu()), dict(axes=None),
        dict(axes=gqa.RopeAxes((16, 17))), dict(pos=None), dict(qk_norm=False),
        dict(q_out=torch.empty_like(q)[:1]), dict(pos0=torch.zeros(3, dtype=torch.int32, device=DEV)),
        dict(n_tok=torch.zeros(2, dtype=torch.int64, device=DEV)),
        dict(status=torch.zeros(1, dtype=torch.int32)), dict(q=q.transpose(1, 2)),
    ]
    for over in bad:
        with pytest.raises((ValueError, TypeError)):
            gqa.gqa_norm_rope_append(**dict(good, **over))
    with pytest.raises(gqa.GqaError):
        gqa.gqa_norm_rope_append(**dict(good, max_pos0=125))
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(gqa.GqaError):
        gqa.gqa_norm_rope_append(**dict(good, pos0=lens, new_len=lens))
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        gqa.gqa_norm_rope_append(**dict(good, q_out=torch.empty_like(q), stream=other))
    dkc = torch.zeros_like(kc)
    with pytest.raises(gqa.GqaError):
        gqa.gqa_norm_rope_append_backward(q, k, q, dkc, dkc, workspace=torch.empty(
            64, dtype=torch.uint8, device=DEV), **kw)
    for over in (dict(q=q[:1]), dict(dk_cache=dkc[:1]), dict(dq=torch.empty_like(k)),
                 dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            gqa.gqa_norm_rope_append_backward(**dict(
                dict(q=q, k=k, dq_out=q, dk_cache=dkc, dv_cache=dkc, **kw), **over))
    torch.cuda.synchronize()
    assert torch.equal(_bits(kc), _bits(c["kc"])), "a refused call wrote to the cache"


def test_gains_that_are_parameters(cuda_lib):
    """A model's gains require gradients: the calls read them all the same."""
    c = _backward_case(61, 2, 6, 4, 2, 64, 128, 1)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    kw = _rope_kw(c)
    for name in ("q_gain", "k_gain"):
        kw[name] = torch.nn.Parameter(kw[name])
    q_out = gqa.gqa_norm_rope_append(_dev(c["q"]), _dev(c["k"]), _dev(c["v"]), kc, vc,
                                     pos0=_dev(c["pos0"]), **kw)
    _check_append(c, q_out, kc, vc)
    _check_backward(c, gqa.gqa_norm_rope_append_backward(
        _dev(c["q"]), _dev(c["k"]), _dev(c["dq_out"]), _dev(c["dkc"]), _dev(c["dvc"]),
        pos0=_dev(c["pos0"]), **kw))


def test_many_sequences_of_one_token(cuda_lib):
    """More sequences than warps, with and without one to write."""
    B = 7001
    c = _case(62, B, 1, 2, 1, 64, 128, 2)
    kc, vc = _dev(c["kc"]), _dev(c["vc"])
    n_tok = (torch.arange(B) % 3 > 0).to(torch.int32)
    before = torch.randn(B, 1, 2, 64).to(BF)
    q_out = _dev(before)
    new_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    gqa.gqa_norm_rope_append(_dev(c["q"]), _dev(c["k"]), _dev(c["v"]), kc, vc,
                             pos0=_dev(c["pos0"]), n_tok=_dev(n_tok), new_len=new_len,
                             q_out=q_out, **_rope_kw(c))
    torch.cuda.synchronize()
    assert torch.equal(new_len.cpu(), c["pos0"] + n_tok)
    want, mag = _want(c, "q")
    on = n_tok.bool()
    _assert_rounded(q_out[on.to(DEV)], want[on], mag[on], "q")
    assert torch.equal(_bits(q_out)[~on], _bits(before)[~on])
    slot = torch.zeros(B, 128, dtype=torch.bool)
    slot[torch.arange(B), c["pos0"].long()] = on
    for got, was in ((kc, c["kc"]), (vc, c["vc"])):
        assert torch.equal(_bits(got)[:, 0][~slot], _bits(was)[:, 0][~slot])
    assert torch.equal(_bits(vc)[:, 0][slot], _bits(c["v"])[:, 0, 0][on])
    want, mag = _want(c, "k")
    _assert_rounded(kc[:, 0].cpu()[slot], want[:, 0, 0][on], mag[:, 0, 0][on], "k")


# ---------------------------------------------------------------------------
# as they are used: a training layer's attention, forward and backward
# ---------------------------------------------------------------------------
def test_training_attention_gradients_through_the_whole_run(cuda_lib):
    """gqa_norm_rope_append -> gqa_prefill_lse -> gqa_attention_backward ->
    gqa_norm_rope_append_backward against float64 autograd of the same chain.

    The attention's gradients come with the roundings of its tensor-core pipeline
    (2e-2 of unit-sized gradients and a bf16 step: the bound its own tests hold it to)
    and pass a linear map whose rows have norm at most r |gain|max, about 2 here for
    unit-variance inputs; q and K enter it rounded to bf16 too."""
    c = _case(51, 2, 150, 6, 2, 64, 256, 3)
    c["q"] = torch.randn(2, 150, 6, 64, generator=torch.Generator().manual_seed(8)).to(BF)
    c["q_gain"], c["k_gain"] = ((1 + 0.1 * torch.randn(
        64, generator=torch.Generator().manual_seed(s))).to(BF) for s in (1, 2))
    kc, vc = torch.zeros_like(c["kc"]).to(DEV), torch.zeros_like(c["vc"]).to(DEV)
    kw = _rope_kw(c)
    q, k, v = (_dev(c[n]) for n in ("q", "k", "v"))
    dout = torch.randn(2, 150, 6, 64, generator=torch.Generator().manual_seed(9)).to(BF)
    q_rot = gqa.gqa_norm_rope_append(q, k, v, kc, vc, **kw)
    out, lse = gqa.gqa_prefill_lse(q_rot, kc, vc)
    dq_rot, dkc, dvc = gqa.gqa_attention_backward(q_rot, kc, vc, out, _dev(dout), lse)
    dq, dk, dv, dqg, dkg = gqa.gqa_norm_rope_append_backward(q, k, dq_rot, dkc, dvc, **kw)

    P = ref.positions(None, 2, 150, c["pos"], c["pair_axis"], 64)
    x = {n: c[n].double().requires_grad_(True) for n in ("q", "k", "v", "q_gain", "k_gain")}
    qr = ref.norm_rope(x["q"], P, x["q_gain"]).transpose(1, 2)
    kr = ref.norm_rope(x["k"], P, x["k_gain"]).transpose(1, 2).repeat_interleave(3, dim=1)
    vv = x["v"].transpose(1, 2).repeat_interleave(3, dim=1)
    s = qr @ kr.transpose(-1, -2) / 8.0
    s = s.masked_fill(torch.ones(150, 150, dtype=torch.bool).triu(1), float("-inf"))
    o = (torch.softmax(s, -1) @ vv).transpose(1, 2)
    (o * dout.double()).sum().backward()
    for got, name in ((dq, "q"), (dk, "k"), (dv, "v")):
        want = x[name].grad
        d = (got.cpu().double() - want).abs()
        assert (d <= 2 * 2e-2 + 2.0 ** -6 * want.abs()).all() and d.mean() <= 2e-3, (
            name, float(d.max()), float(d.mean()))
    for got, name in ((dqg, "q_gain"), (dkg, "k_gain")):
        want = x[name].grad
        rel = (got.cpu().double() - want).norm() / want.norm()
        # each term is off by the mean error above at most, terms of order |w x r| ~ 0.1
        assert rel <= 2e-2, (name, float(rel))
