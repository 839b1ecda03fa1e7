"""GPU parity of the 4-bit cache: its append, its read-back and the decode over it.

Codes and scales are held to the definition exactly (but for the quotients that the
header lets fall to either side), the read-back to the bits, and the decode to the bound
derived in norm_rope_reference.decode.
"""
import math

import pytest
import torch

import rope_gqa_kv_b200 as gqa

import norm_rope_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _random_cache(seed, B, Hkv, L, D):
    """Every byte and scale at random (finite, s >= 0); CPU tensors."""
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (B, Hkv, L, D // 2), generator=g, dtype=torch.uint8)
             for _ in range(2)]
    scales = []
    for _ in range(2):
        s = torch.rand(B, Hkv, L, D // 32, generator=g) * 0.4
        m = -7.5 * s + torch.randn(B, Hkv, L, D // 32, generator=g)
        scales.append(torch.stack((s, m), dim=-1).to(BF))
    return [codes[0], scales[0], codes[1], scales[1]]


def _on_gpu(parts):
    return gqa.Q4Cache(*(t.to(DEV) for t in parts))


def _parts(cache):
    return cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales


def _assert_quantised(codes, scales, x, what):
    """Rows codes [n, D/2], scales [n, D/32, 2] are those of the bf16 rows x [n, D]."""
    c, s, m, near = ref.quantise(x)
    got = ref.unpack_codes(codes.cpu())
    sm = scales.cpu().double()
    assert torch.equal(sm[..., 0], s), what + ": steps"
    assert torch.equal(torch.nan_to_num(sm[..., 1], nan=1e30), torch.nan_to_num(m, nan=1e30)), what
    ok = (got == c) | (near & (got == c - 1))
    assert ok.all(), "%s: %d codes of %d" % (what, int((~ok).sum()), ok.numel())


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 37, 6, 2), (2, 5, 7, 1), (64, 1, 24, 8),
                                        (2, 131, 8, 8), (1, 9, 5, 5)])
def test_append_stores_the_quantised_rows_of_the_bf16_cache(cuda_lib, D, B, T, Hq, Hkv):
    L = 256
    g = torch.Generator().manual_seed(D + T + B)
    q, k, v = (torch.randn(B, T, h, D, generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv))
    gains = [(1 + 0.5 * torch.randn(D, generator=g)).to(BF).to(DEV) for _ in range(2)]
    pos0 = torch.randint(0, L - T + 1, (B,), generator=g).to(torch.int32)
    n_tok = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    n_tok[0] = T
    kc = torch.zeros(B, Hkv, L, D, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    pos = torch.randint(0, 500, (3, B, T), generator=g).to(torch.int32).to(DEV)
    kw = dict(pos0=pos0.to(DEV), n_tok=n_tok.to(DEV), q_gain=gains[0], k_gain=gains[1], pos=pos,
              axes=gqa.RopeAxes((D // 2 - 20, 10, 10)))
    q1 = gqa.gqa_norm_rope_append(q, k, v, kc, vc, q_out=q.clone(), **kw)
    before = _random_cache(5, B, Hkv, L, D)
    cache = _on_gpu(before)
    new_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q2 = gqa.gqa_norm_rope_append_q4(q, k, v, cache, q_out=q.clone(), new_len=new_len,
                                     status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0 and new_len.tolist() == (pos0 + n_tok).tolist()
    assert torch.equal(q1, q2)
    for b in range(B):
        p, n = int(pos0[b]), int(n_tok[b])
        if n:
            for codes, scales, rows in ((cache.k_codes, cache.k_scales, kc),
                                        (cache.v_codes, cache.v_scales, vc)):
                _assert_quantised(codes[b, :, p:p + n].reshape(-1, D // 2),
                                  scales[b, :, p:p + n].reshape(-1, D // 32, 2),
                                  rows[b, :, p:p + n].cpu().reshape(-1, D), "b=%d" % b)
        keep = torch.ones(L, dtype=torch.bool)
        keep[p:p + n] = False
        for got, was in zip(_parts(cache), before):
            assert torch.equal(got[b].cpu()[:, keep], was[b][:, keep])


@pytest.mark.parametrize("D", [64, 96, 128])
def test_quantiser_on_rows_where_it_can_go_wrong(cuda_lib, D):
    g = torch.Generator().manual_seed(D)
    rows = []

    def row(x):
        rows.append(x.to(BF))

    r = lambda: torch.randn(D, generator=g)
    row(torch.zeros(D))
    row(torch.full((D,), -3.25))
    row(torch.arange(D) % 31 * 0.5)                       # quotients n and n + 1/2
    row((torch.arange(D) % 31 * 0.5 - 7.5) * 2.0 ** 40)
    row((torch.arange(D) % 61) * 0.25)
    row(torch.where(torch.arange(D) % 7 == 0, 0.0, 1.0))
    for e in (-140, -133, -130, -126, -122, -60, 60, 100, 120):
        row(r().double() * 2.0 ** e)
    row(r().sign() * 3.38e38)                             # max - min beyond fp32
    row(r() + 2.0 ** 20)
    row(r() * torch.where(torch.arange(D) == 3, 1e30, 1.0))
    row(r() * torch.exp2(-20 * torch.rand(D, generator=g)))
    for bad in (math.nan, math.inf, -math.inf):
        x = r()
        x[5] = bad
        row(x)
        x = r()
        x[D - 1] = bad
        row(x)
    row(torch.full((D,), math.nan))
    row(torch.full((D,), math.inf))
    x = torch.stack(rows + [r().to(BF) for _ in range(200)])
    n = x.shape[0]
    cache = gqa.Q4Cache.zeros(1, 1, 384, D)
    v = x.view(1, n, 1, D).to(DEV)
    k = torch.ones_like(v)
    gqa.gqa_norm_rope_append_q4(None, k, v, cache)
    _assert_quantised(cache.v_codes[0, 0, :n], cache.v_scales[0, 0, :n], x, "D=%d" % D)
    _, got = gqa.kv_cache_read_q4(cache)
    want = ref.values(cache.v_codes.cpu(), cache.v_scales.cpu()).float().to(BF)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.cpu(), nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("B,Hkv,L,Lout", [(1, 1, 128, 1), (3, 2, 256, 256), (2, 3, 384, 77),
                                          (5, 1, 128, 129)])
def test_read_back(cuda_lib, D, B, Hkv, L, Lout):
    parts = _random_cache(D + L, B, Hkv, L, D)
    g = torch.Generator().manual_seed(3)
    first = torch.randint(0, L, (B,), generator=g).to(torch.int32)
    count = torch.minimum(torch.randint(0, Lout + 1, (B,), generator=g), L - first.long())
    first[0], count[0] = 0, min(L, Lout)
    if B > 1:
        count[1] = 0
        first[1] = L
    if B > 2:
        first[2], count[2] = L - 1, 1
    count = count.to(torch.int32)
    was = torch.randn(2, B, Hkv, Lout, D, generator=g).to(BF)
    outs = [was[i].to(DEV) for i in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gqa.kv_cache_read_q4(_on_gpu(parts), *outs, first=first.to(DEV), count=count.to(DEV),
                         status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for i, out in enumerate(outs):
        vals = ref.values(parts[2 * i], parts[2 * i + 1]).float().to(BF)
        for b in range(B):
            f, n = int(first[b]), int(count[b])
            assert torch.equal(out[b, :, :n].cpu(), vals[b, :, f:f + n])
            assert torch.equal(out[b, :, n:].cpu(), was[i][b, :, n:])


def test_read_back_refuses_bad_ranges_on_the_device(cuda_lib):
    cache = _on_gpu(_random_cache(1, 5, 2, 128, 64))
    first = torch.tensor([-1, 0, 100, 0, 0], dtype=torch.int32, device=DEV)
    count = torch.tensor([1, -1, 29, 65, 64], dtype=torch.int32, device=DEV)
    k, v = (torch.full((5, 2, 64, 64), 7.0, dtype=BF, device=DEV) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gqa.kv_cache_read_q4(cache, k, v, first=first, count=count, status=status)
    torch.cuda.synchronize()
    assert status.item() == gqa.GQA_DEV_BAD_LEN | gqa.GQA_DEV_CAPACITY
    assert (k[:4] == 7).all() and (v[:4] == 7).all() and not (k[4] == 7).any()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def _check_decode(q, parts, lens, max_len, what, scale=0.0, **kw):
    dead = torch.arange(parts[0].shape[2]).view(1, 1, -1, 1) >= lens.view(-1, 1, 1, 1)
    dirty = [t.clone() for t in parts]
    for i in (0, 2):                       # rows behind the length: any bytes, NaN scales
        dirty[i].masked_fill_(dead, 0xEE)
        dirty[i + 1].masked_fill_(dead.unsqueeze(-1), math.nan)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gqa.gqa_decode_q4(q.to(DEV), _on_gpu(dirty), lens.to(torch.int32).to(DEV), max_len,
                            scale=scale, status=status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, tol = ref.decode(q, parts, lens, scale if scale > 0 else None)
    d = (out.cpu().double() - want).abs()
    assert (d <= tol).all(), "%s: worst %.3g of the bound, %d elements" % (
        what, float((d / tol).max()), int((d > tol).sum()))
    return out


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (6, 2), (8, 2), (5, 1), (24, 3), (9, 1),
                                    (16, 1), (34, 2), (8, 8)])
def test_decode_groupings(cuda_lib, D, Hq, Hkv):
    lens = torch.tensor([1, 300, 64, 97, 17])
    q = torch.randn(5, Hq, D, generator=torch.Generator().manual_seed(Hq)).to(BF)
    _check_decode(q, _random_cache(D + Hq, 5, Hkv, 384, D), lens, 300, "Hq=%d" % Hq)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("max_len", [64, 128, 512])
def test_decode_lengths_around_tiles_and_chunks(cuda_lib, D, max_len):
    """Lengths one off every tile, warp and chunk edge; max_len decides the cut."""
    every = [1, 2, 3, 4, 5, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 256,
             257, 319, 321, 383, 385, 511, 512]
    lens = torch.tensor([n for n in every if n <= max_len])
    B = lens.numel()
    q = torch.randn(B, 3, D, generator=torch.Generator().manual_seed(1)).to(BF)
    _check_decode(q, _random_cache(D, B, 1, 512, D), lens, max_len, "max_len=%d" % max_len)


@pytest.mark.parametrize("B,Hq,Hkv,L", [(40, 24, 8, 640), (150, 20, 4, 512), (600, 2, 1, 256)])
def test_decode_with_every_tile_count(cuda_lib, B, Hq, Hkv, L):
    """Enough sequences that a CTA takes several tiles per warp."""
    lens = torch.randint(1, L + 1, (B,), generator=torch.Generator().manual_seed(B))
    lens[0], lens[1] = L, 1
    q = torch.randn(B, Hq, 64, generator=torch.Generator().manual_seed(2)).to(BF)
    _check_decode(q, _random_cache(B, B, Hkv, L, 64), lens, L, "B=%d" % B)


@pytest.mark.parametrize("D,n", [(128, 20011), (64, 33000), (96, 2049)])
def test_decode_long_sequences(cuda_lib, D, n):
    """Rows of many chunks: the merge in groups of 32 and by several warps."""
    L = (n + 127) // 128 * 128
    lens = torch.tensor([n, n // 3])
    q = torch.randn(2, 4, D, generator=torch.Generator().manual_seed(n)).to(BF)
    _check_decode(q, _random_cache(n, 2, 1, L, D), lens, n, "n=%d" % n)


def test_decode_peaked_and_scaled_scores(cuda_lib):
    """Scores of some hundreds (one key takes all), and a scale of the caller's."""
    lens = torch.tensor([500, 77])
    q = (40 * torch.randn(2, 6, 128, generator=torch.Generator().manual_seed(4))).to(BF)
    parts = _random_cache(8, 2, 2, 512, 128)
    _check_decode(q, parts, lens, 512, "peaked")
    _check_decode((q / 40).to(BF), parts, lens, 512, "scaled", scale=0.3)


def test_decode_constant_groups_and_nan_keys(cuda_lib):
    """Groups without a step (s = 0) count as their minimum; a NaN group makes the
    heads that read it NaN and no others."""
    parts = _random_cache(9, 2, 2, 128, 64)
    parts[1][0, :, 3:60, :, 0] = 0
    parts[3][0, :, 10:90, 1, 0] = 0
    lens = torch.tensor([100, 128])
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(6)).to(BF)
    _check_decode(q, parts, lens, 128, "constant")
    parts[1][1, 1, 50, 0, 1] = math.nan
    out = gqa.gqa_decode_q4(q.to(DEV), _on_gpu(parts), lens.to(torch.int32).to(DEV), 128).cpu()
    want, tol = ref.decode(q[:1], [t[:1] for t in parts], lens[:1])
    assert ((out[:1].double() - want).abs() <= tol).all()
    assert torch.isnan(out[1, 2:]).all() and torch.isfinite(out[1, :2]).all()


def _times(scales, factor):
    """The (s, m) pairs times powers of two (exact)."""
    return (scales.double() * factor).to(BF)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("n", [60, 700])
def test_decode_far_apart_magnitudes(cuda_lib, D, n):
    """Values whose steps lie 2^30 apart from group to group, grow or shrink by 2^100
    along the sequence, or are very small or large throughout; q and K far from 1."""
    L, lens = 768, torch.tensor([n, n - 13])
    q = torch.randn(2, 6, D, generator=torch.Generator().manual_seed(n)).to(BF)
    base = _random_cache(n + D, 2, 2, L, D)
    ng = D // 32
    groups = torch.exp2(30.0 * torch.arange(ng, dtype=torch.float64) - 45).view(1, 1, 1, ng, 1)
    rows = torch.exp2((100.0 * torch.arange(L, dtype=torch.float64) / n - 50).round())
    rows = rows.view(1, 1, L, 1, 1)
    for what, f in (("groups", groups), ("growing", rows), ("shrinking", 1 / rows),
                    ("small", 2.0 ** -90), ("large", 2.0 ** 100)):
        parts = base[:3] + [_times(base[3], f)]
        _check_decode(q, parts, lens, n, what)
    parts = [base[0], _times(base[1], 2.0 ** -70)] + base[2:]
    _check_decode((q.double() * 2.0 ** 55).to(BF), parts, lens, n, "q", scale=2.0 ** 15 / D ** 0.5)


@pytest.mark.parametrize("max_len", [64, 400])
def test_decode_bad_lengths_give_zeros(cuda_lib, max_len):
    parts = _random_cache(10, 5, 2, 512, 96)
    lens = torch.tensor([0, -3, max_len + 1, 40, 600], dtype=torch.int32, device=DEV)
    q = torch.randn(5, 6, 96, generator=torch.Generator().manual_seed(7)).to(BF)
    out = torch.full((5, 6, 96), 7.0, dtype=BF, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gqa.gqa_decode_q4(q.to(DEV), _on_gpu(parts), lens, max_len, out=out, status=status)
    torch.cuda.synchronize()
    assert status.item() == gqa.GQA_DEV_BAD_LEN | gqa.GQA_DEV_CAPACITY
    assert (out[[0, 1, 2, 4]] == 0).all()
    want, tol = ref.decode(q[3:4], [t[3:4] for t in parts], [40])
    assert ((out[3:4].cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("D,Hq,Hkv,max_len,lens", [
    (128, 6, 2, 8960, [8960, 1, 64, 65]), (64, 3, 1, 12000, [12000] * 3),
    (96, 4, 4, 5000, [4097, 5000, 1, 1, 129, 128]), (128, 24, 8, 4224, [4224, 10, 10, 10, 10, 10]),
    (64, 1, 1, 4500, [1 + 145 * i for i in range(32)]), (128, 9, 1, 30000, [1]),
    (128, 2, 1, 30000, [64, 63]), (96, 5, 1, 6000, [4608] * 27)])
def test_decode_few_rows_share_the_chunks_by_length(cuda_lib, D, Hq, Hkv, max_len, lens):
    """Long capacities with few rows: the cut follows the lengths, on the device."""
    B, L = len(lens), (max_len + 127) // 128 * 128
    q = torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(max_len)).to(BF)
    _check_decode(q, _random_cache(D + B, B, Hkv, L, D), torch.tensor(lens), max_len, str(lens[:4]))


def test_decode_few_rows_with_bad_lengths_and_replayed_with_others(cuda_lib):
    B, Hq, Hkv, D, L, max_len = 5, 6, 2, 64, 9088, 9000
    parts = _random_cache(77, B, Hkv, L, D)
    cache = _on_gpu(parts)
    q = torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(7)).to(BF)
    qd, status = q.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([5000, 0, 9001, 700, -3], dtype=torch.int32, device=DEV)
    ws = gqa.decode_q4_workspace(B, Hq, Hkv, D, max_len, DEV)
    ws.view(torch.float32).fill_(math.nan)
    out = torch.full((B, Hq, D), 7.0, dtype=BF, device=DEV)
    run = lambda: gqa.gqa_decode_q4(qd, cache, lens, max_len, out=out, workspace=ws, status=status)
    run()
    torch.cuda.synchronize()
    assert status.item() == gqa.GQA_DEV_BAD_LEN | gqa.GQA_DEV_CAPACITY
    good = [0, 3]
    want, tol = ref.decode(q[good], [t[good] for t in parts], torch.tensor([5000, 700]), None)
    assert ((out[good].cpu().double() - want).abs() <= tol).all()
    assert (out[[1, 2, 4]] == 0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for n in ([1, 2, 3, 4, 5], [9000, 1, 1, 1, 1], [9000] * 5, [3000, 4000, 64, 65, 8999]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        status.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert status.item() == 0
        replayed = out.clone()
        run()
        assert torch.equal(out, replayed)
        want, tol = ref.decode(q, parts, torch.tensor(n), None)
        assert ((replayed.cpu().double() - want).abs() <= tol).all(), n


def test_offsets_beyond_32_bits(cuda_lib):
    """A cache of more than 2^31 bytes of codes: the last sequence's newest slots are
    written, read back and attended to.  Every other slot is zero (score 0, value 0), so
    the answer has a closed form."""
    B, Hkv, D, L = 2, 8, 128, (1 << 21) + 128
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    cache = gqa.Q4Cache.zeros(B, Hkv, L, D)
    assert cache.k_codes.numel() > 1 << 31
    g = torch.Generator().manual_seed(12)
    k, v = (torch.randn(B, 3, Hkv, D, generator=g).to(BF).to(DEV) for _ in range(2))
    q = (6 * torch.randn(B, Hkv, D, generator=g)).to(BF)
    pos0 = torch.full((B,), L - 3, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    gqa.gqa_norm_rope_append_q4(None, k, v, cache, pos0=pos0, new_len=lens, status=status)
    k3, v3 = (torch.zeros(B, Hkv, 3, D, dtype=BF, device=DEV) for _ in range(2))
    gqa.kv_cache_read_q4(cache, k3, v3, first=pos0, status=status)
    out = gqa.gqa_decode_q4(q.to(DEV), cache, lens, L, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and lens.tolist() == [L, L]
    parts = [t[:, :, L - 3:].cpu() for t in _parts(cache)]
    vals = [ref.values(parts[i], parts[i + 1]) for i in (0, 2)]
    _assert_quantised(parts[2].reshape(-1, 64), parts[3].reshape(-1, 4, 2),
                      v.transpose(1, 2).cpu().reshape(-1, D), "v")
    for got, want in zip((k3, v3), vals):
        assert torch.equal(got.cpu(), want.float().to(BF))
    s = torch.einsum("bhd,bhsd->bhs", q.double(), vals[0]) / math.sqrt(D)
    top = s.amax(-1, keepdim=True).clamp(min=0)
    w = torch.exp(s - top)
    want = torch.einsum("bhs,bhsd->bhd", w, vals[1]) / (w.sum(-1, keepdim=True) +
                                                          (L - 3) * torch.exp(-top))
    # 3 live keys against 2 million: a lane adds a 64th of a chunk's weights (some 1300 of
    # 2^21 / 26 slots) one after the other, which is off by at most as many fp32 units,
    # 1e-4 of the sum; scores of up to ~60 are off by 1e-4
    assert ((out.cpu().double() - want).abs() <= (2.0 ** -8 + 5e-4) * want.abs() + 1e-6).all()
    k3 = v3 = cache = None


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------
def test_two_streams_at_once_and_captured_graphs(cuda_lib):
    parts = _random_cache(20, 8, 2, 2048, 128)
    cache = _on_gpu(parts)
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(1, 2049, (8,), generator=g).to(torch.int32).to(DEV)
    qs = [torch.randn(8, 6, 128, generator=g).to(BF).to(DEV) for _ in range(2)]
    want = [gqa.gqa_decode_q4(q, cache, lens, 2048) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(gqa.gqa_decode_q4(qs[i], cache, lens, 2048, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graphs, outs = [], []
    for q in qs:
        ws = gqa.decode_q4_workspace(8, 6, 2, 128, 2048, DEV)
        out = torch.empty_like(q)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            gqa.gqa_decode_q4(q, cache, lens, 2048, out=out, workspace=ws)
        graphs.append(gr)
        outs.append(out)
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    # the lengths are read at replay: shorter ones give the shorter answer
    lens.clamp_(max=100)
    graphs[0].replay()
    short = gqa.gqa_decode_q4(qs[0], cache, lens, 2048)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], short) and not torch.equal(short, want[0])


def test_binding_refuses_what_does_not_fit(cuda_lib):
    cache = gqa.Q4Cache.zeros(2, 2, 128, 64)
    p = _parts(cache)
    for bad in ((p[0], p[1], p[2], p[3][:1]), (p[0], p[1], p[2].float(), p[3]),
                (p[0], p[1][..., :1].contiguous(), p[2], p[3]),
                (p[0][..., :20].contiguous(), p[1], p[2], p[3]), (p[0], p[1], p[2].cpu(), p[3])):
        with pytest.raises((ValueError, TypeError)):
            gqa.Q4Cache(*bad)
    q = torch.zeros(2, 4, 64, dtype=BF, device=DEV)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    good = dict(q=q, cache=cache, lens=lens, max_len=100)
    for over in (dict(q=q[:1]), dict(q=q.float()), dict(lens=lens[:1]), dict(lens=lens.long()),
                 dict(out=torch.empty_like(q)[:, :2]), dict(cache=p[0]),
                 dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises((ValueError, TypeError)):
            gqa.gqa_decode_q4(**dict(good, **over))
    for over in (dict(max_len=129), dict(max_len=0), dict(q=q[:, :3].contiguous()),
                 dict(workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(gqa.GqaError):
            gqa.gqa_decode_q4(**dict(good, **over))
    with pytest.raises(ValueError):
        gqa.kv_cache_read_q4(cache, k_out=torch.zeros(2, 2, 8, 64, dtype=BF, device=DEV))
    with pytest.raises(ValueError):
        gqa.kv_cache_read_q4(cache, first=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        gqa.DecodeGraph(cache, q, lens, 4)


# ---------------------------------------------------------------------------
# as they are used: a prompt, a continuation chunk and a decode loop
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("axes", [None, (12, 10, 10)])
def test_serving_run_on_a_4_bit_cache(cuda_lib, axes):
    """A prompt and a continuation chunk are written in 4 bits, the chunk attends over
    the prefix read back as bf16, and DecodeGraph generates; every answer against
    float64 on the rows that the cache holds, the graph's steps bit for bit against the
    eager calls."""
    B, Hq, Hkv, D, L, T, C = 2, 6, 2, 64, 256, 70, 33
    g = torch.Generator().manual_seed(30)
    new = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)
    gains = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF).to(DEV) for _ in range(2)]
    ax = None if axes is None else gqa.RopeAxes(axes)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(q_gain=gains[0], k_gain=gains[1], axes=ax, status=status)

    def pos(n):
        if ax is None:
            return None
        return torch.randint(0, 200, (3, B, n), generator=g).to(torch.int32).to(DEV)

    cache = gqa.Q4Cache.zeros(B, Hkv, L, D)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    n_tok = torch.tensor([T, T - 21], dtype=torch.int32, device=DEV)
    gqa.gqa_norm_rope_append_q4(new(B, T, Hq, D), new(B, T, Hkv, D), new(B, T, Hkv, D), cache,
                                n_tok=n_tok, new_len=lens, pos=pos(T), **kw)
    pos0 = lens.clone()
    qc = gqa.gqa_norm_rope_append_q4(new(B, C, Hq, D), new(B, C, Hkv, D), new(B, C, Hkv, D),
                                     cache, pos0=pos0, new_len=lens, pos=pos(C), **kw)
    kb, vb = gqa.kv_cache_read_q4(cache, count=lens, status=status)
    out = gqa.gqa_prefill_chunk(qc, kb, vb, pos0, T, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and lens.tolist() == [T + C, T - 21 + C]
    for b in range(B):
        n0 = int(pos0[b])
        K, V = (t[b, :, :n0 + C].cpu().double().repeat_interleave(3, 0) for t in (kb, vb))
        s = qc[b].cpu().double().transpose(0, 1) @ K.transpose(-1, -2) / 8.0
        late = torch.arange(n0 + C).view(1, -1) > n0 + torch.arange(C).view(-1, 1)
        p = torch.softmax(s.masked_fill(late, -math.inf), -1)
        want = p @ V
        # bf16 probabilities and sums: 2^-8 of sum p |v| and of the result, twice over
        tol = 2.0 ** -7 * (p @ V.abs()) + 2.0 ** -7 * want.abs()
        assert ((out[b].cpu().double().transpose(0, 1) - want).abs() <= tol).all()

    eager = gqa.Q4Cache(*(t.clone() for t in _parts(cache)))
    dg = gqa.DecodeGraph(cache, None, lens, Hq, qk_norm=True, q_gain=gains[0], k_gain=gains[1],
                         axes=ax)
    cur = lens.clone()
    for step in range(9):
        q, k, v, p = new(B, Hq, D), new(B, Hkv, D), new(B, Hkv, D), pos(1)
        dg.q.copy_(q), dg.k.copy_(k), dg.v.copy_(v)
        if p is not None:
            dg.pos.copy_(p[:, :, 0])
        got = dg.step()
        nxt = torch.empty_like(cur)
        qr = gqa.gqa_norm_rope_append_q4(q, k, v, eager, pos0=cur, new_len=nxt,
                                         pos=None if p is None else p, **kw)
        cur = nxt
        want = gqa.gqa_decode_q4(qr, eager, cur, L, status=status)
        torch.cuda.synchronize()
        assert torch.equal(got, want), "step %d" % step
        exact, tol = ref.decode(qr.cpu(), [t.cpu() for t in _parts(eager)], cur.tolist())
        assert ((got.cpu().double() - exact).abs() <= tol).all()
    assert status.item() == 0 and dg.status.item() == 0 and torch.equal(dg.lens, cur)
    for a, b in zip(_parts(cache), _parts(eager)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_decode_graph_with_learned_gains_on_the_bf16_cache(cuda_lib):
    B, Hq, Hkv, D, L = 2, 4, 2, 96, 128
    g = torch.Generator().manual_seed(40)
    new = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)
    gain, ax = (1 + 0.3 * torch.randn(D, generator=g)).to(BF).to(DEV), gqa.RopeAxes((20, 28))
    a = [new(B, Hkv, L, D) for _ in range(2)]
    b = [t.clone() for t in a]
    cur = torch.tensor([3, 60], dtype=torch.int32, device=DEV)
    dg = gqa.DecodeGraph(*a, cur, Hq, qk_norm=True, q_gain=gain, axes=ax)
    for _ in range(4):
        q, k, v = new(B, Hq, D), new(B, Hkv, D), new(B, Hkv, D)
        p = torch.randint(0, 99, (2, B), generator=g).to(torch.int32).to(DEV)
        for buf, t in ((dg.q, q), (dg.k, k), (dg.v, v), (dg.pos, p)):
            buf.copy_(t)
        got = dg.step()
        nxt = torch.empty_like(cur)
        qr = gqa.gqa_norm_rope_append(q, k, v, *b, pos0=cur, new_len=nxt, q_gain=gain, pos=p,
                                      axes=ax)
        cur = nxt
        assert torch.equal(got, gqa.gqa_decode(qr, *b, cur, L))
    assert dg.status.item() == 0
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_checks_in_python_lead_to_the_same_calls(cuda_lib, monkeypatch):
    """What the native argument checks do not take goes through the checks in Python:
    the same results, and a stream of the caller's, either way."""
    from types import SimpleNamespace

    from rope_gqa_kv_b200 import _lib
    g = torch.Generator().manual_seed(50)
    new = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)
    q, k, v = new(2, 5, 4, 64), new(2, 5, 2, 64), new(2, 5, 2, 64)
    gain, ax = new(64), gqa.RopeAxes((10, 22))
    pos = torch.randint(0, 50, (2, 2, 5), generator=g).to(torch.int32).to(DEV)
    pos0 = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    kw = dict(pos0=pos0, q_gain=gain, k_gain=gain, pos=pos, axes=ax)

    def run(stream=None):
        cache = gqa.Q4Cache.zeros(2, 2, 128, 64)
        kc, vc = (torch.zeros(2, 2, 128, 64, dtype=BF, device=DEV) for _ in range(2))
        lens = torch.zeros(2, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        a = gqa.gqa_norm_rope_append(q, k, v, kc, vc, stream=stream, **kw)
        b = gqa.gqa_norm_rope_append_q4(q, k, v, cache, new_len=lens, stream=stream, **kw)
        ko, vo = gqa.kv_cache_read_q4(cache, count=lens, stream=stream)
        out = gqa.gqa_decode_q4(q[:, 4].contiguous(), cache, lens, 20, stream=stream)
        grads = gqa.gqa_norm_rope_append_backward(q, k, q, kc, vc, stream=stream, **kw)
        torch.cuda.synchronize()
        return (a, b, kc, vc, ko, vo, out) + grads + _parts(cache)

    want = run()
    side = torch.cuda.Stream()
    fast = run(side)
    none = lambda *a: None
    monkeypatch.setattr(_lib, "_fast", SimpleNamespace(
        append=none, backward=none, read_back=none, decode=none, cache=none))
    slow = run()
    monkeypatch.setattr(_lib, "_fast_pointers", none)
    slower = run(side)
    for got in (fast, slow, slower):
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("eq,ek", [(12, 0), (28, 0), (31, 0), (40, 0), (60, 0), (60, 50),
                                   (60, 110)])
@pytest.mark.parametrize("D,n", [(64, 100), (96, 700), (128, 4500)])
def test_decode_scores_of_any_size(cuda_lib, eq, ek, D, n):
    """Scores of up to +-2^178, exact in float64, all of one sign: q has one coordinate, +-2^eq,
    and K's rows are constants 2^ek times 141 .. 239 with one 255 (which takes all of the
    heads with a positive q) and one 128 (the others': their scores are all negative)."""
    B, Hq, Hkv, L = 2, 4, 2, (n + 127) // 128 * 128
    g = torch.Generator().manual_seed(n + eq)
    parts = _random_cache(n, B, Hkv, L, D)
    lens = torch.tensor([n, n // 2 + 1])
    m = torch.randint(141, 240, (B, Hkv, L), generator=g).double()
    best = torch.empty(B, Hkv, 2, dtype=torch.long)
    for b in range(B):
        for h in range(Hkv):
            at = torch.randperm(int(lens[b]), generator=g)[:2]
            m[b, h, at[0]], m[b, h, at[1]] = 255, 128
            best[b, h] = at
    parts[1] = torch.stack((torch.zeros(B, Hkv, L, D // 32, dtype=torch.float64),
                            (m * 2.0 ** ek).unsqueeze(-1).expand(B, Hkv, L, D // 32)), -1).to(BF)
    q = torch.zeros(B, Hq, D, dtype=BF)
    q[:, 0::2, 3], q[:, 1::2, 3] = 2.0 ** eq, -2.0 ** eq
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gqa.gqa_decode_q4(q.to(DEV), _on_gpu(parts), lens.to(torch.int32).to(DEV), n,
                            status=status).cpu().double()
    assert status.item() == 0
    # the other weights are below exp(-13 * 2^12 / sqrt(128)) = 0 and the best one's is exactly 1:
    # what is left is p s to fp16, the last sums (as in norm_rope_reference.decode) and bf16
    grp = (torch.arange(D) % (D // 2)) // 16
    vals = ref.values(parts[2], parts[3])
    step, low = parts[3].double()[..., 0][..., grp], parts[3].double()[..., 1][..., grp]
    for b in range(B):
        for h in range(Hq):
            at = (b, h // 2, int(best[b, h // 2, h % 2]))
            want = vals[at]
            tol = 2.0 ** -8 * want.abs() + 1.01 * (2.0 ** -11 * 15 * step[at] + 80 * ref.U32 *
                                                   (15 * step[at] + low[at].abs()))
            assert ((out[b, h] - want).abs() <= tol).all(), (b, h)


@pytest.mark.parametrize("B,Hq,Hkv,D,L,max_len", [(1300, 2, 1, 64, 128, 128),
                                                  (160, 16, 8, 96, 256, 250),
                                                  (400, 6, 3, 128, 128, 64)])
def test_decode_more_rows_than_places(cuda_lib, B, Hq, Hkv, D, L, max_len):
    """More rows than the waves of a call: one chunk each, no second kernel, many rounds."""
    assert gqa.gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, max_len) == 16
    lens = torch.randint(1, max_len + 1, (B,), generator=torch.Generator().manual_seed(B))
    lens[0], lens[1], lens[2] = 1, max_len, 64
    q = torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(3)).to(BF)
    _check_decode(q, _random_cache(B, B, Hkv, L, D), lens, max_len, "B=%d" % B)


@pytest.mark.parametrize("B,Hq,Hkv,D,lengths", [
    (8, 8, 8, 64, [4800, 4736, 4097, 4096, 1500, 64, 1]),      # waves, clusters
    (3, 6, 2, 128, [9088, 9000, 5000, 4160, 4090, 100]),       # shared out by the lengths, clusters
    (40, 8, 4, 96, [1280, 1279, 600, 65]),                     # clusters of two, one chunk
    (125, 8, 8, 64, [384, 320, 129, 64]),                      # waves of many rows
    (1, 2, 1, 64, [33024, 33000, 20000, 4097, 4096])])
def test_one_workspace_for_the_capacity_and_every_shorter_call(cuda_lib, B, Hq, Hkv, D, lengths):
    """The workspace of the longest call, between guard bytes, serves the others: the
    answers are right, and nothing outside of it is written."""
    L = (lengths[0] + 127) // 128 * 128
    size, guard = gqa.gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, lengths[0]), 4096
    buf = torch.empty(guard + size + guard, dtype=torch.uint8, device=DEV)
    parts = _random_cache(B + D, B, Hkv, L, D)
    g = torch.Generator().manual_seed(size % 1000)
    q = torch.randn(B, Hq, D, generator=g).to(BF)
    for n in lengths:
        assert gqa.gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, n) <= size
        lens = torch.randint(1, n + 1, (B,), generator=g)
        lens[-1] = n
        buf.fill_(0xFF)                        # NaN wherever it is read as fp32
        _check_decode(q, parts, lens, n, "max_len=%d" % n, workspace=buf[guard:guard + size])
        assert (buf[:guard] == 0xFF).all() and (buf[guard + size:] == 0xFF).all()


@pytest.mark.parametrize("D,n", [(64, 262144), (96, 131072), (128, 131072)])
def test_decode_sums_of_long_chunks(cuda_lib, D, n):
    """Chunks of 10000 to 20000 keys with equal weights (q = 0).  V's minima take the mean of
    its codes away to 1/4000, so a sum that loses 2^-15 of what it adds up is off by 10 % of
    the answer.  Everything up to the chunks' merge is exact in fp32 by choice of the steps
    (255/128 times a power of two) but for 2^-8 in sums that pass 2^16, a few times in 5000
    keys: 1e-5 of the step's power covers it and the merge, beside the rounding to bf16."""
    Hkv, ng = 32, D // 32
    g = torch.Generator(device=DEV).manual_seed(n + D)
    codes = [torch.randint(0, 256, (1, Hkv, n, D // 2), generator=g, dtype=torch.uint8, device=DEV)
             for _ in range(2)]
    power = torch.exp2(3.0 * torch.arange(ng, device=DEV))
    low = torch.where(torch.arange(n, device=DEV) % 2 == 0, -15.0, -14.875).view(n, 1) * power
    sv = torch.stack((power.expand(n, ng) * (255 / 128), low), -1).to(BF)
    sv = sv.expand(1, Hkv, n, ng, 2).contiguous()
    sk = torch.zeros_like(sv)
    cache = gqa.Q4Cache(codes[0], sk, codes[1], sv)
    q = torch.zeros(1, Hkv, D, dtype=BF, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.full((1,), n, dtype=torch.int32, device=DEV)
    out = gqa.gqa_decode_q4(q, cache, lens, n, status=status)[0].double()
    assert status.item() == 0
    grp = (torch.arange(D, device=DEV) % (D // 2)) // 16
    for h in range(Hkv):
        c = ref.unpack_codes(codes[1][0, h]).double().mean(0)
        want = (c * (255 / 128) - 14.9375) * power.double()[grp]
        tol = 2.0 ** -8 * want.abs() + 1e-5 * power.double()[grp]
        d = (out[h] - want).abs()
        assert (d <= tol).all(), "head %d: %.3g of the bound" % (h, float((d / tol).max()))
    cache = codes = sv = sk = None


@pytest.mark.parametrize("q4", [True, False])
def test_decode_graph_captures_and_replays_on_the_caches_device(cuda_lib, monkeypatch, q4):
    """Whichever device is current (here one that does not exist, as far as DecodeGraph can
    see), the capture's stream and the replay's are the caches' device's."""
    B, Hq, Hkv, D, L = 2, 4, 2, 64, 128
    g = torch.Generator().manual_seed(60)
    new = lambda *s: torch.randn(*s, generator=g).to(BF).to(DEV)
    caches = (gqa.Q4Cache.zeros(B, Hkv, L, D), None) if q4 else (new(B, Hkv, L, D), new(B, Hkv, L, D))
    lens = torch.tensor([3, 60], dtype=torch.int32, device=DEV)
    entered, captured = [], []
    real_device, real_graph = torch.cuda.device, torch.cuda.graph

    class Device(real_device):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

    def graph(cuda_graph, **kw):
        captured.append(kw["stream"].device)
        return real_graph(cuda_graph, **kw)

    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "device", Device)
        m.setattr(torch.cuda, "graph", graph)
        dg = gqa.DecodeGraph(*caches, lens, Hq, qk_norm=True)
        assert captured == [lens.device] * 2 and lens.device.index in entered
        dg.q.copy_(new(B, Hq, D)), dg.k.copy_(new(B, Hkv, D)), dg.v.copy_(new(B, Hkv, D))
        del entered[:]
        m.setattr(torch.cuda, "current_device", lambda: lens.device.index + 1)
        out = dg.step()
        assert entered == [lens.device.index]
    torch.cuda.synchronize()
    assert dg.lens.tolist() == [4, 61] and dg.status.item() == 0
    assert torch.isfinite(out).all() and out.abs().amax(-1).gt(0).all()
