"""The cache operators with learned norms, several position axes and 4-bit storage,
as measured cases: what a case is, its inputs, one pass and its 64-bit answer.

Operators
  append         per-head RMSNorm with a learned gain, rotation by positions on one
                 or three axes, and the write of k and v into the bf16 cache
  append_bwd     the gradients of that pass with respect to q, k, v and the gains
  write_q4       the same pass into a cache held in 4 bits, and the new slots read back
  read_q4        slots of a 4-bit cache read back as bf16
  decode_q4      one query token per sequence against a 4-bit cache

A 4-bit row (one token of one KV head, D values) has D/32 groups; group G holds
the rotation pairs 16 G .. 16 G + 15, that is coordinates i and i + D/2 of each.
With m the group's minimum and s = bf16((max - m) / 15), the code of x is
ceil((x - m) / s - 1/2) and stands for m + s * code.  Pair p's byte has the code of
coordinate p in its low half and that of p + D/2 in its high half and sits at byte
4 * (D/32 * ((p % 16) // 4) + p // 16) + p % 4 of the row.  (s, m) are bf16 pairs.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a training step's prompt batch, 24 query heads on 8 KV heads, image positions
        dict(name="append_prompt_8x2048", op="append", B=8, T=2048, Hq=24, Hkv=8, D=128, axes=3,
             lo=0, hi=0, cap=2048),
        # one decode step of 64 sequences: each appends one token at its own length
        dict(name="append_token_64", op="append", B=64, T=1, Hq=24, Hkv=8, D=128, axes=3,
             lo=256, hi=2048, cap=2176),
        # the training step's way back
        dict(name="append_bwd_8x2048", op="append_bwd", B=8, T=2048, Hq=24, Hkv=8, D=128, axes=3,
             lo=0, hi=0, cap=2048),
        # a small model (8 heads of 96), an odd number of odd-length sequences
        dict(name="append_bwd_3x1001", op="append_bwd", B=3, T=1001, Hq=8, Hkv=8, D=96, axes=1,
             lo=0, hi=0, cap=1024),
        # a continuation chunk written in 4 bits and read back for its attention
        dict(name="write_q4_chunk_8x1024", op="write_q4", B=8, T=1024, Hq=24, Hkv=8, D=128, axes=1,
             lo=512, hi=1536, cap=2560),
        # the decode step's write of 64 sequences
        dict(name="write_q4_token_64", op="write_q4", B=64, T=1, Hq=24, Hkv=8, D=128, axes=1,
             lo=256, hi=2048, cap=2176),
        # cached prefixes of a batch of 16, read back before a chunk's attention
        dict(name="read_q4_16x2048", op="read_q4", B=16, Hkv=8, D=128, lo=1024, hi=2048, cap=2048),
        # one short prefix of a small model
        dict(name="read_q4_1x333", op="read_q4", B=1, Hkv=4, D=64, lo=333, hi=333, cap=384),
        # single-stream generation near the end of its 512 + 100 tokens: latency
        dict(name="decode_q4_1x612", op="decode_q4", B=1, Hq=16, Hkv=4, D=64, lo=612, hi=612,
             cap=640),
        # a small model without shared heads, very uneven lengths
        dict(name="decode_q4_7x1500", op="decode_q4", B=7, Hq=8, Hkv=8, D=96, lo=1, hi=1500,
             cap=1536),
        # the batched serving step
        dict(name="decode_q4_64x2048", op="decode_q4", B=64, Hq=24, Hkv=8, D=128, lo=256, hi=2048,
             cap=2176),
        # few sequences with long contexts: what a smaller cache is for
        dict(name="decode_q4_4x65536", op="decode_q4", B=4, Hq=24, Hkv=8, D=128, lo=49152,
             hi=65536, cap=65536),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cap(n):
    return (n + 127) // 128 * 128


def draw(rng):
    op = rng.choice(("append", "append_bwd", "write_q4", "read_q4", "decode_q4", "decode_q4"))
    D = rng.choice((64, 96, 128))
    Hkv = rng.randint(1, 8)
    g = rng.randint(1, 8)
    if op == "decode_q4":
        tokens = _spread(rng, 300, 200000)          # cached tokens, all sequences together
        B = _spread(rng, 1, min(64, tokens))
        hi = max(1, tokens // B)
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, D=D, lo=max(1, hi // rng.randint(1, 8)),
                    hi=hi, cap=_cap(hi))
    if op == "read_q4":
        tokens = _spread(rng, 300, 30000)
        B = _spread(rng, 1, 32)
        hi = max(1, tokens // B)
        return dict(op=op, B=B, Hkv=Hkv, D=D, lo=max(1, hi // rng.randint(1, 8)), hi=hi,
                    cap=_cap(hi))
    # new tokens, all sequences together; many heads get fewer of them
    tokens = _spread(rng, 1, min(12000, 620000 // (Hkv * (g + 2))))
    B = _spread(rng, 1, min(64, tokens))
    T = max(1, tokens // B)
    lo, hi = (0, 0) if op == "append_bwd" else (0, rng.randint(0, 400))
    return dict(op=op, B=B, T=T, Hq=Hkv * g, Hkv=Hkv, D=D, axes=rng.choice((1, 3)), lo=lo, hi=hi,
                cap=_cap(hi + T))


def work(case):
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    q4_row = D // 2 + D // 8                        # codes and (s, m) of one row
    mean = (case["lo"] + case["hi"]) / 2.0
    if case["op"] == "decode_q4":
        keys = B * mean
        return {"bytes": 2 * keys * Hkv * q4_row + 4 * B * case["Hq"] * D,
                "flops": 4 * keys * case["Hq"] * D}
    if case["op"] == "read_q4":
        return {"bytes": 2 * B * mean * Hkv * (q4_row + 2 * D), "flops": 4 * B * mean * Hkv * D}
    n, Hq = B * case["T"], case["Hq"]
    row = 2 * D
    if case["op"] == "append":
        return {"bytes": n * row * (2 * Hq + 4 * Hkv), "flops": 7 * n * D * (Hq + Hkv)}
    if case["op"] == "append_bwd":
        return {"bytes": n * row * (3 * Hq + 5 * Hkv), "flops": 14 * n * D * (Hq + Hkv)}
    # q in and out, k and v in, their 4-bit rows out and in again, bf16 rows out
    return {"bytes": n * (2 * Hq * row + 2 * Hkv * (2 * row + 2 * q4_row)),
            "flops": n * D * (7 * (Hq + Hkv) + 16 * Hkv)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _sections(D, axes):
    """Rotation pairs per axis: a quarter for time, the rest for height and width."""
    half = D // 2
    return (half,) if axes == 1 else (half - 2 * (half * 3 // 8), half * 3 // 8, half * 3 // 8)


def _positions(case, pos0, g):
    """[axes, B, T] int32: text at pos0 + t, with one image of 16 columns in the middle
    whose rows and columns count on the height and width axes."""
    B, T, axes = case["B"], case["T"], case["axes"]
    t = torch.arange(T, device=DEV)
    seq = pos0.to(torch.int64).view(B, 1) + t.view(1, T)
    if axes == 1:
        return seq.to(torch.int32).view(1, B, T).contiguous()
    a = torch.randint(0, T, (B, 1), device=DEV, generator=g)
    inside = (t.view(1, T) >= a) & (t.view(1, T) < a + T // 2)
    start = pos0.to(torch.int64).view(B, 1) + a
    k = (t.view(1, T) - a).clamp(min=0)
    pos = torch.stack((torch.where(inside, start, seq),
                       torch.where(inside, start + k // 16, seq),
                       torch.where(inside, start + k % 16, seq)))
    return pos.to(torch.int32).contiguous()


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g, dtype=torch.float32)


def _pack(x, D):
    """bf16-valued [..., D] -> (codes uint8 [..., D/2], scales bf16 [..., D/32, 2])."""
    ng = D // 32
    lead = x.shape[:-1]
    y = x.float().view(*lead, 2, ng, 16).transpose(-3, -2)          # [..., ng, 2, 16]
    m = y.amin(dim=(-2, -1), keepdim=True)
    s = ((y.amax(dim=(-2, -1), keepdim=True) - m) / 15).to(torch.bfloat16).float()
    c = torch.where(s > 0, ((y - m) / torch.where(s > 0, s, 1.0) - 0.5).ceil(), 0.0)
    c = c.clamp_(0, 15).to(torch.uint8)
    byte = c[..., 0, :] | (c[..., 1, :] << 4)                       # [..., ng, 16]
    byte = byte.view(*lead, ng, 4, 4).transpose(-3, -2).reshape(*lead, D // 2)
    sm = torch.stack((s[..., 0, 0], m[..., 0, 0]), dim=-1).to(torch.bfloat16)
    return byte.contiguous(), sm.contiguous()


def _cache_q4(case, g, lens):
    """A 4-bit cache as a serving program holds it: keys with a mean per channel, values
    with a scale per channel, rows behind each length left over from other sequences."""
    B, Hkv, L, D = case["B"], case["Hkv"], case["cap"], case["D"]
    k = (_randn(g, B, Hkv, L, D) + _randn(g, 1, Hkv, 1, D)).to(torch.bfloat16)
    kc, ks = _pack(k, D)
    del k
    v = (_randn(g, B, Hkv, L, D) * torch.exp(0.5 * _randn(g, 1, Hkv, 1, D))).to(torch.bfloat16)
    vc, vs = _pack(v, D)
    dead = torch.arange(L, device=DEV).view(1, 1, L, 1) >= lens.view(B, 1, 1, 1)
    kc.masked_fill_(dead, 0xEE)
    vc.masked_fill_(dead, 0xEE)
    ks.masked_fill_(dead.unsqueeze(-1), float("nan"))
    vs.masked_fill_(dead.unsqueeze(-1), float("nan"))
    return kc, ks, vc, vs


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hkv, D, L = case["B"], case["Hkv"], case["D"], case["cap"]
    st = dict(case)
    lens = torch.randint(case["lo"], case["hi"] + 1, (B,), device=DEV, generator=g)
    lens = lens.to(torch.int32)
    st["lens"] = lens
    st["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    bf = torch.bfloat16
    if case["op"] in ("read_q4", "decode_q4"):
        st["cache"] = _cache_q4(case, g, lens)
        if case["op"] == "read_q4":
            st["k_out"] = torch.zeros(B, Hkv, L, D, dtype=bf, device=DEV)
            st["v_out"] = torch.zeros(B, Hkv, L, D, dtype=bf, device=DEV)
        else:
            st["q"] = _randn(g, B, case["Hq"], D).to(bf)
            st["out"] = torch.empty(B, case["Hq"], D, dtype=bf, device=DEV)
            st["workspace"] = None
        return st
    T, Hq = case["T"], case["Hq"]
    st["q"] = _randn(g, B, T, Hq, D).mul_(2.0).to(bf)
    st["k"] = _randn(g, B, T, Hkv, D).to(bf)
    st["v"] = _randn(g, B, T, Hkv, D).to(bf)
    st["q_gain"] = (1.0 + 0.25 * _randn(g, D)).to(bf)
    st["k_gain"] = (1.0 + 0.25 * _randn(g, D)).to(bf)
    st["pos"] = _positions(case, lens, g)
    st["pair_axis"] = torch.cat([torch.full((n,), a, device=DEV) for a, n in
                                 enumerate(_sections(D, case["axes"]))])
    st["axes_plan"] = None
    if case["op"] == "append_bwd":
        st["dq_out"] = _randn(g, B, T, Hq, D).to(bf)
        st["dk_cache"] = _randn(g, B, Hkv, L, D).to(bf)
        st["dv_cache"] = _randn(g, B, Hkv, L, D).to(bf)
        st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[n]) for n in ("q", "k", "v"))
        st["workspace"] = None
        return st
    st["q_out"] = torch.empty_like(st["q"])
    if case["op"] == "append":
        st["k_cache"] = torch.zeros(B, Hkv, L, D, dtype=bf, device=DEV)
        st["v_cache"] = torch.zeros(B, Hkv, L, D, dtype=bf, device=DEV)
    else:
        ng = D // 32
        st["cache"] = tuple(torch.zeros(B, Hkv, L, *tail, dtype=t, device=DEV)
                            for tail, t in 2 * (((D // 2,), torch.uint8), ((ng, 2), bf)))
        st["k_out"] = torch.empty(B, Hkv, T, D, dtype=bf, device=DEV)
        st["v_out"] = torch.empty(B, Hkv, T, D, dtype=bf, device=DEV)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _angles(st):
    """cos, sin [B, T, 1, D/2] of every token's rotation pairs; the angles in 64 bits."""
    half = st["D"] // 2
    theta = BASE ** (-2.0 * torch.arange(half, device=DEV, dtype=torch.float64) / st["D"])
    ang = st["pos"].double()[st["pair_axis"]].permute(1, 2, 0) * theta     # [B, T, half]
    return ang.cos().float().unsqueeze(2), ang.sin().float().unsqueeze(2)


def _norm_rope(x, gain, cos, sin):
    x = x.float()
    u = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    a, b = u.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)


def _slots(st):
    """(sequence, slot) indices [B, 1] and [B, T] of the new tokens."""
    b = torch.arange(st["B"], device=DEV).view(-1, 1)
    return b, st["lens"].long().view(-1, 1) + torch.arange(st["T"], device=DEV).view(1, -1)


def _plain_append(st):
    cos, sin = _angles(st)
    st["q_out"].copy_(_norm_rope(st["q"], st["q_gain"], cos, sin))
    k = _norm_rope(st["k"], st["k_gain"], cos, sin).to(torch.bfloat16)
    b, slot = _slots(st)
    if st["op"] == "append":
        st["k_cache"][b, :, slot] = k
        st["v_cache"][b, :, slot] = st["v"]
        return st["q_out"], st["k_cache"], st["v_cache"]
    kc, ks, vc, vs = st["cache"]
    codes, scales = _pack(k, st["D"])
    kc[b, :, slot], ks[b, :, slot] = codes, scales
    st["k_out"].copy_(_unpack(codes, scales, st["D"]).transpose(1, 2))
    codes, scales = _pack(st["v"], st["D"])
    vc[b, :, slot], vs[b, :, slot] = codes, scales
    st["v_out"].copy_(_unpack(codes, scales, st["D"]).transpose(1, 2))
    return st["q_out"], st["k_out"], st["v_out"]


def _norm_rope_bwd(x, gain, dy, cos, sin):
    """(dx, d gain) of _norm_rope for the output gradient dy."""
    x, gain, dy = x.float(), gain.float(), dy.float()
    a, b = dy.chunk(2, dim=-1)
    w = torch.cat((a * cos + b * sin, b * cos - a * sin), dim=-1)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xr = x * r
    z = gain * w
    dx = r * (z - xr * (xr * z).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (w * xr).sum(dim=(0, 1, 2), dtype=torch.float64).float()


def _plain_append_bwd(st):
    cos, sin = _angles(st)
    T = st["T"]
    dq, dqg = _norm_rope_bwd(st["q"], st["q_gain"], st["dq_out"], cos, sin)
    dk, dkg = _norm_rope_bwd(st["k"], st["k_gain"], st["dk_cache"][:, :, :T].transpose(1, 2),
                             cos, sin)
    st["dq"].copy_(dq)
    st["dk"].copy_(dk)
    st["dv"].copy_(st["dv_cache"][:, :, :T].transpose(1, 2))
    return st["dq"], st["dk"], st["dv"], dqg, dkg


def _unpack(codes, scales, D):
    """The values [..., D] (fp32) that codes and scales stand for."""
    ng = D // 32
    lead = codes.shape[:-1]
    byte = codes.view(*lead, 4, ng, 4).transpose(-3, -2).reshape(*lead, ng, 16)
    c = torch.stack((byte & 15, byte >> 4), dim=-3).float()         # [..., 2, ng, 16]
    s, m = scales.float()[..., 0], scales.float()[..., 1]
    return (m[..., None, :, None] + s[..., None, :, None] * c).reshape(*lead, D)


def _plain_read(st):
    kc, ks, vc, vs = st["cache"]
    live = torch.arange(st["cap"], device=DEV).view(1, 1, -1, 1) < st["lens"].view(-1, 1, 1, 1)
    st["k_out"].copy_(torch.where(live, _unpack(kc, ks, st["D"]).to(torch.bfloat16), st["k_out"]))
    st["v_out"].copy_(torch.where(live, _unpack(vc, vs, st["D"]).to(torch.bfloat16), st["v_out"]))
    return st["k_out"], st["v_out"]


def _plain_decode(st):
    B, Hq, Hkv, D, n = st["B"], st["Hq"], st["Hkv"], st["D"], st["hi"]
    kc, ks, vc, vs = (t[:, :, :n] for t in st["cache"])
    live = torch.arange(n, device=DEV).view(1, 1, 1, n) < st["lens"].view(B, 1, 1, 1)
    q = st["q"].float().view(B, Hkv, Hq // Hkv, D)
    sc = torch.matmul(q, _unpack(kc, ks, D).transpose(-1, -2)) / math.sqrt(D)
    sc = torch.where(live, sc, float("-inf"))
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = torch.where(live.transpose(-1, -2), _unpack(vc, vs, D), 0.0)
    st["out"].copy_(torch.matmul(p, v).view(B, Hq, D))
    return st["out"]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _rope_args(gqa, st):
    if st["axes_plan"] is None:
        st["axes_plan"] = gqa.RopeAxes(_sections(st["D"], st["axes"]))
    return dict(q_gain=st["q_gain"], k_gain=st["k_gain"], pos=st["pos"], axes=st["axes_plan"],
                qk_norm=True, eps=EPS, rope_base=BASE)


def _own(st):
    import rope_gqa_kv_b200 as gqa
    if st["op"] == "append":
        gqa.gqa_norm_rope_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                 pos0=st["lens"], max_pos0=st["hi"], q_out=st["q_out"],
                                 status=st["status"], **_rope_args(gqa, st))
        return st["q_out"], st["k_cache"], st["v_cache"]
    if st["op"] == "append_bwd":
        if st["workspace"] is None:
            st["workspace"] = gqa.norm_rope_backward_workspace(st["D"], st["q"].device)
        return gqa.gqa_norm_rope_append_backward(
            st["q"], st["k"], st["dq_out"], st["dk_cache"], st["dv_cache"], dq=st["dq"],
            dk=st["dk"], dv=st["dv"], workspace=st["workspace"], **_rope_args(gqa, st))
    cache = gqa.Q4Cache(*st["cache"])
    if st["op"] == "write_q4":
        gqa.gqa_norm_rope_append_q4(st["q"], st["k"], st["v"], cache, pos0=st["lens"],
                                    max_pos0=st["hi"], q_out=st["q_out"], status=st["status"],
                                    **_rope_args(gqa, st))
        gqa.kv_cache_read_q4(cache, st["k_out"], st["v_out"], first=st["lens"],
                             status=st["status"])
        return st["q_out"], st["k_out"], st["v_out"]
    if st["op"] == "read_q4":
        return gqa.kv_cache_read_q4(cache, st["k_out"], st["v_out"], count=st["lens"],
                                    status=st["status"])
    if st["workspace"] is None:
        st["workspace"] = gqa.decode_q4_workspace(st["B"], st["Hq"], st["Hkv"], st["D"],
                                                  st["hi"], st["q"].device)
    return gqa.gqa_decode_q4(st["q"], cache, st["lens"], st["hi"], out=st["out"],
                             workspace=st["workspace"], status=st["status"])


def run(state):
    if own:
        return _own(state)
    if state["op"] in ("append", "write_q4"):
        return _plain_append(state)
    if state["op"] == "append_bwd":
        return _plain_append_bwd(state)
    if state["op"] == "read_q4":
        return _plain_read(state)
    return _plain_decode(state)


# ---------------------------------------------------------------------------
# the answer in 64 bits
# ---------------------------------------------------------------------------
def _rotation64(st, b):
    """Complex factors [T, 1, D/2] that turn sequence b's pairs."""
    D = st["D"]
    theta = torch.tensor([BASE ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64,
                         device=DEV)
    parts, at = [], 0
    for a, n in enumerate(_sections(D, st["axes"])):
        parts.append(st["pos"][a, b].to(torch.float64).view(-1, 1) * theta[at:at + n])
        at += n
    ang = torch.cat(parts, dim=1)
    return torch.polar(torch.ones_like(ang), ang).unsqueeze(1)


def _turned64(x, gain, rot):
    """Norm, gain and rotation of [T, H, D] in 64 bits; pairs as complex numbers."""
    x = x.double()
    u = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
    half = x.shape[-1] // 2
    z = torch.complex(u[..., :half], u[..., half:]) * rot
    return torch.cat((z.real, z.imag), dim=-1)


def _stored64(x):
    """The values that the 4-bit rows of x [..., D] (bf16) stand for, in 64 bits."""
    D = x.shape[-1]
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for grp in range(D // 32):
        idx = torch.cat((torch.arange(16 * grp, 16 * grp + 16),
                         torch.arange(16 * grp, 16 * grp + 16) + D // 2)).to(x.device)
        y = x[..., idx].double()
        low = y.min(dim=-1, keepdim=True).values
        step = ((y.max(dim=-1, keepdim=True).values - low) / 15.0).to(torch.bfloat16).double()
        code = torch.where(step > 0, torch.ceil((y - low) / step - 0.5), torch.zeros_like(y))
        out[..., idx] = low + step * code.clamp(0, 15)
    return out


def _values64(codes, scales):
    """The values of 4-bit rows [n, D/2], [n, D/32, 2], byte by byte."""
    D = codes.shape[-1] * 2
    out = torch.empty(codes.shape[0], D, dtype=torch.float64, device=codes.device)
    p = torch.arange(D // 2, device=codes.device)
    grp = p // 16
    at = 4 * (D // 32 * ((p % 16) // 4) + grp) + p % 4
    byte = codes[:, at].to(torch.float64)
    high = torch.floor(byte / 16)
    s, m = scales[:, grp, 0].double(), scales[:, grp, 1].double()
    out[:, :D // 2] = m + s * (byte - 16 * high)
    out[:, D // 2:] = m + s * high
    return out


def exact(case, seed):
    st = prepare(case, seed)
    B, D, Hkv, L = st["B"], st["D"], st["Hkv"], st["cap"]
    lens = st["lens"].tolist()
    f64 = dict(dtype=torch.float64, device=DEV)
    if st["op"] == "decode_q4":
        g = st["Hq"] // Hkv
        out = torch.empty(B, st["Hq"], D, **f64)
        for b in range(B):
            for h in range(Hkv):
                n = lens[b]
                k, v = (_values64(st["cache"][i][b, h, :n], st["cache"][i + 1][b, h, :n])
                        for i in (0, 2))
                q = st["q"][b, h * g:(h + 1) * g].double()
                out[b, h * g:(h + 1) * g] = torch.softmax(q @ k.T / D ** 0.5, dim=-1) @ v
        return out
    if st["op"] == "read_q4":
        k, v = torch.zeros(B, Hkv, L, D, **f64), torch.zeros(B, Hkv, L, D, **f64)
        for b in range(B):
            for h in range(Hkv):
                for i, o in ((0, k), (2, v)):
                    o[b, h, :lens[b]] = _values64(st["cache"][i][b, h, :lens[b]],
                                                  st["cache"][i + 1][b, h, :lens[b]])
        return k, v
    T = st["T"]
    if st["op"] == "append_bwd":
        got = {}
        for name, dy in (("q", st["dq_out"]), ("k", st["dk_cache"][:, :, :T].transpose(1, 2))):
            x, gain = st[name], st[name + "_gain"].double()
            dx, dg = torch.empty(x.shape, **f64), torch.zeros(D, **f64)
            for b in range(B):
                rot = _rotation64(st, b).conj()
                w = torch.complex(dy[b, ..., :D // 2].double(), dy[b, ..., D // 2:].double()) * rot
                w = torch.cat((w.real, w.imag), dim=-1)
                xb = x[b].double()
                n2 = xb.pow(2).sum(-1, keepdim=True) / D + EPS
                dg += (w * xb / n2.sqrt()).sum(dim=(0, 1))
                z = w * gain
                dx[b] = z / n2.sqrt() - xb * (xb * z).sum(-1, keepdim=True) / (D * n2 ** 1.5)
            got[name] = (dx, dg)
        dv = st["dv_cache"][:, :, :T].transpose(1, 2).double()
        return got["q"][0], got["k"][0], dv, got["q"][1], got["k"][1]
    q = torch.empty(st["q"].shape, **f64)
    wide = L if st["op"] == "append" else T
    k, v = torch.zeros(B, Hkv, wide, D, **f64), torch.zeros(B, Hkv, wide, D, **f64)
    for b in range(B):
        rot = _rotation64(st, b)
        q[b] = _turned64(st["q"][b], st["q_gain"], rot)
        kb = _turned64(st["k"][b], st["k_gain"], rot)
        if st["op"] == "append":
            k[b, :, lens[b]:lens[b] + T] = kb.transpose(0, 1)
            v[b, :, lens[b]:lens[b] + T] = st["v"][b].double().transpose(0, 1)
        else:
            k[b] = _stored64(kb.to(torch.bfloat16)).transpose(0, 1)
            v[b] = _stored64(st["v"][b]).transpose(0, 1)
    return q, k, v
