"""Plain float64 forms (torch, CPU) of the learned-norm append, its backward, the 4-bit
row and attention over it, written from the formulas in gqa.h."""
import math

import torch

F64 = torch.float64


# ---------------------------------------------------------------------------
# norm, rotation
# ---------------------------------------------------------------------------
def thetas(D, base=10000.0):
    return base ** (-2.0 * torch.arange(D // 2, dtype=F64) / D)


def positions(pos0, B, T, pos=None, pair_axis=None, D=128):
    """Position [B, T, D/2] of every token's rotation pairs."""
    if pos is None:
        p0 = torch.zeros(B, dtype=F64) if pos0 is None else pos0.to(F64)
        p = p0.view(B, 1) + torch.arange(T, dtype=F64)
        return p.unsqueeze(-1).expand(B, T, D // 2)
    pos = pos.reshape(-1, B, T).to(F64)
    pair_axis = torch.zeros(D // 2, dtype=torch.long) if pair_axis is None else pair_axis
    return pos[pair_axis].permute(1, 2, 0)


def norm_rope(x, P, gain=None, qk_norm=True, eps=1e-6, base=10000.0, mscale=1.0, theta=None):
    """mscale R(P) (gain x (mean x^2 + eps)^-1/2) of x [B, T, H, D]; differentiable."""
    x = x.to(F64)
    D = x.shape[-1]
    if qk_norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if gain is not None:
            x = x * gain.to(F64)
    ang = (P * (thetas(D, base) if theta is None else theta)).unsqueeze(2)
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = x[..., :D // 2], x[..., D // 2:]
    return mscale * torch.cat((a * c - b * s, a * s + b * c), dim=-1)


def norm_rope_grad(x, dy, P, gain=None, qk_norm=True, eps=1e-6, base=10000.0):
    """(dx, d gain) by the formula: w = R^T dy, z = gain w,
    dx = r z - x r^3 mean(x z), d gain = sum w x r."""
    x, dy = x.to(F64), dy.to(F64)
    D = x.shape[-1]
    ang = (P * thetas(D, base)).unsqueeze(2)
    c, s = torch.cos(ang), torch.sin(ang)
    a, b = dy[..., :D // 2], dy[..., D // 2:]
    w = torch.cat((a * c + b * s, b * c - a * s), dim=-1)
    if not qk_norm:
        return w, None
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    z = w if gain is None else w * gain.to(F64)
    dx = r * z - x * r ** 3 * (x * z).mean(-1, keepdim=True)
    return dx, (w * x * r).sum(dim=(0, 1, 2))


# ---------------------------------------------------------------------------
# the 4-bit row
# ---------------------------------------------------------------------------
def group_index(D):
    """[D/32, 32] coordinates of each group."""
    g = torch.arange(D // 32).view(-1, 1) * 16 + torch.arange(16)
    return torch.cat((g, g + D // 2), dim=1)


def byte_of_pair(D):
    """Byte of each rotation pair 0 .. D/2 - 1 within a row."""
    p = torch.arange(D // 2)
    return 4 * (D // 32 * ((p % 16) // 4) + p // 16) + p % 4


def quantise(x):
    """bf16 rows [n, D] -> (c [n, D] int, s, m [n, D/32] float64, near [n, D] bool).
    near: quotients within 2^-19 of themselves above n + 1/2, where c or c - 1 may be
    kept."""
    n, D = x.shape
    idx = group_index(D)
    y = x.to(F64)[:, idx]                                      # [n, D/32, 32]
    ok = torch.isfinite(y).all(-1)
    y = torch.where(ok.unsqueeze(-1), y, torch.zeros_like(y))
    m = y.amin(-1)
    s = ((y.amax(-1) - m) / 15).to(torch.bfloat16).to(F64)
    s = torch.where(s >= 2.0 ** -126, s, torch.zeros_like(s))
    quo = (y - m.unsqueeze(-1)) / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)
    quo = torch.where((s > 0).unsqueeze(-1), quo, torch.zeros_like(quo))
    c = torch.ceil(quo - 0.5).clamp_(min=0)
    over = quo - (c - 0.5)
    near = (over > 0) & (over <= 2.0 ** -19 * quo)
    m = torch.where(ok, m, torch.full_like(m, math.nan))
    s = torch.where(ok, s, torch.zeros_like(s))
    out_c = torch.zeros(n, D, dtype=torch.long)
    out_near = torch.zeros(n, D, dtype=torch.bool)
    out_c[:, idx] = c.long()
    out_near[:, idx] = near
    return out_c, s, m, out_near


def unpack_codes(codes):
    """Code bytes [..., D/2] -> codes [..., D]."""
    D = 2 * codes.shape[-1]
    byte = codes[..., byte_of_pair(D)].long()
    return torch.cat((byte & 15, byte >> 4), dim=-1)


def pack(x):
    """bf16 [..., D] -> (codes uint8 [..., D/2], scales bf16 [..., D/32, 2])."""
    D = x.shape[-1]
    c, s, m, _ = quantise(x.reshape(-1, D))
    codes = torch.empty(c.shape[0], D // 2, dtype=torch.uint8)
    codes[:, byte_of_pair(D)] = (c[:, :D // 2] + 16 * c[:, D // 2:]).to(torch.uint8)
    scales = torch.stack((s, m), dim=-1).to(torch.bfloat16)
    return codes.view(*x.shape[:-1], D // 2), scales.view(*x.shape[:-1], D // 32, 2)


def values(codes, scales):
    """The float64 values [..., D] that codes and scales stand for."""
    D = 2 * codes.shape[-1]
    grp = (torch.arange(D) % (D // 2)) // 16
    s, m = scales[..., 0].to(F64)[..., grp], scales[..., 1].to(F64)[..., grp]
    return m + s * unpack_codes(codes)


# ---------------------------------------------------------------------------
# attention of one token over a 4-bit cache, and what its kernel may be off by
# ---------------------------------------------------------------------------
U32 = 2.0 ** -23           # one unit of an fp32 accumulator that cuts off


def decode(q, cache, lens, scale=None):
    """(out, tolerance) float64 [B, Hq, D]; cache = (k_codes, k_scales, v_codes, v_scales).

    The tolerance counts the roundings of the scheme that the header of the kernel's
    source describes, each at its worst:
      * a score is sum over groups of s sum(q c) + m sum(q): products exact (sum(q) in
        24 bits), at most 36 additions each within U32 of the sum of magnitudes A_q =
        sum |q| (15 s + |m|), so off by d = 36 U32 A_q scale, and a few fp32 units of
        the score in the scaling and the exponential;
      * that moves p by up to 2 d of itself in numerator and denominator together;
      * p s is rounded once to fp16 (11 significant bits: half a step is 2^-11 of the
        value, torch.finfo(torch.float16).eps / 2), 2^-11 of each product p s c with
        c <= 15; additions
        over the keys of a warp (at most 64 at the tests' sizes) and the merges within
        80 U32 of sum p (15 s + |m|);
      * the result's rounding to bf16, 2^-8 of it."""
    kc, ks, vc, vs = cache
    B, Hq, D = q.shape
    Hkv = kc.shape[1]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, tol = torch.zeros(B, Hq, D, dtype=F64), torch.zeros(B, Hq, D, dtype=F64)
    grp = (torch.arange(D) % (D // 2)) // 16
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            K, V = values(kc[b, h, :n], ks[b, h, :n]), values(vc[b, h, :n], vs[b, h, :n])
            x = q[b, h * g:(h + 1) * g].to(F64)
            sc = x @ K.T * scale
            p = torch.softmax(sc, dim=-1)
            o = p @ V
            s_k, m_k = ks[b, h, :n].to(F64)[..., 0][:, grp], ks[b, h, :n].to(F64)[..., 1][:, grp]
            mag = x.abs() @ (15 * s_k + m_k.abs()).T * scale
            d = (36 * U32 * mag + 8 * U32 * (sc.abs() + 1)).amax(-1, keepdim=True)
            s_v, m_v = vs[b, h, :n].to(F64)[..., 0][:, grp], vs[b, h, :n].to(F64)[..., 1][:, grp]
            e = 2 * d * (p @ V.abs()) + 2.0 ** -11 * 15 * (p @ s_v)
            e = e + 80 * U32 * (p @ (15 * s_v + m_v.abs()))
            out[b, h * g:(h + 1) * g] = o
            tol[b, h * g:(h + 1) * g] = 2.0 ** -8 * o.abs() + 1.01 * e
    return out, tol
