"""Plain 64-bit forms of the rotary tables, the norms with the rotation and
their gradients, the quantised append and the decode over 8-bit pages, for the
tests: written from the definitions in include/fa.h, nothing of the library in
them.  Tensors may be on any device; everything is float64."""
import math

import torch

PS = 256
FP8 = torch.float8_e4m3fn


def frequencies(R, base=10000.0, scaling="none", factor=1.0, original=0, low=1.0, high=4.0):
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    out = []
    for i in range(R // 2):
        w = base ** (-2.0 * i / R)
        if scaling == "linear":
            w = w / factor
        elif scaling == "turns":
            a = (original * w / (2 * math.pi) - low) / (high - low)
            a = min(max(a, 0.0), 1.0)
            w = a * w + (1 - a) * w / factor
        elif scaling == "yarn":
            def pair(n):
                return R * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))
            first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), R - 1)
            a = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            w = (1 - a) * w + a * w / factor
        out.append(w)
    return torch.tensor(out, dtype=torch.float64)


def tables(max_pos, R, mscale=1.0, **kw):
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * frequencies(R, **kw)
    return ang.cos() * mscale, ang.sin() * mscale


def rotate(x, cos, sin, interleaved, back=False):
    """x [tokens, heads, d]; cos, sin [tokens, R/2] (of each token's position)."""
    R = 2 * cos.shape[1]
    y = x.clone()
    if R == 0:
        return y
    c, s = cos[:, None].double(), sin[:, None].double()
    if back:
        s = -s
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def norm(x, w, eps):
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def norm_rope(x, w, cos, sin, interleaved, eps):
    return rotate(norm(x.double(), w, eps), cos, sin, interleaved)


def norm_rope_bwd(x, g, w, cos, sin, interleaved, eps):
    """(dx, dw, size of dx's terms, sum of |terms| of dw)."""
    g = rotate(g.double(), cos, sin, interleaved, back=True)
    if w is None:
        return g, None, g.abs(), None
    x, w = x.double(), w.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    hat = x * r
    m = (g * w * hat).mean(-1, keepdim=True)
    dx = r * (g * w - hat * m)
    size = r * ((g * w).abs() + (hat * (g * w * hat).abs().mean(-1, keepdim=True)).abs())
    return dx, (g * hat).sum((0, 1)), size, (g * hat).abs().sum((0, 1))


def bf16_bound(ref):
    """How far a bf16 result computed in fp32 may be from `ref` [..., d]: half a
    bf16 step of the value (2^-8), and the fp32 steps before it.  Those are, of
    2^-24 each: a sum of d squares (12 additions deep, halved by the root), a
    root of 2 ulp (2^-22), the products by the root and the weight, and two
    products and a sum of the rotation: under 2^-20 of |a| + |b|, the pair that
    a value is rotated from, which is at most twice the row's largest value."""
    return 2.0 ** -8 * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True) + 1e-38


def pages_of(lens):
    return [(max(int(n), 0) + PS - 1) // PS for n in lens]


def page_list(table, lens, b):
    """Sequence b's pages, of a packed table or a block table."""
    n = pages_of(lens)
    if table.dim() == 2:
        return table[b, :n[b]].tolist()
    at = sum(n[:b])
    return table[at:at + n[b]].tolist()


def least_scale(a):
    """The least power of two s in [2^-64, 2^64] with a <= 448 s."""
    e = -64
    while e < 64 and a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def e4m3(x):
    """float64 -> the nearest e4m3 code (ties to even), NaN beyond 448."""
    x = torch.where(x.abs() <= 448.0, x, math.nan)
    # the step at |x|: 2^(e-3) in the binade 2^e, 2^-9 below 2^-6; exact in 64 bits
    e = torch.frexp(x.abs())[1].double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return (torch.round(x / step) * step).float().to(FP8)


def gather(pages, scales, page_ids, n):
    """float64 [n, heads, d]: codes times scales of a sequence's first n tokens."""
    ids = torch.tensor(page_ids, dtype=torch.long, device=pages.device)
    x = pages.view(torch.uint8)[ids].view(FP8).double()
    block = PS // scales.shape[2]
    x = x * scales[ids].double().repeat_interleave(block, 2)[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, pages.shape[1], pages.shape[3])[:n]


def decode(q, kp, vp, ks, vs, table, lens, scale):
    """o, lse, and for the bounds: sum of p |v|, and the largest scale * sum |q||k|."""
    B, H, d = q.shape
    Hk = kp.shape[1]
    o = torch.zeros((B, H, d), dtype=torch.float64, device=q.device)
    absv, lse = torch.zeros_like(o), torch.full((B, H), -math.inf, dtype=torch.float64,
                                                device=q.device)
    reach = torch.zeros((B, H), dtype=torch.float64, device=q.device)
    for b, n in enumerate(int(x) for x in lens):
        if n <= 0:
            continue
        ids = page_list(table, lens, b)
        k, v = gather(kp, ks, ids, n), gather(vp, vs, ids, n)
        qb = q[b].double().view(Hk, H // Hk, d)
        s = torch.einsum("hgd,lhd->hgl", qb, k) * scale
        p = torch.softmax(s, -1)
        o[b] = torch.einsum("hgl,lhd->hgd", p, v).reshape(H, d)
        absv[b] = torch.einsum("hgl,lhd->hgd", p, v.abs()).reshape(H, d)
        lse[b] = torch.logsumexp(s, -1).reshape(H)
        reach[b] = (torch.einsum("hgd,lhd->hgl", qb.abs(), k.abs()).amax(-1) *
                    abs(scale)).reshape(H)
    return o, lse, absv, reach
