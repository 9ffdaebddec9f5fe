"""The operators around a serving step with an 8-bit cache and the training step
of its query and key heads, as cases that can be timed and checked:

  rope_table        the cos/sin tables of rotary positions, scaled for long contexts
  qk_norm_rope      norms of queries and keys for each head, with the rotation, and its gradients
  append_rope       new queries and keys normed and rotated, keys and values into a paged cache
  append_fp8        the same into a cache of 8-bit values, a scale for each block of tokens and head
  decode_fp8        attention of one query token per sequence over that 8-bit cache

Where `own` is false, run() computes them with elementary torch operations;
where it is true it calls attn_fwd_04_b200.
"""
import math

import torch

own = False

PAGE = 256
E4M3 = torch.float8_e4m3fn


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # tables at start-up: an ordinary context, and 128K positions with the
        # frequencies blended for a context four times the trained one
        dict(name="table_4k", op="rope_table", max_pos=4096, rot=128, base=10000.0,
             scaling="none", factor=1.0, original=0, low=0.0, high=0.0, mscale=1.0),
        dict(name="table_128k", op="rope_table", max_pos=131072, rot=128, base=500000.0,
             scaling="yarn", factor=4.0, original=32768, low=1.0, high=32.0, mscale=1.1386),
        # one new token of each of 64 sequences: latency
        dict(name="norm_rope_64_rows", op="norm_rope", layout="packed", B=64, N=1, H=32, Hkv=8,
             d=128, rot=128, interleaved=False, norm="bf16", max_pos=32768),
        # the long-prefill layout [1, H, 16384, d] with grouped heads
        dict(name="norm_rope_prefill_16k", op="norm_rope", layout="heads", B=1, N=16384, H=32,
             Hkv=8, d=128, rot=128, interleaved=False, norm="fp32", max_pos=16384),
        # a training step over packed sequences of 1024 to 8192 tokens
        dict(name="norm_rope_bwd_varlen", op="norm_rope_bwd", layout="packed", B=8, N=4600, H=32,
             Hkv=8, d=128, rot=128, interleaved=False, norm="fp32", max_pos=8192),
        # serving, bf16 cache: a decode step of 64 sequences; eight prompts of mixed lengths
        # with an interleaved rotation of half the head
        dict(name="append_rope_64_tokens", op="append_rope", B=64, lo=1, hi=1, lens=5, ctx_lo=1024,
             ctx_hi=4096, H=32, Hkv=8, d=128, rot=128, interleaved=False, norm="bf16",
             table="packed"),
        dict(name="append_rope_prompts", op="append_rope", B=8, lo=1024, hi=8192, lens=5, ctx_lo=0,
             ctx_hi=600, H=32, Hkv=8, d=128, rot=64, interleaved=True, norm="none",
             table="rows"),
        # serving, 8-bit cache: the same step; chunks of 1024 tokens behind cached context
        dict(name="append_fp8_64_tokens", op="append_fp8", B=64, lo=1, hi=1, lens=5, ctx_lo=1024,
             ctx_hi=4096, H=32, Hkv=8, d=128, rot=128, interleaved=False, norm="bf16",
             table="packed", block=64),
        dict(name="append_fp8_chunks", op="append_fp8", B=8, lo=1024, hi=1024, lens=5, ctx_lo=1024,
             ctx_hi=8192, H=32, Hkv=32, d=128, rot=128, interleaved=False, norm="none",
             table="rows", block=64),
        # one user with a short context: latency
        dict(name="decode_fp8_1_user", op="decode_fp8", B=1, lo=777, hi=777, lens=5, H=32,
             Hkv=8, d=128, table="packed", block=64),
        # 64 sequences of 1K to 32K tokens, grouped heads
        dict(name="decode_fp8_64_users", op="decode_fp8", B=64, lo=1024, hi=32768, lens=5,
             H=32, Hkv=8, d=128, table="packed", block=64),
        # a head of the cache for every query head, 1K to 16K tokens: the most to read
        dict(name="decode_fp8_64_users_mha", op="decode_fp8", B=64, lo=1024, hi=16384, lens=5,
             H=32, Hkv=32, d=128, table="rows", block=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope_table", "norm_rope", "norm_rope_bwd", "append_rope", "append_fp8",
                     "decode_fp8", "decode_fp8"])
    if op == "rope_table":
        scaling = rng.choice(["none", "linear", "ntk", "turns", "yarn"])
        low, high = {"turns": (1.0, 4.0), "yarn": (1.0, 32.0)}.get(scaling, (0.0, 0.0))
        return dict(op=op, max_pos=log(16, 131072), rot=16 * rng.randint(2, 8),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 2.5]),
                    original=rng.choice([2048, 4096, 8192]), low=low, high=high,
                    mscale=rng.choice([1.0, 1.2079]))
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 5])
    heads = dict(H=Hkv * rng.choice([1, 2, 3, 4, 7, 8]), Hkv=Hkv, d=d)
    turn = dict(rot=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.4,
                norm=rng.choice(["none", "fp32", "bf16"]))
    table = rng.choice(["packed", "rows"])
    if op in ("norm_rope", "norm_rope_bwd"):
        rows = log(1, 12000)
        B = rng.choice([1, 2, 3, 8])
        return dict(op=op, layout=rng.choice(["packed", "heads"]), B=B, N=max(1, rows // B),
                    **heads, **turn, max_pos=16384)
    if op in ("append_rope", "append_fp8"):
        if rng.random() < 0.5:
            new = dict(B=log(1, 200), lo=1, hi=1)  # a decode step
        else:
            B = log(1, 12)
            new = dict(B=B, lo=0 if B > 2 else 1, hi=log(2, 12000 // B))  # prompts, some empty
        case = dict(op=op, lens=rng.randrange(1000), **new, ctx_lo=0, ctx_hi=log(1, 3000),
                    **heads, **turn, table=table)
        return dict(case, block=rng.choice([16, 32, 64, 128, 256])) if op == "append_fp8" else case
    B = log(1, 64)
    most = min(32768, (1 << 30) // (B * Hkv * d))
    hi = log(1, most)
    lo = rng.choice([0 if B > 2 else 1, 1, max(1, hi // 2), hi])
    return dict(op=op, lens=rng.randrange(1000), B=B, lo=lo, hi=hi,
                H=Hkv * rng.choice([1, 1, 2, 4, 7, 8, 16, 24, 32]), Hkv=Hkv, d=d, table=table,
                block=rng.choice([16, 32, 64, 128, 256]))


# ---- what a user's program has in hand ----------------------------------------

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _lengths(case):
    """The cached tokens and the new ones of each sequence: the case's own,
    whatever the seed, so that its outputs keep their shapes."""
    g, n = _gen(case["lens"], "cpu"), (case["B"],)
    new = torch.randint(case["lo"], case["hi"] + 1, n, generator=g)
    if "ctx_lo" not in case:
        return new, new
    return new + torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, n, generator=g), new


def _bf16(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)


def _tables(max_pos, rot):
    """cos and sin of p * 10000^(-2i/rot), as the caller keeps them."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    p = torch.arange(max_pos, device="cuda", dtype=torch.float64)
    angle = p[:, None] * 10000.0 ** (-2.0 * i / rot)
    return angle.cos().float(), angle.sin().float()


def _weights(case, g):
    if case["norm"] == "none":
        return None, None
    dtype = torch.float32 if case["norm"] == "fp32" else torch.bfloat16
    return tuple((1 + 0.2 * torch.randn(case["d"], generator=g, device="cuda")).to(dtype)
                 for _ in range(2))


def _qkv(total, case, g):
    """Queries, keys and values as views of one projection's output."""
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    qkv = _bf16((total, (H + 2 * Hkv) * d), g)
    return (qkv[:, :H * d].view(total, H, d),
            qkv[:, H * d:(H + Hkv) * d].view(total, Hkv, d),
            qkv[:, (H + Hkv) * d:].view(total, Hkv, d))


def _page_tables(case, lens, seed):
    """The pool's size and the page table: packed, or one row for each sequence."""
    pages = (lens + PAGE - 1) // PAGE
    P = max(1, int(pages.sum()))
    perm = torch.randperm(P, generator=_gen(seed, "cpu")).to(torch.int32)
    if case["table"] == "packed":
        return P, perm.cuda()
    width = max(1, int(pages.max()))
    rows = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages.tolist()):
        rows[b, :n] = perm[at:at + n]
        at += n
    return P, rows.cuda()


def _codes(shape, g):
    """8-bit values as a quantiser leaves them: about normal, the largest near the format's end."""
    out = torch.empty(shape, device="cuda", dtype=E4M3)
    step = max(1, (1 << 26) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        x = torch.randn((n,) + tuple(shape[1:]), generator=g, device="cuda").mul_(110.0)
        out[i:i + n] = x.clamp_(-448.0, 448.0).to(E4M3)
    return out


def prepare(case, seed):
    g = _gen(1000 + seed)
    op, s = case["op"], dict(case)
    if op == "rope_table":
        # the base moves a little with the seed, so that other seeds are other tables
        s["base"] = case["base"] * (1.0 + (seed % 997) * 1e-4)
        return s
    if op in ("norm_rope", "norm_rope_bwd"):
        B, N, H, Hkv, d = (case[k] for k in ("B", "N", "H", "Hkv", "d"))
        s["qw"], s["kw"] = _weights(case, g)
        s["cos"], s["sin"] = _tables(case["max_pos"], case["rot"])
        if case["layout"] == "packed":
            s["q"], s["k"], _ = _qkv(B * N, case, g)
            if N == 1:  # one token each, anywhere in its sequence
                pos = torch.randint(0, case["max_pos"], (B,), generator=g, device="cuda")
            else:
                pos = torch.arange(N, device="cuda").repeat(B)
            s["pos"] = pos.to(torch.int32)
            shapes = (B * N, H, d), (B * N, Hkv, d)
        else:
            shapes = (B, H, N, d), (B, Hkv, N, d)
            s["q"], s["k"], s["pos"] = _bf16(shapes[0], g), _bf16(shapes[1], g), None
        if op == "norm_rope_bwd":
            s["gq"], s["gk"] = _bf16(shapes[0], g, 0.1), _bf16(shapes[1], g, 0.1)
        return s
    Hkv, d, B = case["Hkv"], case["d"], case["B"]
    if op == "decode_fp8":
        lens, _ = _lengths(case)
        P, s["table_t"] = _page_tables(case, lens, seed + 1)
        s["q"] = _bf16((B, case["H"], d), g, 2.0)
        for n in ("k", "v"):
            s[n + "p"] = _codes((P, Hkv, PAGE, d), g)
            u = torch.rand((P, Hkv, PAGE // case["block"]), generator=g, device="cuda")
            s[n + "s"] = (0.004 + 0.008 * u)
        # behind a sequence's end there is whatever was there before: not numbers
        first = torch.cumsum((lens + PAGE - 1) // PAGE, 0) - (lens + PAGE - 1) // PAGE
        for b, n in enumerate(lens.tolist()):
            if n % PAGE:
                t = s["table_t"]
                page = int(t[int(first[b]) + n // PAGE] if t.dim() == 1 else t[b, n // PAGE])
                for m in ("k", "v"):
                    s[m + "p"][page].view(torch.uint8)[:, n % PAGE:] = 0x7F
                    s[m + "s"][page][:, -(-(n % PAGE) // case["block"]):] = math.nan
        s["seq"] = lens.to(torch.int32).cuda()
        return s
    lens, new = _lengths(case)
    P, s["table_t"] = _page_tables(case, lens, seed + 2)
    s["q"], s["k"], s["v"] = _qkv(int(new.sum()), case, g)
    s["qw"], s["kw"] = _weights(case, g)
    s["cos"], s["sin"] = _tables(16384, case["rot"])
    s["seq"] = lens.to(torch.int32).cuda()
    s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).cuda()
    for n in ("k", "v"):
        if op == "append_fp8":
            s[n + "p"] = _codes((P, Hkv, PAGE, d), g)
            # cached blocks of smaller and larger values than the new ones
            e = torch.randint(-9, -5, (P, Hkv, PAGE // case["block"]), generator=g, device="cuda")
            s[n + "s"] = torch.exp2(e.float())
        else:
            s[n + "p"] = _bf16((P, Hkv, PAGE, d), g)
    return s


# ---- one pass -------------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        return _own(op, s)
    return {"rope_table": _table, "norm_rope": _norm_rope, "norm_rope_bwd": _norm_rope_bwd,
            "append_rope": _append_rope, "append_fp8": _append_fp8,
            "decode_fp8": _decode_fp8}[op](s)


def _own(op, s):
    import attn_fwd_04_b200 as fa
    if op == "rope_table":
        return fa.fa_rope_table(s["max_pos"], s["rot"], s["base"], s["scaling"], s["factor"],
                                s["original"], s["low"], s["high"], s["mscale"])
    if op == "norm_rope":
        return fa.fa_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"],
                                  eps=1e-6, interleaved=s["interleaved"])
    if op == "norm_rope_bwd":
        return fa.fa_qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], s["qw"], s["kw"],
                                      s["cos"], s["sin"], s["pos"], eps=1e-6,
                                      interleaved=s["interleaved"])
    if op == "append_rope":
        q = fa.fa_append_paged_rope(s["q"], s["k"], s["v"], s["cu"], s["kp"], s["vp"],
                                    s["table_t"], s["seq"], s["cos"], s["sin"], s["qw"],
                                    s["kw"], eps=1e-6, interleaved=s["interleaved"])
        return q, s["kp"], s["vp"]
    if op == "append_fp8":
        q = fa.fa_append_paged_fp8(s["q"], s["k"], s["v"], s["cu"], s["kp"], s["vp"], s["ks"],
                                   s["vs"], s["table_t"], s["seq"], s["cos"], s["sin"],
                                   s["qw"], s["kw"], eps=1e-6, interleaved=s["interleaved"])
        return q, s["kp"], s["vp"], s["ks"], s["vs"]
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    o = fa.fa_decode_paged_fp8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table_t"],
                               s["seq"], lse=lse)
    return o, lse


def _frequencies(s):
    """The angle of each pair and position, in 64 bits."""
    R, base, f = s["rot"], s["base"], s["factor"]
    i = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    if s["scaling"] == "ntk":
        base = base * f ** (R / (R - 2.0))
    inv = base ** (-2.0 * i / R)
    if s["scaling"] == "linear":
        return inv / f
    if s["scaling"] == "turns":  # by the turns a pair makes within the trained context
        turns = s["original"] * inv / (2 * math.pi)
        keep = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        return inv * (keep + (1 - keep) / f)
    if s["scaling"] == "yarn":  # a ramp over the pairs between two numbers of turns
        def pair(turns):
            return R * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(pair(s["high"])), 0), min(math.ceil(pair(s["low"])), R - 1)
        ramp = ((i - first) / max(last - first, 0.001)).clamp(0, 1)
        return inv * (1 - ramp) + inv / f * ramp
    return inv


def _table(s):
    p = torch.arange(s["max_pos"], device="cuda", dtype=torch.float64)
    angle = p[:, None] * _frequencies(s)
    return (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()


def _turn(x, cos, sin, rot, interleaved):
    """The first `rot` values of each row of x (32 bits) rotated in pairs."""
    part = x[..., :rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _rows(s, name):
    """cos or sin of each token, to go with x[..., pairs]."""
    t = s[name]
    if s["pos"] is None:
        return t[:s["q"].shape[2]]
    return t[s["pos"].long()][:, None]


def _normed(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _norm_rope(s):
    cos, sin = _rows(s, "cos"), _rows(s, "sin")
    q = _turn(_normed(s["q"], s["qw"]), cos, sin, s["rot"], s["interleaved"])
    k = _turn(_normed(s["k"], s["kw"]), cos, sin, s["rot"], s["interleaved"])
    return q.to(torch.bfloat16), k.to(torch.bfloat16)


def _grad(x, g, w, cos, sin, s):
    g = _turn(g.float(), cos, -sin, s["rot"], s["interleaved"])
    if w is None:
        return g.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    gw = g * w.float()
    dx = r * (gw - x * (r * r * (gw * x).mean(-1, keepdim=True)))
    dw = (g * (x * r)).sum(tuple(range(x.dim() - 1)), dtype=torch.float64)
    return dx.to(torch.bfloat16), dw.float()


def _norm_rope_bwd(s):
    cos, sin = _rows(s, "cos"), _rows(s, "sin")
    dq, dqw = _grad(s["q"], s["gq"], s["qw"], cos, sin, s)
    dk, dkw = _grad(s["k"], s["gk"], s["kw"], cos, sin, s)
    return dq, dk, dqw, dkw


def _places(s):
    """Sequence, position, page and slot of each new row."""
    cu, lens, t = s["cu"].long(), s["seq"].long(), s["table_t"]
    new = cu[1:] - cu[:-1]
    total = s["k"].shape[0]
    b = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), new, output_size=total)
    pos = lens[b] - new[b] + torch.arange(total, device="cuda") - cu[b]
    if t.dim() == 1:
        pages = (lens + PAGE - 1) // PAGE
        page = t[(pages.cumsum(0) - pages)[b] + pos // PAGE]
    else:
        page = t[b, pos // PAGE]
    return b, pos, page.long(), pos % PAGE, lens - new, new


def _turned_new(s, pos):
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    q = _turn(_normed(s["q"], s["qw"]), cos, sin, s["rot"], s["interleaved"])
    k = _turn(_normed(s["k"], s["kw"]), cos, sin, s["rot"], s["interleaved"])
    return q.to(torch.bfloat16), k


def _append_rope(s):
    _, pos, page, slot, _, _ = _places(s)
    q, k = _turned_new(s, pos)
    s["kp"][page, :, slot] = k.to(torch.bfloat16)
    s["vp"][page, :, slot] = s["v"]
    return q, s["kp"], s["vp"]


def _append_fp8(s):
    """A block's scale is the least power of two whose 448-fold covers its new
    values; cached values of the block keep their larger scale, or are rounded
    anew where the scale grows."""
    b, pos, page, slot, start, new = _places(s)
    q, k = _turned_new(s, pos)
    _store8(s["kp"], s["ks"], k, b, pos, page, slot, start, new, s)
    _store8(s["vp"], s["vs"], s["v"].float(), b, pos, page, slot, start, new, s)
    return q, s["kp"], s["vp"], s["ks"], s["vs"]


def _store8(pages, scales, x, b, pos, page, slot, start, new, s):
    block = s["block"]
    Hkv, d, P = pages.shape[1], pages.shape[3], pages.shape[0]
    per = PAGE // block
    size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    most = torch.zeros((P * per, Hkv), device="cuda")
    at = page * per + slot // block
    most.scatter_reduce_(0, at[:, None].expand(-1, Hkv), size, "amax")
    m, e = torch.frexp(most)
    e = torch.where(most > 0, e - 8 - (m <= 0.875).int(), -64)
    need = torch.exp2(e.clamp(-64, 64).float())
    touched = torch.zeros(P * per, dtype=torch.bool, device="cuda")
    touched[at] = True
    # the block in which a sequence's new rows begin, where it has cached rows before them
    t = s["table_t"]
    seq = torch.arange(len(start), device="cuda")
    edge = (start // PAGE).clamp(max=(t.shape[-1] - 1))
    if t.dim() == 1:
        n = (s["seq"].long() + PAGE - 1) // PAGE
        first_page = t[(n.cumsum(0) - n + edge).clamp(max=len(t) - 1)].long()
    else:
        first_page = t[seq, edge].long()
    joins = (new > 0) & (start % block > 0)
    first_page = torch.where(joins, first_page, 0)
    join_at = first_page * per + (start % PAGE) // block
    old = torch.zeros((P * per + 1, Hkv), device="cuda")
    old_scale = scales.transpose(1, 2).reshape(P * per, Hkv)
    old[torch.where(joins, join_at, P * per)] = old_scale[join_at]
    old = old[:-1]
    fresh = torch.where(touched[:, None], torch.maximum(old, need), old_scale)
    # the cached rows of such blocks under the new scale
    codes = pages.view(torch.uint8).view(P, Hkv, per, block, d)
    blk = (start % PAGE) // block
    have = codes[first_page, :, blk]
    ratio = (old_scale[join_at] / fresh[join_at])[:, :, None, None]
    moved = (have.view(E4M3).float() * ratio).to(E4M3).view(torch.uint8)
    row = torch.arange(block, device="cuda")
    mine = (joins[:, None] & (row < (start % block)[:, None]))[:, None, :, None]
    w_seq, w_row = torch.nonzero(mine[:, 0, :, 0], as_tuple=True)
    codes[first_page[w_seq], :, blk[w_seq], w_row] = moved[w_seq, :, w_row]
    scales.copy_(fresh.view(P, per, Hkv).transpose(1, 2))
    y = (x / fresh[at][:, :, None]).to(E4M3)
    pages.view(torch.uint8)[page, :, slot] = y.view(torch.uint8)


def _decode_fp8(s):
    lens, t, block = s["seq"].long(), s["table_t"], s["block"]
    B, H, d = s["q"].shape
    Hkv = s["kp"].shape[1]
    L = max(1, s["hi"])
    j = torch.arange(L, device="cuda")
    live = j < lens[:, None]
    if t.dim() == 1:
        n = (lens + PAGE - 1) // PAGE
        entry = (n.cumsum(0) - n)[:, None] + j // PAGE
        page = t[entry.clamp(max=len(t) - 1)].long()
    else:
        page = t[:, (j // PAGE).clamp(max=t.shape[1] - 1)].long()
    page = torch.where(live, page, 0)[:, :, None]
    head, slot = torch.arange(Hkv, device="cuda"), (j % PAGE)[:, None]

    def rows(pages, scales):
        x = pages.view(torch.uint8)[page, head, slot].view(E4M3).float()
        x *= scales[page, head, slot // block][..., None]
        return x.masked_fill_(~live[:, :, None, None], 0.0)

    q = s["q"].float().view(B, Hkv, H // Hkv, d)
    score = torch.einsum("bhgd,blhd->bhgl", q, rows(s["kp"], s["ks"])) * d ** -0.5
    score.masked_fill_(~live[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", p, rows(s["vp"], s["vs"])) / total.clamp(min=1e-30)
    lse = (top + torch.log(total)).view(B, H)
    return o.reshape(B, H, d).to(torch.bfloat16), lse


# ---- what a pass cannot do without -------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope_table":
        n = case["max_pos"] * case["rot"] // 2
        return {"bytes": 8.0 * n, "flops": 4.0 * n}
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if op in ("norm_rope", "norm_rope_bwd"):
        rows = case["B"] * case["N"]
        x = rows * (H + Hkv) * d
        tokens = min(rows, case["max_pos"]) if case["layout"] == "packed" else case["N"]
        table = tokens * case["rot"] * 4.0 + (4.0 * rows if case["layout"] == "packed" else 0)
        if op == "norm_rope":
            return {"bytes": 4.0 * x + table, "flops": 8.0 * x}
        reads = 3 if case["norm"] != "none" else 2  # x, the output's gradient, the input's
        return {"bytes": 2.0 * reads * x + table, "flops": 16.0 * x}
    if op == "decode_fp8":
        tokens = float(_lengths(case)[0].sum())
        return {"bytes": tokens * Hkv * (2.0 * d + 8.0 / case["block"])
                + case["B"] * H * (4.0 * d + 4.0) + tokens / PAGE * 4,
                "flops": 4.0 * tokens * H * d}
    rows = float(_lengths(case)[1].sum())
    q = rows * H * d * 4.0
    table = min(rows, 16384) * case["rot"] * 4.0
    cell = 2.0 if op == "append_rope" else 1.0
    return {"bytes": q + rows * Hkv * d * 2 * (2.0 + cell) + table + case["B"] * 8.0,
            "flops": 8.0 * rows * (H + Hkv) * d}


# ---- the same from the definition, in 64 bits ----------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope_table":
        return _exact_table(s)
    if op in ("norm_rope", "norm_rope_bwd"):
        return _exact_norm_rope(s, op == "norm_rope_bwd")
    if op == "decode_fp8":
        return _exact_decode(s)
    return _exact_append(s, op == "append_fp8")


def _exact_table(s):
    R, f, k = s["rot"], s["factor"], s["scaling"]
    inv = []
    for i in range(R // 2):
        base = s["base"] * (f ** (R / (R - 2)) if k == "ntk" else 1.0)
        w = base ** (-2 * i / R)
        if k == "linear":
            w /= f
        elif k == "turns":
            turns = s["original"] * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - s["low"]) / (s["high"] - s["low"])))
            w = keep * w + (1 - keep) * w / f
        elif k == "yarn":
            at = [R * math.log(s["original"] / (n * 2 * math.pi)) / (2 * math.log(base))
                  for n in (s["high"], s["low"])]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
            share = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            w = w / f * share + w * (1 - share)
        inv.append(w)
    p = torch.arange(s["max_pos"], device="cuda", dtype=torch.float64)
    z = torch.polar(torch.full((s["max_pos"], R // 2), s["mscale"], device="cuda",
                               dtype=torch.float64),
                    torch.outer(p, torch.tensor(inv, device="cuda", dtype=torch.float64)))
    return z.real.contiguous(), z.imag.contiguous()


def _as_complex(x, rot, interleaved):
    """The rotated part of x's rows as complex numbers, a pair each."""
    if interleaved:
        return torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous())
    return torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())


def _exact_turn(x, z, rot, interleaved):
    y = x.clone()
    w = _as_complex(x, rot, interleaved) * z
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    return y


def _exact_norm_rope(s, backward):
    out, sums = [], []
    # tokens first: [tokens, heads, d], the table's row of each token beside it
    packed = s["pos"] is not None
    for n in ("q", "k"):
        x = s[n].double() if packed else s[n].transpose(1, 2).double()
        shape = x.shape
        x = x.reshape(-1, x.shape[-2], x.shape[-1])
        at = s["pos"].long() if packed else torch.arange(shape[1], device="cuda").repeat(shape[0])
        z = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
        w = s[n + "w"].double() if s[n + "w"] is not None else None
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        if not backward:
            y = _exact_turn(x if w is None else x * r * w, z, s["rot"], s["interleaved"])
        else:
            g = s["g" + n].double() if packed else s["g" + n].transpose(1, 2).double()
            g = _exact_turn(g.reshape(x.shape), z.conj(), s["rot"], s["interleaved"])
            if w is None:
                y = g
                sums.append(None)
            else:
                hat = x * r
                sums.append((g * hat).sum((0, 1)))
                y = r * (g * w - hat * (g * w * hat).mean(-1, keepdim=True))
        y = y.view(shape)
        out.append(y if packed else y.transpose(1, 2).contiguous())
    return tuple(out + sums)


def _exact_append(s, eight):
    new = (s["cu"][1:] - s["cu"][:-1]).tolist()
    lens, cu, t = s["seq"].tolist(), s["cu"].tolist(), s["table_t"].cpu()
    z = torch.complex(s["cos"].double(), s["sin"].double())
    qs = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    pools = {}
    for n in ("k", "v"):
        pools[n] = s[n + "p"].double()
    scales = {n: s[n + "s"].double() for n in ("k", "v")} if eight else None
    at = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        count = (L + PAGE - 1) // PAGE
        pages = t[at:at + count].tolist() if t.dim() == 1 else t[b, :count].tolist()
        at += count
        if not n:
            continue
        rows = slice(cu[b], cu[b] + n)
        turn = z[L - n:L][:, None]
        val = {"v": s["v"][rows].double()}
        for m in ("q", "k"):
            x, w = s[m][rows].double(), s[m + "w"]
            if w is not None:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
            val[m] = _exact_turn(x, turn, s["rot"], s["interleaved"])
        qs[rows] = val["q"]
        width = s["block"] if eight else PAGE
        for lo in range((L - n) // width * width, L, width):
            first, last = max(lo, L - n), min(lo + width, L)
            page, o = pages[lo // PAGE], lo % PAGE
            for m in ("k", "v"):
                x = val[m][first - (L - n):last - (L - n)].transpose(0, 1)
                if eight:
                    size = x.abs().amax((1, 2))
                    k = torch.ceil(torch.log2(size / 448)).clamp(-64, 64)
                    sc = torch.exp2(torch.where(size > 448 * torch.exp2(k), k + 1, k))
                    if first > lo:
                        was = scales[m][page, :, o // width]
                        sc = torch.maximum(sc, was)
                        pools[m][page, :, o:o + first - lo] *= (was / sc)[:, None, None]
                    scales[m][page, :, o // width] = sc
                    x = x / sc[:, None, None]
                pools[m][page, :, first % PAGE:first % PAGE + last - first] = x
    if eight:
        return qs, pools["k"], pools["v"], scales["k"], scales["v"]
    return qs, pools["k"], pools["v"]


def _exact_decode(s):
    B, H, d = s["q"].shape
    Hkv, block = s["kp"].shape[1], s["block"]
    o = torch.zeros((B, H, d), device="cuda", dtype=torch.float64)
    lse = torch.full((B, H), -math.inf, device="cuda", dtype=torch.float64)
    t, at = s["table_t"], 0
    for b, L in enumerate(s["seq"].tolist()):
        n = (L + PAGE - 1) // PAGE
        pages = (t[at:at + n] if t.dim() == 1 else t[b, :n]).long()
        at += n
        if not L:
            continue

        def cached(m):
            x = s[m + "p"].view(torch.uint8)[pages].view(E4M3).double()
            x *= s[m + "s"][pages].double().repeat_interleave(block, -1)[..., None]
            return x.transpose(0, 1).reshape(Hkv, n * PAGE, d)[:, :L]

        q = s["q"][b].double().view(Hkv, H // Hkv, d)
        a = torch.matmul(q, cached("k").transpose(1, 2)) / math.sqrt(d)
        lse[b] = torch.logsumexp(a, -1).flatten()
        o[b] = torch.matmul(torch.softmax(a, -1), cached("v")).view(H, d)
    return o, lse
