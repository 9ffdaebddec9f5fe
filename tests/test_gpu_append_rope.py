"""Appends with the norms and the rotation on the way, into bf16 pages and into
8-bit pages with block scales, against 64-bit forms."""
import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref

pytestmark = pytest.mark.gpu
PS = 256
FP8 = torch.float8_e4m3fn


def _ok():
    assert fa.fa_get_device_error() == fa.FA_OK


class Case:
    """New rows of sequences with `new` tokens behind `ctx` cached ones."""

    def __init__(self, new, ctx, H=4, Hk=2, d=128, R=128, weights="fp32", table="packed",
                 block=0, seed=0, max_pos=2048, std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.ctx, self.H, self.Hk, self.d, self.R = new, ctx, H, Hk, d, R
        self.lens = [n + c for n, c in zip(new, ctx)]
        total = sum(new)
        x = (torch.randn((total, (H + 2 * Hk) * d), generator=g) * std).bfloat16().cuda()
        self.q = x[:, :H * d].view(total, H, d)
        self.k = x[:, H * d:(H + Hk) * d].view(total, Hk, d)
        self.v = x[:, (H + Hk) * d:].view(total, Hk, d)
        self.cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0))).int().cuda()
        self.seq = torch.tensor(self.lens).int().cuda()
        pages = ref.pages_of(self.lens)
        P = sum(pages) + 2
        perm = torch.randperm(P, generator=g).int()
        if table == "packed":
            self.table = perm[:sum(pages)].clone()
        else:
            self.table = torch.full((len(new), max(1, max(pages))), -1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(pages):
                self.table[b, :n] = perm[at:at + n]
                at += n
        self.P, self.block = P, block
        shape = (P, Hk, PS, d)
        if block:
            self.kp, self.vp = (torch.randint(0, 255, shape, generator=g).to(torch.uint8)
                                for _ in range(2))
            for t in (self.kp, self.vp):
                t[(t & 127) == 127] = 5  # no NaN among the cached values
            self.kp, self.vp = self.kp.cuda().view(FP8), self.vp.cuda().view(FP8)
            e = torch.randint(-10, -5, (2, P, Hk, PS // block), generator=g)
            self.ks, self.vs = torch.exp2(e.float()).cuda()
        else:
            self.kp, self.vp = (torch.randn(shape, generator=g).bfloat16().cuda()
                                for _ in range(2))
        self.qw = self.kw = None
        if weights != "none":
            dt = torch.float32 if weights == "fp32" else torch.bfloat16
            self.qw, self.kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(dt).cuda()
                                for _ in range(2))
        self.cos, self.sin = fa.fa_rope_table(max_pos, R) if R else (None, None)
        self.pos = torch.cat([torch.arange(c, c + n) for n, c in zip(new, ctx)]).long().cuda() \
            if total else torch.zeros(0, dtype=torch.long, device="cuda")

    def call(self, with_q=True, eps=1e-5, **kw):
        args = dict(rope_cos=self.cos, rope_sin=self.sin, q_weight=self.qw if with_q else None,
                    k_weight=self.kw, eps=eps, **kw)
        q = self.q if with_q else None
        t = self.table.cuda()
        if self.block:
            return fa.fa_append_paged_fp8(q, self.k, self.v, self.cu, self.kp, self.vp, self.ks,
                                          self.vs, t, self.seq, **args)
        return fa.fa_append_paged_rope(q, self.k, self.v, self.cu, self.kp, self.vp, t, self.seq,
                                       **args)

    def turned(self, x, w, interleaved):
        if self.R:
            c, s = self.cos[self.pos], self.sin[self.pos]
        else:
            c = s = torch.empty((len(self.pos), 0), device="cuda")
        return ref.norm_rope(x, w, c, s, interleaved, 1e-5)

    def places(self):
        """(page, slot) of each new row."""
        page = []
        for b, (n, c) in enumerate(zip(self.new, self.ctx)):
            ids = ref.page_list(self.table, self.lens, b)
            page += [ids[p // PS] for p in range(c, c + n)]
        return torch.tensor(page).long().cuda(), self.pos % PS


def _within(y, r):
    over = ((y.double() - r).abs() - ref.bf16_bound(r)).max().item()
    assert over <= 0, over


LENGTHS = [
    ([1], [0]),
    ([1] * 7, [0, 1, 255, 256, 257, 511, 300]),
    ([300, 0, 1, 17, 256], [0, 40, 255, 250, 256]),
    ([0, 33, 600], [0, 223, 1]),
    ([1] * 200, list(range(200))),
]


@pytest.mark.parametrize("table", ["packed", "rows"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,ctx", LENGTHS, ids=range(len(LENGTHS)))
@pytest.mark.parametrize("H,Hk,d,R,weights", [(4, 2, 128, 128, "fp32"), (7, 1, 64, 32, "bf16"),
                                              (5, 5, 128, 48, "none"), (6, 3, 64, 0, "fp32")])
def test_append_rope(table, interleaved, new, ctx, H, Hk, d, R, weights):
    c = Case(new, ctx, H, Hk, d, R, weights, table, seed=len(new) + d)
    before = c.kp.clone(), c.vp.clone()
    q = c.call(interleaved=interleaved)
    _ok()
    _within(q, c.turned(c.q, c.qw, interleaved))
    page, slot = c.places()
    _within(c.kp[page, :, slot], c.turned(c.k, c.kw, interleaved))
    assert torch.equal(c.vp[page, :, slot], c.v)
    before[0][page, :, slot] = c.kp[page, :, slot]  # everything else stays
    before[1][page, :, slot] = c.vp[page, :, slot]
    assert torch.equal(c.kp, before[0]) and torch.equal(c.vp, before[1])


def _check_fp8(c, before, interleaved):
    """Pages and scales after an append against the definition."""
    k, v = c.turned(c.k, c.kw, interleaved), c.v.double()
    fuzz = {0: 2.0 ** -19, 1: 0.0}  # of the row's largest value: fp32 steps (see bf16_bound)
    page, slot = c.places()
    at = 0
    touched = torch.zeros((c.P, PS // c.block), dtype=torch.bool, device="cuda")
    rows = [k, v]
    for b, (n, cx) in enumerate(zip(c.new, c.ctx)):
        ids = ref.page_list(c.table, c.lens, b)
        lo = cx // c.block * c.block
        while n and lo < cx + n:
            first, last = max(lo, cx), min(lo + c.block, cx + n)
            pg, o = ids[lo // PS], lo % PS
            blk = o // c.block
            touched[pg, blk] = True
            for which, (pool, sc, old, olds) in enumerate(
                    ((c.kp, c.ks, before[0], before[2]), (c.vp, c.vs, before[1], before[3]))):
                x = rows[which][at + first - cx:at + last - cx]        # [rows, Hk, d]
                big = x.abs().amax(-1, keepdim=True) * fuzz[which]
                for h in range(c.Hk):
                    a = x[:, h].abs().max().item()
                    s, was = sc[pg, h, blk].item(), olds[pg, h, blk].item()
                    may = {ref.least_scale(a * (1 - 2.0 ** -18)), ref.least_scale(a),
                           ref.least_scale(a * (1 + 2.0 ** -18))}
                    if first > lo:
                        may = {max(was, m) for m in may}
                    assert s in may, (s, may)
                    got = pool[pg, h].view(torch.uint8).view(FP8).double()[o:o + last - lo] * s
                    # new rows: half a step of 4 bits, half the least step below 2^-6
                    y = got[first - lo:]
                    tol = torch.clamp(2.0 ** -4 * x[:, h].abs(), min=2.0 ** -10 * s) + big[:, h]
                    assert ((y - x[:, h]).abs() <= tol).all()
                    # rows before them: exact under the same or the larger scale
                    code = old[pg, h].view(torch.uint8).view(FP8).double()[o:o + first - lo]
                    keep = pool[pg, h].view(torch.uint8)[o:o + first - lo]
                    assert torch.equal(keep.view(FP8).double(), ref.e4m3(code * (was / s)).double())
                # the rest of the block, and the rows outside, stay
            lo += c.block
        at += n
    for pool, sc, old, olds in ((c.kp, c.ks, before[0], before[2]),
                                (c.vp, c.vs, before[1], before[3])):
        now, was = pool.view(torch.uint8).clone(), old.view(torch.uint8).clone()
        was[page, :, slot] = now[page, :, slot]
        for p, blk in torch.nonzero(touched).tolist():
            lo = blk * c.block
            used = [s for q, s in zip(page.tolist(), slot.tolist())
                    if q == p and s // c.block == blk]
            was[p, :, lo:min(used)] = now[p, :, lo:min(used)]  # checked above
        assert torch.equal(now, was)
        still = ~touched[:, None].expand(-1, c.Hk, -1)
        assert torch.equal(sc[still], olds[still])


@pytest.mark.parametrize("table", ["packed", "rows"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,ctx", LENGTHS[:4], ids=range(4))
@pytest.mark.parametrize("H,Hk,d,R,weights,block", [
    (4, 2, 128, 128, "fp32", 64), (7, 1, 64, 32, "bf16", 16), (5, 5, 128, 48, "none", 256),
    (6, 3, 64, 0, "fp32", 32), (2, 1, 128, 128, "bf16", 128)])
def test_append_fp8(table, interleaved, new, ctx, H, Hk, d, R, weights, block):
    c = Case(new, ctx, H, Hk, d, R, weights, table, block, seed=len(new) + d)
    before = [t.clone() for t in (c.kp, c.vp, c.ks, c.vs)]
    q = c.call(interleaved=interleaved)
    _ok()
    _within(q, c.turned(c.q, c.qw, interleaved))
    _check_fp8(c, before, interleaved)


@pytest.mark.parametrize("H,Hk,d,R,weights,block", [
    (5, 5, 128, 128, "fp32", 16), (3, 3, 128, 64, "none", 32), (20, 20, 128, 16, "bf16", 64),
    (9, 9, 64, 64, "fp32", 16), (5, 5, 64, 16, "none", 64), (3, 3, 64, 48, "bf16", 128),
    (2, 2, 64, 64, "fp32", 256), (1, 1, 128, 128, "fp32", 256)])
@pytest.mark.parametrize("new,ctx", [([300, 0, 70, 5], [40, 9, 250, 0]), ([900], [13]),
                                     ([4, 2, 3], [62, 255, 14]),
                                     ([0, 170] + [0] * 60, [3, 40] + [9] * 60)], ids=range(4))
def test_append_fp8_shapes(new, ctx, H, Hk, d, R, weights, block):
    """Every way in which a CTA's rows are divided among a block's tokens and
    heads, heads that are left over, and sequences with a few tokens."""
    c = Case(new, ctx, H, Hk, d, R, weights, "packed", block, seed=Hk + block)
    before = [t.clone() for t in (c.kp, c.vp, c.ks, c.vs)]
    q = c.call()
    _ok()
    _within(q, c.turned(c.q, c.qw, False))
    _check_fp8(c, before, False)


def test_fp8_special_values_on_the_way_of_prompts_and_of_steps():
    """Infinities, NaN, zeros and values beyond the format's reach, with every
    block width: the same codes as the definition's."""
    for block in (16, 32, 64, 128, 256):
        for new, ctx in (([150, 300], [3, 0]), ([1] * 6, [0, 20, 70, 255, 256, 300])):
            c = Case(new, ctx, 1, 3, 128, 0, "none", "rows", block, seed=block)
            g = torch.Generator().manual_seed(block)
            x = c.v.float().cpu()
            pick = torch.rand(x.shape, generator=g)
            x[pick < 0.002] = float("inf")
            x[(pick > 0.002) & (pick < 0.004)] = float("-inf")
            x[(pick > 0.004) & (pick < 0.006)] = float("nan")
            x[(pick > 0.006) & (pick < 0.2)] = 0.0
            c.v = x.bfloat16().cuda()
            old = c.vs.clone()
            c.call(with_q=False)
            _ok()
            page, slot = c.places()
            at = 0
            for b, (n, cx) in enumerate(zip(new, ctx)):
                for lo in range(cx // block * block, cx + n, block):
                    first, last = max(lo, cx), min(lo + block, cx + n)
                    r = slice(at + first - cx, at + last - cx)
                    pg, blk = page[at + first - cx].item(), lo % PS // block
                    for h in range(3):
                        rows = c.v[r, h].double()
                        fin = rows[rows.isfinite()]
                        s = ref.least_scale(fin.abs().max().item() if len(fin) else 0.0)
                        if first > lo:
                            s = max(s, old[pg, h, blk].item())
                        assert c.vs[pg, h, blk].item() == s
                        got = c.vp.view(torch.uint8)[pg, h, first % PS:(last - 1) % PS + 1]
                        want = ref.e4m3(rows / s).view(torch.uint8)
                        nan = (want & 127) == 127
                        assert torch.equal((got & 127) == 127, nan)
                        assert torch.equal(got[~nan], want[~nan])
                at += n


def test_offsets_past_32_bits():
    """A pool whose last pages lie more than 2^32 bytes (8-bit pages: codes) from
    its start."""
    for block in (0, 64):
        c = Case([40, 1], [30, 700], 2, 4, 128, 64, "fp32", "packed", block, seed=1)
        want = c.call()
        small = c.kp.clone(), c.vp.clone()
        d = Case([40, 1], [30, 700], 2, 4, 128, 64, "fp32", "packed", block, seed=1)
        size = 1 if block else 2
        P = (1 << 32) // (4 * PS * 128 * size) + c.P
        far = P - c.P
        for name in ("kp", "vp") + (("ks", "vs") if block else ()):
            t = getattr(d, name)
            big = torch.empty((P,) + t.shape[1:], dtype=t.dtype, device="cuda")
            big[far:].copy_(t) if t.dtype != FP8 else \
                big[far:].view(torch.uint8).copy_(t.view(torch.uint8))
            setattr(d, name, big)
        d.table = d.table + far
        got = d.call()
        _ok()
        assert torch.equal(got, want)
        for a, b in zip((d.kp, d.vp), small):
            assert torch.equal(a[far:].view(torch.uint8), b.view(torch.uint8))
        if block:
            assert torch.equal(d.ks[far:], c.ks) and torch.equal(d.vs[far:], c.vs)
            q = want[[39, 40]].repeat(1, 2, 1)
            o = [fa.fa_decode_paged_fp8(q, x.kp, x.vp, x.ks, x.vs, x.table.cuda(), x.seq)
                 for x in (c, d)]
            _ok()
            assert torch.equal(o[0], o[1])


def test_fp8_many_sequences():
    c = Case([1] * 300, [i % 70 for i in range(300)], 2, 1, 64, 16, "none", "rows", 16, seed=9)
    before = [t.clone() for t in (c.kp, c.vp, c.ks, c.vs)]
    c.call()
    _ok()
    _check_fp8(c, before, False)


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e12])
def test_fp8_scales_follow_the_values(std):
    c = Case([20, 70], [0, 10], 2, 2, 64, 32, "none", "packed", 32, seed=5, std=std)
    before = [t.clone() for t in (c.kp, c.vp, c.ks, c.vs)]
    c.call()
    _ok()
    _check_fp8(c, before, False)


def test_fp8_scale_that_is_no_power_of_two():
    """A block's larger scale stays whatever it is, and the new values are
    divided by it and rounded once."""
    c = Case([3], [5], 1, 1, 64, 0, "none", "packed", 16, seed=5)
    page = int(c.table[0])
    c.ks[page], c.vs[page] = 0.3, 0.7
    c.call()
    _ok()
    for pool, x, s in ((c.kp, c.k, c.ks), (c.vp, c.v, c.vs)):
        s = s[page, 0, 0]
        want = ref.e4m3((x[:, 0].float() / s).double())
        assert torch.equal(pool[page, 0, 5:8].view(torch.uint8), want.view(torch.uint8))


def test_fp8_zeros_infinities_and_nan():
    c = Case([40], [0], 1, 1, 64, 0, "none", "packed", 16, seed=5)
    c.k = c.k.clone()
    c.k[:16] = 0.0
    c.k[16, 0, 3], c.k[17, 0, 4], c.k[20, 0, 60] = float("inf"), float("-inf"), float("nan")
    c.call()
    _ok()
    page = int(c.table[0])
    got = c.kp[page, 0].view(torch.uint8)
    assert (got[:16] & 127 == 0).all() and c.ks[page, 0, 0].item() == 2.0 ** -64
    bad = (got[16:32] & 127) == 127
    assert bad[0, 3] and bad[1, 4] and bad[4, 60] and bad.sum().item() == 3
    x = c.k[16:32, 0].double()
    a = x[x.isfinite()].abs().max().item()
    assert c.ks[page, 0, 1].item() == ref.least_scale(a)


def test_keys_and_values_alone_and_one_weight():
    for block in (0, 32):
        c = Case([9, 30], [100, 0], block=block, seed=2)
        d2 = Case([9, 30], [100, 0], block=block, seed=2)
        c.call()
        assert d2.call(with_q=False) is None
        _ok()
        assert torch.equal(c.kp.view(torch.uint8), d2.kp.view(torch.uint8))
        assert torch.equal(c.vp.view(torch.uint8), d2.vp.view(torch.uint8))
        c = Case([9, 30], [100, 0], block=block, seed=2)
        c.kw = None
        q = c.call()
        _ok()
        _within(q, c.turned(c.q, c.qw, False))


def test_a_rotation_and_append_equal_the_calls_one_by_one():
    """fa_qk_norm_rope and fa_append_paged after it give the same bits."""
    c = Case([70, 5, 300], [3, 250, 0], 4, 2, 128, 64, "bf16", "packed", seed=4)
    kp, vp = c.kp.clone(), c.vp.clone()
    q = c.call(interleaved=True)
    q2, k2 = fa.fa_qk_norm_rope(c.q, c.k, c.qw, c.kw, c.cos, c.sin, c.pos.int(), eps=1e-5,
                                interleaved=True)
    fa.fa_append_paged(k2, c.v.contiguous(), c.cu, kp, vp, c.table.cuda(), c.seq)
    _ok()
    assert torch.equal(q, q2) and torch.equal(c.kp, kp) and torch.equal(c.vp, vp)


@pytest.mark.parametrize("block", [0, 16, 64, 256])
def test_no_epsilon(block):
    """eps = 0 gives what an eps below half a step of any row's mean square gives: the
    rows that a thread's group of tokens or heads lacks are not taken for zeros."""
    for new, ctx in (([3, 1, 2], [60, 0, 255]), ([70, 5, 300], [3, 250, 0])):
        got = []
        for eps in (0.0, 1e-30):
            c = Case(new, ctx, 7, 3, 128, 64, "fp32", "rows", block, seed=6)
            got.append([c.call(eps=eps), c.kp.view(torch.uint8), c.vp.view(torch.uint8)] +
                       ([c.ks, c.vs] if block else []))
        _ok()
        assert all(torch.equal(a, b) for a, b in zip(*got))
        assert torch.isfinite(got[0][0]).all()


@pytest.mark.parametrize("block", [0, 64])
def test_rows_behind_the_last_sequence_are_left(block):
    c = Case([5, 6], [10, 300], block=block, seed=3)
    extra = torch.randn((4, c.H, c.d), device="cuda").bfloat16()
    q, k, v = (torch.cat([t, extra[:, :t.shape[1]]]) for t in (c.q, c.k, c.v))
    whole = Case([5, 6], [10, 300], block=block, seed=3)
    want = whole.call()
    c.q, c.k, c.v = q, k, v
    out = torch.full(q.shape, 7.0, device="cuda").bfloat16()
    c.call(q_out=out)
    _ok()
    assert torch.equal(out[:11], want) and (out[11:] == 7).all()
    assert torch.equal(c.kp.view(torch.uint8), whole.kp.view(torch.uint8))
    assert torch.equal(c.vp.view(torch.uint8), whole.vp.view(torch.uint8))


@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("table", ["packed", "rows"])
def test_bad_lengths_offsets_and_pages_are_reported(block, table):
    def run(change):
        c = Case([4, 5, 6], [10, 300, 50], block=block, table=table, seed=6, max_pos=1024)
        before = c.kp.clone(), c.vp.clone()
        change(c)
        out = torch.full(c.q.shape, 7.0, device="cuda").bfloat16()
        c.call(q_out=out)
        assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
        return c, out, before

    good = Case([4, 5, 6], [10, 300, 50], block=block, table=table, seed=6, max_pos=1024)
    want = good.call()
    _ok()

    def same(a, b):
        return torch.equal(a.view(torch.uint8), b.view(torch.uint8))

    def first_page(c, b):
        return ref.page_list(c.table, good.lens, b)

    def shorter(c):  # fewer tokens than new rows
        c.seq = torch.tensor([14, 3, 56]).int().cuda()
        if table == "packed":
            c.table = torch.cat([c.table[:1], c.table[2:]])

    c, out, before = run(shorter)
    assert (out[4:9] == 0).all()
    assert torch.equal(out[:4], want[:4]) and torch.equal(out[9:], want[9:])
    for p in first_page(good, 1):
        assert same(c.kp[p], before[0][p]) and same(c.vp[p], before[1][p])

    def longer(c):  # behind the rotation's table
        c.cos, c.sin = c.cos[:300].contiguous(), c.sin[:300].contiguous()

    c, out, before = run(longer)
    assert (out[4:9] == 0).all() and torch.equal(out[:4], want[:4])
    for p in first_page(good, 1):
        assert same(c.kp[p], before[0][p]) and same(c.vp[p], before[1][p])

    def no_page(c):  # a page outside the pool
        flat = c.table.view(-1)
        flat[2 if table == "packed" else c.table.shape[1] + 1] = c.P

    c, out, before = run(no_page)
    assert torch.equal(out, want)
    for p in first_page(good, 1):
        assert same(c.kp[p], before[0][p])
    for p in first_page(good, 2):
        assert same(c.kp[p], good.kp[p]) and same(c.vp[p], good.vp[p])

    def huge(c):  # lengths whose pages no table holds
        c.seq = torch.tensor([14, 2 ** 31 - 1, 2 ** 31 - 2]).int().cuda()

    c, out, before = run(huge)
    assert torch.equal(out[:4], want[:4]) and (out[4:] == 0).all()

    def offsets(c):  # rows outside the new ones
        c.cu = torch.tensor([0, 4, 9, 40]).int().cuda()

    c, out, before = run(offsets)
    assert torch.equal(out[:9], want[:9]) and (out[9:] == 7).all()


@pytest.mark.parametrize("block", [0, 64])
def test_a_bad_page_among_many_rows_is_reported(block):
    """Prompts long enough for several tokens a CTA: the page of a single token in
    the middle of one."""
    new, ctx = [2000, 253, 1500], [0, 4, 100]
    good = Case(new, ctx, 2, 1, 64, 32, "none", "packed", block, seed=3)
    want = good.call()
    _ok()
    c = Case(new, ctx, 2, 1, 64, 32, "none", "packed", block, seed=3)
    before = c.kp.clone()
    at = ref.pages_of(good.lens)[0] + 1  # the second sequence's second page: position 256
    page = int(c.table[at])
    c.table[at] = -1
    out = c.call()
    assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
    assert torch.equal(out, want)
    good.kp[page] = before[page]
    assert torch.equal(c.kp.view(torch.uint8), good.kp.view(torch.uint8))


def test_no_new_rows():
    for block in (0, 64):
        c = Case([0, 0], [10, 300], block=block, seed=6)
        before = c.kp.clone()
        q = c.call()
        _ok()
        assert q.shape == (0, c.H, c.d)
        assert torch.equal(c.kp.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.parametrize("block", [0, 64])
def test_captured_and_replayed(block):
    c = Case([1] * 5, [10, 250, 62, 64, 700], block=block, seed=8)
    twin = Case([1] * 5, [10, 250, 62, 64, 700], block=block, seed=8)
    table, out = c.table.cuda(), torch.empty_like(c.q)
    names = ("k", "v", "q")
    rows = [getattr(c, n).contiguous() for n in names]

    def call(x):
        args = (table, x.seq, c.cos, c.sin, c.qw, c.kw)
        if block:
            fa.fa_append_paged_fp8(rows[2], rows[0], rows[1], c.cu, x.kp, x.vp, x.ks, x.vs,
                                   *args, q_out=out)
        else:
            fa.fa_append_paged_rope(rows[2], rows[0], rows[1], c.cu, x.kp, x.vp, *args,
                                    q_out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(c)
    for step in range(3):  # a token each, on the pages the table has
        if step:
            c.seq += 1
            twin.seq += 1
            for r in rows:
                r.mul_(-1.5)
        graph.replay()
        got = out.clone()
        call(twin)
        assert torch.equal(got, out)
    _ok()
    assert torch.equal(c.kp.view(torch.uint8), twin.kp.view(torch.uint8))
    assert torch.equal(c.vp.view(torch.uint8), twin.vp.view(torch.uint8))
