"""The appends with norm and rotation at the ends of what their arguments allow."""
import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref

pytestmark = pytest.mark.gpu
PS = 256
FP8 = torch.float8_e4m3fn


def _ok():
    assert fa.fa_get_device_error() == fa.FA_OK


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("n", [1, 3, 200])
@pytest.mark.parametrize("d,block", [(64, 256), (128, 256), (128, 64), (64, 16)])
def test_a_sequence_of_2_31_tokens(eight, n, d, block):
    """The new rows end at position 2^31 - 2 (a packed table may name one page many
    times); the block's end, one further, is beyond 32 bits.  Only they are written."""
    Hk, L = 2, 2 ** 31 - 1
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn((n, Hk, d), generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.zeros(2 ** 23, dtype=torch.int32, device="cuda")
    table[-1] = 1
    cu, seq = torch.tensor([0, n]).int().cuda(), torch.tensor([L]).int().cuda()
    shape = (2, Hk, PS, d)
    kp, vp = (torch.randn(shape, generator=g).to(FP8 if eight else torch.bfloat16).cuda()
              for _ in range(2))
    before = [t.clone().view(torch.uint8) for t in (kp, vp)]
    rows = slice(255 - n, 255)
    if eight:
        ks, vs = (torch.full((2, Hk, PS // block), 0.25, device="cuda") for _ in range(2))
        fa.fa_append_paged_fp8(None, k, v, cu, kp, vp, ks, vs, table, seq)
    else:
        fa.fa_append_paged_rope(None, k, v, cu, kp, vp, table, seq)
    _ok()
    for t, was, x, s in ((kp, before[0], k, ks if eight else None),
                         (vp, before[1], v, vs if eight else None)):
        x = x.transpose(0, 1)
        if eight:
            # a block that the new rows begin keeps nothing of its old scale
            first = (255 - n) // block * block
            blocks = torch.arange(PS // block)
            touched = blocks >= (255 - n) // block
            for i in blocks[touched].tolist():
                new = x[:, max(i * block - (255 - n), 0):i * block + block - (255 - n)]
                for h in range(Hk):
                    least = ref.least_scale(new[h].abs().max().item())
                    if i * block == first and first < 255 - n:
                        least = max(least, 0.25)
                    assert s[1, h, i].item() == least
            assert (s[0] == 0.25).all() and (s[1, :, ~touched] == 0.25).all()
            scale = s[1].repeat_interleave(block, 1)[:, rows, None].double()
            want = ref.e4m3(x.double() / scale).view(torch.uint8)
            assert torch.equal(t[1, :, rows].view(torch.uint8), want)
        else:
            assert torch.equal(t[1, :, rows], x)
        now = t.view(torch.uint8)
        assert torch.equal(now[0], was[0])
        assert torch.equal(now[1, :, :255 - n], was[1, :, :255 - n])
        assert torch.equal(now[1, :, 255], was[1, :, 255])


@pytest.mark.parametrize("d,block,heads", [(128, 256, 8), (64, 64, 20), (128, 16, 1)])
def test_a_longer_prompt_among_single_tokens(d, block, heads):
    """So few new tokens on average that every block takes the way of a decode step:
    the one prompt's blocks go through it a few rows at a time, and back."""
    new = [1] * 40 + [130] + [1] * 23
    ctx = [(37 * i) % 300 for i in range(64)]
    ctx[40] = 250
    lens = [n + c for n, c in zip(new, ctx)]
    g = torch.Generator().manual_seed(d + block)
    total, P = sum(new), sum(ref.pages_of(lens))
    k, v = ((torch.randn((total, heads, d), generator=g) *
             torch.exp2(torch.randint(-3, 4, (total, heads, 1), generator=g))).bfloat16().cuda()
            for _ in range(2))
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0))).int().cuda()
    table = torch.randperm(P, generator=g).int()
    w = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    cos, sin = fa.fa_rope_table(1024, d)
    shape = (P, heads, PS, d)
    kp, vp = (torch.randn(shape, generator=g).to(FP8).cuda() for _ in range(2))
    # small scales: every block that had tokens grows
    ks, vs = (torch.full((P, heads, PS // block), 2.0 ** -12, device="cuda") for _ in range(2))
    old = [t.float().double() for t in (kp, vp)]
    fa.fa_append_paged_fp8(None, k, v, cu, kp, vp, ks, vs, table.cuda(),
                           torch.tensor(lens).int().cuda(), cos, sin, None, w, eps=1e-5)
    _ok()
    at = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        pos = torch.arange(c, c + n, device="cuda")
        turned = ref.norm_rope(k[at:at + n], w, cos[pos], sin[pos], False, 1e-5)
        pages = ref.page_list(table, lens, b)
        for pool, s, was, x, slack in ((kp, ks, old[0], turned, 2.0 ** -19),
                                       (vp, vs, old[1], v[at:at + n].double(), 0.0)):
            got = ref.gather(pool, s, pages, c + n)
            for lo in range(c // block * block, c + n, block):
                hi, first = min(lo + block, c + n), max(lo, c)
                rows = x[first - c:hi - c]
                scale = s[pages[lo // PS], :, lo % PS // block].double()
                top = rows.abs().amax((0, 2))
                # the least power of two that the block's values need (or one that the
                # fp32 values' own rounding needs)
                least = torch.tensor([ref.least_scale(t) for t in top.tolist()]).cuda().double()
                near = torch.tensor([ref.least_scale(t) for t in (top * (1 + 2 * slack)).tolist()]
                                    ).cuda().double()
                assert ((scale == least) | (scale == near)).all()
                # half a step of 4 bits or of the least codes, and the values' fp32 rounding
                tol = 2.0 ** -4 * rows.abs() + 2.0 ** -10 * scale[:, None] + \
                    slack * rows.abs().amax(-1, keepdim=True)
                assert ((got[first:hi] - rows).abs() <= tol).all()
                kept = was[pages[lo // PS], :, lo % PS:lo % PS + first - lo].transpose(0, 1) * \
                    2.0 ** -12
                tol = 2.0 ** -4 * kept.abs() + 2.0 ** -10 * scale[:, None]
                assert ((got[lo:first] - kept).abs() <= tol).all()
        at += n


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("fault", ["offset", "length"])
def test_a_fault_behind_the_last_new_row_is_reported(eight, with_q, fault):
    """300 sequences, the first 256 with the new rows; something is wrong with one of
    the others, which none of those rows belongs to."""
    B, Hk, d = 300, 2, 64
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((256, h, d), generator=g).bfloat16().cuda() for h in (4, Hk, Hk))
    cu = torch.arange(B + 1).clamp(max=256).int()
    lens = torch.ones(B, dtype=torch.int32)
    lens[256:] = 0
    table = torch.arange(256).int().cuda()
    outs = []
    for bad in (False, True):
        c, n = cu.clone(), lens.clone()
        if bad and fault == "offset":
            c[290] = 257
        if bad and fault == "length":
            n[290] = -3
        dt = FP8 if eight else torch.bfloat16
        kp, vp = (torch.zeros((256, Hk, PS, d), device="cuda").to(dt) for _ in range(2))
        ks, vs = (torch.ones((256, Hk, 4), device="cuda") for _ in range(2))
        a = [q if with_q else None, k, v, c.cuda(), kp, vp, table, n.cuda()]
        if eight:
            a[6:6] = [ks, vs]
        f = fa.fa_append_paged_fp8 if eight else fa.fa_append_paged_rope
        out = f(*a)
        want = fa.FA_ERR_DEVICE_BAD_INPUT if bad else fa.FA_OK
        assert fa.fa_get_device_error() == want
        outs.append([kp.view(torch.uint8), vp.view(torch.uint8), ks, vs] + [out] * with_q)
    for x, y in zip(*outs):
        assert torch.equal(x, y)
