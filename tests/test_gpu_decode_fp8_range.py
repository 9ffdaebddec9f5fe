"""Decode over the 8-bit cache where the blocks' scales lie far apart: what a block
weighs in the output is its softmax weight times its value scale, and neither
alone."""
import math

import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref

pytestmark = pytest.mark.gpu
PS = 256
FP8 = torch.float8_e4m3fn
LOG2E = 1.4426950408889634


def pool(lens, H, Hk, d, block, seed):
    """Queries near one direction u of signs for each K/V head, codes of all kinds."""
    g = torch.Generator().manual_seed(seed)
    P = sum(ref.pages_of(lens))
    u = torch.randint(0, 2, (Hk, d), generator=g) * 2.0 - 1
    q = (u.repeat_interleave(H // Hk, 0) * (1 + 0.25 * torch.rand((len(lens), H, d), generator=g)))
    kp, vp = ((torch.randn((P, Hk, PS, d), generator=g) * 100).clamp(-448, 448).to(FP8)
              for _ in range(2))
    ks = torch.full((P, Hk, PS // block), 0.002)
    vs = 0.01 * torch.exp2(torch.rand((P, Hk, PS // block), generator=g) - 0.5)
    table = torch.randperm(P, generator=g).int()
    return u, q.bfloat16().cuda(), kp.cuda(), vp.cuda(), ks.cuda(), vs.cuda(), table


def block_of(table, lens, b, pos, block):
    """Page and block in it of position pos of sequence b."""
    return ref.page_list(table, lens, b)[pos // PS], pos % PS // block


def check(q, kp, vp, ks, vs, table, lens, bits=11):
    scale = q.shape[2] ** -0.5
    r, rl, absv, reach = ref.decode(q, kp, vp, ks, vs, table, lens, scale)
    # the largest p * vscale of each head, by the same call on codes of one
    ones = torch.ones_like(vp.float()).to(FP8)
    total = ref.decode(q, kp, ones, ks, vs, table, lens, scale)[0].amax(-1)
    n = torch.tensor(lens, device="cuda")[:, None]
    delta = 2.0 ** -16 * reach
    # (scores less a maximum of up to 64 and more lie 2^-17 apart in fp32)
    weights = 2.0 ** -bits + 4 * delta + 2.0 ** -17 + 2.0 ** -22 * n
    # and each weight within 2^-40 of the largest, which is at most their sum, times 448
    tol = 2.0 ** -8 * r.abs() + weights[..., None] * absv + \
        (2.0 ** -40 * 448 * n * total)[..., None]
    # tables of several widths take the kernels' several ways
    for more in (0, 9, 1300):
        t = torch.cat([table, torch.full((more,), -1, dtype=torch.int32)]).cuda()
        lse = torch.empty(q.shape[:2], device="cuda")
        o = fa.fa_decode_paged_fp8(q, kp, vp, ks, vs, t, torch.tensor(lens).int().cuda(), lse=lse)
        assert fa.fa_get_device_error() == fa.FA_OK
        assert torch.isfinite(o).all()
        over = ((o.double() - r).abs() - tol).max().item()
        assert over <= 0, (more, over)
        assert ((lse.double() - rl).abs() <= 2 * delta + 2.0 ** -17 * (1 + rl.abs()) +
                2.0 ** -22 * n).all()
    return r


@pytest.mark.parametrize("H,Hk,d,block", [(4, 1, 128, 32), (8, 2, 64, 16), (16, 1, 128, 16),
                                          (32, 1, 64, 64), (24, 1, 128, 64)])
@pytest.mark.parametrize("ratio", [30, 44, 100, 127])
@pytest.mark.parametrize("at", ["first", "last"])
def test_a_large_block_that_the_softmax_hardly_sees(H, Hk, d, block, ratio, at):
    """One block's value scale 2^ratio times the others', its tokens' weights 2^-ratio
    of theirs (the first sequence: it gives about as much as they do) or less."""
    lens = [700, 5000, 300]
    u, q, kp, vp, ks, vs, table = pool(lens, H, Hk, d, block, seed=ratio)
    vs *= 100 * 2.0 ** -(ratio / 2)
    for b, n in enumerate(lens):
        pos = 0 if at == "first" else (n - 1) // block * block
        p, i = block_of(table, lens, b, pos, block)
        rows = slice(i * block, (i + 1) * block)
        kp[p, :, rows] = (-256.0 * u).to(FP8).cuda()[:, None]
        # (a query's product with it is about 288 d)
        ks[p, :, i] = ratio * (1 + b / 2) / LOG2E / (288 * d ** 0.5)
        vs[p, :, i] = 2.0 ** (ratio / 2)
    check(q, kp, vp, ks, vs, table, lens)


def test_zero_codes_under_a_larger_scale():
    """The small blocks' values come through beside a large block of zeros."""
    lens = [600, 40]
    for shift in (4, 12, 20):
        u, q, kp, vp, ks, vs, table = pool(lens, 4, 1, 128, 16, seed=shift)
        for b in range(2):
            p, i = block_of(table, lens, b, 16, 16)
            vp[p, 0, 16 * i:16 * i + 16] = 0.0
            vs[p, 0, i] = 0.01 * 2.0 ** shift
        check(q, kp, vp, ks, vs, table, lens)


@pytest.mark.parametrize("G", [1, 4, 8, 16, 24, 32])
@pytest.mark.parametrize("d,block", [(128, 16), (64, 64)])
def test_weights_of_22_bits(G, d, block):
    """Zero queries: each weight is its value scale, of 24 random bits.  Two fp16 values
    hold it to 2^-22; the exponential, the division and the sums in fp32 add 2^-22 each,
    the sums once a token.  An output is one of the two bf16 values that the ends of
    that interval round to."""
    lens = [1, 1, 1, 16, 100, 0, 33]
    u, q, kp, vp, ks, vs, table = pool(lens, 2 * G, 2, d, block, seed=G)
    q.zero_()
    r, _, absv, _ = ref.decode(q, kp, vp, ks, vs, table, lens, 1.0)
    n = torch.tensor(lens, device="cuda")[:, None, None]
    off = (2.0 ** -20 + 2.0 ** -22 * n) * absv
    low, high = (r - off).bfloat16(), (r + off).bfloat16()
    for more in (0, 9, 1300):
        t = torch.cat([table, torch.full((more,), -1, dtype=torch.int32)]).cuda()
        o = fa.fa_decode_paged_fp8(q, kp, vp, ks, vs, t, torch.tensor(lens).int().cuda())
        assert fa.fa_get_device_error() == fa.FA_OK
        assert ((low <= o) & (o <= high)).all()


@pytest.mark.parametrize("G", [1, 16])
def test_large_queries_over_small_keys(G):
    """Queries of 2^126 and keys under a scale of 2^-64: the scores, up to 2^80, are in
    fp32's range, and the largest takes all of the weight."""
    lens = [1, 40]
    u, q, kp, vp, ks, vs, table = pool(lens, G, 1, 64, 64, seed=1)
    q = (u.repeat(2, G, 1) * 2.0 ** 126).bfloat16().cuda()
    ks.fill_(2.0 ** -64)
    p = ref.page_list(table, lens, 1)[0]
    kp[p, 0, 17] = (448.0 * u[0]).to(FP8).cuda()
    o = fa.fa_decode_paged_fp8(q, kp, vp, ks, vs, table.cuda(), torch.tensor(lens).int().cuda(),
                               scale=1.0)
    assert fa.fa_get_device_error() == fa.FA_OK
    for b, at in ((0, 0), (1, 17)):
        p = ref.page_list(table, lens, b)[0]
        want = vp[p, 0, at].double() * vs[p, 0, 0].double()
        assert ((o[b].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs()).all()


@pytest.mark.parametrize("H,d", [(1, 64), (16, 64), (4, 128)])
def test_a_sequence_of_2_31_tokens(H, d):
    """2^31 - 1 tokens (a packed table may name one page many times): the last tile
    ends where the sequence does.  The last token, on a page of its own, has weight
    e^34 beside the others' 1, and the slot behind it holds it once more."""
    lens = [2 ** 31 - 1]
    kp, vp = (torch.zeros((2, 1, PS, d), device="cuda").to(FP8) for _ in range(2))
    kp[1, 0, 254:] = torch.tensor(16.0).to(FP8)
    vp[:] = torch.tensor(2.0).to(FP8)
    vp[1, 0, 254:] = torch.tensor(-3.0).to(FP8)
    ks, vs = (torch.ones((2, 1, 1), device="cuda") for _ in range(2))
    table = torch.zeros(2 ** 23, dtype=torch.int32, device="cuda")
    table[-1] = 1
    q = torch.ones((1, H, d), device="cuda").bfloat16()
    lse = torch.empty((1, H), device="cuda")
    scale = 34.0 / (16 * d)
    o = fa.fa_decode_paged_fp8(q, kp, vp, ks, vs, table, torch.tensor(lens).int().cuda(),
                               scale=scale, lse=lse)
    assert fa.fa_get_device_error() == fa.FA_OK
    # 2^31 - 2 weights of 1 and one of e^34 = 5.8e14: 3.7e-6 of the sum
    want = math.log(math.exp(34.0) + 2.0 ** 31 - 2)
    assert (lse.double() - want).abs().max().item() <= 2.0 ** -18 * 35 + 2.0 ** -16 * 34
    assert ((o.double() + 3).abs() <= 3 * 2.0 ** -8 + 2.0 ** -16).all()
