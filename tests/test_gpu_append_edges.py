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
