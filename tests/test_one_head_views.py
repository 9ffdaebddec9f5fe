"""Tensors of one head, whose stride over the heads may be anything: keys of a single
K/V head as [tokens, 1, d] views, transposed or cut out of something wider."""
import pytest
import torch

import attn_fwd_04_b200 as fa
from attn_fwd_04_b200 import build as fa_build

PS = 256
FP8 = torch.float8_e4m3fn


def views(x):
    """[T, 2 d] as [T, 1, d] in several ways; of the first half where it has gaps."""
    T, d = x.shape[0], x.shape[1] // 2
    first = x[:, :d]
    dense = first.contiguous()
    return {"transposed": dense[None].transpose(0, 1),
            "gaps, transposed": first[None].transpose(0, 1),
            "expanded": first.as_strided((T, 1, d), (2 * d, 0, 1)),
            "strange": first.as_strided((T, 1, d), (2 * d, 1 << 40, 1))}


@pytest.fixture
def meta(monkeypatch):
    from attn_fwd_04_b200 import fa as binding

    fa_build.build()
    binding._short()

    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(binding, "_DEVICE_TYPES", ("cuda", "meta"))
    monkeypatch.setattr(binding, "lib", no_library)
    return binding


def test_wrappers_take_them(meta):
    T, d = 70, 128
    x = torch.empty((T, 2 * d), dtype=torch.bfloat16, device="meta")
    q = torch.empty((T, 4, d), dtype=torch.bfloat16, device="meta")
    cu = torch.empty(2, dtype=torch.int32, device="meta")
    one = torch.empty(1, dtype=torch.int32, device="meta")
    pages = torch.empty((3, 1, PS, d), dtype=torch.bfloat16, device="meta")
    for name, k in views(x).items():
        for call in (lambda: meta.fa_qk_norm_rope(q, k),
                     lambda: meta.fa_qk_norm_rope(k, k),
                     lambda: meta.fa_qk_norm_rope_bwd(q, k, q, k),
                     lambda: meta.fa_append_paged_rope(q, k, k, cu, pages, pages, one, one),
                     lambda: meta.fa_append_paged_rope(k, k, k, cu, pages, pages, one, one)):
            with pytest.raises(AssertionError, match="library was called"):
                call()
    # what a single head does not excuse
    odd = torch.empty((T, 2 * d + 4), dtype=torch.bfloat16, device="meta")
    for bad in (odd[:, None, :d], x.as_strided((T, 1, d), (d // 2, d, 1)),
                x.as_strided((T, 1, d), (2 * d, d, 2))):
        with pytest.raises(ValueError):
            meta.fa_qk_norm_rope(q, bad)


@pytest.mark.gpu
@pytest.mark.parametrize("by_hand", [False, True])
def test_results_are_those_of_contiguous_ones(by_hand):
    """By the binding's short way, and by its long one (a stream given by hand)."""
    T, d = 70, 128
    stream = torch.cuda.current_stream() if by_hand else None
    g = torch.Generator().manual_seed(0)
    x = torch.randn((T, 2 * d), generator=g).bfloat16().cuda()
    q = torch.randn((T, 4, d), generator=g).bfloat16().cuda()
    w = torch.rand(d, generator=g).cuda()
    cos, sin = fa.fa_rope_table(512, d)
    cu, seq = torch.tensor([0, T]).int().cuda(), torch.tensor([T + 9]).int().cuda()
    table = torch.zeros(1, dtype=torch.int32, device="cuda")

    def all_of(k):
        out = list(fa.fa_qk_norm_rope(q, k, w, w, cos, sin, stream=stream))
        out += fa.fa_qk_norm_rope(k, k, w, w, cos, sin, stream=stream)
        out += fa.fa_qk_norm_rope_bwd(q, k, q, k, w, w, cos, sin, stream=stream)
        kp, vp = (torch.zeros((1, 1, PS, d), device="cuda").bfloat16() for _ in range(2))
        out += [fa.fa_append_paged_rope(k, k, k, cu, kp, vp, table, seq, cos, sin, w, w,
                                        stream=stream), kp, vp]
        k8, v8 = (torch.zeros((1, 1, PS, d), device="cuda").to(FP8) for _ in range(2))
        ks, vs = (torch.ones((1, 1, 4), device="cuda") for _ in range(2))
        out += [fa.fa_append_paged_fp8(k, k, k, cu, k8, v8, ks, vs, table, seq, cos, sin, w, w,
                                       stream=stream), k8.view(torch.uint8), v8.view(torch.uint8),
                ks, vs]
        assert fa.fa_get_device_error() == fa.FA_OK
        return out

    want = all_of(x[:, None, :d].contiguous())
    for name, k in views(x).items():
        for a, b in zip(want, all_of(k)):
            assert torch.equal(a, b), name
