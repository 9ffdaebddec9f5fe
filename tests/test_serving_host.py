"""Refusals of the calls on tables, norms with the rotation, appends and the
8-bit cache, without a GPU; and the 64-bit forms that their GPU tests use."""
import ctypes
import math

import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref
from attn_fwd_04_b200 import build as fa_build

A, MIS, S = 1 << 20, (1 << 20) + 8, None  # never dereferenced


@pytest.fixture(scope="module")
def L():
    fa_build.build()
    return fa.lib()


def table(L, c=A, s=A, n=64, R=64, base=1e4, kind=0, f=2.0, orig=64, low=1.0, high=4.0, m=1.0):
    return L.fa_rope_table(c, s, n, R, base, kind, f, orig, low, high, m, S)


def norm(L, q=A, k=A, qo=A, ko=A, qw=A, kw=A, wt=1, c=A, s=A, mp=64, R=64, inter=0, pos=A,
         layout=0, B=1, N=8, H=4, Hk=2, d=128, st=(0, 0, 0, 0), eps=1e-6):
    return L.fa_qk_norm_rope(q, k, qo, ko, qw, kw, wt, c, s, mp, R, inter, pos, layout, B, N, H,
                             Hk, d, *st, eps, S)


def norm_bwd(L, q=A, k=A, gq=A, gk=A, dq=A, dk=A, dqw=A, dkw=A, qw=A, kw=A, wt=1, c=A, s=A,
             mp=64, R=64, inter=0, pos=A, layout=0, B=1, N=8, H=4, Hk=2, d=128, st=(0,) * 6,
             eps=1e-6, ws=A, wsb=1 << 30):
    return L.fa_qk_norm_rope_bwd(q, k, gq, gk, dq, dk, dqw, dkw, qw, kw, wt, c, s, mp, R, inter,
                                 pos, layout, B, N, H, Hk, d, *st, eps, ws, wsb, S)


def append(L, eight=False, q=A, k=A, v=A, cu=A, qo=A, kp=A, vp=A, ks=A, vs=A, block=64, t=A,
           tl=8, mpg=0, lens=A, qw=A, kw=A, wt=0, c=A, s=A, mp=64, R=64, inter=0, B=2, H=4, Hk=2,
           total=10, P=8, d=128, ps=256, st=(0, 0, 0), eps=1e-6):
    rest = (t, tl, mpg, lens, qw, kw, wt, c, s, mp, R, inter, B, H, Hk, total, P, d, ps, *st,
            eps, S)
    if eight:
        return L.fa_append_paged_fp8(q, k, v, cu, qo, kp, vp, ks, vs, block, *rest)
    return L.fa_append_paged_rope(q, k, v, cu, qo, kp, vp, *rest)


def decode(L, q=A, kp=A, vp=A, ks=A, vs=A, block=64, t=A, tl=8, mpg=0, lens=A, o=A, lse=A, B=2,
           H=4, Hk=2, P=8, d=128, ps=256, scale=0.1, ws=A, wsb=1 << 30):
    return L.fa_decode_paged_fp8(q, kp, vp, ks, vs, block, t, tl, mpg, lens, o, lse, B, H, Hk, P,
                                 d, ps, scale, ws, wsb, S)


def test_table_errors(L):
    assert table(L, c=None) == fa.FA_ERR_NULL
    for bad in (dict(n=0), dict(R=0), dict(R=31), dict(R=258), dict(base=1.0),
                dict(base=math.inf), dict(m=math.nan), dict(kind=1, f=0.0),
                dict(kind=1, f=math.nan), dict(kind=2, R=2), dict(kind=3, orig=0),
                dict(kind=3, low=4.0), dict(kind=4, low=0.0), dict(kind=4, high=math.inf)):
        assert table(L, **bad) == fa.FA_ERR_SHAPE, bad
    assert table(L, kind=5) == fa.FA_ERR_UNSUPPORTED
    assert table(L, kind=-1) == fa.FA_ERR_UNSUPPORTED
    assert table(L, s=MIS) == fa.FA_ERR_ALIGN


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_norm_errors(L, call):
    assert call(L, q=None) == fa.FA_ERR_NULL
    assert call(L, c=None) == fa.FA_ERR_NULL
    for bad in (dict(N=0), dict(H=0), dict(Hk=-1), dict(B=2), dict(R=144), dict(R=-16),
                dict(mp=0), dict(pos=None, mp=7), dict(eps=-1.0), dict(eps=math.nan),
                dict(layout=1, st=(512,) + (0,) * (3 if call is norm else 5)),
                dict(st=(500,) + (0,) * (3 if call is norm else 5)),
                dict(B=1 << 15, N=1 << 20, layout=1, pos=A)):
        assert call(L, **bad) == fa.FA_ERR_SHAPE, bad
    for bad in (dict(d=96), dict(R=8), dict(R=40), dict(wt=2), dict(layout=2)):
        assert call(L, **bad) == fa.FA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(kw=MIS), dict(c=MIS),
                dict(st=(516,) + (0,) * (3 if call is norm else 5))):
        assert call(L, **bad) == fa.FA_ERR_ALIGN, bad


def test_norm_bwd_errors(L):
    assert norm_bwd(L, gq=None) == fa.FA_ERR_NULL
    assert norm_bwd(L, dqw=None) == fa.FA_ERR_NULL   # a weight without its gradient
    assert norm_bwd(L, kw=None) == fa.FA_ERR_NULL    # a gradient without its weight
    assert norm_bwd(L, gk=MIS) == fa.FA_ERR_ALIGN
    assert norm_bwd(L, ws=MIS) == fa.FA_ERR_ALIGN
    assert norm_bwd(L, wsb=-1) == fa.FA_ERR_SHAPE
    n = ctypes.c_int(0)
    assert L.fa_qk_norm_rope_bwd_workspace(1, 1, 1, 1, 128, None) == fa.FA_ERR_NULL
    assert L.fa_qk_norm_rope_bwd_workspace(1, 0, 1, 1, 128, ctypes.byref(n)) == fa.FA_ERR_SHAPE
    assert L.fa_qk_norm_rope_bwd_workspace(1, 1, 1, 1, 32, ctypes.byref(n)) == \
        fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("eight", [False, True])
def test_append_errors(L, eight):
    for bad in (dict(k=None), dict(cu=None), dict(t=None), dict(lens=None), dict(q=None),
                dict(qo=None), dict(s=None)):
        assert append(L, eight, **bad) == fa.FA_ERR_NULL, bad
    for bad in (dict(B=0), dict(Hk=0), dict(H=0), dict(total=-1), dict(P=0), dict(tl=-1),
                dict(mpg=5), dict(mpg=-1), dict(R=144), dict(mp=0), dict(eps=-1.0),
                dict(st=(0, 200, 0))):
        assert append(L, eight, **bad) == fa.FA_ERR_SHAPE, bad
    for bad in (dict(d=32), dict(ps=128), dict(R=24), dict(wt=7)):
        assert append(L, eight, **bad) == fa.FA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(kp=MIS), dict(qw=MIS), dict(st=(0, 0, 260))):
        assert append(L, eight, **bad) == fa.FA_ERR_ALIGN, bad


def test_append_fp8_errors(L):
    assert append(L, True, ks=None) == fa.FA_ERR_NULL
    for block in (0, 8, 48, 512):
        assert append(L, True, block=block) == fa.FA_ERR_UNSUPPORTED
    assert append(L, True, vs=MIS + 2) == fa.FA_ERR_ALIGN
    assert append(L, True, total=1 << 30, Hk=64, d=64) == fa.FA_ERR_SHAPE  # too many blocks


def test_decode_errors(L):
    for name in ("q", "kp", "vs", "t", "lens", "o"):
        assert decode(L, **{name: None}) == fa.FA_ERR_NULL, name
    for bad in (dict(B=0), dict(H=3), dict(Hk=0), dict(P=0), dict(tl=-1), dict(mpg=5),
                dict(mpg=-1), dict(scale=math.nan), dict(wsb=-1),
                dict(B=1 << 13, H=1 << 14)):
        assert decode(L, **bad) == fa.FA_ERR_SHAPE, bad
    for bad in (dict(d=96), dict(ps=64), dict(block=8), dict(block=96), dict(block=512)):
        assert decode(L, **bad) == fa.FA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=MIS), dict(vp=MIS), dict(ks=MIS + 1), dict(ws=MIS), dict(lse=MIS + 2)):
        assert decode(L, **bad) == fa.FA_ERR_ALIGN, bad
    n = ctypes.c_int(0)
    assert L.fa_decode_paged_fp8_workspace(1, 1, 1, 128, None) == fa.FA_ERR_NULL
    assert L.fa_decode_paged_fp8_workspace(1, 3, 2, 128, ctypes.byref(n)) == fa.FA_ERR_SHAPE
    assert L.fa_decode_paged_fp8_workspace(1, 2, 2, 80, ctypes.byref(n)) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_cuda_errors(L):
    assert table(L) == fa.FA_ERR_CUDA
    assert norm(L) == fa.FA_ERR_CUDA
    assert norm(L, layout=1, B=3) == fa.FA_ERR_CUDA
    assert norm_bwd(L) == fa.FA_ERR_CUDA
    for eight in (False, True):
        assert append(L, eight) == fa.FA_ERR_CUDA
        assert append(L, eight, q=None, qo=None, H=0, mpg=4) == fa.FA_ERR_CUDA
    assert decode(L) == fa.FA_ERR_CUDA
    assert decode(L, lse=None, mpg=4) == fa.FA_ERR_CUDA


# -- the Python wrappers, on meta tensors ------------------------------------------

@pytest.fixture
def meta(monkeypatch):
    from attn_fwd_04_b200 import fa as binding

    fa_build.build()
    binding._short()  # (its short way answers nothing for tensors that are not on a GPU)

    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(binding, "_DEVICE_TYPES", ("cuda", "meta"))
    monkeypatch.setattr(binding, "lib", no_library)
    return binding


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


I32, F32, F8 = torch.int32, torch.float32, torch.float8_e4m3fn


def reaches(f, *a, **kw):
    with pytest.raises(AssertionError, match="library was called"):
        f(*a, **kw)


def test_table_wrapper(meta):
    reaches(meta.fa_rope_table, 16, 64, device="meta")
    for a, kw in (((16, 63), {}), ((0, 64), {}), ((16, 64), dict(scaling="other")),
                  ((16, 64), dict(rope_cos=_m(16, 31, dtype=F32)))):
        with pytest.raises(ValueError):
            meta.fa_rope_table(*a, device="meta", **kw)
    with pytest.raises(TypeError):
        meta.fa_rope_table(16, 64, rope_cos=_m(16, 32), device="meta")


def test_norm_wrapper(meta):
    c = _m(64, 32, dtype=F32)
    x = _m(9, 8 * 128)
    q, k = x[:, :512].view(9, 4, 128), x[:, 512:768].view(9, 2, 128)
    w = _m(128, dtype=F32)
    reaches(meta.fa_qk_norm_rope, q, k, w, w, c, c, _m(9, dtype=I32))
    reaches(meta.fa_qk_norm_rope, _m(2, 4, 9, 128), _m(2, 2, 9, 128), None, None, c, c)
    reaches(meta.fa_qk_norm_rope_bwd, q, k, q, k, w, w, c, c)
    for kw in (dict(positions=_m(8, dtype=I32)), dict(rope_sin=None), dict(q_weight=_m(64, dtype=F32)),
               dict(rope_sin=_m(64, 31, dtype=F32)), dict(q_out=_m(9, 3, 128)),
               dict(q_out=_m(9, 4, 256)[..., :128])):
        args = dict(q_weight=w, k_weight=w, rope_cos=c, rope_sin=c)
        args.update(kw)
        with pytest.raises(ValueError):
            meta.fa_qk_norm_rope(q, k, **args)
    for kw in (dict(positions=_m(9, dtype=torch.int64)), dict(q_weight=_m(128, dtype=torch.float16)),
               dict(q_weight=_m(128))):
        args = dict(q_weight=w, k_weight=w, rope_cos=c, rope_sin=c)
        args.update(kw)
        with pytest.raises(TypeError):
            meta.fa_qk_norm_rope(q, k, **args)
    with pytest.raises(ValueError):
        meta.fa_qk_norm_rope(q, _m(8, 2, 128))
    with pytest.raises(ValueError):  # tokens that overlap
        meta.fa_qk_norm_rope(q[:1].expand(9, 4, 128), k)
    with pytest.raises(TypeError):
        meta.fa_qk_norm_rope(q.float(), k)
    with pytest.raises(TypeError):
        meta.fa_qk_norm_rope_bwd(q, k, None, k)
    with pytest.raises(ValueError):
        meta.fa_qk_norm_rope_bwd(q, k, q, k, dq_weight=w)


def _append_args(eight, P=5, Hk=2, d=128, B=3, total=9):
    dt = F8 if eight else torch.bfloat16
    a = [_m(total, 4, d), _m(total, Hk, d), _m(total, Hk, d), _m(B + 1, dtype=I32),
         _m(P, Hk, 256, d, dtype=dt), _m(P, Hk, 256, d, dtype=dt)]
    if eight:
        a += [_m(P, Hk, 4, dtype=F32), _m(P, Hk, 4, dtype=F32)]
    return a + [_m(7, dtype=I32), _m(B, dtype=I32)]


@pytest.mark.parametrize("eight", [False, True])
def test_append_wrappers(meta, eight):
    f = meta.fa_append_paged_fp8 if eight else meta.fa_append_paged_rope
    n = len(_append_args(eight))
    reaches(f, *_append_args(eight))
    a = _append_args(eight)
    a[-2] = _m(3, 2, dtype=I32)
    reaches(f, *a)
    a[0] = None
    reaches(f, *a)
    with pytest.raises(ValueError):
        f(*a, q_weight=_m(128))
    for i, t in ((0, _m(8, 4, 128)), (2, _m(9, 3, 128)), (5, _append_args(eight, P=6)[5]),
                 (n - 1, _m(4, dtype=I32)), (n - 2, _m(2, 2, dtype=I32)), (1, _m(9, 3, 128))):
        a = _append_args(eight)
        a[i] = t
        with pytest.raises(ValueError):
            f(*a)
    for i, t in ((4, _m(5, 2, 256, 128, dtype=torch.float16)), (3, _m(4, dtype=torch.int64))):
        a = _append_args(eight)
        a[i] = t
        with pytest.raises(TypeError):
            f(*a)
    if eight:
        for t in (_m(5, 2, 3, dtype=F32), _m(5, 1, 4, dtype=F32), _m(4, 2, 4, dtype=F32)):
            a = _append_args(eight)
            a[6] = a[7] = t
            with pytest.raises(ValueError):
                f(*a)


def test_decode_wrapper(meta):
    def args(B=3, H=8, Hk=2, P=5, d=128):
        return [_m(B, H, d), _m(P, Hk, 256, d, dtype=F8), _m(P, Hk, 256, d, dtype=F8),
                _m(P, Hk, 4, dtype=F32), _m(P, Hk, 4, dtype=F32), _m(7, dtype=I32),
                _m(B, dtype=I32)]
    f = meta.fa_decode_paged_fp8
    reaches(f, *args())
    with pytest.raises(ValueError, match="multiple"):
        f(*args(H=7))
    for i, t in ((6, _m(4, dtype=I32)), (5, _m(2, 2, dtype=I32)), (3, _m(5, 2, 8, dtype=F32)),
                 (2, _m(6, 2, 256, 128, dtype=F8))):
        a = args()
        a[i] = t
        with pytest.raises(ValueError):
            f(*a)
    with pytest.raises(TypeError):
        a = args()
        a[1] = _m(5, 2, 256, 128)
        f(*a)
    with pytest.raises(ValueError):
        f(*args(), lse=_m(3, 7, dtype=F32))


# -- the 64-bit forms ------------------------------------------------------------------

def test_e4m3_rounds_as_the_type_does():
    codes = torch.arange(256, dtype=torch.uint8).view(F8).double()
    codes = codes[codes.isfinite()]
    assert torch.equal(ref.e4m3(codes).double(), codes)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 8, (20000,),
                                                                   generator=g).float())
    x = x[x.abs() <= 448]
    assert torch.equal(ref.e4m3(x.double()).view(torch.uint8), x.to(F8).view(torch.uint8))
    assert ref.e4m3(torch.tensor([448.1, math.inf, math.nan]).double()).float().isnan().all()


def test_least_scale():
    assert ref.least_scale(0.0) == 2.0 ** -64 == ref.least_scale(2.0 ** -80)
    assert ref.least_scale(448.0) == 1.0 and ref.least_scale(448.1) == 2.0
    assert ref.least_scale(1e30) == 2.0 ** 64
