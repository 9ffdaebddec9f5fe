"""Rotary tables and the norms of queries and keys with the rotation, forward
and backward, against 64-bit forms.  The tolerances count roundings (see
serving_ref.bf16_bound and the comments here)."""
import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref

pytestmark = pytest.mark.gpu


def _ok():
    assert fa.fa_get_device_error() == fa.FA_OK


def _bf(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).cuda()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _weights(kind, d, g):
    if kind == "none":
        return None, None
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    return tuple((1 + 0.3 * torch.randn(d, generator=g)).to(dt).cuda() for _ in range(2))


# ---- tables ----------------------------------------------------------------------

SCALINGS = [
    dict(),
    dict(base=500000.0),
    dict(scaling="linear", factor=4.0),
    dict(scaling="ntk", factor=8.0),
    dict(scaling="turns", factor=8.0, original=8192, low=1.0, high=4.0, base=500000.0),
    dict(scaling="yarn", factor=4.0, original=4096, low=1.0, high=32.0, mscale=1.1386),
    dict(scaling="yarn", factor=2.0, original=16, low=1.0, high=2.0),
]


@pytest.mark.parametrize("kw", SCALINGS, ids=[str(i) for i in range(len(SCALINGS))])
@pytest.mark.parametrize("max_pos,R", [(1, 128), (777, 64), (513, 30), (5, 256), (131072, 128)])
def test_table(kw, max_pos, R):
    names = {"original": "original_len"}
    c, s = fa.fa_rope_table(max_pos, R, **{names.get(k, k): v for k, v in kw.items()})
    _ok()
    rc, rs = ref.tables(max_pos, R, **kw)
    assert c.shape == s.shape == (max_pos, R // 2) and c.dtype == torch.float32
    # the reduced angle (under pi/4) rounded to fp32, a sine or cosine of 2 ulp,
    # mscale rounded and multiplied: under 8 roundings of 2^-24
    tol = 2.0 ** -21 * kw.get("mscale", 1.0)
    assert (c.cpu().double() - rc).abs().max().item() <= tol
    assert (s.cpu().double() - rs).abs().max().item() <= tol


def test_table_is_what_the_harness_builds():
    from attn_fwd_04_b200 import workloads as W
    c, s = fa.fa_rope_table(4096, 128)
    rc, rs = W.rope_tables(4096, 128, device="cuda")
    assert (c - rc).abs().max().item() <= 2.0 ** -21
    assert (s - rs).abs().max().item() <= 2.0 ** -21


# ---- forward ---------------------------------------------------------------------

def _inputs(layout, tokens, H, Hk, d, seed):
    """q, k (packed: parts of one projection), positions and the packed views."""
    g = _gen(seed)
    if layout == "packed":
        qkv = _bf(g, tokens, (H + 2 * Hk) * d)
        q = qkv[:, :H * d].view(tokens, H, d)
        k = qkv[:, H * d:(H + Hk) * d].view(tokens, Hk, d)
        pos = torch.randint(0, 700, (tokens,), generator=g, dtype=torch.int32).cuda()
        return q, k, pos, pos
    B = 2
    q, k = _bf(g, B, H, tokens, d), _bf(g, B, Hk, tokens, d)
    return q, k, None, torch.arange(tokens, dtype=torch.int32).repeat(B).cuda()


def _packed(x):
    """[B, heads, N, d] as [B * N, heads, d]; packed tensors as they are."""
    return x if x.dim() == 3 else x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])


def _close(y, r):
    y = _packed(y).double()
    assert torch.isfinite(y).all()
    over = ((y - r).abs() - ref.bf16_bound(r)).max().item()
    assert over <= 0, over


@pytest.mark.parametrize("layout", ["packed", "heads"])
@pytest.mark.parametrize("weights", ["none", "bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R,tokens,H,Hk", [(128, 128, 1, 32, 8), (128, 64, 3, 5, 5),
                                             (128, 16, 33, 3, 1), (64, 64, 17, 7, 1),
                                             (64, 48, 300, 4, 2), (128, 0, 9, 2, 2),
                                             (64, 16, 1, 1, 1)])
def test_forward(layout, weights, interleaved, d, R, tokens, H, Hk):
    q, k, pos, at = _inputs(layout, tokens, H, Hk, d, seed=d + R + tokens)
    wq, wk = _weights(weights, d, _gen(5))
    c, s = fa.fa_rope_table(700, R) if R else (None, None)
    yq, yk = fa.fa_qk_norm_rope(q, k, wq, wk, c, s, pos, eps=1e-5, interleaved=interleaved)
    _ok()
    cr = c[at.long()] if R else torch.empty((len(at), 0), device="cuda")
    sr = s[at.long()] if R else cr
    _close(yq, ref.norm_rope(_packed(q), wq, cr, sr, interleaved, 1e-5))
    _close(yk, ref.norm_rope(_packed(k), wk, cr, sr, interleaved, 1e-5))
    if R < d and weights == "none":  # the part that is not rotated is copied
        assert torch.equal(yq[..., R:], q[..., R:])


def test_one_weight_only():
    q, k, pos, at = _inputs("packed", 21, 3, 2, 128, seed=1)
    wq, wk = _weights("fp32", 128, _gen(2))
    c, s = fa.fa_rope_table(700, 128)
    cr, sr = c[at.long()], s[at.long()]
    for a, b in ((wq, None), (None, wk)):
        yq, yk = fa.fa_qk_norm_rope(q, k, a, b, c, s, pos)
        _ok()
        _close(yq, ref.norm_rope(q, a, cr, sr, False, 1e-6))
        _close(yk, ref.norm_rope(k, b, cr, sr, False, 1e-6))


def test_extreme_rows():
    """A row of zeros stays zero (eps under the root), huge and tiny rows are
    normed like others, and a row that holds an infinity or NaN spoils no other."""
    q, k, pos, at = _inputs("packed", 6, 2, 2, 64, seed=3)
    q = q.clone()
    q[0] = 0.0
    q[1] *= 1e18
    q[2] *= 1e-18
    w = torch.ones(64, device="cuda")
    c, s = fa.fa_rope_table(700, 64)
    yq, _ = fa.fa_qk_norm_rope(q, k, w, w, c, s, pos, eps=1e-30)
    r = ref.norm_rope(q, w, c[at.long()], s[at.long()], False, 1e-30)
    assert (yq[0] == 0).all()
    _close(yq, r)
    q[4, 0, 5], q[4, 1, 60] = float("inf"), float("nan")
    y2, _ = fa.fa_qk_norm_rope(q, k, w, w, c, s, pos, eps=1e-30)
    _ok()
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(y2[keep], yq[keep])
    assert y2[4, 1].isnan().all() and not y2[4].isfinite().all()


def test_in_place_strided_and_rotation_only_equals_the_fused_forward():
    """Without a norm this is fa_fwd_rope's rotation bit for bit, so attention
    on rotated copies equals the fused call; in place gives the same bits."""
    g = _gen(9)
    q, k, v = _bf(g, 2, 4, 300, 128), _bf(g, 2, 2, 300, 128), _bf(g, 2, 2, 300, 128)
    c, s = fa.fa_rope_table(512, 128)
    qr, kr = fa.fa_qk_norm_rope(q, k, None, None, c, s)
    o, lse = fa.fa_fwd_gqa(qr, kr, v, True)
    o2, lse2 = fa.fa_fwd_rope(q, k, v, c, s, True)
    _ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    q3, k3 = q.clone(), k.clone()
    fa.fa_qk_norm_rope(q3, k3, None, None, c, s, q_out=q3, k_out=k3)
    assert torch.equal(q3, qr) and torch.equal(k3, kr)
    # packed and strided, in place: the values beside them stay
    q, k, pos, _ = _inputs("packed", 40, 4, 2, 128, seed=4)
    whole = q._base if q._base is not None else q
    before = whole.clone()
    want = fa.fa_qk_norm_rope(q, k, None, None, c, s, pos % 512)
    fa.fa_qk_norm_rope(q, k, None, None, c, s, pos % 512, q_out=q, k_out=k)
    _ok()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(whole[:, 6 * 128:], before[:, 6 * 128:])


def test_positions_out_of_range_are_reported():
    q, k, pos, at = _inputs("packed", 8, 3, 1, 128, seed=6)
    c, s = fa.fa_rope_table(700, 128)
    w = torch.ones(128, device="cuda")
    good = fa.fa_qk_norm_rope(q, k, w, w, c, s, pos)
    pos = pos.clone()
    pos[2], pos[5] = -1, 700
    yq, yk = fa.fa_qk_norm_rope(q, k, w, w, c, s, pos)
    assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(yq[keep], good[0][keep]) and torch.equal(yk[keep], good[1][keep])
    assert (yq[[2, 5]] == 0).all() and (yk[[2, 5]] == 0).all()
    g = torch.randn(q.shape, device="cuda").bfloat16()
    gk = torch.randn(k.shape, device="cuda").bfloat16()
    out = fa.fa_qk_norm_rope_bwd(q, k, g, gk, w, w, c, s, pos)
    assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
    part = fa.fa_qk_norm_rope_bwd(q[keep], k[keep], g[keep], gk[keep], w, w, c, s, pos[keep])
    _ok()
    assert (out[0][[2, 5]] == 0).all() and torch.equal(out[0][keep], part[0])
    assert (out[2] - part[2]).abs().max().item() <= 1e-4


def test_no_epsilon():
    """eps = 0: rows that a thread's group of heads lacks, and tokens out of range,
    are no zeros to be normed."""
    for layout in ("packed", "heads"):
        q, k, pos, at = _inputs(layout, 7, 3, 1, 128, seed=9)
        c, s = fa.fa_rope_table(700, 128)
        w = torch.linspace(0.5, 1.5, 128, device="cuda")
        g, gk = torch.randn_like(q), torch.randn_like(k)
        yq, yk = fa.fa_qk_norm_rope(q, k, w, w, c, s, pos, eps=0.0)
        out = fa.fa_qk_norm_rope_bwd(q, k, g, gk, w, w, c, s, pos, eps=0.0)
        _ok()
        for x, y, gx, dx, dw in ((q, yq, g, out[0], out[2]), (k, yk, gk, out[1], out[3])):
            cr, sr = c[at.long()], s[at.long()]
            _close(y, ref.norm_rope(_packed(x), w, cr, sr, False, 0.0))
            rx, rw, size, sums = ref.norm_rope_bwd(_packed(x), _packed(gx), w, cr, sr, False, 0.0)
            tol = 2.0 ** -8 * rx.abs() + 2.0 ** -18 * size.amax(-1, keepdim=True)
            assert ((_packed(dx).double() - rx).abs() <= tol).all()
            assert ((dw.double() - rw).abs() <= 2.0 ** -15 * sums).all()
    q, k, pos, at = _inputs("packed", 7, 3, 1, 128, seed=9)
    pos = pos.clone()
    pos[3] = 700
    out = fa.fa_qk_norm_rope_bwd(q, k, q, k, w, w, c, s, pos, eps=0.0)
    assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
    assert all(torch.isfinite(t).all() for t in out) and (out[0][3] == 0).all()


def test_no_tokens():
    q, k = torch.empty((0, 4, 128)).bfloat16().cuda(), torch.empty((0, 2, 128)).bfloat16().cuda()
    w = torch.ones(128, device="cuda")
    yq, yk = fa.fa_qk_norm_rope(q, k, w, w)
    assert yq.shape == (0, 4, 128) and yk.shape == (0, 2, 128)
    _, _, dw, dw2 = fa.fa_qk_norm_rope_bwd(q, k, q, k, w, w)
    assert (dw == 0).all() and (dw2 == 0).all()


# ---- backward --------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["packed", "heads"])
@pytest.mark.parametrize("weights", ["none", "bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R,tokens,H,Hk", [(128, 128, 1, 4, 1), (128, 64, 33, 5, 3),
                                             (64, 64, 300, 7, 1), (64, 16, 9, 2, 2),
                                             (128, 0, 17, 3, 3), (128, 128, 5000, 8, 2)])
def test_backward(layout, weights, interleaved, d, R, tokens, H, Hk):
    q, k, pos, at = _inputs(layout, tokens, H, Hk, d, seed=d + R + tokens)
    g = _gen(7)
    gq, gk = _bf(g, *q.shape, std=0.1), _bf(g, *k.shape, std=0.1)
    wq, wk = _weights(weights, d, _gen(5))
    c, s = fa.fa_rope_table(5000, R) if R else (None, None)
    got = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, wq, wk, c, s, pos, eps=1e-5,
                                 interleaved=interleaved)
    _ok()
    cr = c[at.long()] if R else torch.empty((len(at), 0), device="cuda")
    sr = s[at.long()] if R else cr
    for x, gx, w, dx, dw in ((q, gq, wq, got[0], got[2]), (k, gk, wk, got[1], got[3])):
        rx, rw, size, sums = ref.norm_rope_bwd(_packed(x), _packed(gx), w, cr, sr, interleaved,
                                               1e-5)
        # half a bf16 step, and under 40 fp32 steps (2^-18) of the terms of dx,
        # the pair's two among them (hence the largest of the row)
        tol = 2.0 ** -8 * rx.abs() + 2.0 ** -18 * size.amax(-1, keepdim=True) + 1e-38
        over = ((_packed(dx).double() - rx).abs() - tol).max().item()
        assert over <= 0, over
        if w is None:
            assert dw is None
        else:
            # fp32 sums of at most 256 rows a thread and 16 threads, each term
            # and each addition a few steps of 2^-24: 2^-15 of the terms' sum
            assert dw.dtype == torch.float32
            over = ((dw.double() - rw).abs() - 2.0 ** -15 * sums).max().item()
            assert over <= 0, over


def test_backward_is_the_derivative():
    """The 64-bit formula against central differences of the 64-bit forward."""
    g = _gen(11)
    x = torch.randn((3, 2, 64), generator=g, dtype=torch.float64)
    gy = torch.randn((3, 2, 64), generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(64, generator=g, dtype=torch.float64)
    for inter in (False, True):
        c, s = ref.tables(3, 32)
        dx, dw, _, _ = ref.norm_rope_bwd(x, gy, w, c, s, inter, 1e-5)

        def loss(x_, w_):
            return (ref.norm_rope(x_, w_, c, s, inter, 1e-5) * gy).sum()

        h = 1e-6
        for idx in [(0, 0, 0), (1, 1, 17), (2, 0, 40), (2, 1, 63)]:
            e = torch.zeros_like(x)
            e[idx] = h
            num = (loss(x + e, w) - loss(x - e, w)) / (2 * h)
            assert abs(num.item() - dx[idx].item()) <= 1e-7
        for i in (0, 16, 63):
            e = torch.zeros_like(w)
            e[i] = h
            num = (loss(x, w + e) - loss(x, w - e)) / (2 * h)
            assert abs(num.item() - dw[i].item()) <= 1e-7


def test_backward_repeats_bit_for_bit_in_place_and_replayed():
    q, k, pos, _ = _inputs("packed", 900, 6, 2, 128, seed=8)
    g = _gen(8)
    gq, gk = _bf(g, *q.shape, std=0.1), _bf(g, *k.shape, std=0.1)
    w = torch.linspace(0.5, 1.5, 128, device="cuda")
    c, s = fa.fa_rope_table(700, 128)
    want = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, w, w, c, s, pos)
    again = fa.fa_qk_norm_rope_bwd(q, k, gq, gk, w, w, c, s, pos)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    g2, g3 = gq.clone(), gk.clone()
    into = fa.fa_qk_norm_rope_bwd(q, k, g2, g3, w, w, c, s, pos, dq=g2, dk=g3)
    assert all(torch.equal(a, b) for a, b in zip(want, into))
    # two captured graphs of one stream, replayed in turn on new inputs
    side = torch.cuda.Stream()
    ins = [(q.clone(), k.clone()) for _ in range(2)]
    graphs, outs = [], []
    side.wait_stream(torch.cuda.current_stream())
    for a, b in ins:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append(fa.fa_qk_norm_rope_bwd(a, b, gq, gk, w, w, c, s, pos))
        graphs.append(graph)
    ins[1][0].mul_(2.0)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(want, outs[0]))
    other = fa.fa_qk_norm_rope_bwd(ins[1][0], k, gq, gk, w, w, c, s, pos)
    assert all(torch.equal(a, b) for a, b in zip(other, outs[1]))


def test_library_workspace_is_refused_in_a_capture_and_serves_outside_one():
    """The C call without scratch: the library's workspace, but not in a graph."""
    L = fa.lib()
    q, k, pos, _ = _inputs("packed", 50, 2, 2, 64, seed=2)
    q, k = q.contiguous(), k.contiguous()
    w = torch.ones(64, device="cuda")
    c, s = fa.fa_rope_table(700, 64)
    want = fa.fa_qk_norm_rope_bwd(q, k, q, k, w, w, c, s, pos)
    dq, dk, dw, dv = (torch.empty_like(x) for x in (q, k, w, w))

    def call(stream):
        return L.fa_qk_norm_rope_bwd(
            q.data_ptr(), k.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(), dk.data_ptr(),
            dw.data_ptr(), dv.data_ptr(), w.data_ptr(), w.data_ptr(), 1, c.data_ptr(),
            s.data_ptr(), 700, 64, 0, pos.data_ptr(), 0, 1, 50, 2, 2, 64, 0, 0, 0, 0, 0, 0, 1e-6,
            None, 0, stream)

    assert call(torch.cuda.current_stream().cuda_stream) == fa.FA_OK
    _ok()
    assert torch.equal(dq, want[0]) and torch.equal(dw, want[2])
    got = []
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        x = torch.zeros(1, device="cuda")  # a graph of something
        got.append(call(torch.cuda.current_stream().cuda_stream))
        x += 1
    assert got == [fa.FA_ERR_UNSUPPORTED]


def test_other_stream_orders_outputs():
    """Outputs made on the call's stream, read there; inputs ready before."""
    q, k, pos, _ = _inputs("packed", 2000, 8, 2, 128, seed=12)
    c, s = fa.fa_rope_table(700, 128)
    want = fa.fa_qk_norm_rope(q, k, None, None, c, s, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.fa_qk_norm_rope(q, k, None, None, c, s, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
