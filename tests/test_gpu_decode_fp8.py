"""Decode over the 8-bit paged cache against the 64-bit form, and the whole
path of a token: tables, appends, decode."""
import math

import pytest
import torch

import attn_fwd_04_b200 as fa
import serving_ref as ref

pytestmark = pytest.mark.gpu
PS = 256
FP8 = torch.float8_e4m3fn


def _ok():
    assert fa.fa_get_device_error() == fa.FA_OK


class Cache:
    def __init__(self, lens, H, Hk, d, block, table, seed=0, spread=1.0, qstd=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens = lens
        B = len(lens)
        pages = ref.pages_of(lens)
        P = sum(pages) + 2
        perm = torch.randperm(P, generator=g).int()
        if table == "packed":
            self.table = perm[:sum(pages)].clone()
        else:
            self.table = torch.full((B, max(1, max(pages))), -7, dtype=torch.int32)
            at = 0
            for b, n in enumerate(pages):
                self.table[b, :n] = perm[at:at + n]
                at += n
        self.q = (torch.randn((B, H, d), generator=g) * qstd).bfloat16().cuda()
        shape = (P, Hk, PS, d)
        self.kp, self.vp = ((torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(FP8)
                            .view(torch.uint8) for _ in range(2))
        sc = (P, Hk, PS // block)
        self.ks, self.vs = (0.01 * torch.exp2(spread * (torch.rand(sc, generator=g) - 0.5))
                            for _ in range(2))
        # whatever is behind the last token is not a number
        for b, n in enumerate(lens):
            if n > 0 and n % PS:
                p = ref.page_list(self.table, lens, b)[-1]
                for pool, s in ((self.kp, self.ks), (self.vp, self.vs)):
                    pool[p, :, n % PS:] = 0x7F
                    s[p, :, -(-(n % PS) // block):] = math.nan
        self.kp, self.vp = self.kp.cuda().view(FP8), self.vp.cuda().view(FP8)
        self.ks, self.vs = self.ks.cuda(), self.vs.cuda()
        self.seq = torch.tensor(lens).int().cuda()
        self.scale = d ** -0.5

    def call(self, more=0, **kw):
        """`more`: entries of the table that no sequence has a use for; a few pages
        a row take another way through the kernels than many, and very many yet
        another where more than 16 query heads share a K/V head."""
        table = self.table
        if more:
            shape = (more,) if table.dim() == 1 else (len(table), more)
            table = torch.cat([table, torch.full(shape, -1, dtype=torch.int32)], -1)
        lse = torch.full(self.q.shape[:2], 9.0, device="cuda")
        o = torch.full(self.q.shape, math.nan, device="cuda").bfloat16()
        fa.fa_decode_paged_fp8(self.q, self.kp, self.vp, self.ks, self.vs, table.cuda(),
                               self.seq, scale=self.scale, o=o, lse=lse, **kw)
        return o, lse

    def both(self):
        for more in (0, 9, 1300):
            o, lse = self.call(more)
            _ok()
            self.check(o, lse)

    def check(self, o, lse):
        r, rl, absv, reach = ref.decode(self.q, self.kp, self.vp, self.ks, self.vs, self.table,
                                        self.lens, self.scale)
        assert torch.isfinite(o).all()
        n = torch.tensor([max(x, 1) for x in self.lens], device="cuda")[:, None]
        # a score is a sum of d products in fp32 (one rounding of 2^-23 for each
        # at most) and three factors: under 2^-16 of `reach`, its terms' sum.
        # exp2 turns that into as much relative to a weight.  Weights are held
        # to 11 bits (2^-11), the sums over tokens in fp32 (2^-24 each).
        delta = 2.0 ** -16 * reach
        weights = 2.0 ** -11 + 4 * delta + 2.0 ** -18 + 2.0 ** -22 * n
        tol = 2.0 ** -8 * r.abs() + weights[..., None] * absv + 1e-30
        over = ((o.double() - r).abs() - tol).max().item()
        assert over <= 0, over
        empty = torch.tensor([x <= 0 for x in self.lens], device="cuda")
        assert (lse[empty] == -math.inf).all() and (o[empty] == 0).all()
        live = ~empty
        if live.any():
            tl = 2 * delta + 2.0 ** -20 * (1 + rl.abs()) + 2.0 ** -22 * n
            assert ((lse.double() - rl).abs() <= tl)[live].all()


LENS = [
    [1],
    [777],
    [0, 1, 15, 16, 17, 31, 32, 33, 255, 256, 257, 511, 512, 513, 0],
    [4103, 1, 0, 2048, 3000],
    [0, 0],
    [1] * 130,
]


@pytest.mark.parametrize("table", ["packed", "rows"])
@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
@pytest.mark.parametrize("H,Hk,d,block", [(8, 2, 128, 64), (5, 5, 64, 16), (7, 1, 128, 32),
                                          (16, 2, 64, 128), (16, 1, 128, 256), (2, 1, 128, 16)])
def test_decode(table, lens, H, Hk, d, block):
    c = Cache(lens, H, Hk, d, block, table, seed=len(lens) + d)
    c.both()


@pytest.mark.parametrize("G", [3, 9, 11, 12, 16, 17, 24, 32, 33, 48, 272])
@pytest.mark.parametrize("d", [64, 128])
def test_group_sizes(G, d):
    c = Cache([300, 0, 1, 1025], 2 * G, 2, d, 64, "rows", seed=G)
    c.both()


@pytest.mark.parametrize("G", [12, 32, 40])
@pytest.mark.parametrize("d,block", [(64, 16), (128, 32), (64, 128)])
def test_wide_groups_over_long_and_many_sequences(G, d, block):
    for lens, Hk, table in (([9000, 1, 0, 2500], 1, "packed"),
                            ([(i * 61) % 700 for i in range(150)], 2, "rows")):
        c = Cache(lens, G * Hk, Hk, d, block, table, seed=G, spread=4.0)
        c.both()


def test_long_sequences_beside_short_ones():
    c = Cache([40000, 3, 9000], 8, 1, 128, 64, "packed", seed=1)
    c.both()


def test_many_sequences():
    lens = [(i * 37) % 70 for i in range(3000)]
    c = Cache(lens, 2, 1, 64, 16, "packed", seed=2)
    c.both()


@pytest.mark.parametrize("qstd", [0.0, 1e-20, 30.0])
@pytest.mark.parametrize("spread", [1.0, 24.0])
def test_magnitudes(qstd, spread):
    """Scales that differ by 2^24 over a cache, queries that are tiny, zero, or
    make the softmax one-hot."""
    c = Cache([700, 2000, 31], 8, 2, 128, 16, "packed", seed=3, spread=spread, qstd=qstd)
    c.both()


def test_growing_scales_and_scores():
    """Each block larger than all before it, in both caches; and zero scales."""
    c = Cache([1500], 4, 1, 128, 32, "packed", seed=3)
    for i, p in enumerate(ref.page_list(c.table, c.lens, 0)):
        blk = torch.arange(8, device="cuda") + 8 * i
        n = min(8, -(-(1500 - 256 * i) // 32))
        c.vs[p, 0, :n] = torch.exp2(blk.float() - 30)[:n]
        c.ks[p, 0, :n] = (0.001 * 1.05 ** blk.float())[:n]
    c.both()
    p = ref.page_list(c.table, c.lens, 0)
    c.vs[p[0]], c.ks[p[1]] = 0.0, 0.0
    c.both()
    for i in p:
        c.vs[i, :, :2] = 0.0
        c.vs[i] = torch.where(c.vs[i].isnan(), math.nan, 0.0)
    o, lse = c.call()
    _ok()
    assert (o == 0).all()


def test_scales_at_the_ends_of_their_range():
    c = Cache([600], 4, 2, 64, 64, "packed", seed=3)
    keep = c.vs.isnan()
    for s in (2.0 ** -64, 2.0 ** 64):
        c.vs = torch.where(keep, math.nan, s)
        c.both()
    c.vs = torch.where(keep, math.nan, 0.01)
    c.ks = torch.where(c.ks.isnan(), math.nan, 2.0 ** 64)
    c.q = (c.q.float() * 2.0 ** -70).bfloat16()
    c.both()


def test_every_code_and_a_query_of_wide_range():
    c = Cache([512], 8, 1, 64, 64, "packed", seed=4)
    codes = torch.arange(256, dtype=torch.uint8)
    codes[(codes & 127) == 127] = 0
    for p in range(c.kp.shape[0]):
        c.kp.view(torch.uint8)[p, 0] = codes[:, None].cuda()
        c.vp.view(torch.uint8)[p, 0] = codes[:, None].roll(p, 0).cuda()
    c.q *= torch.exp2(torch.linspace(-12, 0, 64, device="cuda")).bfloat16()
    c.both()


def test_lse_is_optional_and_calls_repeat_bit_for_bit():
    c = Cache([400, 100, 1257], 16, 4, 128, 64, "rows", seed=5)
    for more in (9, 0):
        o, lse = c.call(more)
        for _ in range(3):
            a, b = c.call(more)
            assert torch.equal(a, o) and torch.equal(b, lse)
    alone = fa.fa_decode_paged_fp8(c.q, c.kp, c.vp, c.ks, c.vs, c.table.cuda(), c.seq)
    _ok()
    assert torch.equal(alone, o)


def test_bad_input_is_reported():
    c = Cache([300, 200, 600], 4, 2, 128, 64, "packed", seed=6)
    want, _ = c.call()
    _ok()
    c.seq[0] = -5
    c.table = c.table[2:].clone()
    o, lse = c.call()
    assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
    assert (o[0] == 0).all() and (lse[0] == -math.inf).all()
    assert (o[1:].float() - want[1:].float()).abs().max().item() <= 2.0 ** -6
    # longer than the table's entries: cut to them
    c = Cache([300, 200, 512], 4, 2, 128, 64, "packed", seed=6)
    want, wl = c.call()
    _ok()
    for n in (513, 9000, 2 ** 31 - 1):
        c.seq[2] = n
        o, lse = c.call()
        assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
        assert (lse - wl).abs().max().item() <= 1e-4
        assert (o.float() - want.float()).abs().max().item() <= 2.0 ** -6
    c.seq[:] = 2 ** 31 - 1  # the sum of their pages passes 32 bits many times
    c.seq = c.seq.repeat(400)
    c.q = c.q.repeat(400, 1, 1)
    c.lens = [1] * 1200
    o, lse = c.call()
    assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
    assert (o[1:] == 0).all() and (lse[1:] == -math.inf).all()
    # a page outside the pool
    for table in ("packed", "rows"):
        c = Cache([300, 200, 600], 4, 2, 128, 64, table, seed=6)
        want, _ = c.call()
        _ok()
        for bad in (-1, c.kp.shape[0], 2 ** 31 - 1):
            t = c.table.clone()
            c.table.view(-1)[3 if table == "packed" else 6] = bad
            o, _ = c.call()
            assert fa.fa_get_device_error() == fa.FA_ERR_DEVICE_BAD_INPUT
            assert (o[:2].float() - want[:2].float()).abs().max().item() <= 2.0 ** -6
            c.table = t


def test_two_streams_and_two_graphs():
    """Calls that overlap have scratch of their own, graphs too."""
    a = Cache([9000, 20, 3000], 8, 2, 128, 64, "packed", seed=7)
    b = Cache([5000, 7000, 1], 8, 2, 128, 32, "rows", seed=8)
    want = [a.call(), b.call()]
    _ok()
    tables = [a.table.cuda(), b.table.cuda()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]

    def call(i, stream=None):
        c = (a, b)[i]
        fa.fa_decode_paged_fp8(c.q, c.kp, c.vp, c.ks, c.vs, tables[i], c.seq, o=outs[i][0],
                               lse=outs[i][1], stream=stream)

    torch.cuda.synchronize()
    for _ in range(50):
        for i, s in enumerate(streams):
            call(i, s)
    torch.cuda.synchronize()
    _ok()
    for w, x in zip(want, outs):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
        x[0].zero_()
        x[1].zero_()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            call(i)
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    _ok()
    for w, x in zip(want, outs):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])


def test_library_workspace_is_refused_in_a_capture_and_serves_outside_one():
    c = Cache([9000, 300], 8, 2, 128, 64, "packed", seed=7)
    want, wl = c.call()
    table, o = c.table.cuda(), torch.empty_like(c.q)

    def call():
        return fa.lib().fa_decode_paged_fp8(
            c.q.data_ptr(), c.kp.data_ptr(), c.vp.data_ptr(), c.ks.data_ptr(), c.vs.data_ptr(),
            64, table.data_ptr(), len(table), 0, c.seq.data_ptr(), o.data_ptr(), None, 2, 8, 2,
            c.kp.shape[0], 128, PS, c.scale, None, 0, torch.cuda.current_stream().cuda_stream)

    assert call() == fa.FA_OK
    _ok()
    assert torch.equal(o, want)
    got = []
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        x = torch.zeros(1, device="cuda")
        got.append(call())
        x += 1
    assert got == [fa.FA_ERR_UNSUPPORTED]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("table", ["packed", "rows"])
def test_a_token_all_the_way(interleaved, table):
    """Prompts, then tokens one by one: table, norm and rotation, append into
    8-bit pages, decode -- against attention in 64 bits over the keys and values
    themselves.  What lies between is the cache's rounding: values are off by
    at most half a step of 4 bits (2^-4 of the value, 2^-10 of the block's
    scale, itself at most 2^-8 of the block's largest magnitude: 2^-18 of it)."""
    H, Hk, d, block, B = 8, 2, 128, 32, 3
    g = torch.Generator().manual_seed(1)
    cos, sin = fa.fa_rope_table(1024, 64, 500000.0, "yarn", 4.0, 256, 1.0, 32.0, 1.1)
    qw, kw = (1 + 0.2 * torch.randn(d, generator=g).cuda() for _ in range(2))
    P = 12
    kp, vp = (torch.full((P, Hk, PS, d), 0x7F, dtype=torch.uint8, device="cuda").view(FP8)
              for _ in range(2))
    ks, vs = (torch.full((P, Hk, PS // block), math.nan, device="cuda") for _ in range(2))
    rows = torch.randperm(P, generator=g).int().view(B, 4)
    lens = [0] * B
    keys, vals = [[] for _ in range(B)], [[] for _ in range(B)]
    for new in ([250, 40, 300],) + ([1, 1, 1],) * 12:
        total = sum(new)
        x = torch.randn((total, (H + 2 * Hk) * d), generator=g).bfloat16().cuda()
        q, k, v = (t.view(total, -1, d) for t in x.split([H * d, Hk * d, Hk * d], 1))
        cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0))).int().cuda()
        pos = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, new)]).cuda()
        lens = [n + m for n, m in zip(lens, new)]
        seq = torch.tensor(lens).int().cuda()
        t = rows if table == "rows" else torch.cat([rows[b, :n] for b, n in
                                                    enumerate(ref.pages_of(lens))])
        t = t.cuda()
        qr = fa.fa_append_paged_fp8(q, k, v, cu, kp, vp, ks, vs, t, seq, cos, sin, qw, kw,
                                    interleaved=interleaved)
        kr = ref.norm_rope(k, kw, cos[pos], sin[pos], interleaved, 1e-6)
        for b in range(B):
            keys[b].append(kr[cu[b]:cu[b + 1]])
            vals[b].append(v[cu[b]:cu[b + 1]].double())
    lse = torch.empty((B, H), device="cuda")
    o = fa.fa_decode_paged_fp8(qr, kp, vp, ks, vs, t, seq, lse=lse)
    _ok()
    for b in range(B):
        k, v = torch.cat(keys[b]), torch.cat(vals[b])
        qb = qr[b].double().view(Hk, H // Hk, d)
        s = torch.einsum("hgd,lhd->hgl", qb, k) * d ** -0.5
        # a key's element may be off by 2^-4 of it (twice, where its block's scale
        # grew later) and 2^-17 of the block's largest
        step = 2.0 ** -3 * k.abs() + 2.0 ** -16 * k.abs().max()
        off = torch.einsum("hgd,lhd->hgl", qb.abs(), step) * d ** -0.5
        most = torch.exp(2 * off.amax(-1))  # of a weight, up or down
        p = torch.softmax(s, -1)
        want = torch.einsum("hgl,lhd->hgd", p, v)
        size = torch.einsum("hgl,lhd->hgd", p, v.abs())
        worst = (most - 1)[..., None] * size + most[..., None] * (2.0 ** -3 * size + 2.0 ** -6)
        err = (o[b].double().view_as(want) - want).abs()
        assert (err <= worst + 2.0 ** -8 * want.abs()).all()
        # errors are of both signs: far below the worst, over all elements
        rms = err.square().mean().sqrt() / want.square().mean().sqrt()
        assert rms <= 2.0 ** -3
        assert ((lse[b].double().view(Hk, -1) - torch.logsumexp(s, -1)).abs() <=
                off.amax(-1) + 1e-3).all()


def test_the_binding_s_two_ways_agree():
    """A call on the current stream takes the binding's short way, one with the
    stream given by hand the long one: same bits, outputs given or not."""
    g = torch.Generator().manual_seed(3)
    T, H, Hk, d = 70, 6, 2, 128
    x = torch.randn((T, (H + 2 * Hk) * d), generator=g).bfloat16().cuda()
    q, k, v = (t.view(T, -1, d) for t in x.split([H * d, Hk * d, Hk * d], 1))
    w = torch.nn.Parameter(1 + 0.2 * torch.randn(d, generator=g).cuda())
    here = torch.cuda.current_stream()
    pairs = []

    def both(f, *a, **kw):
        out = [f(*a, **kw), f(*a, stream=here, **kw)]
        _ok()
        pairs.append([o if isinstance(o, tuple) else (o,) for o in out])
        return out[0]

    cos, sin = both(fa.fa_rope_table, 512, 64, 1e4, "linear", 2.0)
    pos = torch.randint(0, 512, (T,), generator=g).int().cuda()
    both(fa.fa_qk_norm_rope, q, k, w, w, cos, sin, pos, interleaved=True)
    both(fa.fa_qk_norm_rope, q.transpose(0, 1)[None].contiguous(),
         k.transpose(0, 1)[None].contiguous(), None, w, cos, sin)
    both(fa.fa_qk_norm_rope, q, k, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    both(fa.fa_qk_norm_rope_bwd, q, k, q, k, w, None, cos, sin, pos)
    cu = torch.tensor([0, 50, 70]).int().cuda()
    c = Cache([300, 100], H, Hk, d, 64, "packed", seed=2)
    t = c.table.cuda()
    for dt in (torch.bfloat16, FP8):
        pools = []
        for stream in (None, here):
            kp, vp = (torch.zeros((5, Hk, PS, d), device="cuda").to(dt) for _ in range(2))
            ks, vs = (torch.ones((5, Hk, 4), device="cuda") for _ in range(2))
            a = (q, k, v, cu, kp, vp) + (() if dt is torch.bfloat16 else (ks, vs))
            f = fa.fa_append_paged_rope if dt is torch.bfloat16 else fa.fa_append_paged_fp8
            out = f(*a, t, c.seq, cos, sin, w, w, stream=stream)
            f(None, *a[1:], t, c.seq, cos, sin, None, w, stream=stream)
            _ok()
            pools.append((out, kp.view(torch.uint8), vp.view(torch.uint8), ks, vs))
        pairs.append(pools)
    for table in (t, torch.stack([t[:2], t[2:3].expand(2)]).contiguous()):
        both(fa.fa_decode_paged_fp8, c.q, c.kp, c.vp, c.ks, c.vs, table, c.seq)
        both(fa.fa_decode_paged_fp8, c.q, c.kp, c.vp, c.ks, c.vs, table, c.seq, scale=0.3,
             lse=torch.empty(c.q.shape[:2], device="cuda"), o=torch.empty_like(c.q))
    for a, b in pairs:
        assert len(a) == len(b)
        for y, z in zip(a, b):
            assert (y is None and z is None) or torch.equal(y, z)
    for bad in (dict(eps=-1.0), dict(q_weight=w[:64])):
        for stream in (None, here):
            with pytest.raises((fa.FaError, ValueError)):
                fa.fa_qk_norm_rope(q, k, rope_cos=cos, rope_sin=sin, stream=stream, **bad)


def test_a_decode_step_captured_once_and_replayed():
    """Append and decode in one graph, the lengths counted on the device, over the
    borders of blocks and pages: the same bits as the calls made one by one."""
    H, Hk, d, block, B = 8, 2, 128, 16, 3
    g = torch.Generator().manual_seed(4)
    cos, sin = fa.fa_rope_table(1024, d)
    w = 1 + 0.2 * torch.randn(d, generator=g).cuda()
    rows = torch.randperm(4 * B, generator=g).int().view(B, 4).cuda()
    cu = torch.arange(B + 1).int().cuda()
    prompt = torch.randn((3 * 14, (H + 2 * Hk) * d), generator=g).bfloat16().cuda()

    def parts(x):
        return [t.view(len(x), -1, d) for t in x.split([H * d, Hk * d, Hk * d], 1)]

    class State:
        def __init__(self):
            self.kp, self.vp = (torch.zeros((4 * B, Hk, PS, d), device="cuda").to(FP8)
                                for _ in range(2))
            self.ks, self.vs = (torch.ones((4 * B, Hk, PS // block), device="cuda")
                                for _ in range(2))
            self.seq = torch.tensor([14, 250, 14]).int().cuda()
            self.x = torch.zeros((B, prompt.shape[1]), device="cuda").bfloat16()
            first = torch.tensor([0, 14, 28, 42]).int().cuda()
            fa.fa_append_paged_fp8(*parts(prompt), first, self.kp, self.vp, self.ks, self.vs,
                                   rows, self.seq, cos, sin, w, w)

        def step(self):
            self.seq += 1
            q = fa.fa_append_paged_fp8(*parts(self.x), cu, self.kp, self.vp, self.ks, self.vs,
                                       rows, self.seq, cos, sin, w, w)
            return fa.fa_decode_paged_fp8(q, self.kp, self.vp, self.ks, self.vs, rows, self.seq)

    # (the second sequence's earlier tokens are zeros: never written)
    a, b = State(), State()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = a.step()
    for i in range(12):
        x = (torch.randn(a.x.shape, generator=g) * 2.0 ** (i % 5 - 2)).bfloat16().cuda()
        a.x.copy_(x)
        b.x.copy_(x)
        graph.replay()
        assert torch.equal(out, b.step()), i
    _ok()
    for n in ("kp", "vp", "ks", "vs"):
        assert torch.equal(getattr(a, n).view(torch.uint8), getattr(b, n).view(torch.uint8))


def test_library_workspaces_of_two_streams():
    """Calls on the current stream take the library's workspace of that stream."""
    a = Cache([9000, 20, 3000], 8, 2, 128, 64, "packed", seed=7)
    b = Cache([5000, 7000, 1], 24, 1, 64, 32, "rows", seed=8)
    tables = [a.table.cuda(), b.table.cuda()]

    def call(c, t):
        return fa.fa_decode_paged_fp8(c.q, c.kp, c.vp, c.ks, c.vs, t, c.seq)

    want = [call(a, tables[0]), call(b, tables[1])]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):
        for i, (c, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                got[i].append(call(c, tables[i]))
    torch.cuda.synchronize()
    _ok()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
