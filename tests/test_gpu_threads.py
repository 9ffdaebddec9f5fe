"""Several host threads that call on one stream share its workspace: each call's
launches stay together, and a call that needs more waits for those being made."""
import threading

import pytest
import torch

import attn_fwd_04_b200 as fa

pytestmark = pytest.mark.gpu
PS = 256
FP8 = torch.float8_e4m3fn


def test_calls_of_several_threads_on_one_stream():
    g = torch.Generator().manual_seed(0)

    def cache(B, H, Hk, d, dtype, pages):
        shape = (B * pages, Hk, PS, d)
        kp, vp = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
        table = torch.randperm(B * pages, generator=g).int().cuda()
        lens = torch.full((B,), pages * PS - 5).int().cuda()
        return torch.randn((B, H, d), generator=g).bfloat16().cuda(), kp, vp, table, lens

    # an older call, of growing sizes: its workspace is freed and allocated again
    olds = [cache(B, 8, 2, 128, torch.bfloat16, 12) for B in (1, 3, 9, 30)]
    jobs = [lambda out, c=c: [fa.fa_decode_paged_gqa(*c, o=out and out[0])] for c in olds]
    # decodes over 8-bit pages: through the binding, and with the library's workspace
    # from C (without Python's lock)
    news = []
    for B, H, Hk in ((3, 16, 4), (20, 8, 8)):
        q, kp, vp, table, lens = cache(B, H, Hk, 128, FP8, 14)
        ks, vs = (torch.rand((kp.shape[0], Hk, 4), generator=g).cuda() for _ in range(2))
        news.append((q, kp, vp, ks, vs, table, lens))
    jobs += [lambda out, c=c: [fa.fa_decode_paged_fp8(*c, o=out and out[0])] for c in news]

    def from_c(out, c=news[0]):
        q, kp, vp, ks, vs, table, lens = c
        o = out[0] if out else torch.empty_like(q)
        rc = fa.lib().fa_decode_paged_fp8(
            q.data_ptr(), kp.data_ptr(), vp.data_ptr(), ks.data_ptr(), vs.data_ptr(), 64,
            table.data_ptr(), len(table), 0, lens.data_ptr(), o.data_ptr(), None, q.shape[0],
            q.shape[1], kp.shape[1], kp.shape[0], 128, PS, 128 ** -0.5, None, 0,
            torch.cuda.current_stream().cuda_stream)
        assert rc == fa.FA_OK
        return [o]

    jobs.append(from_c)
    # gradients of the norms, whose partial sums are in the workspace
    x = torch.randn((700, 10, 128), generator=g).bfloat16().cuda()
    w = torch.rand(128, generator=g).cuda()

    def norms(out):
        more = dict(zip(("dq", "dk", "dq_weight", "dk_weight"), out)) if out else {}
        return list(fa.fa_qk_norm_rope_bwd(x[:, :8], x[:, 8:], x[:, :8], x[:, 8:], w, w, **more))

    jobs.append(norms)

    wants = [job(None) for job in jobs]
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == fa.FA_OK
    outs = [[[torch.empty_like(t) for t in want] for _ in range(60)] for want in wants]
    failed = []
    start = threading.Barrier(len(jobs))

    def work(job, mine):
        try:
            torch.cuda.set_device(0)
            start.wait()
            for out in mine:
                job(out)
        except BaseException as e:
            failed.append(e)

    for _ in range(3):
        for mine in outs:
            for out in mine:
                for t in out:
                    t.zero_()
        torch.cuda.synchronize()
        threads = [threading.Thread(target=work, args=a) for a in zip(jobs, outs)]
        for t in threads:
            t.start()
        fa.fa_release_workspace()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        assert fa.fa_get_device_error() == fa.FA_OK
        for want, mine in zip(wants, outs):
            for out in mine:
                assert all(torch.equal(a, b) for a, b in zip(want, out))
