"""The training-side calls from several host threads at the same time (ctypes
lets go of the interpreter's lock during a call)."""
import threading

import pytest
import torch

import dual_view_diffusion_b200 as pkg

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _run(jobs, rounds):
    """Each job in a thread and on a stream of its own, `rounds` times; what any of
    them raised."""
    raised, start = [], threading.Barrier(len(jobs))

    def work(job):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(rounds):
                    job()
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 (handed to the test's thread)
            raised.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return raised


def test_embed_grad_pieces_of_two_lengths():
    """Calls whose sorted rows are cut into pieces of 4096 and of 2048 ask for
    different shared memory of the same kernel."""
    jobs, want = [], []
    for n in (2500000, 1500000):
        g = torch.Generator(device=DEV)
        g.manual_seed(n)
        dout = torch.randn((n, 8), generator=g, device=DEV).bfloat16()
        ids = torch.randint(0, 1000, (n,), generator=g, device=DEV, dtype=torch.int32)
        out = torch.empty((1000, 8), dtype=torch.bfloat16, device=DEV)
        want.append((out, pkg.orthrus_embed_grad(dout, ids, 1000)))
        jobs += [lambda d=dout, i=ids, o=out: pkg.orthrus_embed_grad(d, i, 1000, out=o)]
    torch.cuda.synchronize()
    assert _run(jobs, 300) == []
    torch.cuda.synchronize()
    for got, w in want:
        assert torch.equal(got, w)


def test_losses_and_rows_in_threads():
    """Every operator from four threads at once: each as alone."""
    def inputs(seed, n, d, V, dt):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        w = (0.1 * torch.randn((V, d), generator=g, device=DEV)).to(dt)
        h = torch.randn((n, d), generator=g, device=DEV).to(dt)
        t = torch.randint(-1, V, (n,), generator=g, device=DEV, dtype=torch.int32)
        return h, w, t, torch.randn((n,), generator=g, device=DEV) / n

    def step(h, w, t, up):
        gain = torch.ones(h.shape[1], dtype=h.dtype, device=DEV)
        loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
        return (loss, lse, *pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up),
                pkg.orthrus_kl_lm_head_grad(h, h.flip(0).contiguous(), w, lse, lse.flip(0).contiguous(), up),
                pkg.orthrus_embed_rows(w, t), pkg.orthrus_embed_grad(h, t, w.shape[0]),
                pkg.orthrus_rmsnorm(h, gain, 1e-6), *pkg.orthrus_rmsnorm_grad(h, gain, h, 1e-6))

    cases = [inputs(1, 40, 256, 3000, torch.bfloat16), inputs(2, 400, 512, 5000, torch.bfloat16),
             inputs(3, 17000, 24, 300, torch.bfloat16), inputs(4, 70, 64, 500, torch.float32)]
    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def job(c, w):
        got = step(*c)
        if not all(torch.equal(a, b) for a, b in zip(got, w)):
            bad.append(c[0].shape)

    assert _run([lambda c=c, w=w: job(c, w) for c, w in zip(cases, want)], 20) == []
    assert bad == []
