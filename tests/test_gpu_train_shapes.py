"""Shapes that carry the training-side operators in earnest and that small cases
do not reach: wide rows whose runs cross pieces in several column slabs, the
widest hidden rows, the most rows and ids, and rows without a share on every
path of the losses."""
import math

import pytest
import torch

import dual_view_diffusion_b200 as pkg

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
DEV = "cuda"


def half(dt):
    return torch.finfo(dt).eps / 2


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dt,odt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("n,d,V,kind", [(2000, 4096, 300, "blocks"), (20000, 1536, 300, "blocks"), (8192, 4096, 2000, "blocks"),
                                        (3000, 2056, 40, "any"), (5000, 1032, 5000, "one"), (2000, 4095, 300, "blocks")])
def test_embed_grad_runs_across_pieces_of_wide_rows(dt, odt, n, d, V, kind):
    g = gen(80)
    dout = torch.randn((n, d), generator=g, device=DEV).to(dt)
    ids = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    if kind == "blocks":
        ids[torch.arange(n, device=DEV) % 32 != 0] = V - 1
    elif kind == "one":
        ids.fill_(V // 2)
    ids[5] = -1
    live = ids >= 0
    x, idx = dout.to(F64)[live], ids[live].long()
    want = torch.zeros((V, d), dtype=F64, device=DEV).index_add_(0, idx, x)
    mag = torch.zeros((V, d), dtype=F64, device=DEV).index_add_(0, idx, x.abs())
    cnt = torch.bincount(idx, minlength=V).to(F64)[:, None]
    tol = half(odt) * want.abs() + (cnt + 3) * U * mag
    got = pkg.orthrus_embed_grad(dout, ids, V, 1.0, odt)
    e = (got.to(F64) - want).abs()
    assert bool((e <= tol).all()), float((e / tol.clamp_min(1e-300)).max())
    assert torch.equal(got, pkg.orthrus_embed_grad(dout, ids, V, 1.0, odt))
    base = torch.randn((V, d), generator=g, device=DEV)
    out = base.clone()
    pkg.orthrus_embed_grad(dout, ids, V, 1.0, out=out, accumulate=True)
    want += base.to(F64)
    e = (out.to(F64) - want).abs()
    assert bool((e <= 2 * U * want.abs() + (cnt + 4) * U * mag).all())
    assert torch.equal(out[cnt[:, 0] == 0], base[cnt[:, 0] == 0])


# (narrow and wide cross entropy; narrow and wide interleaved rows of the KL: 2 n against 256; SIMT)
@pytest.mark.parametrize("dt,n,d", [(BF, 60, 64), (BF, 128, 72), (BF, 129, 72), (BF, 256, 64), (BF, 257, 64), (BF, 700, 136),
                                    (BF, 300, 60), (F32, 300, 64)])
def test_rows_without_a_share_hold_anything(dt, n, d):
    V = 900
    g = gen(81)
    w = (0.3 * torch.randn((V, d), generator=g, device=DEV)).to(dt)
    h = torch.randn((n, d), generator=g, device=DEV).to(dt)
    h2 = (h.float() + 0.5 * torch.randn((n, d), generator=g, device=DEV)).to(dt)
    t = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    up = torch.randn((n,), generator=g, device=DEV) / n
    r = torch.arange(n, device=DEV)
    ignored, zero = r % 5 == 1, r % 7 == 3
    t[ignored] = -1
    up[zero] = 0
    dead = ignored | zero
    lse, lse2 = pkg.orthrus_ce_lm_head(h, w, t)[1], pkg.orthrus_ce_lm_head(h2, w, t)[1]
    want = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    zup = torch.where(dead, torch.zeros_like(up), up)
    wantk = pkg.orthrus_kl_lm_head_grad(h, h2, w, lse, lse2, zup)
    for fill in (float("nan"), float("inf"), -float("inf"), torch.finfo(dt).min):
        b, b2, bl, bl2, bu = h.clone(), h2.clone(), lse.clone(), lse2.clone(), up.clone()
        for x in (b, b2, bl, bl2):
            x[dead] = fill
        bu[ignored] = fill
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        tz = torch.where(dead, torch.full_like(t, -1), t)
        loss, l = pkg.orthrus_ce_lm_head(b, w, tz, err=err)
        assert int(err) == 0 and torch.equal(l[~dead], lse[~dead]) and torch.count_nonzero(loss[dead]) == 0
        got = pkg.orthrus_ce_lm_head_grad(b, w, t, bl, bu)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.count_nonzero(got[0][dead]) == 0
        assert torch.equal(pkg.orthrus_ce_lm_head_grad(b, w, t, bl, bu, weight_grad=False)[0], want[0])
        assert torch.equal(pkg.orthrus_kl_lm_head_grad(b, b2, w, bl, bl2, zup), wantk)


def _check_losses(dt, n, d, V, rows, ids, seed=82):
    """Loss, lse, and gradients of the rows and head rows given, in fp64."""
    g = gen(seed)
    w = (torch.randn((V, d), generator=g, device=DEV) * (1.5 / math.sqrt(d))).to(dt)
    h = torch.randn((n, d), generator=g, device=DEV).to(dt)
    h2 = (h.float() + 0.5 * torch.randn((n, d), generator=g, device=DEV)).to(dt)
    t = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    t[torch.arange(n, device=DEV) % 6 == 4] = -1
    t[rows] = torch.randint(0, V, (len(rows),), generator=g, device=DEV, dtype=torch.int32)
    up = torch.randn((n,), generator=g, device=DEV)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    lse2 = pkg.orthrus_ce_lm_head(h2, w, t)[1]
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    dk = pkg.orthrus_kl_lm_head_grad(h, h2, w, lse, lse2, up)
    W, H, H2 = w.to(F64), h[rows].to(F64), h2[rows].to(F64)
    z, z2 = H @ W.T, H2 @ W.T
    L = torch.logsumexp(z, 1)
    mag = float((H.abs() @ W.abs().T).max())
    zerr = 2 * U * max(d / 16, 8) * mag            # as many truncated additions (or fp32 sums in groups of 128)
    assert float((lse[rows].to(F64) - L).abs().max()) <= zerr + 2.0 ** -18 + 4 * U * float(L.abs().max())
    zt = z.gather(1, t[rows].long()[:, None])[:, 0]
    want = torch.nn.functional.softplus(torch.logsumexp(z.scatter(1, t[rows].long()[:, None], -math.inf), 1) - zt)
    assert float(((loss[rows].to(F64) - want) / want.clamp_min(1e-3)).abs().max()) <= 2 * zerr + 2.0 ** -17 or V == 1
    p = torch.softmax(z, 1)
    s = up[rows].to(F64)[:, None]
    # two roundings of bf16 (fp32: the exponentials'), and the logits' own errors
    tol = (2 * half(BF) if dt == BF else 1e-5) + 4 * zerr
    dz = p.scatter_add(1, t[rows].long()[:, None], -torch.ones((len(rows), 1), dtype=F64, device=DEV)) * s
    for got, x in ((dh, dz), (dk, (torch.softmax(z2, 1) - p) * s)):
        want = x @ W
        floor = 1e-4 * (s * W.norm(dim=1).max())[:, 0].abs()    # (rows whose dz all but cancels)
        assert bool(((got[rows].to(F64) - want).norm(dim=1) <= tol * want.norm(dim=1) + tol * floor).all())
    pi = torch.exp(h.to(F64) @ W[ids].T - lse.to(F64)[:, None]) - (t.long()[:, None] == ids[None, :]).to(F64)
    wantw = (pi * (up.to(F64) * (t >= 0))[:, None]).T @ h.to(F64)
    e = (dw[ids].to(F64) - wantw).norm(dim=1) / wantw.norm(dim=1)
    assert float(e.max()) <= tol, float(e.max())


@pytest.mark.parametrize("dt,n,d,V", [(BF, 3, 65536, 300), (BF, 300, 65536, 70), (BF, 3, 65535, 300), (F32, 3, 65536, 300),
                                      (F32, 70, 16000, 130)])
def test_losses_of_the_widest_rows(dt, n, d, V):
    rows = torch.tensor([0, 1, n - 1], device=DEV)
    _check_losses(dt, n, d, V, rows, torch.tensor([0, 1, V // 2, V - 1], device=DEV))


@pytest.mark.parametrize("dt", [BF, F32])
def test_losses_of_the_most_rows(dt):
    n, d, V = 4000000, 8, 70
    rows = torch.tensor([0, 1, 255, 256, 2000000, n - 2, n - 1], device=DEV)
    _check_losses(dt, n, d, V, rows, torch.tensor([0, 1, 63, 64, V - 1], device=DEV))


@pytest.mark.parametrize("dt,n", [(BF, 2), (BF, 200), (F32, 2)])
def test_losses_of_the_most_ids(dt, n):
    d, V = 16, 4000000
    rows = torch.tensor([0, n - 1], device=DEV)
    _check_losses(dt, n, d, V, rows, torch.tensor([0, 255, 2097152, V - 1], device=DEV))
