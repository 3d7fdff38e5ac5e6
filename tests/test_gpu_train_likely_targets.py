"""The losses of a model that is partly trained: rows whose target is already
likely, where 1 - p is the whole answer.  Against fp64, with a bound per row."""
import math

import pytest
import torch

import dual_view_diffusion_b200 as pkg

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
DEV = "cuda"
WANTED = [0.9, 0.99, 0.999, 0.9999]


def half(dt):
    return torch.finfo(dt).eps / 2


def likely_rows(n, d, V, dt, seed=50):
    """Hidden rows that give their target about the wanted probability: noise,
    moved along the target's head row."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    w = (torch.randn((V, d), generator=g, device=DEV) / math.sqrt(d) * 1.3).to(dt)
    t = torch.randperm(V, generator=g, device=DEV)[:n].to(torch.int32)
    h = torch.randn((n, d), generator=g, device=DEV).to(F64)
    W, wt = w.to(F64), w[t.long()].to(F64)
    p = torch.tensor([WANTED[i % len(WANTED)] for i in range(n)], dtype=F64, device=DEV)
    zt = torch.logsumexp(h @ W.T, 1) + torch.log(p / (1 - p))
    h = h + ((zt - (h * wt).sum(1)) / wt.square().sum(1))[:, None] * wt
    up = torch.randn((n,), generator=g, device=DEV) / n
    return h.to(dt), w, t, up


def rel_rows(got, want):
    return (got.to(F64) - want).norm(dim=1) / want.norm(dim=1)


# (rows as columns beside the head's, and as rows of their own; d % 8 != 0 and fp32: the SIMT path)
SHAPES = [(BF, 24, 2048, 5000), (BF, 200, 4096, 20000), (BF, 300, 1024, 5000), (BF, 600, 4096, 20000),
          (BF, 40, 1023, 3000), (F32, 48, 512, 3000)]


@pytest.mark.parametrize("dt,n,d,V", SHAPES)
def test_gradient_of_likely_targets(dt, n, d, V):
    """The gradient's formula at the log-sum-exp it is given (in fp32, so that its
    own rounding is no part of the bound)."""
    h, w, t, up = likely_rows(n, d, V, dt)
    H, W, ti = h.to(F64), w.to(F64), t.long()[:, None]
    z = H @ W.T
    lse = torch.logsumexp(z, 1).float()
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    x = z - lse.to(F64)[:, None]
    one_minus = -torch.expm1(x.gather(1, ti))[:, 0]
    assert float(one_minus.min()) < 2e-4 and float(one_minus.max()) > 0.05
    dz = torch.exp(x).scatter(1, ti, -one_minus[:, None]) * up.to(F64)[:, None]
    # roundings of dz and of the result, relative to the row (the head rows and the
    # hidden rows are nearly orthogonal, so errors of single ids add in squares);
    # a truncated logit moves the other probabilities by 1e-4 of themselves; the
    # target's logit is a sum of d fp32 products, its part of 1 - p the last term
    tol = (2 * half(dt) if dt == BF else 1e-5) + (1e-4 if dt == BF else 2 * d * U)
    # fp32 products of |h||w|: groups of 128 added up, on the SIMT path
    zerr = 4 * U * z.gather(1, ti)[:, 0].abs() + (0 if dt == BF and d % 8 == 0 else 8 * U * (H.abs() * W[t.long()].abs()).sum(1))
    e = rel_rows(dh, dz @ W)
    assert bool((e <= tol + zerr / one_minus).all()), float((e / (tol + zerr / one_minus)).max())
    e = rel_rows(dw[t.long()], dz[:, t.long()].T @ H)
    assert bool((e <= tol + zerr / one_minus).all()), float((e / (tol + zerr / one_minus)).max())
    only, _ = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up, weight_grad=False)
    assert torch.equal(only, dh)


@pytest.mark.parametrize("n", [20, 300])
def test_target_logit_of_one_sign(n):
    """All products of the target's logit positive, so that truncated sums lose
    the most; every other logit is zero, so the loss and the gradient hold the
    target's logit alone."""
    d, V, t0 = 4096, 3000, 17
    g = torch.Generator(device=DEV)
    g.manual_seed(51)
    w = torch.zeros((V, d), dtype=BF, device=DEV)
    w[t0] = (0.5 + torch.rand((d,), generator=g, device=DEV)).to(BF)
    h = (0.5 + torch.rand((n, d), generator=g, device=DEV))
    h = (h * torch.linspace(8, 17, n, device=DEV)[:, None] / (h @ w[t0].float())[:, None]).to(BF)
    t = torch.full((n,), t0, dtype=torch.int32, device=DEV)
    zt = h.to(F64) @ w[t0].to(F64)
    lse = torch.log(torch.exp(zt) + (V - 1)).float()
    up = torch.ones(n, device=DEV)
    dh, _ = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up, weight_grad=False)
    one_minus = -torch.expm1(zt - lse.to(F64))
    want = -one_minus[:, None] * w[t0].to(F64)
    tol = 2 * half(BF) + 4 * U * zt / one_minus
    e = rel_rows(dh, want)
    assert bool((e <= tol).all()), float((e / tol).max())


@pytest.mark.parametrize("dt,n,d,V", SHAPES)
def test_loss_of_likely_targets(dt, n, d, V):
    """The loss of a likely target is small: its own digits count, not lse's."""
    h, w, t, up = likely_rows(n, d, V, dt)
    H, W, ti = h.to(F64), w.to(F64), t.long()[:, None]
    z = H @ W.T
    zt = z.gather(1, ti)[:, 0]
    rest = torch.logsumexp(z.scatter(1, ti, -math.inf), 1)
    want = torch.nn.functional.softplus(rest - zt)
    assert float(want.min()) < 2e-4 and float(want.max()) > 0.05
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    # |d loss / loss| is at most the error of rest - z_t: of the other logits (bf16:
    # d / 16 truncated additions; else fp32 sums in groups of 128), of z_t, of the
    # exponentials' sum (2^-18) and of the logarithm
    mag = (H.abs() @ W.abs().T).amax(1)
    tc = dt == BF and d % 8 == 0
    rerr = (2 * U * d / 16 if tc else 8 * U) * mag
    zerr = 4 * U * zt.abs() if tc else 8 * U * (H.abs() * W[t.long()].abs()).sum(1)
    tol = rerr + zerr + 2.0 ** -18 + 4 * U * (rest.abs() + zt.abs())
    e = (loss.to(F64) - want).abs() / want
    assert bool((e <= tol).all()), (float((e / tol).max()), float(e.max()))
    L = torch.logsumexp(z, 1)
    tol = U * L.abs() + zerr + tol * want
    e = (lse.to(F64) - L).abs()
    assert bool((e <= tol).all()), float((e / tol).max())
    # what the gradient makes of it: 1 - p off by lse's half step and no more
    dh, _ = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up, weight_grad=False)
    p = torch.softmax(z, 1)
    one_minus = -torch.expm1(zt - L)
    dz = p.scatter(1, ti, -one_minus[:, None]) * up.to(F64)[:, None]
    # (z_t's error enters through lse as well as in the gradient's own z - lse)
    tol = (2 * half(dt) + 1e-4 if dt == BF else 1e-5 + 2 * d * U) + (U * L.abs() + 2 * zerr + 2.0 ** -23) / one_minus
    e = rel_rows(dh, dz @ W)
    assert bool((e <= tol).all()), float((e / tol).max())


@pytest.mark.parametrize("n", [20, 300])
def test_loss_of_one_sign(n):
    """As test_target_logit_of_one_sign: all of the loss's error is z_t's, which
    the tensor cores' truncated sum would put 1e-5 of z_t off."""
    d, V, t0 = 4096, 3000, 17
    g = torch.Generator(device=DEV)
    g.manual_seed(52)
    w = torch.zeros((V, d), dtype=BF, device=DEV)
    w[t0] = (0.5 + torch.rand((d,), generator=g, device=DEV)).to(BF)
    h = (0.5 + torch.rand((n, d), generator=g, device=DEV))
    h = (h * torch.linspace(-4, 17, n, device=DEV)[:, None] / (h @ w[t0].float())[:, None]).to(BF)
    t = torch.full((n,), t0, dtype=torch.int32, device=DEV)
    zt = h.to(F64) @ w[t0].to(F64)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    a = math.log(V - 1) - zt
    want = torch.nn.functional.softplus(a)
    e = (loss.to(F64) - want).abs() / want
    # a in fp32 (two roundings of at most |z| + log V), log and exp two steps each
    tol = U * (2 * zt.abs() + 4 * math.log(V) + 8)
    assert bool((e <= tol).all()), float((e / tol).max())
    L = zt + want
    assert bool(((lse.to(F64) - L).abs() <= U * (L.abs() + 16)).all())


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 60), (F32, 64)])
@pytest.mark.parametrize("n", [3, 270])
def test_losses_at_the_ends(dt, d, n):
    """One id; a target or all else at -inf; every id at -inf; a target at +inf."""
    inf = math.inf
    h = torch.zeros((n, d), dtype=dt, device=DEV)
    h[:, 0] = 1
    t = torch.zeros(n, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    one = torch.zeros((1, d), dtype=dt, device=DEV)
    one[0, 0] = 3
    loss, lse = pkg.orthrus_ce_lm_head(h, one, t, err=err)
    assert bool((loss == 0).all()) and bool((lse == 3).all()) and int(err) == 0
    w = torch.zeros((70, d), dtype=dt, device=DEV)
    w[0, 0] = -inf
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t, err=err)
    assert bool((loss == inf).all()) and bool(((lse - math.log(69)).abs() < 1e-6).all()) and int(err) == 0
    w[:, 0] = -inf
    w[0, 0] = 2
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t, err=err)
    assert bool((loss == 0).all()) and bool((lse == 2).all()) and int(err) == 0
    w[0, 0] = -inf
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t, err=err)
    assert bool((lse == -inf).all()) and bool(loss.isnan().all()) and int(err) == 4
    err.zero_()
    w[0, 0] = inf
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t, err=err)
    assert bool((lse == inf).all()) and bool(loss.isnan().all()) and int(err) == 4
    # an ignored row's lse is of the whole vocabulary
    w[:, 0] = 0
    w[0, 0] = 4
    lse = pkg.orthrus_ce_lm_head(h, w, torch.full_like(t, -1))[1]
    assert bool(((lse - math.log(math.exp(4) + 69)).abs() < 1e-5).all())
