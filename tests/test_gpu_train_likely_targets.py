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
