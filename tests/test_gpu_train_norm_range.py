"""RMSNorm and its gradient over the range of x and eps that the calls take:
rows far from one, where powers of 1 / rms leave fp32 and the result does
not, and row counts at which every width goes over its rows more than once."""
import pytest
import torch

import dual_view_diffusion_b200 as pkg

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24
DEV = "cuda"
TYPES = [(F32, BF), (BF, BF), (F32, F32)]


def half(dt):
    return torch.finfo(dt).eps / 2


def case(n, d, xdt, dt, rms, seed=60):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = (torch.randn((n, d), generator=g, device=DEV, dtype=F64) * rms).to(xdt)
    gain = (1 + 0.2 * torch.randn((d,), generator=g, device=DEV)).to(dt)
    dy = (0.1 * torch.randn((n, d), generator=g, device=DEV)).to(dt)
    return x, gain, dy


def check(x, gain, dy, eps):
    n, d = x.shape
    y = pkg.orthrus_rmsnorm(x, gain, eps)
    dx, dgain = pkg.orthrus_rmsnorm_grad(x, gain, dy, eps)
    # a thread adds at most d / 32 terms of a row's sums in a row, then trees; 64
    # covers the rest of the formula (see the tests of the ordinary range)
    k = (d / 32 + 64) * U
    X, G, D = x.to(F64), gain.to(F64), dy.to(F64)
    r = (X.square().mean(1, keepdim=True) + eps).rsqrt()
    xn, u = X * r, D * G
    want = xn * G
    # (results below the type's normal numbers are off by half of its smallest one)
    tiny = {BF: 2.0 ** -134, F32: 2.0 ** -150}
    assert bool(((y.to(F64) - want).abs() <= (half(gain.dtype) + k) * want.abs() + tiny[gain.dtype]).all())
    c = (u * xn).mean(1, keepdim=True)
    wx = r * (u - xn * c)
    mag = r * (u.abs() + xn.abs() * (u * xn).abs().mean(1, keepdim=True))
    tol = half(x.dtype) * wx.abs() + 2 * k * mag + tiny[x.dtype]
    e = (dx.to(F64) - wx).abs()
    assert bool((e <= tol).all()), float((e / tol).max())
    # dgain: a block adds its rows up, then at most 296 blocks
    wg, gmag = (D * xn).sum(0), (D * xn).abs().sum(0)
    assert bool(((dgain.to(F64) - wg).abs() <= (n * U + 2 * k) * gmag).all())
    again = pkg.orthrus_rmsnorm_grad(x, gain, dy, eps)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgain)


@pytest.mark.parametrize("xdt,dt", TYPES)
@pytest.mark.parametrize("n,d", [(5, 64), (3, 1000), (4, 511), (3, 4096), (2, 8191), (2, 9000)])
@pytest.mark.parametrize("rms,eps", [(1e-14, 0.0), (1e-16, 0.0), (1e-13, 1e-30), (1e14, 1e-6), (1e15, 1e-6), (1e16, 1e-6),
                                     (1e-3, 0.0), (1e-14, 1e-6), (1.0, 1e4)])
def test_rmsnorm_gradient_far_from_one(xdt, dt, n, d, rms, eps):
    check(*case(n, d, xdt, dt, rms), eps)


def test_rows_of_different_scales():
    """A row's scale is its own."""
    x, gain, dy = case(40, 300, F32, F32, 1.0)
    x *= 10.0 ** torch.linspace(-16, 16, 40, device=DEV)[:, None]
    check(x, gain, dy, 0.0)


@pytest.mark.parametrize("xdt,dt", TYPES)
@pytest.mark.parametrize("n,d", [(700, 4096), (650, 8192), (650, 8191), (1500, 2047), (5000, 200), (3000, 513), (600, 3000)])
def test_every_width_over_many_rows(xdt, dt, n, d):
    """More rows than the grid takes at once: the next row's loads, the alternating
    buffers and dgain's sum over rows."""
    check(*case(n, d, xdt, dt, 2.0), 1e-6)
