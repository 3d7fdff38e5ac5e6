"""The training-side operators against their definitions in fp64: the token
embedding and its gradient, RMSNorm and its gradient, the cross entropy
through the LM head and its gradients, and the gradient of the forward KL.

Tolerances are bounds: half a step of the output's type for the last
rounding, and for what comes before it a count of fp32 roundings (u = 2^-24)
times the sum of the absolute values that were added up."""
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


def normal(g, shape, dt=F32, std=1.0):
    return torch.empty(shape, dtype=F32, device=DEV).normal_(0.0, std, generator=g).to(dt)


def within(got, want, tol, what=""):
    d = (got.to(F64) - want).abs()
    ok = bool((d <= tol).all())
    assert ok, (what, float((d / tol.clamp_min(1e-300)).max()), int((d > tol).sum()), d.numel())


def misaligned(x):
    """The same values in a contiguous tensor whose storage starts one element
    off a 16-byte boundary."""
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)
    y = buf[1:].view(x.shape)
    y.copy_(x)
    return y


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("dt,odt", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("n,d,V", [(1, 1, 1), (3, 8, 5), (33, 2048, 300), (7, 100, 11), (2, 4095, 9), (5, 20000, 4)])
def test_embed_rows(dt, odt, n, d, V):
    g = gen(1)
    table = normal(g, (V, d), dt)
    ids = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    if n > 2:
        ids[1] = -1
    scale = math.sqrt(d)
    got = pkg.orthrus_embed_rows(table, ids, scale, odt)
    want = table.to(F64)[ids.long().clamp_min(0)] * torch.tensor(scale, dtype=F32).item()
    want[ids < 0] = 0
    assert got.dtype == odt and got.shape == (n, d)
    within(got, want, (half(odt) + 2 * U) * want.abs())


def test_embed_rows_equals_the_decode_path():
    """scale 1 and fp32 out is the residual row the decode path starts from:
    the table's values unchanged."""
    g = gen(2)
    table = normal(g, (50, 64), BF)
    ids = torch.arange(50, device=DEV, dtype=torch.int32)
    assert torch.equal(pkg.orthrus_embed_rows(table, ids), table.float())
    assert torch.equal(pkg.orthrus_embed_rows(misaligned(table), ids), table.float())


def test_embed_bad_ids_are_reported_and_left_out():
    g = gen(3)
    table = normal(g, (10, 16), BF)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = torch.tensor([3, 10, -5, 2 ** 31 - 1, 9], dtype=torch.int32, device=DEV)
    out = pkg.orthrus_embed_rows(table, ids, err=err)
    assert int(err) == 1
    assert torch.equal(out[[1, 2, 3]], torch.zeros(3, 16, device=DEV))
    assert torch.equal(out[[0, 4]], table[[3, 9]].float())
    err.zero_()
    dout = torch.full((5, 16), float("nan"), dtype=BF, device=DEV)
    dout[0], dout[4] = 1.0, 2.0
    grad = pkg.orthrus_embed_grad(dout, ids, 10, err=err)
    assert int(err) == 1
    want = torch.zeros((10, 16), dtype=BF, device=DEV)
    want[3], want[9] = 1.0, 2.0
    assert torch.equal(grad, want)
    err.zero_()
    pkg.orthrus_embed_rows(table, ids[[0, 2]], err=err)       # padding alone is no error
    pkg.orthrus_embed_grad(dout[[0, 2]], ids[[0, 2]], 10, err=err)
    assert int(err) == 0


def _embed_grad_case(n, d, V, dt, kind, seed=4):
    g = gen(seed)
    dout = normal(g, (n, d), dt)
    ids = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    if kind == "blocks":       # one anchor, 31 mask tokens
        ids[torch.arange(n, device=DEV) % 32 != 0] = V - 1
    elif kind == "one":
        ids.fill_(V // 2)
    elif kind == "padded":
        ids[torch.arange(n, device=DEV) % 3 == 1] = -1
    return dout, ids


def _embed_grad_want(dout, ids, V, scale):
    n, d = dout.shape
    live = ids >= 0
    want = torch.zeros((V, d), dtype=F64, device=DEV)
    mag, cnt = torch.zeros_like(want), torch.zeros(V, dtype=F64, device=DEV)
    x = dout.to(F64)[live] * scale
    idx = ids[live].long()
    want.index_add_(0, idx, x)
    mag.index_add_(0, idx, x.abs())
    cnt.index_add_(0, idx, torch.ones_like(idx, dtype=F64))
    return want, mag, cnt


@pytest.mark.parametrize("dt,odt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("n,d,V,kind", [
    (1, 8, 1, "any"), (2, 16, 7, "one"), (31, 24, 5, "any"), (33, 7, 40, "padded"), (1000, 64, 256, "blocks"),
    (1024, 520, 2, "any"), (4097, 40, 70000, "blocks"), (8192, 16, 300, "any"), (8193, 16, 300, "blocks"),
    (9001, 9, 3, "padded"), (40000, 8, 151936, "blocks"), (70001, 8, 100, "any")])
def test_embed_grad(dt, odt, n, d, V, kind):
    dout, ids = _embed_grad_case(n, d, V, dt, kind)
    scale = 3.0
    got = pkg.orthrus_embed_grad(dout, ids, V, scale, odt)
    want, mag, cnt = _embed_grad_want(dout, ids, V, scale)
    within(got, want, half(odt) * want.abs() + (cnt[:, None] + 3) * U * mag)
    assert torch.equal(got, pkg.orthrus_embed_grad(dout, ids, V, scale, odt))     # the same bits again
    # untouched ids hold exact zeros
    assert torch.count_nonzero(got[cnt == 0]) == 0


def test_embed_grad_huge_vocabulary_keys():
    """Token ids up to the largest vocabulary."""
    n, d, V = 5000, 1, 3999999
    dout, ids = _embed_grad_case(n, d, V, F32, "any")
    ids[:100] = V - 1
    got = pkg.orthrus_embed_grad(dout, ids, V)
    want, mag, cnt = _embed_grad_want(dout, ids, V, 1.0)
    within(got, want, half(F32) * want.abs() + (cnt[:, None] + 3) * U * mag)


@pytest.mark.parametrize("n", [63, 65, 1023, 1025, 2048, 3000, 4096, 5000, 11000, 16383, 16384, 16385])
@pytest.mark.parametrize("V", [50, 3999999])
def test_embed_grad_sorts(n, V):
    """Rows around the edges of the counting sort's blocks and its end, where the
    radix sort takes over."""
    d = 3
    dout, ids = _embed_grad_case(n, d, V, F32, "padded")
    got = pkg.orthrus_embed_grad(dout, ids, V)
    want, mag, cnt = _embed_grad_want(dout, ids, V, 1.0)
    within(got, want, half(F32) * want.abs() + (cnt[:, None] + 3) * U * mag)


@pytest.mark.parametrize("n,d,V,dt,odt,kind", [
    (300, 1000, 40000, BF, BF, "any"), (9000, 129, 151936, BF, F32, "blocks"), (2500, 33, 1100000, F32, BF, "padded"),
    (5, 4096, 9000, BF, BF, "one"), (9000, 1000, 134217, BF, BF, "any"), (9000, 1500, 151936, BF, BF, "blocks"), (20000, 129, 151936, BF, F32, "blocks"),
    (70000, 8, 2200000, BF, F32, "any"), (3, 65536, 600, F32, BF, "any")])
def test_embed_grad_large_tables(n, d, V, dt, odt, kind):
    """Tables whose zeros are written beside the sums, whatever they held."""
    dout, ids = _embed_grad_case(n, d, V, dt, kind)
    ids[0] = 0
    ids[-1] = V - 1
    want, mag, cnt = _embed_grad_want(dout, ids, V, 1.0)
    tol = half(odt) * want.abs() + (cnt[:, None] + 3) * U * mag
    del mag
    for out in (torch.full((V, d), float("nan"), dtype=odt, device=DEV),
                misaligned(torch.full((V, d), float("nan"), dtype=odt, device=DEV))):
        got = pkg.orthrus_embed_grad(dout, ids, V, out=out)
        within(got, want, tol)
        assert torch.count_nonzero(got[cnt == 0]) == 0
    base = torch.ones((V, d), dtype=odt, device=DEV)
    pkg.orthrus_embed_grad(dout, ids, V, out=base, accumulate=True)
    assert bool((base[cnt == 0] == 1).all())


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,d", [(1500000, 8), (2500000, 8), (4000000, 3)])
def test_embed_grad_most_rows(dt, n, d):
    """The longest pieces of the sorted rows, up to the most rows there may be."""
    dout, ids = _embed_grad_case(n, d, 1000, dt, "blocks")
    got = pkg.orthrus_embed_grad(dout, ids, 1000)
    want, mag, cnt = _embed_grad_want(dout, ids, 1000, 1.0)
    # a piece adds at most 4096 rows in a row, the pieces come to at most 1024
    # partials in 8 strands: no longer chain of additions than their sum
    within(got, want, half(dt) * want.abs() + (4096 + 1024 / 8 + 8 + 3) * U * mag)


@pytest.mark.parametrize("n,V", [(100, 64), (9000, 64), (17000, 64)])
def test_embed_grad_accumulates(n, V):
    d = 48
    dout, ids = _embed_grad_case(n, d, V, BF, "padded")
    ids[ids == 5] = 6
    base = normal(gen(5), (V, d), F32)
    out = base.clone()
    r = pkg.orthrus_embed_grad(dout, ids, V, 0.5, out=out, accumulate=True)
    assert r.data_ptr() == out.data_ptr()
    want, mag, cnt = _embed_grad_want(dout, ids, V, 0.5)
    want += base.to(F64)
    within(out, want, 2 * U * want.abs() + (cnt[:, None] + 4) * U * mag)
    assert torch.equal(out[cnt == 0], base[cnt == 0])          # rows of absent ids as they were
    out2 = torch.full_like(base, float("nan"))
    pkg.orthrus_embed_grad(dout, ids, V, 0.5, out=out2)        # overwritten whole
    assert torch.equal(out2, pkg.orthrus_embed_grad(dout, ids, V, 0.5, F32))


def test_embed_grad_unaligned_and_empty():
    dout, ids = _embed_grad_case(200, 64, 20, BF, "any")
    a = pkg.orthrus_embed_grad(dout, ids, 20)
    assert torch.equal(a, pkg.orthrus_embed_grad(misaligned(dout), ids, 20))
    out = misaligned(torch.full((20, 64), 7.0, dtype=BF, device=DEV))
    assert torch.equal(a, pkg.orthrus_embed_grad(dout, ids, 20, out=out))
    z = pkg.orthrus_embed_grad(dout[:0], ids[:0], 20)
    assert torch.count_nonzero(z) == 0 and z.shape == (20, 64)
    one = torch.ones((20, 64), dtype=BF, device=DEV)
    pkg.orthrus_embed_grad(dout[:0], ids[:0], 20, out=one, accumulate=True)
    assert bool((one == 1).all())
    assert pkg.orthrus_embed_rows(a, ids[:0]).shape == (0, 64)


# ------------------------------------------------------------------ RMSNorm
EPS = 1e-6
NORM_TYPES = [(F32, BF), (BF, BF), (F32, F32)]
NORM_SHAPES = [(1, 1), (1, 8), (3, 64), (2, 100), (5, 511), (4, 512), (3, 1000), (300, 1024), (7, 2047), (700, 2048),
               (2, 4096), (1300, 72), (3, 8192), (2, 8191), (3, 8200), (2, 20001)]


def _norm_want(x, gain, dy, eps=EPS):
    x, g = x.to(F64), gain.to(F64)
    r = (x.square().mean(1, keepdim=True) + eps).rsqrt()
    y = x * r * g
    if dy is None:
        return y
    dy = dy.to(F64)
    u = dy * g
    B = (u * x).mean(1, keepdim=True)
    dx = r * u - r ** 3 * B * x
    mag = (r * u).abs() + r ** 3 * (u * x).abs().mean(1, keepdim=True) * x.abs()
    return dx, mag, (dy * x * r).sum(0), (dy * x * r).abs().sum(0)


@pytest.mark.parametrize("xdt,dt", NORM_TYPES)
@pytest.mark.parametrize("n,d", NORM_SHAPES)
def test_rmsnorm_and_gradient(xdt, dt, n, d):
    g = gen(10)
    x = normal(g, (n, d), xdt, 2.0)
    gain = (1 + normal(g, (d,), F32, 0.2)).to(dt)
    dy = normal(g, (n, d), dt, 0.1)
    # roundings behind a row's sum of d positive terms: a thread adds at most
    # d / 32 of them in a row, then trees; 64 covers the rest of the formula
    k = (d / 32 + 64) * U
    y = pkg.orthrus_rmsnorm(x, gain, EPS)
    want = _norm_want(x, gain, None)
    within(y, want, (half(dt) + k) * want.abs(), "y")
    dx, dgain = pkg.orthrus_rmsnorm_grad(x, gain, dy, EPS)
    wx, mag, wg, gmag = _norm_want(x, gain, dy)
    assert dx.dtype == xdt and dgain.dtype == F32
    within(dx, wx, half(xdt) * wx.abs() + 2 * k * mag, "dx")
    within(dgain, wg, (n * U + 2 * k) * gmag, "dgain")
    dx2, dgain2 = pkg.orthrus_rmsnorm_grad(x, gain, dy, EPS)
    assert torch.equal(dx, dx2) and torch.equal(dgain, dgain2)


def test_rmsnorm_edges():
    gain = torch.ones(64, dtype=BF, device=DEV)
    z = torch.zeros((2, 64), device=DEV)
    assert torch.count_nonzero(pkg.orthrus_rmsnorm(z, gain, EPS)) == 0
    dx, dg = pkg.orthrus_rmsnorm_grad(z, gain, gain.expand(2, 64).contiguous(), EPS)
    assert torch.allclose(dx, torch.full_like(dx, EPS ** -0.5), rtol=1e-5) and torch.count_nonzero(dg) == 0
    x = normal(gen(11), (5, 64))
    dy = normal(gen(12), (5, 64), BF)
    a, ga = pkg.orthrus_rmsnorm_grad(x, gain, dy, EPS)
    b, gb = pkg.orthrus_rmsnorm_grad(misaligned(x), gain, misaligned(dy), EPS)
    assert torch.allclose(a, b, rtol=1e-5, atol=1e-6) and torch.allclose(ga, gb, rtol=1e-5, atol=1e-6)
    e, ge = pkg.orthrus_rmsnorm_grad(x[:0], gain, dy[:0], EPS)
    assert e.shape == (0, 64) and torch.count_nonzero(ge) == 0
    assert pkg.orthrus_rmsnorm(x[:0], gain, EPS).shape == (0, 64)
    # a row that is not finite stays its own
    bad = x.clone()
    bad[2] = float("inf")
    y = pkg.orthrus_rmsnorm(bad, gain, EPS)
    keep = [0, 1, 3, 4]
    assert torch.equal(y[keep], pkg.orthrus_rmsnorm(x, gain, EPS)[keep])


# ------------------------------------------------------------------- losses
# (rows, hidden, vocabulary): the fp32 path and bf16 rows of a multiple of 8
# and not, vocabularies around the tiles' edges, one row to several tiles
LOSS_SHAPES = [(1, 8, 1), (1, 64, 2), (2, 16, 63), (5, 7, 65), (31, 64, 256), (33, 72, 257), (127, 128, 1000),
               (128, 64, 512), (130, 200, 300), (257, 64, 129), (300, 136, 2049), (64, 1, 40), (513, 512, 700)]


def _loss_case(n, d, V, dt, seed=20, pad=True):
    g = gen(seed)
    w = normal(g, (V, d), dt, 0.5 / math.sqrt(d) * 4)
    h = normal(g, (n, d), dt)
    t = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    if pad and n > 2:
        t[1::5] = -1
    up = normal(g, (n,)) / n
    return h, w, t, up


def _logits(h, w):
    z = h.to(F64) @ w.to(F64).T
    # fp32 products and sums: at most d roundings of partial sums of |h||w|
    # (2 u each: the tensor cores may truncate instead of rounding)
    dz = 2 * h.shape[1] * U * (h.to(F64).abs() @ w.to(F64).abs().T)
    return z, dz


def _lse_tol(dz, lse, V):
    # the logits' own errors, exponentials good to 2^-20, sums of V terms in
    # strands (tiles of up to 256 ids, then their count), fp32 results
    return dz.amax(1) + 2.0 ** -20 + (256 + V / 256) * U + 4 * U * lse.abs()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,d,V", LOSS_SHAPES)
def test_ce_lm_head(dt, n, d, V):
    h, w, t, _ = _loss_case(n, d, V, dt)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t, err=err)
    z, dz = _logits(h, w)
    want = torch.logsumexp(z, 1)
    tol = _lse_tol(dz, want, V)
    within(lse, want, tol, "lse")
    live = t >= 0
    zt = z.gather(1, t.long().clamp_min(0)[:, None])[:, 0]
    within(loss[live], (want - zt)[live], (tol + dz.amax(1) + 2 * U * (want.abs() + zt.abs()))[live], "loss")
    assert torch.count_nonzero(loss[~live]) == 0
    assert int(err) == 0
    again = pkg.orthrus_ce_lm_head(h, w, t)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


def _grad_tol(p_err, dz, out, m, dt, inner):
    """Bound of |sum_k dz_k m_k| errors: the probabilities' own errors, dz's
    rounding to the operand type on the bf16 path, the sum's fp32 roundings."""
    e = (half(BF) * 1.01 if dt == BF else 2 * U) + 2 * inner * U
    return half(dt) * out.abs() + p_err @ m.abs() + e * (dz.abs() @ m.abs()) + 1e-30


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,d,V", LOSS_SHAPES)
def test_ce_lm_head_grad(dt, n, d, V):
    h, w, t, up = _loss_case(n, d, V, dt)
    _, lse = pkg.orthrus_ce_lm_head(h, w, t)
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    z, zerr = _logits(h, w)
    L = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    g = (up.to(F64) * (t >= 0))[:, None]
    dz = p.clone().scatter_add_(1, t.long().clamp_min(0)[:, None], torch.full((n, 1), -1.0, dtype=F64, device=DEV)) * g
    # error of a probability: of its logit and lse, and of the exponential
    perr = g.abs() * p * (zerr + _lse_tol(zerr, L, V)[:, None] + 2.0 ** -19 + 8 * U * (z.abs() + L.abs()[:, None]))
    H, W = h.to(F64), w.to(F64)
    want = dz @ W
    within(dh, want, _grad_tol(perr, dz, want, W, dt, V), "dh")
    wantw = dz.T @ H
    within(dw, wantw, _grad_tol(perr.T, dz.T, wantw, H, dt, n), "dw")
    dead = (t < 0) if n > 2 else torch.zeros_like(t, dtype=torch.bool)
    assert torch.count_nonzero(dh[dead]) == 0
    only, none = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up, weight_grad=False)
    assert none is None and torch.equal(only, dh)          # the same bits without dw, and again
    again = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n,d,V", LOSS_SHAPES)
def test_kl_lm_head_grad(dt, n, d, V):
    h, w, t, up = _loss_case(n, d, V, dt)
    h2 = (h.float() + normal(gen(21), (n, d), F32, 0.5)).to(dt)
    _, la = pkg.orthrus_ce_lm_head(h, w, t)
    _, ld = pkg.orthrus_ce_lm_head(h2, w, t)
    if n > 3:
        up[2] = 0
    got = pkg.orthrus_kl_lm_head_grad(h, h2, w, la, ld, up)
    W = w.to(F64)
    perr, ps = 0, []
    g = up.to(F64)[:, None]
    for x in (h2, h):
        z, zerr = _logits(x, w)
        L = torch.logsumexp(z, 1)
        p = torch.softmax(z, 1)
        perr = perr + g.abs() * p * (zerr + _lse_tol(zerr, L, V)[:, None] + 2.0 ** -19 +
                                     8 * U * (z.abs() + L.abs()[:, None]))
        ps.append(p)
    dz = g * (ps[0] - ps[1])
    want = dz @ W
    within(got, want, _grad_tol(perr, dz, want, W, dt, V), "dh_diff")
    if n > 3:
        assert torch.count_nonzero(got[2]) == 0
    assert torch.equal(got, pkg.orthrus_kl_lm_head_grad(h, h2, w, la, ld, up))


@pytest.mark.parametrize("dt,d", [(BF, 64), (BF, 60), (F32, 64)])
def test_losses_ignore_what_padded_rows_hold(dt, d):
    """Hidden rows of ignored tokens (or of a zero upstream gradient) may hold
    infinities and NaN: nothing of them reaches a loss or a gradient."""
    n, V = 150, 500
    h, w, t, up = _loss_case(n, d, V, dt)
    clean = pkg.orthrus_ce_lm_head(h, w, t)
    dead = t < 0
    up[7] = 0.0
    t[7] = 3
    bad = h.clone()
    bad[dead] = float("nan")
    bad[1] = float("inf")
    bad[7] = float("nan")
    live = ~dead
    live[7] = False
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    t2 = t.clone()
    t2[7] = -1
    loss, lse = pkg.orthrus_ce_lm_head(bad, w, t2, err=err)
    assert int(err) == 0
    assert torch.equal(lse[live], clean[1][live]) and torch.count_nonzero(loss[~live]) == 0
    a = pkg.orthrus_ce_lm_head_grad(h, w, t, clean[1], up)
    b = pkg.orthrus_ce_lm_head_grad(bad, w, t, lse, up)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(b[0].isfinite().all()) and bool(b[1].isfinite().all())
    k0 = pkg.orthrus_kl_lm_head_grad(h, h, w, clean[1], clean[1], up)
    h2 = (h.float() * 1.5).to(dt)
    ld = pkg.orthrus_ce_lm_head(h2, w, t)[1]
    zero = torch.where(live, up, torch.zeros_like(up))
    k1 = pkg.orthrus_kl_lm_head_grad(h, h2, w, clean[1], ld, zero)
    h2b = h2.clone()
    h2b[~live] = float("inf")
    k2 = pkg.orthrus_kl_lm_head_grad(bad, h2b, w, lse, pkg.orthrus_ce_lm_head(h2b, w, t)[1], zero)
    assert torch.count_nonzero(k0) == 0                     # equal views
    assert torch.equal(k1, k2)


def test_losses_report_bad_targets_and_rows():
    h, w, t, up = _loss_case(40, 64, 100, BF, pad=False)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    t[3] = 100
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t, err=err)
    assert int(err) == 1 and float(loss[3]) == 0
    err.zero_()
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up, err=err)
    assert int(err) == 1 and torch.count_nonzero(dh[3]) == 0
    t2 = t.clone()
    t2[3] = -1
    a = pkg.orthrus_ce_lm_head_grad(h, w, t2, lse, up)
    assert torch.equal(a[0], dh) and torch.equal(a[1], dw)
    err.zero_()
    h[5, 0] = float("nan")
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t2, err=err)
    assert int(err) == 4 and bool(loss[5].isnan()) and int(loss.isnan().sum()) == 1


@pytest.mark.parametrize("dt,d", [(BF, 64), (F32, 48)])
def test_losses_extreme_logits(dt, d):
    """Logits of hundreds, one id far above the rest, ids at -inf (a head row of
    the type's lowest values)."""
    n, V = 20, 300
    h = torch.ones((n, d), dtype=dt, device=DEV)
    w = torch.zeros((V, d), dtype=dt, device=DEV)
    w[:, 0] = torch.linspace(-400, 400, V, device=DEV).to(dt)
    w[17] = torch.finfo(dt).min
    t = torch.arange(n, device=DEV, dtype=torch.int32) + 100
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    z = h.to(F64) @ w.to(F64).T
    want = torch.logsumexp(z, 1)
    within(lse, want, 4 * U * want.abs() + 2.0 ** -19)
    within(loss, want - z.gather(1, t.long()[:, None])[:, 0], 16 * U * want.abs() + 2.0 ** -19)
    assert bool(loss.isfinite().all())


def test_losses_empty_batch():
    h, w, t, up = _loss_case(4, 64, 100, BF)
    loss, lse = pkg.orthrus_ce_lm_head(h[:0], w, t[:0])
    assert loss.shape == lse.shape == (0,)
    dh, dw = pkg.orthrus_ce_lm_head_grad(h[:0], w, t[:0], lse, up[:0])
    assert dh.shape == (0, 64) and torch.count_nonzero(dw) == 0 and dw.shape == w.shape
    assert pkg.orthrus_kl_lm_head_grad(h[:0], h[:0], w, lse, lse, up[:0]).shape == (0, 64)


def test_losses_unaligned_buffers():
    """bf16 rows that TMA cannot address take the SIMT path: the same result
    within the two paths' rounding."""
    h, w, t, up = _loss_case(70, 64, 333, BF)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    l2, s2 = pkg.orthrus_ce_lm_head(misaligned(h), misaligned(w), t)
    assert torch.allclose(loss, l2, rtol=1e-5, atol=1e-5) and torch.allclose(lse, s2, rtol=1e-5, atol=1e-5)
    a = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    b = pkg.orthrus_ce_lm_head_grad(misaligned(h), misaligned(w), t, lse, up)
    for x, y in zip(a, b):
        assert float((x.float() - y.float()).norm() / x.float().norm()) < 2 * half(BF)


def test_losses_full_vocabulary_rows():
    """The model shapes' vocabulary and a ragged training batch, sampled rows and
    head rows in fp64."""
    n, d, V = 777, 512, 151936
    h, w, t, up = _loss_case(n, d, V, BF, seed=23)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    rows = torch.tensor([0, 2, 127, 128, 255, 256, 600, 776], device=DEV)
    W = w.to(F64)
    z, zerr = _logits(h[rows], w)
    L = torch.logsumexp(z, 1)
    within(lse[rows], L, _lse_tol(zerr, L, V), "lse")
    g = (up.to(F64) * (t >= 0))
    p = torch.softmax(z, 1)
    dz = p.scatter_add(1, t[rows].long().clamp_min(0)[:, None], torch.full((8, 1), -1.0, dtype=F64, device=DEV))
    dz *= g[rows][:, None]
    want = dz @ W
    rel = (dh[rows].to(F64) - want).norm() / want.norm()
    assert float(rel) < 2 * half(BF)
    ids = torch.cat([t[t >= 0][:6].long(), torch.tensor([0, 255, 256, V - 1], device=DEV)])
    zi = h.to(F64) @ W[ids].T
    pi = torch.exp(zi - lse.to(F64)[:, None])
    hit = (t.long()[:, None] == ids[None, :]).to(F64)
    wantw = ((pi - hit) * g[:, None]).T @ h.to(F64)
    rel = (dw[ids].to(F64) - wantw).norm(dim=1) / wantw.norm(dim=1)
    assert float(rel.max()) < 3 * half(BF)


@pytest.mark.parametrize("dt,n,d,V", [(BF, 4000, 72, 40001), (F32, 5000, 16, 4000)])
def test_losses_in_several_pieces(dt, n, d, V):
    """So many rows that the vocabulary is gone over in pieces, with a ragged
    last piece: every element."""
    test_ce_lm_head(dt, n, d, V)
    test_ce_lm_head_grad(dt, n, d, V)
    test_kl_lm_head_grad(dt, n, d, V)


def test_offsets_past_32_bits():
    """A head and a table of more than 2^31 elements: the last ids' rows."""
    n, d, V = 3, 4104, 530000
    assert V * d > 1 << 31
    g = gen(40)
    w = torch.empty((V, d), dtype=BF, device=DEV).normal_(0.0, 0.03, generator=g)
    h = normal(g, (n, d), BF)
    t = torch.tensor([V - 1, 7, V - 3], dtype=torch.int32, device=DEV)
    up = torch.tensor([0.5, -1.0, 2.0], device=DEV)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    h2 = (h.float() + normal(g, (n, d), F32, 0.5)).to(BF)
    ld = pkg.orthrus_ce_lm_head(h2, w, t)[1]
    dk = pkg.orthrus_kl_lm_head_grad(h, h2, w, lse, ld, up)
    H, H2 = h.to(F64), h2.to(F64)
    z = torch.cat([H @ c.to(F64).T for c in w.split(65536)], 1)
    z2 = torch.cat([H2 @ c.to(F64).T for c in w.split(65536)], 1)
    L = torch.logsumexp(z, 1)
    # (the logits here are below 10: d roundings of sums of that size, twice)
    assert float(z.abs().max()) < 16
    assert float((lse.to(F64) - L).abs().max()) < 2 * d * U * 16
    assert float((loss.to(F64) - (L - z.gather(1, t.long()[:, None])[:, 0])).abs().max()) < 4 * d * U * 16
    p = torch.softmax(z, 1)
    dz = p.scatter_add(1, t.long()[:, None], torch.full((n, 1), -1.0, dtype=F64, device=DEV)) * up.to(F64)[:, None]
    dk_z = (torch.softmax(z2, 1) - p) * up.to(F64)[:, None]
    for got, x in ((dh, dz), (dk, dk_z)):
        want = sum(x[:, i:i + 65536] @ w[i:i + 65536].to(F64) for i in range(0, V, 65536))
        assert float((got.to(F64) - want).norm() / want.norm()) < 2 * half(BF)
    ids = torch.tensor([0, 7, 255, 256, 523265, V - 257, V - 3, V - 2, V - 1], device=DEV)
    wantw = dz[:, ids].T @ H
    assert float(((dw[ids].to(F64) - wantw).norm(dim=1) / wantw.norm(dim=1)).max()) < 3 * half(BF)
    del dw
    rows = pkg.orthrus_embed_rows(w, t, 2.0)
    assert torch.equal(rows, 2.0 * w[t.long()].float())
    gt = pkg.orthrus_embed_grad(rows, t, V, dtype=BF)
    assert torch.equal(gt[t.long()], rows.to(BF)) and not bool(gt[: V - 3].view(-1)[-8 * d:].any())


def test_two_calls_at_once():
    """Losses on two streams at the same time: each as alone."""
    a, b = _loss_case(600, 256, 30000, BF, seed=41), _loss_case(40, 512, 60000, BF, seed=42)
    pkg_lse = [pkg.orthrus_ce_lm_head(*x[:3])[1] for x in (a, b)]

    def one(x, lse):
        h, w, t, up = x
        return (*pkg.orthrus_ce_lm_head(h, w, t), *pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up),
                pkg.orthrus_embed_grad(h, t, w.shape[0]))

    alone = [one(x, lse) for x, lse in zip((a, b), pkg_lse)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, x, lse in zip(streams, (a, b), pkg_lse):
            with torch.cuda.stream(s):
                got.append(one(x, lse))
        torch.cuda.synchronize()
        for g, w in zip(got, alone):
            assert all(torch.equal(i, j) for i, j in zip(g, w))


def test_loss_gradients_against_differences():
    """Central differences of the losses themselves, fp32 path, and of the KL
    forward entry point's definition."""
    n, d, V = 6, 24, 50
    h, w, t, up = _loss_case(n, d, V, F32, pad=False)
    _, lse = pkg.orthrus_ce_lm_head(h, w, t)
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)

    def total(hh, ww):
        z = hh.to(F64) @ ww.to(F64).T
        return float(((torch.logsumexp(z, 1) - z.gather(1, t.long()[:, None])[:, 0]) * up.to(F64)).sum())

    def kl(hh):
        a, b = torch.log_softmax(h.to(F64) @ w.to(F64).T, 1), torch.log_softmax(hh.to(F64) @ w.to(F64).T, 1)
        return float(((a.exp() * (a - b)).sum(1) * up.to(F64)).sum())

    e = 1e-5
    h2 = h + 0.3
    ld = pkg.orthrus_ce_lm_head(h2, w, t)[1]
    dk = pkg.orthrus_kl_lm_head_grad(h, h2, w, lse, ld, up)
    H, W, H2 = h.to(F64), w.to(F64), h2.to(F64)
    for r, c in ((0, 0), (3, 11), (5, 23)):
        D = torch.zeros_like(H)
        D[r, c] = e
        num = (total(H + D, W) - total(H - D, W)) / (2 * e)
        assert abs(num - float(dh[r, c])) < 1e-5 * float(dh.abs().max()) + 1e-7
        num = (kl(H2 + D) - kl(H2 - D)) / (2 * e)
        assert abs(num - float(dk[r, c])) < 1e-5 * float(dk.abs().max()) + 1e-7
    for v, c in ((int(t[0]), 3), (49, 20)):
        D = torch.zeros_like(W)
        D[v, c] = e
        num = (total(H, W + D) - total(H, W - D)) / (2 * e)
        assert abs(num - float(dw[v, c])) < 1e-5 * float(dw.abs().max()) + 1e-7


# ------------------------------------------------------------ used together
def _chain(ids, table, gain, head, t):
    """Embedding, norm, head and loss with their gradients, as a training step
    runs them; the embedding and the head are separate tables here."""
    scale = 2.0
    x = pkg.orthrus_embed_rows(table, ids, scale)
    y = pkg.orthrus_rmsnorm(x, gain, EPS)
    loss, lse = pkg.orthrus_ce_lm_head(y, head, t)
    up = torch.full_like(loss, 1.0 / loss.numel())
    dy, dhead = pkg.orthrus_ce_lm_head_grad(y, head, t, lse, up)
    dx, dgain = pkg.orthrus_rmsnorm_grad(x, gain, dy, EPS)
    dtable = pkg.orthrus_embed_grad(dx, ids, table.shape[0], scale, table.dtype)
    return loss, dtable, dgain, dhead


def _chain_inputs(dt, n=200, d=64, V=300):
    g = gen(30)
    table, head = normal(g, (V, d), dt), normal(g, (V, d), dt, 0.3)
    gain = (1 + normal(g, (d,), F32, 0.1)).to(dt)
    ids = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    ids[torch.arange(n, device=DEV) % 32 != 0] = V - 1
    t = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    t[::9] = -1
    return ids, table, gain, head, t


@pytest.mark.parametrize("dt", [F32, BF])
def test_training_step_of_the_two_ends(dt):
    ids, table, gain, head, t = _chain_inputs(dt)
    loss, dtable, dgain, dhead = _chain(ids, table, gain, head, t)
    tb, gn, hd = (x.to(F64).requires_grad_() for x in (table, gain, head))
    x = 2.0 * tb[ids.long()]
    y = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * gn
    ls = torch.nn.functional.cross_entropy(y @ hd.T, t.long().clamp_min(0), reduction="none") * (t >= 0)
    (ls.sum() / t.numel()).backward()
    # bf16: the norm's output, its gradient and dz are rounded on the way (three
    # half steps, relative to each tensor's norm), then the result
    rel = 1e-5 if dt == F32 else 5 * half(BF)
    for got, want in ((loss, ls.detach()), (dtable, tb.grad), (dgain, gn.grad), (dhead, hd.grad)):
        assert float((got.to(F64) - want).norm() / want.norm()) < rel


@pytest.mark.parametrize("dt", [F32, BF])
def test_training_step_on_a_side_stream_and_captured(dt):
    """The same bits on another stream, and from a captured graph replayed on new
    inputs; two graphs of the same calls keep their workspaces apart."""
    ids, table, gain, head, t = _chain_inputs(dt)
    want = _chain(ids, table, gain, head, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _chain(ids, table, gain, head, t)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    sid, st = ids.clone(), t.clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_chain(sid, table, gain, head, st))
        graphs.append(g)
    ids2 = ids.flip(0).contiguous()
    t2 = t.roll(1)
    want2 = _chain(ids2, table, gain, head, t2)
    sid.copy_(ids2)
    st.copy_(t2)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(want2, o))
    sid.copy_(ids)
    st.copy_(t)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    a.wait_stream(torch.cuda.current_stream())
    b.wait_stream(torch.cuda.current_stream())
    for _ in range(3):                                    # both at once
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(x, y) for x, y in zip(want, o))


def test_engine_methods_and_the_kl_forward():
    """The engine's methods run on its own weights: a distillation step's loss
    (kl_lm_head) and its gradient, and the cross entropy on the same rows."""
    import dataclasses

    import synth
    s = dataclasses.replace(synth.QWEN3_8B, n_layers=1, hidden=256, n_q_heads=2, n_kv_heads=1, head_dim=128, ffn=64,
                            vocab=1000)
    eng = pkg.Engine(s, synth.make_weights(s, 0, n_layers=1), max_batch=2, max_block=32, max_seq=128, split_tokens=64)
    n = 31
    ids = torch.full((n,), s.vocab - 1, dtype=torch.int32, device=DEV)
    x = eng.embed_rows(ids, 10.0)
    assert torch.equal(x, (eng.embed[ids.long()].float() * 10.0))
    xa, xd = x + normal(gen(40), (n, 256)), x + normal(gen(41), (n, 256))
    ha, hd = eng.final_norm_rows(xa), eng.final_norm_rows(xd)
    kl, la, ld = eng.kl_lm_head(ha, hd)
    up = torch.full((n,), 1.0 / n, device=DEV)
    dhd = eng.kl_lm_head_grad(ha, hd, la, ld, up)
    dx, dgain = eng.final_norm_grad(xd, dhd)
    H, W = hd.to(F64).requires_grad_(), eng.lm_head.to(F64)
    p = torch.log_softmax(ha.to(F64) @ W.T, 1)
    q = torch.log_softmax(H @ W.T, 1)
    want = (p.exp() * (p - q)).sum(1)
    assert torch.allclose(kl.to(F64), want.detach(), rtol=1e-3, atol=1e-5)
    (want.sum() / n).backward()
    # dz rounded to bf16, the forward's log-sum-exps (good to 1e-4) and the result
    assert float((dhd.to(F64) - H.grad).norm() / H.grad.norm()) < 3 * half(BF)
    assert dx.shape == (n, 256) and dgain.shape == (256,)
    t = torch.arange(n, dtype=torch.int32, device=DEV)
    loss, lse = eng.ce_lm_head(hd, t)
    assert torch.allclose(lse, ld, rtol=1e-4, atol=1e-4)
    dh, dw = eng.ce_lm_head_grad(hd, t, lse, up)
    assert dw.shape == eng.lm_head.shape
    dt_ = eng.embed_grad(dx, ids, 10.0)
    assert torch.count_nonzero(dt_[:-1]) == 0 and torch.count_nonzero(dt_[-1]) > 0
    assert eng.check_train_error() == 0 and eng.check_error()[1] == 0
    eng.embed_rows(torch.tensor([s.vocab], dtype=torch.int32))
    assert eng.check_train_error() == 1 and eng.check_train_error() == 0


def test_binding_refusals_on_device():
    h, w, t, up = _loss_case(4, 64, 100, BF)
    lse = torch.zeros(4, device=DEV)
    with pytest.raises(TypeError):
        pkg.orthrus_ce_lm_head(h, w, t.long())
    with pytest.raises(TypeError):
        pkg.orthrus_ce_lm_head(h, w.float(), t)
    with pytest.raises(ValueError):
        pkg.orthrus_ce_lm_head(h, w[:, :32].contiguous(), t)
    with pytest.raises(TypeError):
        pkg.orthrus_ce_lm_head(h[:, :32], w[:, :32], t)               # not contiguous
    with pytest.raises(TypeError):
        pkg.orthrus_ce_lm_head_grad(h, w, t, lse.double(), up)
    with pytest.raises(ValueError):
        pkg.orthrus_ce_lm_head_grad(h, w, t, lse[:3], up)
    with pytest.raises(TypeError):
        pkg.orthrus_embed_rows(w.half(), t)
    with pytest.raises(ValueError):
        pkg.orthrus_embed_grad(h, t, 100, accumulate=True)
    for vocab in (0, -1, (1 << 32) + 100):
        with pytest.raises(ValueError):
            pkg.orthrus_embed_grad(h, t, vocab)
    with pytest.raises(pkg.OrthrusError):
        pkg.orthrus_rmsnorm(h, torch.ones(64, device=DEV), EPS)       # bf16 rows, fp32 gain
