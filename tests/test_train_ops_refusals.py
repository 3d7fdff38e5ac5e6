"""The training-side operators refuse what they do not take, on the host,
before anything is enqueued (no GPU needed): the C entry points' checks of
sizes, pointers, types and workspaces, and the binding's checks of tensors."""
import ctypes as C

import pytest
import torch

import synth  # noqa: F401  (puts the repository root on the path through conftest)

OK, INVALID, UNSUPPORTED, CAPACITY = 0, 1, 2, 3
BF16, FP32 = 0, 1
MOST = 4000000


@pytest.fixture(scope="module")
def pkg():
    from dual_view_diffusion_b200 import build
    build.build()
    import dual_view_diffusion_b200 as p
    return p


@pytest.fixture(scope="module")
def lib(pkg):
    return pkg.lib()


# never dereferenced: every call below is refused first
P = C.c_void_p(4096)
ODD = C.c_void_p(4097)


def size(fn, *args):
    n = C.c_size_t(12345)
    return fn(*args, C.byref(n)), n.value


def test_workspace_sizes(lib):
    for name, args in (("orthrus_embed_grad_workspace", (100, 64, 256)), ("orthrus_rmsnorm_grad_workspace", (100, 64)),
                       ("orthrus_ce_lm_head_workspace", (100, 64, 256, BF16)),
                       ("orthrus_ce_lm_head_grad_workspace", (100, 64, 256, BF16, 1)),
                       ("orthrus_kl_lm_head_grad_workspace", (100, 64, 256, BF16))):
        fn = getattr(lib, name)
        st, n = size(fn, *args)
        assert st == OK and n > 0 and n % 256 == 0, name
        assert size(fn, 0, *args[1:]) == (OK, 0), name           # no rows, no scratch
        assert size(fn, -1, *args[1:])[0] == INVALID, name
        assert size(fn, args[0], 0, *args[2:])[0] == INVALID, name
        assert size(fn, MOST + 1, *args[1:])[0] == CAPACITY, name
        assert size(fn, args[0], 65537, *args[2:])[0] == CAPACITY, name
        assert fn(*args, None) == INVALID, name
    assert size(lib.orthrus_ce_lm_head_workspace, 1, 64, MOST + 1, BF16)[0] == CAPACITY
    assert size(lib.orthrus_ce_lm_head_workspace, 1, 64, 256, 2)[0] == INVALID
    assert size(lib.orthrus_ce_lm_head_grad_workspace, 1, 64, 256, BF16, 2)[0] == INVALID


def test_loss_scratch_does_not_grow_with_the_vocabulary(lib):
    """The gradient's scratch is a piece of the vocabulary's, not [rows][vocab]."""
    a = size(lib.orthrus_ce_lm_head_grad_workspace, 4096, 4096, 151936, BF16, 0)[1]
    b = size(lib.orthrus_ce_lm_head_grad_workspace, 4096, 4096, 4 * 151936, BF16, 0)[1]
    assert a == b
    assert a < 4096 * 151936 * 2


def test_embed_rows(lib):
    f = lib.orthrus_embed_rows
    assert f(None, BF16, 8, 4, P, 1, 1.0, P, FP32, None, None) == INVALID
    assert f(P, BF16, 8, 4, None, 1, 1.0, P, FP32, None, None) == INVALID
    assert f(P, BF16, 8, 4, P, 1, 1.0, None, FP32, None, None) == INVALID
    assert f(P, 5, 8, 4, P, 1, 1.0, P, FP32, None, None) == INVALID
    assert f(P, BF16, 8, 4, P, 1, 1.0, P, 5, None, None) == INVALID
    assert f(ODD, BF16, 8, 4, P, 1, 1.0, P, FP32, None, None) == INVALID
    assert f(P, BF16, 8, 4, P, 1, 1.0, P, FP32, ODD, None) == INVALID
    assert f(P, BF16, 0, 4, P, 1, 1.0, P, FP32, None, None) == INVALID
    assert f(P, BF16, MOST + 1, 4, P, 1, 1.0, P, FP32, None, None) == CAPACITY
    assert f(None, BF16, 8, 4, None, 0, 1.0, None, FP32, None, None) == OK


def test_embed_grad(lib):
    f = lib.orthrus_embed_grad
    n = size(lib.orthrus_embed_grad_workspace, 3, 4, 8)[1]
    assert f(P, BF16, P, 3, 4, 8, 1.0, 0, P, BF16, P, n - 1, None, None) == CAPACITY
    assert f(P, BF16, P, 3, 4, 8, 1.0, 0, P, BF16, None, n, None, None) == INVALID
    assert f(P, BF16, P, 3, 4, 8, 1.0, 0, P, BF16, C.c_void_p(4096 + 128), n, None, None) == INVALID
    assert f(P, BF16, P, 3, 4, 8, 1.0, 2, P, BF16, P, n, None, None) == INVALID
    assert f(P, BF16, P, 3, 4, 8, 1.0, 0, None, BF16, P, n, None, None) == INVALID
    assert f(None, BF16, P, 3, 4, 8, 1.0, 0, P, BF16, P, n, None, None) == INVALID
    assert f(P, BF16, None, 3, 4, 8, 1.0, 0, P, BF16, P, n, None, None) == INVALID
    assert f(None, BF16, None, 0, 4, 8, 1.0, 1, P, BF16, None, 0, None, None) == OK   # adds nothing


def test_rmsnorm(lib):
    f = lib.orthrus_rmsnorm
    assert f(None, FP32, P, BF16, 1, 4, 1e-6, P, None) == INVALID
    assert f(P, FP32, None, BF16, 1, 4, 1e-6, P, None) == INVALID
    assert f(P, FP32, P, BF16, 1, 4, 1e-6, None, None) == INVALID
    assert f(P, FP32, P, BF16, 1, 4, -1.0, P, None) == INVALID
    assert f(P, FP32, P, BF16, 1, 4, float("nan"), P, None) == INVALID
    assert f(P, BF16, P, FP32, 1, 4, 1e-6, P, None) == UNSUPPORTED
    assert f(None, FP32, P, BF16, 0, 4, 1e-6, None, None) == OK
    g = lib.orthrus_rmsnorm_grad
    n = size(lib.orthrus_rmsnorm_grad_workspace, 2, 4)[1]
    assert g(P, FP32, P, P, BF16, 2, 4, 1e-6, P, P, P, n - 1, None) == CAPACITY
    assert g(P, FP32, P, P, BF16, 2, 4, 1e-6, None, P, P, n, None) == INVALID
    assert g(P, FP32, P, P, BF16, 2, 4, 1e-6, P, None, P, n, None) == INVALID
    assert g(P, FP32, P, None, BF16, 2, 4, 1e-6, P, P, P, n, None) == INVALID
    assert g(P, BF16, P, P, FP32, 2, 4, 1e-6, P, P, P, n, None) == UNSUPPORTED


def test_losses(lib):
    f = lib.orthrus_ce_lm_head
    n = size(lib.orthrus_ce_lm_head_workspace, 2, 8, 16, BF16)[1]
    good = [P, P, BF16, P, 2, 8, 16, P, P, P, n, None, None]
    for i, bad, want in ((0, None, INVALID), (0, ODD, INVALID), (1, None, INVALID), (2, 3, INVALID), (3, None, INVALID),
                         (4, -1, INVALID), (5, 0, INVALID), (6, 0, INVALID), (6, MOST + 1, CAPACITY), (7, None, INVALID),
                         (8, None, INVALID), (9, None, INVALID), (10, n - 1, CAPACITY), (11, ODD, INVALID)):
        a = list(good)
        a[i] = bad
        assert f(*a) == want, (i, bad)
    assert f(None, None, BF16, None, 0, 8, 16, None, None, None, 0, None, None) == OK
    g = lib.orthrus_ce_lm_head_grad
    n = size(lib.orthrus_ce_lm_head_grad_workspace, 2, 8, 16, BF16, 1)[1]
    good = [P, P, BF16, P, P, P, 2, 8, 16, P, P, P, n, None, None]
    for i, bad, want in ((0, None, INVALID), (1, None, INVALID), (3, None, INVALID), (4, None, INVALID),
                         (5, None, INVALID), (9, None, INVALID), (10, ODD, INVALID), (11, None, INVALID),
                         (12, n - 1, CAPACITY)):
        a = list(good)
        a[i] = bad
        assert g(*a) == want, (i, bad)
    k = lib.orthrus_kl_lm_head_grad
    n = size(lib.orthrus_kl_lm_head_grad_workspace, 2, 8, 16, BF16)[1]
    good = [P, P, P, BF16, P, P, P, 2, 8, 16, P, P, n, None, None]
    for i, bad, want in ((0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (4, None, INVALID),
                         (5, None, INVALID), (6, None, INVALID), (10, None, INVALID), (11, None, INVALID),
                         (12, n - 1, CAPACITY), (3, 9, INVALID)):
        a = list(good)
        a[i] = bad
        assert k(*a) == want, (i, bad)
    assert k(None, None, None, BF16, None, None, None, 0, 8, 16, None, None, 0, None, None) == OK


def test_binding_refuses_host_tensors(pkg):
    """No CPU fallback: host tensors raise before the library is called."""
    h = torch.zeros((2, 8), dtype=torch.bfloat16)
    w = torch.zeros((16, 8), dtype=torch.bfloat16)
    i, f = torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    gain = torch.ones(8, dtype=torch.bfloat16)
    for call in (lambda: pkg.orthrus_embed_rows(w, i), lambda: pkg.orthrus_embed_grad(h, i, 16),
                 lambda: pkg.orthrus_rmsnorm(h, gain, 1e-6), lambda: pkg.orthrus_rmsnorm_grad(h, gain, h, 1e-6),
                 lambda: pkg.orthrus_ce_lm_head(h, w, i), lambda: pkg.orthrus_ce_lm_head_grad(h, w, i, f, f),
                 lambda: pkg.orthrus_kl_lm_head_grad(h, h, w, f, f, f)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_binding_refuses_extents_past_31_bits(pkg):
    """An extent that the C entry's int32 would cut short is an error."""
    class Rows:
        is_cuda, dtype, device = True, torch.int32, torch.device("cuda", 0)

        def __init__(self, *shape):
            self.shape = torch.Size(shape)

        def is_contiguous(self):
            return True

    assert tuple(pkg._need_rows("ids", Rows((1 << 31) - 1), (torch.int32,), (None,))) == ((1 << 31) - 1,)
    for shape in ((1 << 31,), ((1 << 32) + 5,)):
        with pytest.raises(ValueError, match="2\\^31"):
            pkg._need_rows("ids", Rows(*shape), (torch.int32,), (None,))
    with pytest.raises(ValueError):
        pkg._need_rows("x", Rows(4, 8), (torch.int32,), (4,))
    with pytest.raises(ValueError):
        pkg._need_rows("x", Rows(4, 8), (torch.int32,), (4, 9))
