"""What only the device can see is never lost: calls that name no error word of
their own collect their bits in the library's word of the device."""
import ctypes as C
import subprocess
import sys
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pkg():
    from dual_view_diffusion_b200 import build
    build.build()
    import dual_view_diffusion_b200 as p
    return p


def test_refusals(pkg):
    assert pkg.lib().orthrus_train_check_error(None, None) == 1
    with pytest.raises(ValueError, match="CUDA"):
        pkg.orthrus_train_check_error("cpu")
    # calls of no rows raise nothing and need no device
    assert pkg.lib().orthrus_embed_rows(None, 0, 8, 4, None, 0, 1.0, None, 1, None, None) == 0
    assert pkg.lib().orthrus_ce_lm_head(None, None, 0, None, 0, 8, 16, None, None, None, 0, None, None) == 0


def _inputs(dt=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(70)
    h = torch.randn((6, 64), generator=g, device="cuda").to(dt)
    w = torch.randn((50, 64), generator=g, device="cuda").to(dt)
    t = torch.tensor([0, 1, -1, 3, 49, 5], dtype=torch.int32, device="cuda")
    return h, w, t, torch.ones(6, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_bits_without_a_word(pkg, dt):
    h, w, t, up = _inputs(dt)
    pkg.orthrus_train_check_error()
    lse = pkg.orthrus_ce_lm_head(h, w, t)[1]
    pkg.orthrus_ce_lm_head_grad(h, w, t, lse, up)
    pkg.orthrus_embed_rows(w, t)
    pkg.orthrus_embed_grad(h, t, 50)
    assert pkg.orthrus_train_check_error() == 0          # padding is no error
    bad = t.clone()
    bad[3] = 50
    for call in (lambda: pkg.orthrus_embed_rows(w, bad), lambda: pkg.orthrus_embed_grad(h, bad, 50),
                 lambda: pkg.orthrus_ce_lm_head(h, w, bad), lambda: pkg.orthrus_ce_lm_head_grad(h, w, bad, lse, up)):
        call()
        assert pkg.orthrus_train_check_error("cuda") == 1
        assert pkg.orthrus_train_check_error(h.device) == 0
    nan = h.clone()
    nan[0, 0] = float("nan")
    pkg.orthrus_ce_lm_head(nan, w, bad)
    assert pkg.orthrus_train_check_error() == 5
    # a word of the caller's keeps the bits to itself
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.orthrus_ce_lm_head(nan, w, bad, err=err)
    assert int(err) == 5 and pkg.orthrus_train_check_error() == 0
    # the C entry's status
    bits = C.c_uint32()
    pkg.orthrus_ce_lm_head(h, w, bad)
    torch.cuda.synchronize()
    assert pkg.lib().orthrus_train_check_error(None, C.byref(bits)) == 5 and bits.value == 1
    pkg.orthrus_ce_lm_head(nan, w, t)
    torch.cuda.synchronize()
    assert pkg.lib().orthrus_train_check_error(None, C.byref(bits)) == 6 and bits.value == 4


_FIRST_CALL = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import dual_view_diffusion_b200 as pkg
w = torch.randn((50, 64), device="cuda").bfloat16()
t = torch.tensor([0, 50, 7], dtype=torch.int32, device="cuda")
h = torch.randn((3, 64), device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    rows = pkg.orthrus_embed_rows(w, t)
    loss, lse = pkg.orthrus_ce_lm_head(h, w, t)
    dh, dw = pkg.orthrus_ce_lm_head_grad(h, w, t, lse, torch.ones_like(lse))
torch.cuda.synchronize()
assert pkg.orthrus_train_check_error() == 0      # captured, not run
for _ in range(2):
    g.replay()
    assert pkg.orthrus_train_check_error() == 1
assert pkg.orthrus_train_check_error() == 0
assert torch.equal(rows[[0, 2]], w[[0, 7]].float()) and not bool(rows[1].any()) and float(loss[1]) == 0
print("ok")
"""


@pytest.mark.gpu
def test_a_process_whose_first_calls_are_captured():
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]
