"""Token ids given to the engine's training-side methods in 64 bits."""
import dataclasses

import pytest
import torch

import dual_view_diffusion_b200 as pkg
import synth

pytestmark = pytest.mark.gpu


def test_ids_past_32_bits_are_out_of_range():
    """An id of 2^32 + 5 is no token: reported and left out, not taken for id 5."""
    s = dataclasses.replace(synth.QWEN3_8B, n_layers=1, hidden=256, n_q_heads=2, n_kv_heads=1, head_dim=128, ffn=64,
                            vocab=1000)
    eng = pkg.Engine(s, synth.make_weights(s, 0, n_layers=1), max_batch=2, max_block=32, max_seq=128, split_tokens=64)
    wide = torch.tensor([7, (1 << 32) + 5, -(1 << 33) + 3, -100, 999], device="cuda")
    ids = torch.tensor([7, 1000, -1, -1, 999], dtype=torch.int32, device="cuda")
    assert torch.equal(eng.embed_rows(wide), eng.embed_rows(ids)) and eng.check_train_error() == 1
    h = torch.randn((5, 256), device="cuda").bfloat16()
    assert torch.equal(eng.embed_grad(h, wide), eng.embed_grad(h, ids)) and eng.check_train_error() == 1
    a, b = eng.ce_lm_head(h, wide), eng.ce_lm_head(h, ids)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and eng.check_train_error() == 1
    up = torch.ones(5, device="cuda")
    a, b = eng.ce_lm_head_grad(h, wide, a[1], up), eng.ce_lm_head_grad(h, ids, b[1], up)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and eng.check_train_error() == 1
    assert torch.equal(eng.embed_rows([7, 999]), eng.embed_rows(ids[[0, 4]])) and eng.check_train_error() == 0
