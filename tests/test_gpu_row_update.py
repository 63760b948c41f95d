"""The pipelined row update (many rows of one K slice) with the GPU full.

Its ring's stages are refilled by bulk copies while other rows are reduced: a
stage handed back before its words have been read would show as rows that
change from call to call.
"""

import numpy as np
import pytest
import torch

from tests.gpu_util import assert_parity, build, inputs, oracle, oracle_cache, to_np

pytestmark = pytest.mark.gpu

# (d_model, query heads, rows): 8, 5 and 3 stages of two vectors, 8, 3 and 2 of three
SHAPES = [(256, 4, 6000), (2560, 40, 2500), (4096, 64, 1500)]


def model_of(d, hq, **over):
    return build("tiny", seed=5, d_model=d, n_q_heads=hq, n_kv_heads=hq // 4, head_dim=64, d_ff=256,
                 n_in_blocks=1, n_rec_blocks=1, n_out_blocks=1, window=64, **over)


@pytest.mark.parametrize("d,hq,n", SHAPES)
def test_update_repeats_itself(d, hq, n):
    """Without re-injection: one MLP sublayer over and over on the same rows."""
    cfg, prov, model = model_of(d, hq)
    _, h = inputs(cfg, 31, 128)
    start = torch.from_numpy(np.tile(h, (n // 128 + 1, 1))[:n].astype(np.float32)).cuda()
    # rows of all sizes, so that a row read in place of another one shows
    start *= torch.linspace(0.5, 2.0, n, device="cuda")[:, None]
    first = start.clone()
    model.mlp_sublayer(0, first)
    for _ in range(40):
        again = start.clone()
        model.mlp_sublayer(0, again)
        assert torch.equal(again, first)
    assert model.device_status() == 0
    model.close()


@pytest.mark.parametrize("d,hq,n", SHAPES)
def test_update_with_reinjection_repeats_itself(d, hq, n):
    """A prefill of three loops: the later ones add the saved stream to every row."""
    cfg, prov, model = model_of(d, hq)
    x, h = inputs(cfg, 32, n)
    kv = model.kv_cache("last_loop", 1, n, k_max=3)
    first = model.prefill(kv, x, 3).clone()
    for _ in range(15):
        assert torch.equal(model.prefill(kv, x, 3), first)
    assert model.device_status() == 0
    m = 160   # rows of the prefix do not depend on those behind it
    ref = oracle(cfg, prov).forward(h[:m], 0, 3, oracle_cache(cfg, "last_loop", k_max=3))
    assert_parity(to_np(first[:m]), ref, what=f"prefill d {d}")
    kv.free()
    model.close()
