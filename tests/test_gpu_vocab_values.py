"""Values and sizes of the operators around the vocabulary in every kernel form:
infinities and NaN, and more answers than groups of logits.
"""

import math

import numpy as np
import pytest
import torch

from tests.test_gpu_vocab_ops import (OV, cuda, distill_bounds, distill_case, lse_bound, make_vocab,
                                      top_rows)

pytestmark = pytest.mark.gpu

# (n, V): a warp, a CTA of 128 and of 256 threads, a cluster per row
FORMS = [(2, 256), (3, 2048), (3, 2304), (400, 16384), (160, 50432), (1, 131072)]


@pytest.mark.parametrize("n,V", FORMS)
def test_top_of_rows_with_nan_and_infinity(n, V):
    """The log-sum-exp is NaN wherever a NaN stands, beside +inf too; +inf without
    a NaN gives +inf."""
    model, voc = make_vocab(V)
    rng = np.random.default_rng(V)
    for inf_at, nan_at in ((9, 10), (10, 9), (0, V - 1), (V - 1, 0), (V // 2, V // 2 + 127), (5, 5 + V // 2)):
        z = rng.standard_normal((n, V)).astype(np.float32)
        z[:, inf_at] = np.inf
        values, tokens, lse = voc.top(cuda(z), 2)
        assert (tokens[:, 0] == inf_at).all() and (values[:, 0] == math.inf).all() and (lse == math.inf).all()
        z[0, nan_at] = np.nan
        values, tokens, lse = voc.top(cuda(z), 2)
        assert (tokens[:, 0] == inf_at).all() and (values[:, 0] == math.inf).all()
        assert torch.isfinite(values[:, 1]).all() and (tokens[:, 1] != nan_at)[0]
        assert torch.isnan(lse[0]) and (lse[1:] == math.inf).all()
    assert model.device_status() == 0


@pytest.mark.parametrize("V", [512, 16384, 33280, 131072])
def test_distill_of_infinite_logits(V):
    """+inf on either side: no softmax, so the row's loss and gradient are NaN; the
    other rows are what they are without it."""
    model, voc = make_vocab(V)
    c = distill_case(V, 4, V, 6, weights=False)
    rl, rz = OV.distill(**c)
    bl, bz = distill_bounds(c, 1.0, None, 1.0, False)
    c["z"][1, V // 3] = np.inf
    c["teacher_logits"][2, 0] = np.inf
    loss, dz = voc.distill(**{k: cuda(v) for k, v in c.items()})
    assert torch.isnan(loss[1:3]).all() and torch.isnan(dz[1]).all()
    assert torch.isnan(dz[2, cuda(c["teacher_tokens"][2].astype(np.int64))]).all()
    for i in (0, 3):
        assert abs(float(loss[i]) - rl[i]) <= bl[i]
        assert np.all(np.abs(dz[i].double().cpu().numpy() - rz[i]) <= bz[i])
    assert model.device_status() == 0


@pytest.mark.parametrize("n,V", FORMS)
def test_top_of_rows_with_fewer_numbers_than_answers(n, V):
    """Answers that reach into the NaNs: by ascending token, wherever they stand
    (scattered, whole groups, all but a few)."""
    model, voc = make_vocab(V)
    rng = np.random.default_rng(V + 1)
    for k in (5, 70, 256):
        z = np.full((n, V), np.nan, np.float32)
        z[0, rng.permutation(V)[: k // 2]] = rng.standard_normal(k // 2)
        z[-1, :k // 2] = -np.inf
        if n > 2:
            z[1] = rng.standard_normal(V)
            z[1, rng.random(V) < 0.9] = np.nan
            z[1, V // 2:] = np.nan
        values, tokens, lse = voc.top(cuda(z), k)
        rv, rt, _ = OV.top_logits(z, k)
        assert np.array_equal(tokens.cpu().numpy(), rt), k
        assert np.array_equal(values.double().cpu().numpy(), rv, equal_nan=True)
        assert torch.isnan(lse).all()
    assert model.device_status() == 0


@pytest.mark.parametrize("n,V,k", [(3, 2304, 256), (3, 4096, 200), (200, 4096, 129), (3, 7936, 249)])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "none", "few", "up", "down", "cluster", "zeros",
                                  "wide"])
def test_top_with_more_answers_than_groups(n, V, k, kind):
    """Rows of fewer groups of 32 logits than answers: every logit is a candidate."""
    model, voc = make_vocab(V)
    z = top_rows(kind, n, V, V + k)
    values, tokens, lse = voc.top(cuda(z), k)
    rv, rt, rl = OV.top_logits(z, k)
    assert np.array_equal(tokens.cpu().numpy(), rt)
    assert np.array_equal(values.double().cpu().numpy(), rv)
    got = lse.double().cpu().numpy()
    if kind == "none":
        assert np.all(got == -np.inf)
    else:
        assert np.all(np.abs(got - rl) <= lse_bound(V, rl))
    assert model.device_status() == 0
