"""The forms in which the vocabulary's tables are taken and the devices a model takes,
on a host without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

V, D = 256, 128
BITS = (np.arange(V * D, dtype=np.uint32) * 40503 >> 3).astype(np.uint16).reshape(V, D)
SCALE = np.linspace(1, 2, V, dtype=np.float32)


@pytest.fixture
def create(monkeypatch):
    """Vocab(model, tables) with the library replaced by a copy of what it is given."""
    from looped_ngpt_transformer_fwd_b200 import model as M

    class Model:
        device, handle, cfg_struct = torch.device("cpu"), None, None
        cfg = dict(d_model=D)

    given = {}

    def copy(handle, size, emb_in, emb_out, scale, buf, nbytes, stream):
        at = [p.value if isinstance(p, ctypes.c_void_p) else p for p in (emb_in, emb_out, scale)]
        given["tables"] = [ctypes.string_at(at[0], 2 * V * D), ctypes.string_at(at[1], 2 * V * D),
                           ctypes.string_at(at[2], 4 * V)]

    monkeypatch.setattr(M.B, "dory_vocab_bytes", lambda *a: 64)
    monkeypatch.setattr(M.B, "dory_vocab_create", copy)
    monkeypatch.setattr(M, "_stream", lambda s: None)
    monkeypatch.setattr(M.torch.cuda, "synchronize", lambda *a: None)

    def run(emb_in=BITS, emb_out=BITS, logit_scale=SCALE, **more):
        M.Vocab(Model, dict(emb_in=emb_in, emb_out=emb_out, logit_scale=logit_scale, **more))
        return given.pop("tables")
    return run


TORCH_BITS = torch.from_numpy(BITS.view(np.int16).copy())
FORMS = dict(uint16=BITS, int16=BITS.view(np.int16), torch_int16=TORCH_BITS,
             torch_uint16=TORCH_BITS.view(torch.uint16), torch_bf16=TORCH_BITS.view(torch.bfloat16),
             flat=BITS.reshape(-1), heads=BITS.reshape(V, 2, D // 2),
             columns=np.asfortranarray(BITS), torch_columns=TORCH_BITS.t().contiguous().t())


@pytest.mark.parametrize("form", FORMS)
def test_tables_in_every_form(create, form):
    want = [BITS.tobytes(), BITS.tobytes(), SCALE.tobytes()]
    assert create(emb_in=FORMS[form], emb_out=FORMS[form]) == want
    assert create(emb_in=FORMS[form], logit_scale=torch.from_numpy(SCALE)) == want


def test_other_entries_are_not_looked_at(create):
    assert create(name="tables", extra=np.zeros(3)) == [BITS.tobytes(), BITS.tobytes(), SCALE.tobytes()]


@pytest.mark.parametrize("kw", [
    dict(emb_in=BITS[:-1]), dict(emb_out=BITS[:, :-2]), dict(emb_in=np.ascontiguousarray(BITS.T)),
    dict(emb_out=BITS.reshape(V // 2, 2 * D)), dict(emb_in=TORCH_BITS[: V // 2]),
    dict(emb_in=np.zeros((V, D), np.float32)), dict(emb_out=np.zeros((V, D), np.float16)),
    dict(emb_in=torch.zeros(V, D)), dict(emb_out=torch.zeros(V, D, dtype=torch.float16)),
    dict(emb_in=np.zeros((V, D), np.int64)), dict(logit_scale=SCALE.astype(np.float64)),
    dict(logit_scale=torch.ones(V, dtype=torch.bfloat16)), dict(logit_scale=np.ones(V, np.uint16)),
    dict(logit_scale=np.ones((V, 2), np.float32)), dict(emb_in=np.zeros((V, D // 2), np.float32)),
])
def test_refused_tables(create, kw):
    with pytest.raises(ValueError):
        create(**kw)


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
def test_a_model_is_on_a_cuda_device(device):
    from looped_ngpt_transformer_fwd_b200.model import DoryModel
    from synthetic import load_config
    with pytest.raises(ValueError):
        DoryModel(load_config("tiny"), lambda b: pytest.fail("weights were asked for"), device=device)
