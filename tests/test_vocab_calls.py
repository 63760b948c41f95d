"""What the vocabulary's methods hand to the library, on a host without a GPU."""

import pytest
import torch

I32 = torch.int32


@pytest.fixture
def voc(monkeypatch):
    """A vocabulary of 512 tokens on the CPU that records the call of dory_adjust_logits."""
    from looped_ngpt_transformer_fwd_b200 import model as M

    class Model:
        device = torch.device("cpu")
        cfg = dict(d_model=128)

    v = object.__new__(M.Vocab)
    v.model, v.size, v.handle = Model, 512, None
    v.calls = []
    monkeypatch.setattr(M, "_stream_of", lambda stream, device: 0)
    monkeypatch.setattr(M.B, "dory_adjust_logits", lambda h, z, n, c, out, s: v.calls.append((n, c)))
    return v


def test_an_empty_history_is_no_history(voc):
    z = torch.zeros(2, 512)
    allowed = torch.zeros(2, 16, dtype=I32)
    voc.adjust(z, torch.zeros(2, 0, dtype=I32), torch.zeros(2, dtype=I32), torch.zeros(2, dtype=I32),
               torch.ones(2), torch.ones(2), torch.ones(2), torch.zeros(2, 3, dtype=I32), torch.zeros(2, 3),
               allowed)
    n, c = voc.calls.pop()
    assert n == 2 and c.n_bias == 3 and c.allowed == allowed.data_ptr() and c.bias_values
    for part in ("history", "history_len", "prompt_len", "repetition", "frequency", "presence"):
        assert getattr(c, part) is None, part
    with pytest.raises(ValueError):   # the other arguments are checked all the same
        voc.adjust(z, torch.zeros(2, 0, dtype=I32), torch.zeros(3, dtype=I32))


def test_a_history_is_handed_over(voc):
    z, h, n = torch.zeros(2, 512), torch.zeros(2, 4, dtype=I32), torch.full((2,), 4, dtype=I32)
    r = torch.ones(2)
    voc.adjust(z, h, n, repetition=r)
    _, c = voc.calls.pop()
    assert (c.history, c.history_ld, c.history_len, c.repetition) == (h.data_ptr(), 4, n.data_ptr(), r.data_ptr())
    assert c.prompt_len is None and c.n_bias == 0
