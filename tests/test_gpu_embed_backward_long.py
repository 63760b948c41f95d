"""The embedding gradient of many rows, long runs of one token, and buffers that
overlap."""

import numpy as np
import pytest
import torch

from tests.test_gpu_vocab_ops import U, make_vocab

pytestmark = pytest.mark.gpu


def reference(E, tok, dh, was=None):
    """float64 on the GPU: the sums by token, projected off the row's direction."""
    e = E.double()
    G = torch.zeros_like(e).index_add_(0, tok.long(), dh.double())
    norm2 = e.square().sum(1, keepdim=True)
    out = (G - e * ((e * G).sum(1, keepdim=True) / norm2)) / norm2.sqrt()
    return out if was is None else out + was.double()


def bound(E, tok, dh, ref, was):
    """G: at most 64 rows (and the entries of one window) are added one after the
    other in fp32, 63 roundings, the join in float64 and one rounding to fp32;
    |G| is at most the sum of |dh|.  e . G: products, d / 128 + 12 additions and
    G's own; a division, a product, a subtraction, the scaling (three) and,
    accumulating, an addition."""
    e = E.double()
    d = e.shape[1]
    size = torch.zeros_like(e).index_add_(0, tok.long(), dh.double().abs())
    depth = 64
    norm = e.norm(dim=1, keepdim=True)
    proj = (e.abs() * size).sum(1, keepdim=True) / norm ** 2
    o = U * depth * size + e.abs() * proj * U * (depth + 2 * (d / 128 + 12) + 8) + 8 * U * (size + e.abs() * proj)
    return o / norm * (1 + 1e-6) + 2 * U * (ref.abs() + was.double().abs())


@pytest.mark.parametrize("n", [150016, 300000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_run_is_joined_without_drift(n, accumulate):
    """One token; of each 32 rows (a window) only the first is not zero, so that every
    window's sum is exact.  Its value is one whose addition in 32 bits would round
    down by nearly half a step each time once 256 of them are summed.  Joined in 64
    bits the sum is exact, and the result is rounded once; along the row's own
    direction (column 0) the gradient is 0."""
    V, d = 256, 128
    E = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    E[:, 0] = 1.0
    model, voc = make_vocab(V, d, emb=E)
    value = 1 + 2.0 ** -16 - 2.0 ** -23
    dh = torch.zeros(n, d, device="cuda")
    dh[::32, 1:] = value
    tok = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    out = torch.zeros(V, d, device="cuda")
    got = voc.embed_backward(tok, dh, out=out, accumulate=accumulate).double()
    want = ((n + 31) // 32) * value
    assert (got[77, 1:] - want).abs().max() <= U * want
    assert got[77, 0] == 0 and not got[:77].any() and not got[78:].any()
    assert model.device_status() == 0


@pytest.mark.parametrize("n", [200003, 330000])
@pytest.mark.parametrize("kind", ["one", "zipf"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_many_rows_of_nonzero_mean(n, kind, accumulate):
    V, d = 1024, 128
    g = torch.Generator(device="cuda").manual_seed(n)
    E = torch.randn(V, d, device="cuda", generator=g)
    E = (E / E.norm(dim=1, keepdim=True)).bfloat16()
    model, voc = make_vocab(V, d, emb=E)
    tok = torch.full((n,), 5, dtype=torch.int32, device="cuda") if kind == "one" else (
        V * torch.rand(n, device="cuda", generator=g) ** 4).int()
    dh = 1 + torch.randn(n, d, device="cuda", generator=g)
    was = torch.randn(V, d, device="cuda", generator=g)
    got = voc.embed_backward(tok, dh, out=was.clone(), accumulate=accumulate)
    was = was if accumulate else torch.zeros_like(was)
    ref = reference(E, tok, dh, was)
    over = (got.double() - ref).abs() - bound(E, tok, dh, ref, was)
    assert over.max() <= 0, over.max()
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[tok.long()] = False
    assert torch.equal(got[absent], was[absent])
    again = voc.embed_backward(tok, dh, out=was.clone(), accumulate=accumulate)
    assert torch.equal(again, got)
    assert model.device_status() == 0


@pytest.mark.parametrize("n", [8200, 262150])
@pytest.mark.parametrize("accumulate", [False, True])
def test_tokens_of_three_sort_passes(n, accumulate):
    """A vocabulary of 2^18 tokens: 19 bits of key, three passes."""
    V, d = 1 << 18, 128
    g = torch.Generator(device="cuda").manual_seed(n)
    E = torch.randn(V, d, device="cuda", generator=g).bfloat16()
    model, voc = make_vocab(V, d, emb=E)
    tok = (V * torch.rand(n, device="cuda", generator=g) ** 3).int()
    tok[::7], tok[1::50], tok[-1] = 4099, V - 1, 0
    dh = torch.randn(n, d, device="cuda", generator=g)
    was = torch.randn(V, d, device="cuda", generator=g)
    got = voc.embed_backward(tok, dh, out=was.clone(), accumulate=accumulate)
    was = was if accumulate else torch.zeros_like(was)
    ref = reference(E, tok, dh, was)
    assert ((got.double() - ref).abs() - bound(E, tok, dh, ref, was)).max() <= 0
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[tok.long()] = False
    assert torch.equal(got[absent], was[absent])
    assert model.device_status() == 0


def test_overlapping_buffers_are_refused():
    """The table's gradient in the place of an input or of the workspace, whole or in part."""
    from looped_ngpt_transformer_fwd_b200 import binding as B
    V, d, n = 256, 128, 256
    model, voc = make_vocab(V, d)
    row = d * 4
    need = B.dory_embed_backward_workspace_bytes(voc.handle, n)
    buf = torch.zeros(2 * V * row + n * row + n * 4 + 2 * need + 1024, dtype=torch.uint8, device="cuda")
    p = (buf.data_ptr() + 255) // 256 * 256
    table, dh, tok, ws = p, p + V * row, p + V * row + n * row, p + V * row + n * row + n * 4

    def call(tok=tok, dh=dh, table=table, ws=ws, size=need):
        return B.lib().dory_embed_backward(voc.handle, tok, n, dh, table, 0, ws, size, None)
    assert call(dh=table) == -1 and call(dh=table + V * row - 16) == -1 and call(table=dh + 16) == -1
    assert call(tok=table + 4) == -1 and call(tok=ws) == -1 and call(dh=ws) == -1
    assert call(ws=table) == -1 and call(ws=dh + n * row - 256) == -1 and call(ws=tok - 256) == -1
    torch.cuda.synchronize()
    assert not buf.any()
    assert call() == 0 and model.device_status() == 0      # neighbours, none overlapping
    dh = torch.ones(n, d, device="cuda")
    with pytest.raises(B.DoryError):
        voc.embed_backward(torch.zeros(n, dtype=torch.int32, device="cuda"), dh, out=dh)
    assert (dh == 1).all()
