"""combine_rows_backward of more tokens than one launch takes, as combine_rows takes
them (CPU only: the calls that it makes)."""
import pytest
import torch

from moe_expert_ffn_persistent_amd import ops

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture
def made(monkeypatch):
    calls = []
    monkeypatch.setattr(ops, "_first_call", lambda name, check, args, *rest: calls.append((name, check(*args), args)))
    monkeypatch.setattr(ops, "_MAX_TOKENS", 100)
    return calls


@pytest.mark.parametrize("tokens,pieces", [(100, [100]), (101, [100, 1]), (230, [100, 100, 30])])
def test_more_tokens_go_in_pieces(made, tokens, pieces):
    dy, rows, out = torch.zeros(tokens, 32, dtype=BF)[:, :16], torch.zeros(8, 16, dtype=BF), torch.zeros(8, 16, dtype=BF)
    at, w, dw = torch.zeros(tokens, 3, dtype=I32), torch.rand(tokens, 3), torch.empty(tokens, 3)
    got = ops.combine_rows_backward(dy, rows, at, w, out=out, dweights=dw)
    assert got[0] is out and got[1] is dw
    assert [p.tokens for _, p, _ in made] == pieces and {n for n, _, _ in made} == {"moe_combine_rows_backward"}
    first = 0
    for n, (_, p, (dyi, rowsi, ati, wi, outi, dwi)) in zip(pieces, made):
        assert rowsi is rows and outi is out and p.ld_dy == (32 if n > 1 else 16)
        assert dyi.data_ptr() == dy[first:].data_ptr() and wi.data_ptr() == w[first:].data_ptr() and dwi.data_ptr() == dw[first:].data_ptr()
        assert ati.data_ptr() == at[first:].data_ptr() and ati.numel() == 3 * n and len(wi) == len(dwi) == len(dyi) == n
        first += n
    assert first == tokens


def test_every_version_moves(made):
    rows, w, dw = torch.zeros(8, 16, dtype=BF), torch.rand(230, 3), torch.empty(230, 3)
    ops.combine_rows_backward(torch.zeros(230, 16, dtype=F32), rows, torch.zeros(690, dtype=I32), w, out=rows, dweights=dw)   # over the rows
    assert all(a[4] is rows for _, _, a in made)
    assert all(a[5]._base is dw for _, _, a in made)   # views: what they write counts as dw's


def test_other_faults_of_many_tokens_are_refused(made):
    dy, rows, at, w = torch.zeros(230, 16, dtype=BF), torch.zeros(8, 16, dtype=BF), torch.zeros(690, dtype=I32), torch.rand(230, 3)
    for bad in (dict(pair_row=at[:-1]), dict(weights=w[:, :2]), dict(out=rows.float()), dict(dweights=torch.empty(229, 3)), dict(dy=dy[:, :15])):
        with pytest.raises(ValueError):
            ops.combine_rows_backward(**{**dict(dy=dy, rows=rows, pair_row=at, weights=w, out=torch.zeros_like(rows), dweights=torch.empty(230, 3)), **bad})
    assert not made
