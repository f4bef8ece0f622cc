"""What the binding of include/qgemv_mx.h refuses on the host (no GPU)."""
from __future__ import annotations

import pytest

import quantized_gemv_gguf_amd as q


@pytest.fixture
def on_device(monkeypatch):
    """CPU tensors pass for device tensors; the calls below are refused before any of them is used."""
    torch = pytest.importorskip("torch")
    q._torch_names()
    monkeypatch.setattr(q, "_here", lambda t, name: 0x1000)
    monkeypatch.setattr(q, "_here_stream", lambda stream: 0)
    return torch


def matrix(torch, rows, k):
    return q.Matrix(torch.zeros(rows * (k // 32) * 17, dtype=torch.uint8), q.MXFP4, rows, k)


@pytest.mark.parametrize("pair", [False, True])
def test_slots_need_the_number_of_choices(on_device, pair):
    """Without it a slot would be taken for a token."""
    torch = on_device
    x, y = torch.zeros(4, 64), torch.zeros(8, 8)
    offsets, slots = torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    ws = [matrix(torch, 16, 64)] * (1 + pair)
    call = q.qgemv_expert_mx_swiglu if pair else q.qgemv_expert_mx
    with pytest.raises(ValueError, match="n_sel"):
        call(*ws, 2, x, offsets, y, slots=slots)
    with pytest.raises(q.QgemvError, match="QG_E_ARG"):
        call(*ws, 2, x, offsets, y, slots=slots, n_sel=0)
    # without slots the number is not looked at: four rows of x for eight places
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        call(*ws, 2, x, offsets, y)


def test_weights_by_choice_are_not_taken_transposed(on_device):
    """(choices, tokens) holds as many values as (tokens, choices)."""
    torch = on_device
    tok, sel = 6, 4
    y, out = torch.zeros(tok * sel, 8), torch.zeros(tok, 7)  # (7 columns: refused by the library after the binding)
    pos, w = torch.zeros(tok, sel, dtype=torch.int32), torch.zeros(tok, sel)
    wrong = torch.zeros(sel, tok)
    with pytest.raises(ValueError, match="choices"):
        q.qgemv_expert_combine(y, pos, out, w=wrong)
    with pytest.raises(ValueError, match="choices"):
        q.qgemv_expert_combine_grad(out, y, pos, wrong, torch.zeros_like(y), w)
    with pytest.raises(ValueError, match="choices"):
        q.qgemv_expert_combine_grad(out, y, pos, w, torch.zeros_like(y), wrong)
    for fine in (None, w, w.flatten(), torch.zeros(tok + 3, sel)):
        with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
            q.qgemv_expert_combine(y, pos, out, w=fine)
    for fine in (w, w.flatten()):
        with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
            q.qgemv_expert_combine_grad(out, y, pos, fine, torch.zeros_like(y), w)


def test_choices_past_32_bits(on_device):
    """Numbers of choices that a C int does not hold are refused, not cut to their low bits."""
    torch = on_device
    n = 2 ** 32 + 1
    many = torch.empty((1, n), dtype=torch.int32, device="meta")
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_expert_sort(many, 2, torch.zeros(3, dtype=torch.int32), many, many)
    y, out, w = torch.zeros(8, 8), torch.zeros(1, 8), torch.empty((1, n), device="meta")
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE"):
        q.qgemv_expert_combine(y, many, out, w=w)
    with pytest.raises(q.QgemvError, match="QG_E_SHAPE|QG_E_ARG"):
        q.qgemv_expert_combine_grad(out, y, many, w, y, w)
    slots = torch.zeros(8, dtype=torch.int32)
    for bad in (-2 ** 32 + 1, -1, 0):
        with pytest.raises(q.QgemvError, match="QG_E_ARG"):
            q.qgemv_expert_gather(y, slots, bad, y)
        with pytest.raises(q.QgemvError, match="QG_E_ARG"):
            q.qgemv_expert_mx(matrix(torch, 16, 64), 2, torch.zeros(4, 64), slots, y, slots=slots, n_sel=bad)
