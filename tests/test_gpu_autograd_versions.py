"""Tensors of the caller that the adapter, checkpoint and input-gradient calls write, beside
autograd: their versions rise, and what it could not follow is refused."""

import pytest
import torch

import _adapters as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _args(s):
    return s["A"], s["B"], s["scaling"], s["starts"], s["adapter"]


def _small():
    s = R.make(BF, 128, 64, 16, 2, [3, 5], [0, 1], 1)
    V = torch.zeros(8, 16, device="cuda")
    return s, V


def _calls(s, V):
    """(call, tensors that it writes) of every operator that updates tensors of the caller."""
    from post_weight_quantization_23_b200 import (act_checkpoint, act_restore, lora_add, lora_backward,
                                                  quant_matmul_dgrad)
    a = _args(s)
    out, dX2 = torch.empty_like(s["Y"]), torch.empty_like(s["dX"])
    dA, dB = torch.empty_like(s["A"]), torch.empty_like(s["B"])
    codes = torch.zeros(8, 128, dtype=torch.int8, device="cuda")
    sc = torch.zeros(8, 1, device="cuda")
    qw = torch.zeros(64, 16, dtype=torch.int32, device="cuda")
    gs, gz = torch.ones(64, 1, device="cuda"), torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    return [
        (lambda: lora_add(s["Y"], s["X"], *a, V=V), [s["Y"], V]),
        (lambda: lora_add(s["Y"], s["X"], *a, out=out), [out]),
        (lambda: lora_backward(s["dY"], s["X"], V, *a, s["dX"], dA=dA, dB=dB), [s["dX"], dA, dB]),
        (lambda: lora_backward(s["dY"], s["X"], V, *a, s["dX"], out=dX2), [dX2]),
        (lambda: act_checkpoint(s["X"], codes, sc), [codes, sc]),
        (lambda: act_restore(codes, sc, out=s["X"]), [s["X"]]),
        (lambda: quant_matmul_dgrad(s["dY"], qw, gs, gz, 4, 128, 128, out=dX2), [dX2]),
    ]


def test_updates_in_place_raise_the_version():
    s, V = _small()
    every = [*s.values(), V]
    for call, written in _calls(s, V):
        before = [(t, t._version) for t in every]
        mine = [(t, t._version) for t in written]
        call()
        for t, v in mine:
            assert t._version > v
        for t, v in before:  # what a call only reads keeps its version
            assert any(t is w for w in written) or t._version == v


def test_saved_tensor_overwritten_is_an_error():
    # exp keeps its result for its own backward pass
    from post_weight_quantization_23_b200 import lora_add
    s, V = _small()
    w = s["Y"].clone().requires_grad_()
    Y = w.exp()
    with torch.no_grad():
        lora_add(Y, s["X"], *_args(s))
    with pytest.raises(RuntimeError, match="inplace"):
        Y.sum().backward()


def test_written_tensors_that_require_grad_are_refused():
    # the calls record nothing: under grad mode their update would be missing from the gradients
    from post_weight_quantization_23_b200 import GptqError
    s, V = _small()
    for call, written in _calls(s, V):
        for t in written:
            if not t.is_floating_point():
                continue
            was = t.clone().view(torch.uint8)  # bits: some are uninitialised
            t.requires_grad_()
            with pytest.raises(GptqError, match="requires grad"):
                call()
            assert torch.equal(t.detach().view(torch.uint8), was)
            with torch.no_grad():
                call()
            t.requires_grad_(False)
    # inputs that require grad (parameters) are no obstacle
    from post_weight_quantization_23_b200 import lora_add
    s["A"].requires_grad_()
    s["B"].requires_grad_()
    lora_add(s["Y"], s["X"], *_args(s))


def test_inference_tensors():
    from post_weight_quantization_23_b200 import lora_add
    s, V = _small()
    want = lora_add(s["Y"].clone(), s["X"], *_args(s))
    with torch.inference_mode():
        Y = s["Y"].clone()
        lora_add(Y, s["X"], *_args(s))
    assert torch.equal(Y, want)
    lora_add(Y, s["X"], *_args(s))  # also outside: nothing records it
    assert torch.equal(Y, lora_add(want, s["X"], *_args(s)))
