"""Operands and results of the adapter, checkpoint and input-gradient calls as ranges of columns
of one buffer: they share no element, so the calls take them; real overlaps are refused."""

import pytest
import torch

import _adapters as R

pytestmark = pytest.mark.gpu

H, BF = torch.float16, torch.bfloat16


def _args(s):
    return s["A"], s["B"], s["scaling"], s["starts"], s["adapter"]


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("lens", [[3, 1, 4], [400, 1, 350]], ids=["decode", "long"])
def test_column_ranges_of_one_buffer(lens, dtype):
    # operands and results side by side in one buffer share no element
    from post_weight_quantization_23_b200 import (GptqError, act_checkpoint, act_restore, lora_add,
                                                  lora_backward, quant_matmul_dgrad)
    k, n, m = 136, 72, sum(lens)
    s = R.make(dtype, k, n, 16, 2, lens, [1, -1, 0], 6)
    V = torch.zeros(m, 16, device="cuda")
    want = lora_add(s["Y"], s["X"], *_args(s), out=torch.empty_like(s["Y"]), V=V)
    buf = torch.full((m, 8 + k + 2 * n), 3.0, dtype=dtype, device="cuda")
    X, Y, out = buf[:, 8:8 + k], buf[:, 8 + k:8 + k + n], buf[:, 8 + k + n:]
    X.copy_(s["X"])
    Y.copy_(s["Y"])
    lora_add(Y, X, *_args(s), out=out)
    assert torch.equal(out, want) and torch.equal(X, s["X"]) and torch.equal(Y, s["Y"])
    lora_add(Y, X, *_args(s))
    assert torch.equal(Y, want) and (buf[:, :8] == 3.0).all()
    with pytest.raises(GptqError):
        lora_add(Y, X, *_args(s), out=buf[:, 8 + k + n - 8:8 + k + 2 * n - 8])
    # backward: dY, dX and out in one buffer
    dX, dA, dB = lora_backward(s["dY"], s["X"], V, *_args(s), s["dX"], out=torch.empty_like(s["dX"]))
    buf = torch.full((m, n + 2 * k), 3.0, dtype=dtype, device="cuda")
    dY, dXi, o = buf[:, :n], buf[:, n:n + k], buf[:, n + k:]
    dY.copy_(s["dY"])
    dXi.copy_(s["dX"])
    got = lora_backward(dY, s["X"], V, *_args(s), dXi, out=o)
    for g, w in zip(got, (dX, dA, dB)):
        assert torch.equal(g, w)
    assert torch.equal(dY, s["dY"]) and torch.equal(dXi, s["dX"])
    # the gradient through packed weights
    g = torch.Generator(device="cuda").manual_seed(1)
    qw = torch.randint(-2 ** 31, 2 ** 31, (n, 128 // 8), generator=g, device="cuda").to(torch.int32)
    a = (qw, torch.rand(n, 4, generator=g, device="cuda") * 0.01,
         torch.full((n, 4), 8, dtype=torch.int32, device="cuda"), 4, 32, 128)
    want = quant_matmul_dgrad(s["dY"], *a)
    assert torch.equal(quant_matmul_dgrad(dY, *a, out=buf[:, n:n + 128]), want)
    assert torch.equal(dY, s["dY"])
    with pytest.raises(GptqError):
        quant_matmul_dgrad(dY, *a, out=buf[:, n - 8:n + 120])
    # a checkpoint beside its activations: 2 k bytes of values and k of codes in each row
    codes, sc = act_checkpoint(s["X"])
    raw = torch.zeros(m, 3 * k, dtype=torch.int8, device="cuda")
    x, c = raw.view(dtype)[:, :k], raw[:, 2 * k:]
    x.copy_(s["X"])
    act_checkpoint(x, c)
    assert torch.equal(c, codes) and torch.equal(x, s["X"])
    act_restore(c, sc, out=x)
    assert torch.equal(x, act_restore(codes, sc, dtype)) and torch.equal(c, codes)
    with pytest.raises(GptqError):
        act_checkpoint(x, raw[:, 2 * k - 8:3 * k - 8])
