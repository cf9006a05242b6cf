"""Infinities that meet the padding of the adapters' rank, and batches at the sizes where another
kernel takes over."""

import pytest
import torch

import _adapters as R

pytestmark = pytest.mark.gpu

H, BF, D = torch.float16, torch.bfloat16, torch.float64


def _args(s):
    return s["A"], s["B"], s["scaling"], s["starts"], s["adapter"]


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 72, 128])
@pytest.mark.parametrize("lens", [[3, 2, 4], [300, 5, 600]], ids=["decode", "long"])
def test_infinity_in_a_row(lens, rank, dtype):
    # positive factors: an infinity in x (dY) is an infinity in every value of V and out (dX),
    # never NaN, whatever the rank is padded to; other rows are as without it
    from post_weight_quantization_23_b200 import lora_add, lora_backward
    s = R.make(dtype, 264, 200, rank, 2, lens, [0, -1, 1], 3)
    m = sum(lens)
    s["A"], s["B"] = s["A"].abs() + 0.01, s["B"].abs() + 0.01
    hit = [1, lens[0] + 1, m - 1]  # the second is a row without an adapter
    for name, cols in (("X", (5, 263)), ("dY", (7, 199))):
        s[name][hit[0], cols[0]] = float("inf")
        s[name][hit[1], cols[0]] = float("inf")
        s[name][hit[2], cols[1]] = float("-inf")
    V = torch.zeros(m, rank, device="cuda")
    out = lora_add(s["Y"], s["X"], *_args(s), out=torch.empty_like(s["Y"]), V=V)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[hit] = False
    inf = float("inf")
    for row, want in ((hit[0], inf), (hit[2], -inf)):
        assert (V[row] == want).all() and (out[row] == want).all()
    assert torch.equal(out[hit[1]], s["Y"][hit[1]]) and (V[hit[1]] == 0).all()
    clean = dict(s)
    clean["X"], clean["dY"] = s["X"].clone(), s["dY"].clone()
    clean["X"][hit], clean["dY"][hit] = 0, 0
    ref, bound, Vr, bv, _ = R.add_ref(clean, dtype)
    R.check(out[keep], ref[keep], bound[keep], "out")
    R.check(V[keep], Vr[keep], bv[keep], "V")
    got = lora_backward(s["dY"], clean["X"], Vr.float(), *_args(s), s["dX"],
                        out=torch.empty_like(s["dX"]))[0]
    clean["V"] = Vr.float()
    ref, bound = R.backward_ref(clean, dtype, clean["X"].to(D))["out"]
    for row, want in ((hit[0], inf), (hit[2], -inf)):
        assert (got[row] == want).all()
    R.check(got[keep], ref[keep], bound[keep], "dX")


@pytest.mark.parametrize("rank,rows", [(8, 512), (16, 512), (32, 512), (64, 256), (128, 192)])
@pytest.mark.parametrize("several", [False, True])
def test_batches_at_the_rule(rank, rows, several):
    # on both sides of the number of rows where the tensor-core kernel takes over
    from post_weight_quantization_23_b200 import lora_add
    edges = [rows, rows + 1] if rank > 16 or not several else [704, 705]
    for m in edges:
        lens, ids = ([m - 100, 99, 1], [1, 0, 1]) if several else ([m], [1])
        s = R.make(BF, 512, 328, rank, 2, lens, ids, m)
        ref, bound, Vr, bv, _ = R.add_ref(s, BF)
        V = torch.zeros(m, rank, device="cuda")
        out = lora_add(s["Y"], s["X"], *_args(s), out=torch.empty_like(s["Y"]), V=V)
        R.check(out, ref, bound, "out")
        R.check(V, Vr, bv, "V")
