"""A quantized layer that carries adapters, as a training step and a serving step use it:
GptqPlan's packed weights, the shared product, the adapters, the 8-bit checkpoint and the
two gradients, against the same chain in 64 bits."""

import pytest
import torch

import _adapters as R

pytestmark = pytest.mark.gpu

D = torch.float64


def _plan(r, k, seed, act_order=False, bits=4):
    from post_weight_quantization_23_b200 import GptqPlan, QuantConfig
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = torch.randn(r, k, generator=g, device="cuda").half() * 0.02
    X = torch.randn(1024, k, generator=g, device="cuda").half()
    plan = GptqPlan(r, k, QuantConfig(bits=bits, group_size=128, act_order=act_order), "cuda",
                    deq_dtype=torch.float32)
    plan.hessian_add(X, 1024)
    plan.run_after_hessian(W)
    plan.check()
    return plan


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,ids", [([1] * 9, [0, 1, 2, 0, -1, 1, 1, 0, 0]), ([300, 1, 129], [1, 0, 2])])
def test_layer_forward_and_backward(dtype, lens, ids):
    from post_weight_quantization_23_b200 import act_checkpoint, lora_add, lora_backward
    n, k, r = 384, 512, 16
    plan = _plan(n, k, 1)
    s = R.make(dtype, k, n, r, 3, lens, ids, 4)
    m = sum(lens)
    a = (s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    W = plan.deq.to(D)
    u = R.U[dtype]
    # forward: the shared product, the adapters in place, what the backward pass keeps
    V = torch.zeros(m, r, device="cuda")
    Y = plan.matmul(s["X"])
    lora_add(Y, s["X"], *a, V=V)
    codes, xs = act_checkpoint(s["X"])
    s["Y"] = torch.zeros_like(Y)
    d, ed, Vr, bv, _ = R.add_ref(s, dtype)
    base = s["X"].to(D) @ W.T
    mag = s["X"].to(D).abs() @ W.abs().T
    # the product's weights are rounded twice to the type (3 u with the square), its result once,
    # the sum once; ed holds one rounding of the adapters' part too
    R.check(Y, base + d, 3 * u * mag + 2 * u * (base.abs() + d.abs()) + ed + 2.0 ** -24, "Y")
    # backward: through the packed weights, then the adapters on top
    s["V"] = V
    s["dX"] = plan.matmul_dgrad(s["dY"])
    gb = s["dY"].to(D) @ W
    gm = s["dY"].to(D).abs() @ W.abs()
    R.check(s["dX"], gb, 2 * u * gm + 2 * u * gb.abs() + 2.0 ** -24, "dX of the weights")
    Xd = codes.to(D) * xs.to(D).repeat_interleave(128, 1)
    ref = R.backward_ref(s, dtype, Xd)
    out, dA, dB = lora_backward(s["dY"], codes, V, *a, s["dX"].clone(), x_scales=xs)
    R.check(out, *ref["out"], "dX")
    R.check(dA, *ref["dA"], "dA")
    R.check(dB, *ref["dB"], "dB")


def test_gradients_of_the_whole_layer_against_differences():
    # the loss sum(G * Y) of the 64-bit layer is linear in X, A and B each: its differences
    # are exact, the kernels' gradients within their roundings
    from post_weight_quantization_23_b200 import lora_add, lora_backward
    n, k, r = 256, 256, 8
    plan = _plan(n, k, 2)
    s = R.make(torch.float16, k, n, r, 2, [40, 90], [1, 0], 6)
    a = (s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    V = torch.zeros(130, r, device="cuda")
    lora_add(plan.matmul(s["X"]), s["X"], *a, V=V)
    dX, dA, dB = lora_backward(s["dY"], s["X"], V, *a, plan.matmul_dgrad(s["dY"]))
    W, G = plan.deq.to(D), s["dY"].to(D)
    v = {q: s[q].to(D) for q in ("X", "A", "B")}

    def loss(w):
        t = (G * (w["X"] @ W.T)).sum()
        for b, e, i in R.spans(s, 2):
            low = (w["X"][b:e] @ w["A"][i].T) * s["scaling"][i].to(D)
            t = t + (G[b:e] * (low @ w["B"][i].T)).sum()
        return t

    gen = torch.Generator().manual_seed(3)
    for name, grad in (("X", dX), ("A", dA), ("B", dB)):
        top = grad.to(D).abs().max()
        for _ in range(10):
            i = tuple(int(torch.randint(0, z, (1,), generator=gen)) for z in v[name].shape)
            hi, lo = dict(v), dict(v)
            hi[name], lo[name] = v[name].clone(), v[name].clone()
            hi[name][i] += 1e-2
            lo[name][i] -= 1e-2
            num = (loss(hi) - loss(lo)) / 2e-2
            # two roundings to f16 and 2^-11 of every weight in sums of a few hundred products,
            # whose magnitudes stay below a few times the largest gradient
            assert abs(num - grad[i].to(D)) <= 2.0 ** -9 * abs(num) + 2.0 ** -9 * top, (name, i)


def test_plan_dgrad_takes_act_order_groups():
    plan = _plan(128, 256, 5, act_order=True)
    dY = torch.randn(33, 128, device="cuda").half()
    got = plan.matmul_dgrad(dY)
    ref = dY.to(D) @ plan.deq.to(D)
    mag = dY.to(D).abs() @ plan.deq.to(D).abs()
    R.check(got, ref, 2.0 ** -11 * ref.abs() + 2.0 ** -14 * mag + 2.0 ** -24, "dX")
    out = torch.empty_like(got)
    assert plan.matmul_dgrad(dY, out=out) is out and torch.equal(out, got)
