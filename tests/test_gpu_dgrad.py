"""The gradient of the inference product with respect to its input (gptq_gemm_dgrad)
against the 64-bit product of the oracle's weights.

Bound: each weight is the fp32 scale times the exact code - zero (one fp32
rounding), on the tensor-core path rounded once to the 16-bit type (u); products
exact or once rounded, fp32 sums over the n rows (twice over, in case an adder
truncates), one rounding of the result (u) and half f16's subnormal spacing.  The
tensor-core path adds the scale's low half as a 16-bit value: f16 holds it to
2^-25 absolutely, times |code - zero| (included below).
"""

import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

H, BF = torch.float16, torch.bfloat16
U = {H: 2.0 ** -11, BF: 2.0 ** -8}

# (n, k, bits, group, m, dtype, g_idx passed, act-order)
CASES = [
    (64, 64, 4, 32, 1, H, False, False),
    (1, 32, 4, 32, 1, BF, False, False),
    (256, 1024, 4, 128, 1, H, False, False),
    (300, 1056, 4, 128, 17, BF, False, False),    # ragged rows, a short last group
    (512, 768, 4, 64, 130, H, False, False),
    (1000, 320, 4, -1, 300, BF, False, False),    # one group per row
    (200, 416, 4, 8, 65, H, False, False),         # groups of 8
    (4096, 256, 4, 128, 513, BF, False, False),
    (72, 4128, 4, 1024, 257, H, False, False),
    (33, 256, 4, 128, 40, H, False, False),        # odd n: rows of dY off 16 bytes
    (128, 256, 4, 12, 40, H, False, False),        # groups that straddle words
    (96, 512, 2, 64, 70, BF, False, False),
    (64, 1024, 3, 128, 33, H, False, False),
    (70, 512, 8, 32, 129, BF, False, False),
    (80, 1024, 4, 128, 90, BF, True, True),        # act-order groups
    (48, 512, 4, 128, 20, H, True, False),
    # few tiles: the rows of W split over a cluster of 2, 4 or 8
    (2200, 1024, 4, 128, 1, H, False, False),
    (4104, 128, 4, -1, 200, BF, False, False),
    (520, 384, 4, 32, 90, BF, False, False),
    (1000, 2048, 4, 64, 250, H, False, False),
]


def _inputs(n, k, bits, G, m, dtype, act, seed):
    g = torch.Generator().manual_seed(seed)
    Gk = k if G == -1 else G
    ng = (k + Gk - 1) // Gk
    codes = torch.randint(0, 2 ** bits, (n, k), generator=g)
    scales = (torch.rand(n, ng, generator=g) * 0.02 + 1e-3).float()
    zeros = torch.randint(0, 2 ** bits, (n, ng), generator=g, dtype=torch.int32)
    g_idx = (torch.arange(k) // Gk).to(torch.int32)
    if act:
        g_idx = g_idx[torch.randperm(k, generator=g)]
    dY = (torch.randn(m, n, generator=g) * 0.1).to(dtype)
    return codes, scales, zeros, g_idx.contiguous(), dY, torch.from_numpy(O.pack(codes.numpy(), bits))


def _check(got, dY, codes, scales, zeros, g_idx, dtype, tc):
    d = torch.float64
    s, z = scales.to(d)[:, g_idx.long()], zeros.to(d)[:, g_idx.long()]
    W = s * (codes.to(d) - z)
    y = dY.to(d)
    ref, mag = y @ W, y.abs() @ W.abs()
    u, n = U[dtype], dY.shape[1]
    e = 2 * (n + 8) * 2.0 ** -24 * mag
    if tc:
        e = e + (u + u * u) * mag + 2.0 ** -25 * (y.abs() @ (codes.to(d) - z).abs())
    bound = u * ref.abs() + (1 + u) * e + 2.0 ** -25
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= bound).all(), float((err / bound).max())
    return float((err / bound).max()) if err.numel() else 0.0


@pytest.mark.parametrize("case", CASES, ids=[f"n{c[0]}_k{c[1]}_b{c[2]}_g{c[3]}_m{c[4]}{'_act' if c[7] else ''}"
                                              for c in CASES])
def test_dgrad(case):
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    n, k, bits, G, m, dtype, pass_gidx, act = case
    codes, scales, zeros, g_idx, dY, qw = _inputs(n, k, bits, G, m, dtype, act, n + k + m)
    a = (qw.cuda(), scales.cuda(), zeros.cuda(), bits, G, k)
    got = quant_matmul_dgrad(dY.cuda(), *a, g_idx.cuda() if pass_gidx else None)
    tc = bits == 4 and not pass_gidx and (G == -1 or G % 8 == 0) and n % 8 == 0
    print("max err / bound", _check(got, dY, codes, scales, zeros, g_idx, dtype, tc))
    # padded leading dimensions, the padding kept; one call after another gives the same bits
    yp = torch.full((m, n + 8), float("nan"), dtype=dtype, device="cuda")
    yp[:, :n] = dY.cuda()
    xp = torch.full((m, k + 5), 3.0, dtype=dtype, device="cuda")
    quant_matmul_dgrad(yp[:, :n], *a, g_idx.cuda() if pass_gidx else None, out=xp[:, :k])
    _check(xp[:, :k], dY, codes, scales, zeros, g_idx, dtype, True)
    assert (xp[:, k:] == 3.0).all()
    assert torch.equal(quant_matmul_dgrad(dY.cuda(), *a, g_idx.cuda() if pass_gidx else None), got)


def test_dgrad_is_the_transpose_of_the_product():
    # <dY, X W^T> = <dY W, X>: the two products read the same packed weights
    from post_weight_quantization_23_b200 import quant_matmul, quant_matmul_dgrad
    codes, scales, zeros, g_idx, dY, qw = _inputs(512, 1024, 4, 128, 64, H, False, 3)
    X = torch.randn(64, 1024, generator=torch.Generator().manual_seed(1)).half()
    Y = quant_matmul(X.cuda(), qw.cuda(), scales.cuda(), zeros.cuda(), 4, 128)
    dX = quant_matmul_dgrad(dY.cuda(), qw.cuda(), scales.cuda(), zeros.cuda(), 4, 128, 1024)
    a = (dY.double().cuda() * Y.double()).sum()
    b = (dX.double() * X.double().cuda()).sum()
    # both sums carry independent relative errors of a few u per element
    mag = (dY.double().cuda().abs() * Y.double().abs()).sum()
    assert abs(a - b) <= 8 * 2.0 ** -11 * mag


def test_dgrad_bad_gidx_is_nan():
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    codes, scales, zeros, g_idx, dY, qw = _inputs(64, 256, 4, 128, 5, H, False, 3)
    for bad in (-1, 2, 1 << 30):
        gi = g_idx.clone()
        gi[7] = bad
        got = quant_matmul_dgrad(dY.cuda(), qw.cuda(), scales.cuda(), zeros.cuda(), 4, 128, 256, gi.cuda())
        assert got[:, 7].isnan().all()
        keep = [c for c in range(256) if c != 7]
        gi[7] = 0
        _check(got[:, keep], dY, codes[:, keep], scales, zeros, gi[keep], H, False)


@pytest.mark.parametrize("m", [3, 200])
def test_dgrad_nan_rows_stay(m):
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    codes, scales, zeros, g_idx, dY, qw = _inputs(128, 256, 4, 128, m, BF, False, 3)
    y = dY.clone()
    y[1] = float("nan")
    got = quant_matmul_dgrad(y.cuda(), qw.cuda(), scales.cuda(), zeros.cuda(), 4, 128, 256)
    assert got[1].isnan().all()
    keep = [t for t in range(m) if t != 1]
    _check(got[keep], dY[keep], codes, scales, zeros, g_idx, BF, True)


def test_dgrad_full_size():
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    n, k, m = 4096, 4096, 1024
    codes, scales, zeros, g_idx, dY, qw = _inputs(n, k, 4, 128, m, BF, False, 5)
    got = quant_matmul_dgrad(dY.cuda(), qw.cuda(), scales.cuda(), zeros.cuda(), 4, 128, k)
    _check(got, dY, codes, scales, zeros, g_idx, BF, True)


def test_dgrad_empty_and_refusals():
    from post_weight_quantization_23_b200 import GptqError, quant_matmul_dgrad
    codes, scales, zeros, g_idx, dY, qw = _inputs(64, 256, 4, 128, 5, H, False, 3)
    a = [t.cuda() for t in (qw, scales, zeros)]
    y = dY.cuda()
    assert quant_matmul_dgrad(y[:0], *a, 4, 128, 256).shape == (0, 256)
    for call in (lambda: quant_matmul_dgrad(y.float(), *a, 4, 128, 256),
                 lambda: quant_matmul_dgrad(y, *a, 5, 128, 256),
                 lambda: quant_matmul_dgrad(y, *a, 4, 64, 256),
                 lambda: quant_matmul_dgrad(y, *a, 4, 128, 224),
                 lambda: quant_matmul_dgrad(y[:, :32], *a, 4, 128, 256),
                 lambda: quant_matmul_dgrad(y.cpu(), *a, 4, 128, 256),
                 lambda: quant_matmul_dgrad(y, *a, 4, 128, 256, out=y),
                 lambda: quant_matmul_dgrad(y, *a, 4, 128, 256, g_idx.cuda()[:200]),
                 lambda: quant_matmul_dgrad(y, *a, 4, 128, 256, out=torch.zeros(5, 256, device="cuda"))):
        with pytest.raises(GptqError):
            call()


@pytest.mark.parametrize("n,k,m", [(2048, 2048, 700), (2048, 4096, 2048)])
def test_dgrad_repeats_under_load(n, k, m):
    # many calls back to back give the same bits (copies land in every order)
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    codes, scales, zeros, g_idx, dY, qw = _inputs(n, k, 4, 128, m, BF, False, 7)
    a = (dY.cuda(), qw.cuda(), scales.cuda(), zeros.cuda(), 4, 128, k)
    first = quant_matmul_dgrad(*a)
    _check(first, dY, codes, scales, zeros, g_idx, BF, True)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(500):
        bad += (quant_matmul_dgrad(*a) != first).any()
    assert int(bad) == 0
