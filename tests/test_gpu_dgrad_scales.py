"""The input gradient of the packed weights (gptq_gemm_dgrad) over the range of scales and
zeros that its arrays can hold, and over the tensor-core kernel's tile shapes, against the
64-bit product.

Bounds.  General kernel: fp32 weights (one rounding) and fp32 sums over the n rows, counted
twice in case an adder truncates; one rounding of the result (u) and half f16's subnormal
spacing.  Tensor-core kernel: besides, each weight is rounded once to the 16-bit type (u, with
the square for the two-part scale).  In f16 the scales of a group's column are brought into
the type's range by one power of two per group: what the range still costs is an absolute
error of at most (|code - zero| + 2) half steps of f16's subnormals, 2^-25 before the power of
two is taken back, and that power is at most 2^6 times the group's largest scale.
"""

import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

H, BF, D = torch.float16, torch.bfloat16, torch.float64
U = {H: 2.0 ** -11, BF: 2.0 ** -8}

# (n, k, group, m) and the tile shape they are here for
ONE = (304, 1056, 128, 17)        # one 128-column tile per CTA
SPLIT = (4104, 384, 64, 200)      # the rows of W shared by the CTAs of a cluster
TWO = (1000, 7200, 96, 1000)      # two 128-column tiles per CTA, ragged everywhere
GENERAL = (301, 320, 32, 33)      # odd n: rows of dY off 16 bytes


def _cdiv(a, b):
    return -(-a // b)


def _shape(n, k, m):
    """The kernel's choice of column tiles, tokens and split (launch_shape)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ns, best, got = _cdiv(n, 64), 0, None
    for mt in (1, 2):
        for nn in range(16, 257, 16):
            tiles = _cdiv(k, mt * 128) * _cdiv(m, nn)
            stage = max(2 * mt * nn, nn * (1 + mt) + 320 * mt)
            sp = 1
            while sp <= (8 if mt == 1 else 1) and sp * 4 <= max(ns, 4):
                if sp > 1 and tiles * sp > sms:
                    break
                cost = _cdiv(tiles * sp, sms) * _cdiv(ns, sp) * stage + (8000 + 24 * nn if sp > 1 else 0)
                if best == 0 or cost < best:
                    best, got = cost, (mt, nn, sp)
                sp *= 2
    return got


def _inputs(n, k, G, m, dtype, scales, seed, y_scale=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 16, (n, k), generator=g, device="cuda")
    zeros = torch.randint(0, 16, scales.shape, generator=g, device="cuda", dtype=torch.int32)
    dY = (torch.randn(m, n, generator=g, device="cuda") * y_scale).to(dtype)
    qw = torch.from_numpy(O.pack(codes.cpu().numpy(), 4)).cuda()
    return dY, qw, codes, zeros


def _scales(n, k, G, seed, lo, hi):
    """Log-uniform in [lo, hi]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ng = 1 if G == -1 else _cdiv(k, G)
    e = torch.rand(n, ng, generator=g, device="cuda", dtype=D)
    return (lo * (hi / lo) ** e).float()


def _ref(dY, codes, scales, zeros, G, dtype, tc):
    """The product in 64 bits and its bound."""
    k = codes.shape[1]
    col = torch.arange(k, device="cuda") // (k if G == -1 else G)
    s, d = scales.to(D)[:, col], codes.to(D) - zeros.to(D)[:, col]
    W, y, u, n = s * d, dY.to(D), U[dtype], dY.shape[1]
    ref, mag = y @ W, y.abs() @ W.abs()
    e = 2 * (n + 8) * 2.0 ** -24 * mag
    if tc:
        e = e + (u + u * u) * mag
        if dtype == H:
            top = s.abs().amax(0)
            e = e + 2.0 ** -19 * (y.abs() @ (d.abs() + 2)) * top
    return ref, u * ref.abs() + (1 + u) * e + 2.0 ** -25


def _check(got, ref, bound):
    assert torch.isfinite(got).all()
    err = (got.to(D) - ref).abs()
    assert (err <= bound).all(), float((err / bound).max())
    print("max err / bound", float((err / bound).max()))


def _run(dY, qw, scales, zeros, G, k):
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    return quant_matmul_dgrad(dY, qw, scales, zeros, 4, G, k)


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("scale", [2e-8, 3e-6, 1e-5, 3e-5, 1e-4, 1e-3, 0.02, 1.0, 40.0, 7e4])
@pytest.mark.parametrize("case", [ONE, SPLIT, TWO, GENERAL], ids=["one", "split", "two", "general"])
def test_scales_of_every_size(case, scale, dtype):
    n, k, G, m = case
    if case is not GENERAL:
        mt, _, split = _shape(n, k, m)
        assert (mt == 2) == (case is TWO) and (split > 1) == (case is SPLIT)
    scales = _scales(n, k, G, 1, 0.6 * scale, 1.4 * scale)
    # results of a common size, gradients within f16
    dY, qw, codes, zeros = _inputs(n, k, G, m, dtype, scales, 2, min(max(0.01 / scale, 1e-6), 1e4))
    ref, bound = _ref(dY, codes, scales, zeros, G, dtype, case is not GENERAL)
    _check(_run(dY, qw, scales, zeros, G, k), ref, bound)


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("scale", [2e-8, 3e-6, 1e-5, 3e-5, 1e-4, 1e-3, 0.02, 1.0, 40.0, 7e4])
def test_weights_one_by_one(scale, dtype):
    # rows of dY with a single power of two give the weights themselves: one rounding each
    n, k, G = 256, 512, 64
    scales = _scales(n, k, G, 13, 0.6 * scale, 1.4 * scale)
    _, qw, codes, zeros = _inputs(n, k, G, 1, dtype, scales, 14)
    y = 2.0 ** max(-14, min(14, round(-torch.tensor(scale).log2().item())))
    dY = (torch.eye(n, device="cuda") * y).to(dtype)
    col = torch.arange(k, device="cuda") // G
    s, d = scales.to(D)[:, col], codes.to(D) - zeros.to(D)[:, col]
    u = U[dtype]
    # the two-part scale's square, the range's share (f16), and half a step of f16's subnormals
    # where the result itself is that small
    bound = (u + 2 * u * u) * (s * d * y).abs() + 2.0 ** -25
    if dtype == H:
        bound = bound + 2.0 ** -19 * (d.abs() + 2) * s.amax(0) * y
    _check(_run(dY, qw, scales, zeros, G, k), s * d * y, bound)


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("case", [ONE, SPLIT, TWO, GENERAL], ids=["one", "split", "two", "general"])
def test_scales_of_mixed_sizes(case, dtype):
    # within a group from 1e-7 to 1, rows of scale zero, and groups far apart from each other
    n, k, G, m = case
    scales = _scales(n, k, G, 3, 1e-7, 1.0)
    scales[::7] = 0.0
    scales[:, 1] *= 1e-4
    scales[:, -1] *= 3.0
    scales[:, 0] = 0.0
    dY, qw, codes, zeros = _inputs(n, k, G, m, dtype, scales, 4)
    ref, bound = _ref(dY, codes, scales, zeros, G, dtype, case is not GENERAL)
    got = _run(dY, qw, scales, zeros, G, k)
    _check(got, ref, bound)
    assert (got[:, :G] == 0).all()
    for _ in range(20):
        assert torch.equal(_run(dY, qw, scales, zeros, G, k), got)


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("case", [ONE, SPLIT, TWO, GENERAL], ids=["one", "split", "two", "general"])
@pytest.mark.parametrize("scale", [0.01, 1e-6])
def test_zeros_out_of_range(case, scale, dtype):
    # the tensor-core kernel holds zeros up to +-127 exactly; a group that has another is NaN.
    # The general kernel takes any.
    n, k, G, m = case
    scales = _scales(n, k, G, 5, 0.6 * scale, 1.4 * scale)
    dY, qw, codes, zeros = _inputs(n, k, G, m, dtype, scales, 6, min(0.01 / scale, 1e3))
    ng = zeros.shape[1]
    zeros[n - 1, 0] = 127
    zeros[3, 0] = -127
    zeros[5, 1] = 300
    zeros[n // 2, ng - 1] = -128
    zeros[7, ng - 2] = 1 << 30
    got = _run(dY, qw, scales, zeros, G, k)
    ref, bound = _ref(dY, codes, scales, zeros, G, dtype, case is not GENERAL)
    if case is GENERAL:
        ok = ref.abs() < 6e4
        _check(got[ok], ref[ok], bound[ok])
        return
    bad = torch.zeros(k, dtype=torch.bool, device="cuda")
    for g in (1, ng - 2, ng - 1):
        bad[g * G:(g + 1) * G] = True
    assert got[:, bad].isnan().all()
    _check(got[:, ~bad], ref[:, ~bad], bound[:, ~bad])


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("case", [ONE, SPLIT, TWO, GENERAL], ids=["one", "split", "two", "general"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_nonfinite_scales_stay_in_their_group(case, bad, dtype):
    n, k, G, m = case
    scales = _scales(n, k, G, 7, 1e-3, 2e-2)
    dY, qw, codes, zeros = _inputs(n, k, G, m, dtype, scales, 8)
    dY[dY == 0] = 0.125
    ref, bound = _ref(dY, codes, scales, zeros, G, dtype, case is not GENERAL)
    scales[9, 1] = bad
    got = _run(dY, qw, scales, zeros, G, k)
    mine = torch.zeros(k, dtype=torch.bool, device="cuda")
    mine[G:2 * G] = True
    _check(got[:, ~mine], ref[:, ~mine], bound[:, ~mine])
    want, _ = _ref(dY, codes, scales, zeros, G, dtype, False)
    want = want[:, mine]
    assert not torch.isfinite(want).any()
    assert torch.equal(got[:, mine].isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[:, mine][inf].to(D), want[inf])


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("n,k,G,m", [
    (712, 7200, 32, 1000), (712, 7200, 96, 1000), (1000, 4896, -1, 1200), (520, 2336, 32, 2000),
    (1000, 5792, 160, 1100), (1000, 9376, 128, 700), (8, 11008, -1, 333), (72, 16672, 4192, 400)])
def test_two_column_tiles(n, k, G, m, dtype):
    # every one of these takes two 128-column tiles per CTA, most with the second one part-filled
    assert _shape(n, k, m)[0] == 2
    scales = _scales(n, k, G, 9, 1e-3, 2e-2)
    dY, qw, codes, zeros = _inputs(n, k, G, m, dtype, scales, 10)
    ref, bound = _ref(dY, codes, scales, zeros, G, dtype, True)
    got = _run(dY, qw, scales, zeros, G, k)
    _check(got, ref, bound)
    # rows padded, the padding kept
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    xp = torch.full((m, k + 5), 3.0, dtype=dtype, device="cuda")
    quant_matmul_dgrad(dY, qw, scales, zeros, 4, G, k, out=xp[:, :k])
    assert torch.equal(xp[:, :k], got) and (xp[:, k:] == 3.0).all()


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("n,k,G,m,gidx", [(300, 416, 8, 65, False), (33, 256, 128, 40, False),
                                          (128, 256, 12, 40, False), (80, 1024, 128, 90, True)])
def test_general_kernel_keeps_fp32_weights(n, k, G, m, gidx, dtype):
    # groups that are no multiple of 32, odd rows, g_idx: no 16-bit rounding of the weights
    from post_weight_quantization_23_b200 import quant_matmul_dgrad
    scales = _scales(n, k, G, 11, 1e-3, 2e-2)
    dY, qw, codes, zeros = _inputs(n, k, G, m, dtype, scales, 12)
    ref, bound = _ref(dY, codes, scales, zeros, G, dtype, False)
    gi = (torch.arange(k, device="cuda") // G).to(torch.int32) if gidx else None
    _check(quant_matmul_dgrad(dY, qw, scales, zeros, 4, G, k, gi), ref, bound)
    if gidx or G % 32:  # and with rows of dY on 16-byte boundaries
        yp = torch.full((m, _cdiv(n, 8) * 8 + 8), float("nan"), dtype=dtype, device="cuda")
        yp[:, :n] = dY
        _check(quant_matmul_dgrad(yp[:, :n], qw, scales, zeros, 4, G, k, gi), ref, bound)
