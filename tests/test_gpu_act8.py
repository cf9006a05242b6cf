"""8-bit activation checkpoints (gptq_act_checkpoint, gptq_act_restore) against the
definition in 64 bits: codes and scales bit for bit, restored values rounded once."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = [torch.float32, torch.float16, torch.bfloat16]


def _ref(X):
    """codes, scales, restored values in 64 bits (scale and factor are fp32 by definition)."""
    x = X.double()
    m, k = x.shape
    codes = torch.zeros(m, k, dtype=torch.int64, device=X.device)
    scales = []
    vals = torch.zeros_like(x)
    for c in range(0, k, 128):
        b = x[:, c:c + 128]
        top = b.abs().amax(1, keepdim=True).float()
        one = torch.full_like(top, 127.0)
        tiny = top < 2.0 ** -100
        inv = torch.where(tiny, torch.zeros_like(top), one / top)
        sc = torch.where(tiny, torch.zeros_like(top), top / one)
        q = (b * inv.double()).round()  # the product of two fp32 values is exact in 64 bits
        codes[:, c:c + 128] = q.long()
        vals[:, c:c + 128] = q * sc.double()
        scales.append(sc)
    return codes, torch.cat(scales, 1), vals


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (1, 128), (5, 129), (64, 4096), (33, 1000),
                                 (2, 11008), (700, 264), (1, 100000)])
def test_round_trip(m, k, dtype):
    from post_weight_quantization_23_b200 import act_checkpoint, act_restore
    g = torch.Generator(device="cuda").manual_seed(m * 7 + k)
    X = (torch.randn(m, k, generator=g, device="cuda") *
         torch.exp(2 * torch.randn(k, generator=g, device="cuda"))).to(dtype)
    # halves: every block holds half of its largest value (a code of 63.5 before rounding)
    c = torch.arange(0, k, 128, device="cuda")
    top = torch.full((m, len(c)), 127.0, device="cuda", dtype=dtype) * 2
    X[:, c] = top
    X[:, (c + 1).clamp_max(k - 1)] = top / 2
    codes, scales = act_checkpoint(X)
    rc, rs, rv = _ref(X)
    assert torch.equal(codes.long(), rc) and torch.equal(scales, rs)
    for out in DT:
        got = act_restore(codes, scales, out)
        # one fp32 product, one rounding to the type: exactly the rounding of the fp32 product
        assert torch.equal(got, (rc.float() * rs.repeat_interleave(128, 1)[:, :k]).to(out))
        err = (got.double() - rv).abs()
        u = torch.finfo(out).eps / 2
        assert (err <= (u + 2.0 ** -23) * rv.abs() + 2.0 ** -25).all()
    # half a step, and |x| times how far scale * factor is from 1 (two roundings): 127 * 2^-23 steps
    step = rs.double().repeat_interleave(128, 1)[:, :k]
    assert ((rv - X.double()).abs() <= 0.5 * step * (1 + 2.0 ** -14)).all()


def test_largest_value_and_half_ties():
    # top = 254: scale 2 and factor 1/2 exactly, odd values sit on halves and go to even codes
    from post_weight_quantization_23_b200 import act_checkpoint
    X = torch.arange(-127, 128, device="cuda").float()[None, :128].half()
    X[0, 127] = 254
    codes, scales = act_checkpoint(X)
    assert scales.item() == 2.0
    assert torch.equal(codes.double(), (X.double() / 2).round())


@pytest.mark.parametrize("dtype", DT)
def test_special_blocks(dtype):
    from post_weight_quantization_23_b200 import act_checkpoint, act_restore
    X = torch.ones(6, 260, device="cuda", dtype=dtype)
    X[0] = 0                       # zeros
    X[1, 5] = float("nan")         # NaN in the first block only
    X[2, 200] = float("-inf")      # infinity in the second
    if dtype != torch.float16:
        X[3] = 1e-38               # below 2^-100: stored as zeros
    X[4] = torch.finfo(dtype).max
    X[5] = -torch.finfo(dtype).max
    codes, scales = act_checkpoint(X)
    back = act_restore(codes, scales, torch.float32)
    assert not back[0].any() and not scales[0].any()
    assert back[1, :128].isnan().all() and (back[1, 128:] == 1).all()
    assert (back[2, :128] == 1).all() and back[2, 128:256].isnan().all() and (back[2, 256:] == 1).all()
    if dtype != torch.float16:
        assert not back[3].any()
    top = float(torch.finfo(dtype).max)
    assert ((back[4].double() / top - 1).abs() <= 2.0 ** -23).all()
    assert (codes[4] == 127).all() and (codes[5] == -127).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("pads", [(8, 16, 8), (1, 3, 5)])
def test_strides(dtype, pads):
    from post_weight_quantization_23_b200 import act_checkpoint, act_restore
    m, k = 37, 300
    xp, cp, op = pads
    X = torch.randn(m, k + xp, device="cuda").to(dtype)
    codes = torch.full((m, k + cp), 99, dtype=torch.int8, device="cuda")
    c, s = act_checkpoint(X[:, 1:1 + k] if xp == 1 else X[:, :k], codes=codes[:, :k])
    rc, rs, _ = _ref((X[:, 1:1 + k] if xp == 1 else X[:, :k]).contiguous())
    assert torch.equal(codes[:, :k].long(), rc) and torch.equal(s, rs)
    assert (codes[:, k:] == 99).all()
    out = torch.full((m, k + op), 5.0, dtype=dtype, device="cuda")
    act_restore(codes[:, :k], s, out=out[:, :k])
    assert torch.equal(out[:, :k], (rc.float() * rs.repeat_interleave(128, 1)[:, :k]).to(dtype))
    assert (out[:, k:] == 5.0).all()


def test_offsets_past_32_bits():
    from post_weight_quantization_23_b200 import act_checkpoint, act_restore
    m, k = 140000, 16384  # 2.3e9 elements
    X = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    X[-3:] = torch.randn(3, k, device="cuda").bfloat16()
    codes, scales = act_checkpoint(X)
    rc, rs, _ = _ref(X[-3:])
    assert torch.equal(codes[-3:].long(), rc) and torch.equal(scales[-3:], rs)
    assert not codes[:-3].any()
    del X
    back = act_restore(codes, scales, torch.bfloat16)
    assert torch.equal(back[-3:], (rc.float() * rs.repeat_interleave(128, 1)).bfloat16())


def test_empty_and_refusals():
    from post_weight_quantization_23_b200 import GptqError, act_checkpoint, act_restore
    c, s = act_checkpoint(torch.zeros(0, 64, device="cuda"))
    assert c.shape == (0, 64) and act_restore(c, s).shape == (0, 64)
    X = torch.zeros(4, 64, device="cuda")
    codes, scales = act_checkpoint(X)
    for call in (lambda: act_checkpoint(X.double()), lambda: act_checkpoint(X.cpu()),
                 lambda: act_checkpoint(X.T), lambda: act_checkpoint(X, codes=codes[:3]),
                 lambda: act_checkpoint(X, codes=codes.float()),
                 lambda: act_checkpoint(X, scales=scales.half()),
                 lambda: act_restore(codes, scales[:3]), lambda: act_restore(codes, scales, torch.int8),
                 lambda: act_restore(codes, scales, out=torch.zeros(4, 63, device="cuda")),
                 lambda: act_checkpoint(codes)):
        with pytest.raises(GptqError):
            call()
