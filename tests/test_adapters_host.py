"""CPU checks of the adapter, checkpoint and input-gradient operators: the C ABI's
refusals (no device work), the extension module's, and the integer steps of the kernels."""

import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import post_weight_quantization_23_b200 as P
from post_weight_quantization_23_b200 import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 4, 5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from post_weight_quantization_23_b200 import build
        build.build()
    return _lib.load()


def p(v):
    return ctypes.c_void_p(v)  # never dereferenced: every call below ends at a host check


A, B, X, Y, OUT, S, ST, AD, V = (p((i + 1) << 32) for i in range(9))


def _add(lib, **kw):
    v = dict(Y=Y, ldy=64, X=X, dt=1, m=4, k=64, ldx=64, A=A, B=B, S=S, na=2, r=16, st=ST, ad=AD,
             nreq=2, n=64, out=OUT, ldo=64, V=None)
    v.update(kw)
    return lib.gptq_lora_add(v["Y"], v["ldy"], v["X"], v["dt"], v["m"], v["k"], v["ldx"], v["A"], v["B"],
                             v["S"], v["na"], v["r"], v["st"], v["ad"], v["nreq"], v["n"], v["out"],
                             v["ldo"], v["V"], None)


def test_lora_add_refusals(lib):
    for kw, want in (
            (dict(dt=0), UNSUPPORTED), (dict(dt=9), INVALID), (dict(r=4), UNSUPPORTED),
            (dict(r=20), UNSUPPORTED), (dict(r=136), UNSUPPORTED), (dict(m=-1), INVALID),
            (dict(m=1 << 27), INVALID), (dict(k=0), INVALID), (dict(n=-1), INVALID),
            (dict(na=0), INVALID), (dict(na=65536), INVALID), (dict(nreq=-1), INVALID),
            (dict(nreq=4 + 65537), INVALID), (dict(X=None), INVALID), (dict(A=None), INVALID),
            (dict(B=None), INVALID), (dict(S=None), INVALID), (dict(st=None), INVALID),
            (dict(ad=None), INVALID), (dict(out=None), INVALID), (dict(ldx=63), INVALID),
            (dict(ldo=63), INVALID), (dict(ldy=63), INVALID), (dict(X=p(3)), INVALID),
            (dict(V=p(6)), INVALID), (dict(st=p(2)), INVALID),
            (dict(out=X), INVALID),                       # out over X
            (dict(out=p((4 << 32) + 64)), INVALID),       # out over part of Y
            (dict(out=Y, ldo=72), INVALID),               # in place with another row stride
            (dict(m=0), OK), (dict(n=0), OK), (dict(nreq=0), OK)):
        assert _add(lib, **kw) == want, kw


def test_lora_backward_refusals(lib):
    def back(**kw):
        v = dict(dY=Y, dt=2, m=4, n=64, ldy=64, X=X, ldx=128, xs=None, k=128, V=V, A=A, B=B, S=S, na=2,
                 r=16, st=ST, ad=AD, nreq=2, dX=OUT, ldd=128, out=OUT, ldo=128, dA=p(11 << 32),
                 dB=p(12 << 32), ws=p(13 << 32), nb=1 << 20)
        v.update(kw)
        return lib.gptq_lora_backward(v["dY"], v["dt"], v["m"], v["n"], v["ldy"], v["X"], v["ldx"],
                                      v["xs"], v["k"], v["V"], v["A"], v["B"], v["S"], v["na"], v["r"],
                                      v["st"], v["ad"], v["nreq"], v["dX"], v["ldd"], v["out"], v["ldo"],
                                      v["dA"], v["dB"], v["ws"], v["nb"], None)

    for kw, want in (
            (dict(dt=0), UNSUPPORTED), (dict(r=12), UNSUPPORTED), (dict(n=0), INVALID),
            (dict(dY=None), INVALID), (dict(X=None), INVALID), (dict(V=None), INVALID),
            (dict(dA=None), INVALID), (dict(dB=None), INVALID), (dict(ldy=63), INVALID),
            (dict(ldx=127), INVALID), (dict(ldo=127), INVALID), (dict(ldd=127), INVALID),
            (dict(out=Y, dX=None, ldo=128), INVALID),     # out over dY
            (dict(out=X, dX=None), INVALID),              # out over X
            (dict(dX=p((5 << 32) + 256)), INVALID),       # out over part of dX
            (dict(ws=None), WORKSPACE), (dict(nb=128), WORKSPACE), (dict(ws=p(100)), WORKSPACE)):
        assert back(**kw) == want, kw
    assert _lib.workspace_size(_lib.OP_LORA_BACKWARD, 16, 0, 100, None) == 6400
    assert _lib.workspace_size(_lib.OP_LORA_BACKWARD, 16, 0, 1, None) == 256
    assert _lib.workspace_size(_lib.OP_LORA_BACKWARD, 16, 0, 1 << 27, None) == 0


def test_checkpoint_refusals(lib):
    f = lib.gptq_act_checkpoint
    assert f(X, 7, 4, 64, 64, A, 64, S, None) == INVALID
    assert f(None, 1, 4, 64, 64, A, 64, S, None) == INVALID
    assert f(X, 1, 4, 64, 63, A, 64, S, None) == INVALID
    assert f(X, 1, 4, 64, 64, A, 63, S, None) == INVALID
    assert f(X, 1, 4, 64, 64, X, 64, S, None) == INVALID  # codes over X
    assert f(X, 1, 1 << 27, 64, 64, A, 64, S, None) == INVALID
    assert f(X, 1, 0, 64, 64, A, 64, S, None) == OK
    assert f(X, 1, 4, 0, 0, A, 0, S, None) == OK
    f = lib.gptq_act_restore
    assert f(A, 64, S, 4, 64, 5, X, 64, None) == INVALID
    assert f(A, 64, None, 4, 64, 1, X, 64, None) == INVALID
    assert f(A, 63, S, 4, 64, 1, X, 64, None) == INVALID
    assert f(A, 64, S, 4, 64, 1, A, 64, None) == INVALID
    assert f(A, 64, S, 0, 64, 1, X, 64, None) == OK


def test_dgrad_refusals(lib):
    def d(dY=Y, dt=1, m=4, n=64, ldy=64, qw=A, sc=S, ze=B, gi=None, k=256, bits=4, G=128, ng=2, dX=OUT,
          ldx=256):
        return lib.gptq_gemm_dgrad(dY, dt, m, n, ldy, qw, sc, ze, gi, k, bits, G, ng, dX, ldx, None)

    for kw, want in (
            (dict(dt=0), UNSUPPORTED), (dict(bits=5), UNSUPPORTED), (dict(k=250), INVALID),
            (dict(m=-1), INVALID), (dict(m=131071), INVALID), (dict(G=0), INVALID), (dict(G=-2), INVALID),
            (dict(ng=3), INVALID), (dict(ldy=63), INVALID), (dict(ldx=255), INVALID),
            (dict(dX=None), INVALID), (dict(dY=None), INVALID), (dict(qw=None), INVALID),
            (dict(sc=None), INVALID), (dict(ze=None), INVALID), (dict(dX=Y), INVALID),
            (dict(m=0), OK), (dict(k=0, ldx=0, ng=0), OK)):
        assert d(**kw) == want, kw


def test_python_refuses_cpu_tensors_and_wrong_arguments(lib):
    z = torch.zeros(4, 64).half()
    ad = dict(A=torch.zeros(2, 16, 64).half(), B=torch.zeros(2, 64, 16).half(), scaling=torch.ones(2),
              starts=torch.zeros(3, dtype=torch.int32), adapter=torch.zeros(2, dtype=torch.int32))
    for call in (lambda: P.act_checkpoint(z), lambda: P.act_restore(z.char(), torch.zeros(4, 1)),
                 lambda: P.lora_add(z, z, **ad), lambda: P.lora_add(z, None, **ad),
                 lambda: P.lora_add("y", z, **ad),
                 lambda: P.lora_backward(z, z, torch.zeros(4, 16), **ad, dX=z),
                 lambda: P.quant_matmul_dgrad(z, z, z, z, 4, 128, 64),
                 lambda: P.quant_matmul_dgrad(z, z, z, z, "4", 128, 64),
                 lambda: P.act_restore(z.char(), torch.zeros(4, 1), "float16")):
        with pytest.raises(P.GptqError):
            call()
    try:
        P.act_checkpoint(z)
    except P.GptqError as e:
        assert e.status == INVALID and "gptq_act_checkpoint" in str(e) and "X" in str(e)


# ---------------------------------------------------------------- integer steps of the kernels


def test_division_by_multiplication():
    # the checkpoint kernels' quotient by the vectors of a row: exact below 2^31
    g = np.random.default_rng(0)
    for d in [1, 2, 3, 7, 16, 48, 1376, 1 << 16, (1 << 16) + 16, 131072, (1 << 30) + 5]:
        shift = 0
        while (1 << shift) < d:
            shift += 1
        mul = ((1 << 32) * ((1 << shift) - d)) // d + 1
        assert mul < 1 << 32
        n = np.concatenate([g.integers(0, 1 << 31, 20000), np.arange(0, 3 * d if d < 1000 else 1000),
                            (np.arange(1, 2000) * d)[np.arange(1, 2000) * d < (1 << 31)],
                            (np.arange(1, 2000) * d - 1)[np.arange(1, 2000) * d < (1 << 31)],
                            [(1 << 31) - 1]]).astype(object)
        q = [(((mul * int(x)) >> 32) + int(x)) >> shift for x in n]
        assert q == [int(x) // d for x in n], d


def test_codes_to_bf16_pairs():
    # 128 + low seven bits minus 128 or 256 in bf16: every int8 exactly
    for c in range(-128, 128):
        b = c & 0xFF
        h = torch.tensor([0x4300 | (b & 0x7F)], dtype=torch.int16).view(torch.bfloat16)
        z = torch.tensor([0x4300 | (b & 0x80)], dtype=torch.int16).view(torch.bfloat16)
        assert float(h - z) == c


def test_codes_by_the_rounding_constant():
    # x * inv + 1.5 * 2^23 rounded once (spacing 1 there, the constant even) is the nearest
    # integer, halves to even, and its low byte the code; in exact fractions, since neither
    # fp32 nor fp64 holds the sum
    g = np.random.default_rng(1)
    top = np.float32(g.uniform(0.5, 2, 4000))
    x = (top * g.choice([1.0, 0.5, -0.5, 1.0 / 127, 63.5 / 127, 0.3], 4000)).astype(np.float32)
    inv = (np.float32(127) / top).astype(np.float32)
    for xi, fi in zip(x, inv):
        exact = Fraction(float(xi)) * Fraction(float(fi))
        fused = np.float32(float(round(exact + 12582912)))  # an integer below 2^24: exact
        assert abs(round(exact)) <= 127
        assert int(fused.view(np.int32)) - 0x4B400000 == round(exact)
        assert np.uint8(int(fused.view(np.int32)) & 0xFF).view(np.int8) == round(exact)


def test_scale_split_gives_one_rounding():
    # w = fl(d * hi + fl(d * lo)) with s = hi + lo to 16 bits more: within a rounding of d * s
    g = torch.Generator().manual_seed(0)
    for dt, u in ((torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -8)):
        s = torch.rand(20000, generator=g) * 0.02 + 1e-3
        d = torch.randint(-15, 16, (20000,), generator=g).double()
        hi = s.to(dt).float()
        lo = (s - hi).to(dt)
        t = (d * lo.double()).to(dt).double()
        w = (d * hi.double() + t).to(dt).double()  # a fused multiply-add rounds once
        # f16 holds lo to 2^-25 absolutely
        assert ((w - d * s.double()).abs() <= (u + u * u) * (d * s.double()).abs()
                + 2.0 ** -25 * d.abs() + 2.0 ** -25).all()


def _pieces(starts, adapter, m, na, lo, hi):
    """The decode kernel's pieces (windows of 256 requests, eight rows of one adapter each)."""
    out = []
    for q0 in range(0, len(adapter), 256):
        before, rows = {}, {}
        for q in range(q0, min(q0 + 256, len(adapter))):
            b, e = (min(max(v, 0), m) for v in starts[q:q + 2])
            n = e - b if lo <= e - b <= hi else 0
            a = adapter[q] if 0 <= adapter[q] < na else -1
            rows.setdefault(a, []).extend(range(b, b + n))
            before[q] = (a, len(rows[a]) - n, n, b)
        # each request owns the pieces whose first row (rank 8 i) is its own
        for q, (a, r0, n, b) in before.items():
            own = -(-(r0 + n) // 8) - -(-r0 // 8) if n > 0 else 0
            for i in range(own):
                first = (-(-r0 // 8) + i) * 8
                out.append((a, rows[a][first:first + 8]))
    return out


def test_decode_pieces_cover_every_row_once():
    g = np.random.default_rng(2)
    for nreq in (1, 7, 64, 255, 256, 257, 900):
        lens = g.integers(0, 30, nreq)
        starts = [3, *(3 + np.cumsum(lens))]
        adapter = g.integers(-2, 9, nreq).tolist()
        m = starts[-1] + 5
        for lo, hi in ((1, m), (1, 24), (25, m)):
            got = sorted(r for _, rows in _pieces(starts, adapter, m, 8, lo, hi) for r in rows)
            want = sorted(r for q in range(nreq) if lo <= lens[q] <= hi
                          for r in range(starts[q], starts[q + 1]))
            assert got == want
            owner = {r: adapter[q] if 0 <= adapter[q] < 8 else -1 for q in range(nreq)
                     for r in range(starts[q], starts[q + 1])}
            assert all(owner[r] == a for a, rows in _pieces(starts, adapter, m, 8, lo, hi) for r in rows)
            # the grid of the launch is a bound on their number
            n = len(_pieces(starts, adapter, m, 8, lo, hi))
            assert n <= min(m, m // 8 + nreq, nreq * -(-min(hi, m) // 8))
