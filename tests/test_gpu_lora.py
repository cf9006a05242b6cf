"""The adapters of many requests (gptq_lora_add, gptq_lora_backward) against plain
64-bit implementations, with bounds derived from the kernels' arithmetic
(tests/_adapters.py)."""

import pytest
import torch

import _adapters as R

pytestmark = pytest.mark.gpu

H, BF = torch.float16, torch.bfloat16

# (dtype, k, n, rank, adapters, request lengths, adapter of each, rows before, rows behind)
CASES = [
    (BF, 4096, 4096, 16, 8, [1], [3], 0, 0),                      # one token
    (H, 64, 64, 8, 1, [1], [0], 0, 0),                            # the smallest rank
    (H, 512, 768, 16, 4, [1] * 13, [0, 1, 2, 3, -1, 4, 0, 0, 1, 7, -5, 2, 3], 0, 0),  # decode, some bare
    (BF, 1024, 520, 32, 3, [0, 1, 0, 0, 9, 8, 7, 0], [0, 1, 2, 0, 1, 2, 0, 1], 3, 5),  # empty requests
    (H, 72, 33, 24, 2, [17, 1, 40], [1, 0, 1], 2, 9),             # odd n: rows off 16 bytes
    (BF, 4136, 1000, 40, 2, [5, 130, 1], [0, 1, -1], 1, 1),       # rank 40, ragged k and n
    (H, 2048, 640, 64, 3, [300, 1, 1, 129], [2, 0, 1, 2], 0, 7),
    (BF, 768, 2056, 128, 2, [128, 64, 257], [1, 0, 1], 0, 0),     # the largest rank
    (H, 136, 264, 72, 2, [70, 3], [0, 1], 0, 2),                  # rank 72
    (BF, 8, 8, 8, 1, [3], [0], 0, 0),                             # the narrowest layer
    (BF, 11008, 256, 16, 1, [600], [0], 0, 0),
    (H, 256, 11008, 16, 5, [33] * 9 + [1] * 40, [i % 6 - 1 for i in range(49)], 4, 4),
    (BF, 320, 320, 48, 4, [1000], [2], 0, 24),
]
IDS = [f"{'f16' if c[0] == H else 'bf16'}_k{c[1]}_n{c[2]}_r{c[3]}_m{sum(c[5])}" for c in CASES]


def _make(c, seed=0):
    dtype, k, n, r, na, lens, ids, first, tail = c
    return R.make(dtype, k, n, r, na, lens, ids, seed + k + n + r, first, tail)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_add(case):
    from post_weight_quantization_23_b200 import lora_add
    s = _make(case)
    ref, bound, Vr, bv, cov = R.add_ref(s, case[0])
    out = torch.full_like(s["Y"], 7.0)
    V = torch.full((s["Y"].shape[0], case[3]), 5.0, device="cuda")
    before = {k: v.clone() for k, v in s.items()}
    lora_add(s["Y"], s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"], out=out, V=V)
    torch.cuda.synchronize()
    r = R.check(out[cov], ref[cov], bound[cov], "out")
    r2 = R.check(V[cov], Vr[cov], bv[cov], "V")
    print("max err / bound", r, r2)
    assert (out[~cov] == 7.0).all() and (V[~cov] == 5.0).all()  # rows of no request
    for k, v in before.items():
        assert torch.equal(s[k], v), k
    # in place, without V: the same bits
    Y = s["Y"].clone()
    got = lora_add(Y, s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    assert got is Y
    assert torch.equal(Y[cov], out[cov]) and torch.equal(Y[~cov], s["Y"][~cov])


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_add_without_y(case):
    from post_weight_quantization_23_b200 import lora_add
    s = _make(case, 1)
    ref, bound, _, _, cov = R.add_ref(s, case[0], with_y=False)
    out = torch.full_like(s["Y"], 7.0)
    lora_add(None, s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"], out=out)
    R.check(out[cov], ref[cov], bound[cov], "out")
    assert (out[~cov] == 7.0).all()


@pytest.mark.parametrize("xoff,ypad", [(0, 8), (0, 3), (3, 5), (8, 0)])
@pytest.mark.parametrize("lens", [[1, 4, 2], [200, 1, 77]])
def test_add_strided(xoff, ypad, lens):
    # padded rows: X on and off 16-byte boundaries, Y and out with odd strides, the padding kept
    from post_weight_quantization_23_b200 import lora_add
    s = R.make(BF, 264, 72, 16, 2, lens, [1, -1, 0], 5)
    ref, bound, _, _, cov = R.add_ref(s, BF)
    m = s["X"].shape[0]
    Xp = torch.full((m, 264 + xoff), float("nan"), dtype=BF, device="cuda")
    Xp[:, :264] = s["X"]
    Yp = torch.full((m, 72 + ypad), 3.0, dtype=BF, device="cuda")
    Yp[:, :72] = s["Y"]
    lora_add(Yp[:, :72], Xp[:, :264], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    R.check(Yp[:, :72][cov], ref[cov], bound[cov], "out")
    assert (Yp[:, 72:] == 3.0).all()


@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("lens", [[2, 1, 3], [140, 30, 150]])
def test_add_nonfinite_neighbours(dtype, lens):
    # NaN and infinity in one request's rows, in uncovered rows and in another adapter stay there
    from post_weight_quantization_23_b200 import lora_add
    s = R.make(dtype, 128, 136, 16, 3, lens, [0, 1, 0], 9, first=2, tail=3)
    ref, bound, _, _, cov = R.add_ref(s, dtype)
    b1, e1 = 2 + lens[0], 2 + lens[0] + lens[1]
    s["X"][b1:e1] = float("nan")
    s["X"][:2] = float("inf")
    s["X"][e1 + lens[2]:] = float("nan")
    s["A"][2] = float("nan")
    s["B"][2] = float("inf")
    out = lora_add(s["Y"].clone(), s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    keep = cov.clone()
    keep[b1:e1] = False
    R.check(out[keep], ref[keep], bound[keep], "out")
    assert out[b1:e1].isnan().all()
    assert torch.equal(out[~cov], s["Y"][~cov])


@pytest.mark.parametrize("lens", [[1, 1], [150, 90]])
def test_add_f16_range(lens):
    # V far above and far below f16's range: each row is scaled by its own power of two
    from post_weight_quantization_23_b200 import lora_add
    s = R.make(H, 256, 64, 16, 2, lens, [0, 1], 3)
    s["X"] *= 100
    s["scaling"] = torch.tensor([3.0e5, 3.0e-9], device="cuda")
    s["B"][0] *= 1e-4
    s["Y"].zero_()
    ref, bound, _, _, cov = R.add_ref(s, H)
    out = lora_add(s["Y"].clone(), s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    R.check(out, ref, bound, "out")


def test_add_repeats_bit_for_bit():
    from post_weight_quantization_23_b200 import lora_add
    s = R.make(BF, 2048, 512, 32, 4, [1] * 20 + [300, 77], [i % 4 for i in range(22)], 2)
    a = (s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    first = lora_add(s["Y"].clone(), *a)
    for _ in range(5):
        assert torch.equal(lora_add(s["Y"].clone(), *a), first)


def test_add_bad_requests_stay_inside():
    # starts outside [0, m], descending: no row outside the batch is touched
    from post_weight_quantization_23_b200 import lora_add
    for lens in ([5, 4], [150, 40]):
        m = sum(lens)
        s = R.make(H, 64, 64, 16, 2, lens, [0, 1], 4)
        for bad in ([-7, 3, m + 9], [m, 2, 1], [m + 5, m + 6, m + 7], [-9, -8, -1]):
            st = torch.tensor(bad, dtype=torch.int32, device="cuda")
            big = torch.full((m + 8, 64), 2.0, dtype=H, device="cuda")
            big[4:4 + m] = s["Y"]
            lora_add(big[4:4 + m], s["X"], s["A"], s["B"], s["scaling"], st, s["adapter"])
            torch.cuda.synchronize()
            assert (big[:4] == 2.0).all() and (big[4 + m:] == 2.0).all()


def test_add_offsets_past_32_bits():
    # rows whose element offset passes 2^31
    from post_weight_quantization_23_b200 import lora_add
    m, n, k = 70000, 32768, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    Y = torch.zeros(m, n, dtype=BF, device="cuda")
    X = torch.randn(m, k, generator=g, device="cuda").to(BF)
    A = (torch.randn(1, 16, k, generator=g, device="cuda") / 8).to(BF)
    B = (torch.randn(1, n, 16, generator=g, device="cuda") * 0.05).to(BF)
    sc = torch.ones(1, device="cuda")
    st = torch.tensor([m - 300, m - 4, m - 1], dtype=torch.int32, device="cuda")
    ad = torch.zeros(2, dtype=torch.int32, device="cuda")
    lora_add(Y, X, A, B, sc, st, ad)
    s = dict(X=X[-300:], Y=torch.zeros(300, n, device="cuda"), A=A, B=B, scaling=sc, starts=st - (m - 300),
             adapter=ad)
    ref, bound, _, _, cov = R.add_ref(s, BF)
    R.check(Y[-300:][cov], ref[cov], bound[cov], "out")
    assert (Y[-1] == 0).all()
    assert not Y[:m - 300].any()


# ---------------------------------------------------------------- backward

BCASES = [
    (BF, 1024, 512, 16, 1, [300], [0], 0, 0),
    (H, 512, 1024, 8, 3, [65, 1, 200, 0, 31], [0, 2, -1, 1, 0], 2, 5),
    (BF, 256, 2056, 64, 2, [129, 64], [1, 1], 0, 3),
    (H, 4128, 256, 32, 2, [1], [1], 0, 0),
    (BF, 136, 72, 128, 2, [190, 70], [0, 1], 1, 0),
    (H, 320, 264, 40, 4, [7, 8, 9, 500], [3, 3, 0, 3], 0, 0),
    (BF, 2048, 2048, 24, 1, [1500], [0], 0, 0),
    (H, 72, 33, 16, 2, [20, 50], [1, 0], 0, 1),   # odd n: dY rows off 16 bytes
    (BF, 8, 8, 8, 1, [3], [0], 0, 0),
]
BIDS = [f"{'f16' if c[0] == H else 'bf16'}_k{c[1]}_n{c[2]}_r{c[3]}_m{sum(c[5])}" for c in BCASES]


def _with_v(s, dtype):
    V = torch.zeros(s["X"].shape[0], s["A"].shape[1], dtype=R.D, device="cuda")
    for b, e, a in R.spans(s, s["A"].shape[0]):
        if a >= 0 and e > b:
            V[b:e] = R.low(s["X"][b:e], s["A"][a], float(s["scaling"][a].double()), False)[0]
    s["V"] = V.float()


@pytest.mark.parametrize("saved", [16, 8])
@pytest.mark.parametrize("case", BCASES, ids=BIDS)
def test_backward(case, saved):
    from post_weight_quantization_23_b200 import act_checkpoint, lora_backward
    dtype = case[0]
    s = _make(case)
    _with_v(s, dtype)
    X, xs, Xd = s["X"], None, s["X"].to(R.D)
    if saved == 8:
        X, xs = act_checkpoint(s["X"])
        Xd = X.to(R.D) * xs.to(R.D).repeat_interleave(128, 1)[:, :case[1]]
    ref = R.backward_ref(s, dtype, Xd)
    out = torch.full_like(s["dX"], 7.0)
    dA, dB = torch.full_like(s["A"], 9.0), torch.full_like(s["B"], 9.0)
    lora_backward(s["dY"], X, s["V"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"],
                  s["dX"], x_scales=xs, out=out, dA=dA, dB=dB)
    torch.cuda.synchronize()
    cov = R.add_ref(s, dtype)[4]
    rs = [R.check(out[cov], ref["out"][0][cov], ref["out"][1][cov], "out"),
          R.check(dA, *ref["dA"], "dA"), R.check(dB, *ref["dB"], "dB")]
    print("max err / bound", rs)
    assert (out[~cov] == 7.0).all()
    # in place, and without an input gradient: the same bits
    dX = s["dX"].clone()
    o2, a2, b2 = lora_backward(s["dY"], X, s["V"], s["A"], s["B"], s["scaling"], s["starts"],
                               s["adapter"], dX, x_scales=xs)
    assert o2 is dX and torch.equal(dX[cov], out[cov]) and torch.equal(dX[~cov], s["dX"][~cov])
    assert torch.equal(a2, dA) and torch.equal(b2, dB)
    o3, a3, b3 = lora_backward(s["dY"], X, s["V"], s["A"], s["B"], s["scaling"], s["starts"],
                               s["adapter"], None, x_scales=xs)
    assert o3 is None and torch.equal(a3, dA) and torch.equal(b3, dB)


def test_backward_against_differences():
    # d/dA, d/dB, d/dX of sum(G * out) by central differences of the 64-bit forward formula
    from post_weight_quantization_23_b200 import lora_add, lora_backward
    s = R.make(H, 64, 40, 8, 2, [70, 9], [1, 0], 8)
    s["A"], s["B"] = s["A"].clone(), s["B"].clone()
    V = torch.zeros(79, 8, device="cuda")
    lora_add(s["Y"].clone(), s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"], V=V)
    dX, dA, dB = lora_backward(s["dY"], s["X"], V, s["A"], s["B"], s["scaling"], s["starts"],
                               s["adapter"], torch.zeros_like(s["X"]))
    G = s["dY"].double()
    v = {k: s[k].double() for k in ("X", "A", "B", "scaling", "Y")}

    def f(w):
        t = 0.0
        for b, e, a in R.spans(s, 2):
            t = t + (G[b:e] * ((w["X"][b:e] @ w["A"][a].T) * w["scaling"][a] @ w["B"][a].T)).sum()
        return t

    g = torch.Generator().manual_seed(0)
    for name, grad in (("X", dX), ("A", dA), ("B", dB)):
        top = grad.double().abs().max()
        for _ in range(12):
            i = tuple(int(torch.randint(0, d, (1,), generator=g)) for d in v[name].shape)
            h = 1e-3
            w = dict(v)
            w[name] = v[name].clone()
            w[name][i] += h
            hi = f(w)
            w[name][i] -= 2 * h
            num = (hi - f(w)) / (2 * h)  # linear in each input: exact up to 64-bit rounding
            # one rounding to f16 and the fp32 sums of at most a few hundred products
            assert abs(num - grad[i].double()) <= 2.0 ** -10 * abs(num) + 2.0 ** -12 * top, (name, i)


@pytest.mark.parametrize("saved", [16, 8])
def test_backward_nonfinite_neighbours(saved):
    # NaN rows of uncovered tokens and of another adapter's request do not leak
    from post_weight_quantization_23_b200 import act_checkpoint, lora_backward
    s = R.make(BF, 256, 128, 16, 3, [70, 33, 90], [0, 1, 0], 3, first=3, tail=4)
    _with_v(s, BF)
    cov = R.add_ref(s, BF)[4]
    bad = torch.ones_like(cov)
    bad[3:73] = bad[106:196] = False
    for name in ("X", "dY", "V"):
        s[name][bad] = float("nan")
    X, xs, Xd = s["X"], None, s["X"].to(R.D)
    if saved == 8:
        X, xs = act_checkpoint(s["X"])
        Xd = X.to(R.D) * xs.to(R.D).repeat_interleave(128, 1)
    ref = R.backward_ref(s, BF, Xd)
    out, dA, dB = lora_backward(s["dY"], X, s["V"], s["A"], s["B"], s["scaling"], s["starts"],
                                s["adapter"], s["dX"].clone(), x_scales=xs)
    good = ~bad
    R.check(out[good], ref["out"][0][good], ref["out"][1][good], "out")
    for i, (got, name) in enumerate(((dA, "dA"), (dB, "dB"))):
        R.check(got[0], ref[name][0][0], ref[name][1][0], name)
        assert got[1].isnan().all() and not got[2].any()


def test_backward_no_requests():
    from post_weight_quantization_23_b200 import lora_backward
    s = R.make(H, 64, 64, 8, 2, [4], [0], 3)
    s["V"] = torch.zeros(4, 8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ad = torch.zeros(0, dtype=torch.int32, device="cuda")
    dX = s["dX"].clone()
    out, dA, dB = lora_backward(s["dY"], s["X"], s["V"], s["A"], s["B"], s["scaling"], st, ad, dX)
    assert torch.equal(dX, s["dX"]) and not dA.any() and not dB.any()


@pytest.mark.parametrize("lens", [[1, 3], [400, 200]])
def test_capture_and_streams(lens):
    # forward and backward captured into a graph, replayed on new data; and on a side stream
    from post_weight_quantization_23_b200 import act_checkpoint, lora_add, lora_backward
    s = R.make(BF, 512, 256, 16, 2, lens, [0, 1], 1)
    m = sum(lens)
    V = torch.zeros(m, 16, device="cuda")
    out, dout = torch.zeros_like(s["Y"]), torch.zeros_like(s["dX"])
    dA, dB = torch.zeros_like(s["A"]), torch.zeros_like(s["B"])
    a = (s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])

    def step():
        codes, xs = act_checkpoint(s["X"])
        lora_add(s["Y"], s["X"], *a, out=out, V=V)
        lora_backward(s["dY"], codes, V, *a, s["dX"], x_scales=xs, out=dout, dA=dA, dB=dB)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (11, 12):
        new = R.make(BF, 512, 256, 16, 2, lens, [1, 0], seed)
        for k in ("X", "Y", "dY", "dX", "A", "B", "scaling", "adapter"):
            s[k].copy_(new[k])
        g.replay()
        got = [t.clone() for t in (out, dout, dA, dB, V)]
        step()
        for x, y in zip(got, (out, dout, dA, dB, V)):
            assert torch.equal(x, y)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        o2 = lora_add(s["Y"].clone(), s["X"], *a, stream=side)
    side.synchronize()
    assert torch.equal(o2, got[0])


def test_refusals():
    from post_weight_quantization_23_b200 import GptqError, lora_add, lora_backward
    s = R.make(H, 64, 64, 16, 2, [4], [0], 3)
    s["V"] = torch.zeros(4, 16, device="cuda")

    def add(**kw):
        v = dict(s, out=None)
        v.update(kw)
        return lora_add(v["Y"], v["X"], v["A"], v["B"], v["scaling"], v["starts"], v["adapter"],
                        out=v["out"])

    def back(**kw):
        v = dict(s, out=None, xs=None)
        v.update(kw)
        return lora_backward(v["dY"], v["X"], v["V"], v["A"], v["B"], v["scaling"], v["starts"],
                             v["adapter"], v["dX"], x_scales=v["xs"], out=v["out"], ws=v.get("ws"))

    f = torch.float32
    for kw in (dict(X=s["X"].float()), dict(A=s["A"].bfloat16()), dict(A=s["A"][:, :12], B=s["B"][:, :, :12]),
               dict(scaling=s["scaling"].half()), dict(starts=s["starts"].long()),
               dict(adapter=s["adapter"][:0]), dict(Y=s["Y"][:3]), dict(Y=s["Y"].T), dict(Y=None),
               dict(X=s["X"].cpu()), dict(out=s["X"]), dict(A=s["A"][:, :, :56]),
               dict(A=s["A"].transpose(1, 2).contiguous().transpose(1, 2)),
               dict(A=s["A"][:, :4], B=s["B"][:, :, :4].contiguous()), dict(out=s["Y"].float())):
        with pytest.raises(GptqError):
            add(**kw)
    for kw in (dict(V=s["V"].half()), dict(V=s["V"][:3]), dict(xs=torch.zeros(4, 1, device="cuda")),
               dict(X=s["X"].to(torch.int8)), dict(dY=s["dY"].to(f)), dict(out=s["dY"]),
               dict(X=s["X"].to(torch.int8), xs=torch.zeros(4, 2, device="cuda")),
               dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda")),
               dict(dX=s["dX"][:, :8])):
        with pytest.raises(GptqError):
            back(**kw)


@pytest.mark.parametrize("dtype,r", [(BF, 16), (BF, 64), (H, 16), (H, 128)])
def test_repeats_under_load(dtype, r):
    # many calls back to back give the same bits (copies land in every order)
    from post_weight_quantization_23_b200 import act_checkpoint, lora_add, lora_backward
    s = R.make(dtype, 2048, 2048, r, 2, [500, 300, 224], [0, 1, 0], r)
    s["V"] = torch.zeros(1024, r, device="cuda")
    a = (s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
    out = torch.empty_like(s["Y"])
    lora_add(s["Y"], s["X"], *a, out=out, V=s["V"])
    first_y, V = out.clone(), s["V"].clone()
    codes, xs = act_checkpoint(s["X"])
    first = {}
    for saved, (X, sc) in ((16, (s["X"], None)), (8, (codes, xs))):
        o = torch.empty_like(s["dX"])
        first[saved] = lora_backward(s["dY"], X, V, *a, s["dX"], x_scales=sc, out=o)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        lora_add(s["Y"], s["X"], *a, out=out, V=s["V"])
        saved, (X, sc) = ((16, (s["X"], None)), (8, (codes, xs)))[i % 2]
        got = lora_backward(s["dY"], X, V, *a, s["dX"], x_scales=sc, out=torch.empty_like(s["dX"]))
        for x, y in zip(got + (out, s["V"]), first[saved] + (first_y, V)):
            bad += (x != y).any()
    assert int(bad) == 0


# ---------------------------------------------------------------- long and crowded batches


@pytest.mark.parametrize("r,m,k,n", [(8, 140000, 64, 64), (128, 10000, 64, 136), (64, 20000, 72, 64)])
def test_many_pieces_per_cluster(r, m, k, n):
    # more pieces than the clusters take at once, more tiles than one look-up holds
    from post_weight_quantization_23_b200 import act_checkpoint, lora_add, lora_backward
    lens = [m // 2 + 1, 3, m - m // 2 - 4 - 77, 77]
    s = R.make(BF, k, n, r, 2, lens, [0, 1, 1, 0], r)
    ref, bound, Vr, bv, cov = R.add_ref(s, BF)
    V = torch.zeros(m, r, device="cuda")
    out = lora_add(s["Y"], s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"],
                   out=torch.empty_like(s["Y"]), V=V)
    R.check(out, ref, bound, "out")
    R.check(V, Vr, bv, "V")
    s["V"] = V
    for saved in (16, 8):
        X, xs, Xd = s["X"], None, s["X"].to(R.D)
        if saved == 8:
            X, xs = act_checkpoint(s["X"])
            Xd = X.to(R.D) * xs.to(R.D).repeat_interleave(128, 1)[:, :k]
        b = R.backward_ref(s, BF, Xd)
        got = lora_backward(s["dY"], X, V, s["A"], s["B"], s["scaling"], s["starts"], s["adapter"],
                            s["dX"], x_scales=xs, out=torch.empty_like(s["dX"]))
        for g, name in zip(got, ("out", "dA", "dB")):
            R.check(g, *b[name], name)


@pytest.mark.parametrize("dtype", [H, BF])
def test_add_many_requests(dtype):
    # 1001 requests over 37 adapters: several windows of the decode kernel, pieces that gather
    # tokens of many requests, some long ones among them
    from post_weight_quantization_23_b200 import lora_add
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 4, (1001,), generator=g).tolist()
    lens[500], lens[77] = 300, 40
    ids = torch.randint(-1, 38, (1001,), generator=g).tolist()
    s = R.make(dtype, 256, 328, 16, 37, lens, ids, 3, first=1, tail=2)
    ref, bound, Vr, bv, cov = R.add_ref(s, dtype)
    V = torch.full((s["X"].shape[0], 16), 5.0, device="cuda")
    out = torch.full_like(s["Y"], 7.0)
    lora_add(s["Y"], s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"], out=out, V=V)
    R.check(out[cov], ref[cov], bound[cov], "out")
    R.check(V[cov], Vr[cov], bv[cov], "V")
    assert (out[~cov] == 7.0).all() and (V[~cov] == 5.0).all()


def test_backward_many_requests_and_adapters():
    from post_weight_quantization_23_b200 import lora_backward
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    ids = torch.randint(-1, 10, (300,), generator=g).tolist()
    s = R.make(H, 136, 200, 16, 9, lens, ids, 5)
    _with_v(s, H)
    ref = R.backward_ref(s, H, s["X"].to(R.D))
    got = lora_backward(s["dY"], s["X"], s["V"], s["A"], s["B"], s["scaling"], s["starts"],
                        s["adapter"], s["dX"], out=torch.empty_like(s["dX"]))
    for x, name in zip(got, ("out", "dA", "dB")):
        R.check(x, *ref[name], name)


def test_backward_unaligned_v():
    # V on a 4-byte boundary: the general gradient kernel
    from post_weight_quantization_23_b200 import lora_backward
    s = R.make(BF, 128, 64, 8, 1, [90], [0], 5)
    _with_v(s, BF)
    buf = torch.zeros(90 * 8 + 1, device="cuda")
    V = buf[1:].view(90, 8)
    V.copy_(s["V"])
    ref = R.backward_ref(s, BF, s["X"].to(R.D))
    got = lora_backward(s["dY"], s["X"], V, s["A"], s["B"], s["scaling"], s["starts"], s["adapter"],
                        s["dX"].clone())
    for x, name in zip(got, ("out", "dA", "dB")):
        R.check(x, *ref[name], name)


def test_two_streams_at_once():
    # two backward passes and a forward call side by side, each with its own workspace
    from post_weight_quantization_23_b200 import lora_add, lora_backward
    ss = []
    for i in range(2):
        s = R.make(BF, 1024, 1024, 32, 2, [700, 400], [0, 1], i)
        _with_v(s, BF)
        a = (s["A"], s["B"], s["scaling"], s["starts"], s["adapter"])
        want = lora_backward(s["dY"], s["X"], s["V"], *a, s["dX"], out=torch.empty_like(s["dX"]))
        y = lora_add(s["Y"], s["X"], *a, out=torch.empty_like(s["Y"]))
        ss.append((s, a, want, y))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for (s, a, want, y), st in zip(ss, streams):
            with torch.cuda.stream(st):
                o = lora_backward(s["dY"], s["X"], s["V"], *a, s["dX"], out=torch.empty_like(s["dX"]))
                got.append(o + (lora_add(s["Y"], s["X"], *a, out=torch.empty_like(s["Y"])),))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        _, _, want, y = ss[i % 2]
        for p, q in zip(o, want + (y,)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype,r", [(BF, 64), (H, 32), (BF, 8), (H, 16)])
@pytest.mark.parametrize("m", [1920, 2180, 3111, 4200, 5290])
def test_cluster_sizes(dtype, r, m):
    # as many pieces as make clusters of 8, 6, 5, 4 and 3 CTAs the choice; the last piece and
    # the last owner's rows of it ragged; once one request, once three and rows of none
    from post_weight_quantization_23_b200 import lora_add, lora_backward
    k, n = 456, 328
    for lens, ids, first, tail in (([m], [0], 0, 0), ([m - 533, 412, 121], [0, 2, 1], 2, 3)):
        s = R.make(dtype, k, n, r, 2, lens, ids, m + r, first, tail)
        ref, bound, Vr, bv, cov = R.add_ref(s, dtype)
        V = torch.full((s["Y"].shape[0], r), 5.0, device="cuda")
        out = torch.full_like(s["Y"], 7.0)
        lora_add(s["Y"], s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"], out=out,
                 V=V)
        R.check(out[cov], ref[cov], bound[cov], "out")
        R.check(V[cov], Vr[cov], bv[cov], "V")
        assert (out[~cov] == 7.0).all() and (V[~cov] == 5.0).all()
        s["V"] = V
        b = R.backward_ref(s, dtype, s["X"].to(R.D))
        dX = torch.full_like(s["dX"], 7.0)
        got = lora_backward(s["dY"], s["X"], V, s["A"], s["B"], s["scaling"], s["starts"],
                            s["adapter"], s["dX"], out=dX)
        R.check(dX[cov], b["out"][0][cov], b["out"][1][cov], "dX")
        R.check(got[1], *b["dA"], "dA")
        R.check(got[2], *b["dB"], "dB")
        assert (dX[~cov] == 7.0).all()


# the tests above again with batches long enough for the tensor-core kernel at every rank

@pytest.mark.parametrize("case", [
    (H, 512, 768, 16, 4, [300] + [1] * 40 + [33] * 9 + [257, 25, 24, 0, 140],
     [i % 6 - 1 for i in range(55)], 4, 4),
    (BF, 1024, 520, 32, 3, [0, 1, 129, 0, 500, 8, 7, 333], [0, 1, 2, 0, 1, 2, 0, 1], 3, 5),
    (H, 136, 264, 8, 2, [127, 650, 2], [1, 0, 1], 1, 2),
    (BF, 11008, 256, 16, 1, [800], [0], 0, 0),
    (H, 8, 8, 8, 1, [777], [0], 0, 9),
], ids=lambda c: f"r{c[3]}_m{sum(c[5])}")
def test_add_long(case):
    test_add(case)
    test_add_without_y(case)


@pytest.mark.parametrize("xoff,ypad", [(0, 8), (0, 3), (3, 5), (8, 0)])
def test_add_long_strided(xoff, ypad):
    test_add_strided(xoff, ypad, [600, 1, 177])


@pytest.mark.parametrize("dtype", [H, BF])
def test_add_long_nonfinite_neighbours(dtype):
    test_add_nonfinite_neighbours(dtype, [540, 30, 250])


def test_add_long_f16_range_and_capture():
    test_add_f16_range([650, 190])
    test_capture_and_streams([800, 200])
