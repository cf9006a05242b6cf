"""Operators around a quantized layer that carries low-rank adapters, as cases that can be
timed and compared: the adapters of many requests beside the shared projection, their
backward pass, activation checkpoints in 8 bits, and the gradient through the packed weights.

``run`` computes an operator either in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where ``own`` is set, by this package's call.
"""

import random

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}
_BLOCK = 128  # columns that share one scale of an 8-bit checkpoint


def listed():
    return [
        # one token of one request, the smallest call of a serving loop (4096-wide q/o projection)
        dict(name="add_1_token", op="add", dtype="bf16", k=4096, n=4096, rank=16, adapters=8,
             decode=1, prompts=0, tokens=1, bare=False, layout=1, keep=False),
        # a decode step of 64 requests over 16 adapters, some without one, beside the stacked qkv
        dict(name="add_64_decode", op="add", dtype="f16", k=4096, n=12288, rank=16, adapters=16,
             decode=64, prompts=0, tokens=64, bare=True, layout=2, keep=False),
        # prompt chunks of odd lengths and decode tokens in one batch (down projection)
        dict(name="add_mixed_2027", op="add", dtype="bf16", k=11008, n=4096, rank=32, adapters=24,
             decode=89, prompts=7, tokens=2027, bare=True, layout=3, keep=False),
        # the forward of a training step: one adapter, 8192 tokens (up projection); it keeps
        # the low-rank activations V for the backward pass
        dict(name="add_train_8192", op="add", dtype="bf16", k=4096, n=11008, rank=64, adapters=1,
             decode=0, prompts=1, tokens=8192, bare=False, layout=4, keep=True),
        # backward of a short training step from the 16-bit activations
        dict(name="backward_1024", op="backward", dtype="bf16", k=4096, n=4096, rank=16, adapters=1,
             decode=0, prompts=1, tokens=1024, bare=False, layout=5, saved=16),
        # backward of a longer step from the 8-bit checkpoint (up projection)
        dict(name="backward_8bit_4096", op="backward", dtype="bf16", k=4096, n=11008, rank=64,
             adapters=1, decode=0, prompts=1, tokens=4096, bare=False, layout=6, saved=8),
        # several adapters trained at once on sequences of odd lengths, 8-bit checkpoint
        dict(name="backward_ragged_3001", op="backward", dtype="f16", k=11008, n=4096, rank=8,
             adapters=3, decode=0, prompts=7, tokens=3001, bare=True, layout=7, saved=8),
        # a checkpoint of a small batch, saved and restored
        dict(name="checkpoint_64", op="checkpoint", dtype="f16", k=4096, tokens=64),
        # a checkpoint of the widest input of a block, saved and restored
        dict(name="checkpoint_8192", op="checkpoint", dtype="bf16", k=11008, tokens=8192),
        # gradient through the packed weights: a short step on the 4096-wide projection
        dict(name="dgrad_512", op="dgrad", dtype="f16", k=4096, n=4096, tokens=512, group=128),
        # an odd number of tokens through the down projection
        dict(name="dgrad_down_333", op="dgrad", dtype="bf16", k=11008, n=4096, tokens=333, group=128),
        # the stacked gate and up projection of a training step
        dict(name="dgrad_gate_up_4096", op="dgrad", dtype="bf16", k=4096, n=22016, tokens=4096,
             group=128),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step between lo and hi, even over its logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["add", "add", "backward", "backward", "checkpoint", "dgrad"])
    dtype = rng.choice(["f16", "bf16"])
    k = _log(rng, 512, 12288, 32)
    if op == "checkpoint":
        return dict(op=op, dtype=dtype, k=k, tokens=_log(rng, 1, 7001))
    n = _log(rng, 512, 12288, 8)
    if op == "dgrad":
        return dict(op=op, dtype=dtype, k=k, n=n, tokens=_log(rng, 1, 4001),
                    group=rng.choice([32, 64, 128, -1]))
    case = dict(op=op, dtype=dtype, k=k, n=n, rank=rng.choice([8, 16, 24, 32, 64]),
                bare=rng.random() < 0.5, layout=rng.randrange(1 << 20))
    if op == "add":
        case["adapters"] = _log(rng, 1, 32)
        case["decode"] = rng.choice([0, _log(rng, 1, 200)])
        case["prompts"] = rng.randrange(0 if case["decode"] else 1, 6)
        case["tokens"] = case["decode"] + (_log(rng, 8, 4001) if case["prompts"] else 0)
        case["keep"] = rng.random() < 0.3
    else:
        case["adapters"] = rng.randrange(1, 5)
        case["decode"] = 0
        case["prompts"] = rng.randrange(1, 8)
        case["tokens"] = _log(rng, 65, 4001)
        case["saved"] = rng.choice([8, 16])
    return case


def _requests(case):
    """Lengths and adapters of the requests: single tokens among prompts of uneven lengths."""
    rng = random.Random(case["layout"])
    left = case["tokens"] - case["decode"]
    share = [0.2 + rng.random() for _ in range(case["prompts"])]
    lens = [max(1, int(left * s / sum(share))) for s in share]
    if lens:
        lens[-1] += left - sum(lens)
    lens += [1] * case["decode"]
    rng.shuffle(lens)
    ids = [i % case["adapters"] for i in range(len(lens))]
    rng.shuffle(ids)
    if case["bare"] and len(ids) > 1:
        for i in range(0, len(ids), 5):
            ids[i] = -1
    return lens, ids


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, m, k, dt):
    """Tokens whose channels have lognormal scales, one in a hundred of them an outlier."""
    scale = torch.exp(_randn(gen, k))
    scale = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01, 20 * scale, scale)
    return (_randn(gen, m, k) * (0.3 * scale)).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, k, m = _DT[case["dtype"]], case["k"], case["tokens"]
    s = dict(case=dict(case), dt=dt)
    if case["op"] == "checkpoint":
        s["X"] = _activations(gen, m, k, dt)
        return s
    n = case["n"]
    if case["op"] == "dgrad":
        ng = 1 if case["group"] == -1 else -(-k // case["group"])
        s["dY"] = (_randn(gen, m, n) * 0.05).to(dt)
        s["qweight"] = torch.randint(-(1 << 31), 1 << 31, (n, k // 8), generator=gen, device="cuda",
                                     dtype=torch.int64).to(torch.int32)
        s["scales"] = (0.5 + torch.rand(n, ng, generator=gen, device="cuda")) * 0.0053
        s["zeros"] = torch.randint(6, 10, (n, ng), generator=gen, device="cuda", dtype=torch.int32)
        return s
    na, r = case["adapters"], case["rank"]
    lens, ids = _requests(case)
    at = [0]
    for v in lens:
        at.append(at[-1] + v)
    s["starts"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    s["adapter"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    s["token_adapter"] = torch.repeat_interleave(
        s["adapter"].long(), torch.tensor(lens, device="cuda"), output_size=m)
    s["A"] = (_randn(gen, na, r, k) / k ** 0.5).to(dt)
    s["B"] = (_randn(gen, na, n, r) * 0.02).to(dt)
    s["scaling"] = 0.5 + 1.5 * torch.rand(na, generator=gen, device="cuda")
    X = _activations(gen, m, k, dt)
    if case["op"] == "add":
        s["X"] = X
        s["Y"] = _randn(gen, m, n).to(dt)
        s["out"] = torch.zeros_like(s["Y"])
        return s
    # backward: what the forward left (V = scaling X A^T, the saved activations) and the
    # gradients that arrive from the layer above and through the packed weights
    s["V"] = _low(X, s)
    s["dY"] = (_randn(gen, m, n) * 0.05).to(dt)
    s["dX"] = (_randn(gen, m, k) * 0.05).to(dt)
    s["out"] = torch.zeros_like(s["dX"])
    if case["saved"] == 8:
        codes, scale, _ = _quantized(X)
        s["X"], s["x_scales"] = codes.to(torch.int8), scale
    else:
        s["X"], s["x_scales"] = X, None
    return s


# ---------------------------------------------------------------- the plain forms


def _member(s):
    """(tokens, adapters * rank) truth values: the rank rows of each token's own adapter."""
    na, r = s["A"].shape[:2]
    own_rows = torch.arange(na, device="cuda").repeat_interleave(r)
    return s["token_adapter"][:, None] == own_rows[None, :]


def _scale_rows(s):
    return s["scaling"].repeat_interleave(s["A"].shape[1])[None, :]


def _low(X, s):
    """V = scaling (X A^T) of each token's adapter, 32 bits, zero where it has none."""
    na, r, k = s["A"].shape
    every = X.float() @ s["A"].float().reshape(na * r, k).T
    every = torch.where(_member(s), every * _scale_rows(s), 0.0)
    return every.reshape(-1, na, r).sum(1)


def _spread(V, s):
    """V (tokens, rank) placed at the rank rows of each token's adapter."""
    return torch.where(_member(s), V.repeat(1, s["A"].shape[0]), 0.0)


def _quantized(X):
    """8-bit codes and scales of blocks of 128 columns: scale = max|x| / 127, codes = x * (127 /
    max|x|) to the nearest, halves to even, the product taken in 64 bits so that no second
    rounding moves a half."""
    m, k = X.shape
    nb = -(-k // _BLOCK)
    x = torch.nn.functional.pad(X.float(), (0, nb * _BLOCK - k)).reshape(m, nb, _BLOCK)
    top = x.abs().amax(2)
    scale = top / 127.0
    inv = torch.where(top > 0, 127.0 / top, 0.0)
    codes = (x.double() * inv.double()[:, :, None]).round()
    values = codes.float() * scale[:, :, None]
    return codes.reshape(m, -1)[:, :k], scale, values.reshape(m, -1)[:, :k]


def _weights(s):
    """(n, k) weights in 32 bits from the packed 4-bit codes."""
    k, g = s["case"]["k"], s["case"]["group"]
    g = k if g == -1 else g
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    codes = ((s["qweight"][:, :, None] >> shifts) & 15).reshape(-1, k)
    col = torch.arange(k, device="cuda") // g
    return s["scales"][:, col] * (codes - s["zeros"][:, col]).float()


def _plain(s):
    op, dt = s["case"]["op"], s["dt"]
    if op == "checkpoint":
        _, scale, values = _quantized(s["X"])
        return {"values": values.to(dt), "scales": scale}
    if op == "dgrad":
        return (s["dY"].float() @ _weights(s)).to(dt)
    na, r, k = s["A"].shape
    n = s["B"].shape[1]
    rows = s["A"].float().reshape(na * r, k)
    cols = s["B"].float().permute(0, 2, 1).reshape(na * r, n)
    if op == "add":
        V = _low(s["X"], s)
        Y = (s["Y"].float() + _spread(V, s) @ cols).to(dt)
        return {"Y": Y, "V": V} if s["case"]["keep"] else {"Y": Y}
    dY = s["dY"].float()
    X = s["X"].float()
    if s["x_scales"] is not None:
        X = X * s["x_scales"].repeat_interleave(_BLOCK, 1)[:, :k]
    U = torch.where(_member(s), (dY @ cols.T) * _scale_rows(s), 0.0)
    dA = (U.T @ X).reshape(na, r, k)
    dB = (_spread(s["V"], s).T @ dY).reshape(na, r, n).permute(0, 2, 1)
    return {"dX": (s["dX"].float() + U @ rows).to(dt), "dA": dA.to(dt), "dB": dB.to(dt)}


# ---------------------------------------------------------------- the package's calls


def _own(s):
    import post_weight_quantization_23_b200 as P

    c = s["case"]
    if c["op"] == "checkpoint":
        codes, scales = P.act_checkpoint(s["X"])
        return {"values": P.act_restore(codes, scales, s["dt"]), "scales": scales}
    if c["op"] == "dgrad":
        return P.quant_matmul_dgrad(s["dY"], s["qweight"], s["scales"], s["zeros"], 4, c["group"],
                                    c["k"])
    if c["op"] == "add":
        V = torch.zeros(c["tokens"], c["rank"], device="cuda") if c["keep"] else None
        Y = P.lora_add(s["Y"], s["X"], s["A"], s["B"], s["scaling"], s["starts"], s["adapter"],
                       out=s["out"], V=V)
        return {"Y": Y, "V": V} if c["keep"] else {"Y": Y}
    dX, dA, dB = P.lora_backward(s["dY"], s["X"], s["V"], s["A"], s["B"], s["scaling"],
                                 s["starts"], s["adapter"], s["dX"], x_scales=s["x_scales"],
                                 out=s["out"])
    return {"dX": dX, "dA": dA, "dB": dB}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, m, k = case["op"], case["tokens"], case["k"]
    blocks = -(-k // _BLOCK)
    if op == "checkpoint":  # X in, codes and scales out; those in, the values out
        return {"bytes": m * k * (2 + 1 + 1 + 2) + 2 * 4 * m * blocks, "flops": 3 * m * k}
    n = case["n"]
    if op == "dgrad":
        ng = 1 if case["group"] == -1 else -(-k // case["group"])
        return {"bytes": n * k // 2 + 8 * n * ng + 2 * m * (n + k), "flops": 2 * m * n * k}
    lens, ids = _requests(case)
    r = case["rank"]
    used = len({i for i in ids if i >= 0})
    with_one = sum(v for v, i in zip(lens, ids) if i >= 0)
    both = 2 * used * r * (n + k)
    if op == "add":  # X of the tokens with an adapter, Y in and out, V out, the adapters in use
        low = 4 * m * r if case["keep"] else 0
        return {"bytes": 2 * with_one * k + 4 * m * n + low + both,
                "flops": 2 * with_one * r * (n + k)}
    saved = with_one * k * 2 if case["saved"] == 16 else with_one * (k + 4 * blocks)
    return {"bytes": saved + 2 * with_one * n + 4 * m * k + 4 * with_one * r + both
            + 2 * case["adapters"] * r * (n + k),
            "flops": 4 * with_one * r * (n + k)}


# ---------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "checkpoint":
        # the scale is stored in 32 bits and the codes are taken with the 32-bit 127 / max|x|
        X = s["X"].to(d)
        m, k = X.shape
        values = torch.empty_like(X)
        scales = []
        for c0 in range(0, k, _BLOCK):
            x = X[:, c0:c0 + _BLOCK]
            top = x.abs().max(dim=1, keepdim=True).values.float()
            factor = torch.where(top > 0, torch.tensor(127.0, device="cuda") / top,
                                 torch.zeros_like(top)).to(d)
            step = (top / 127).to(d)
            values[:, c0:c0 + _BLOCK] = torch.round(x * factor) * step
            scales.append(step)
        return {"values": values, "scales": torch.cat(scales, 1)}
    if op == "dgrad":
        n, k = case["n"], case["k"]
        g = k if case["group"] == -1 else case["group"]
        W = torch.empty(n, k, dtype=d, device="cuda")
        words = s["qweight"].long() & 0xFFFFFFFF
        for j in range(8):
            W[:, j::8] = (words // (16 ** j) % 16).to(d)
        for i, c0 in enumerate(range(0, k, g)):
            W[:, c0:c0 + g] = (W[:, c0:c0 + g] - s["zeros"][:, i:i + 1]) * s["scales"][:, i:i + 1].to(d)
        return torch.matmul(s["dY"].to(d), W)
    lens, ids = _requests(case)
    A, B, sc = s["A"].to(d), s["B"].to(d), s["scaling"].to(d)
    X = s["X"].to(d)
    if op == "backward" and s["x_scales"] is not None:
        for b in range(s["x_scales"].shape[1]):
            X[:, b * _BLOCK:(b + 1) * _BLOCK] *= s["x_scales"][:, b:b + 1].to(d)
    if op == "add":
        Y = s["Y"].to(d)
        V = torch.zeros(X.shape[0], A.shape[1], dtype=d, device="cuda")
        t = 0
        for v, a in zip(lens, ids):
            if a >= 0:
                V[t:t + v] = sc[a] * torch.einsum("tk,rk->tr", X[t:t + v], A[a])
                Y[t:t + v] += torch.einsum("tr,nr->tn", V[t:t + v], B[a])
            t += v
        return {"Y": Y, "V": V} if case["keep"] else {"Y": Y}
    dY, dX, V = s["dY"].to(d), s["dX"].to(d), s["V"].to(d)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    t = 0
    for v, a in zip(lens, ids):
        if a >= 0:
            U = sc[a] * torch.einsum("tn,nr->tr", dY[t:t + v], B[a])
            dX[t:t + v] += torch.einsum("tr,rk->tk", U, A[a])
            dA[a] += torch.einsum("tr,tk->rk", U, X[t:t + v])
            dB[a] += torch.einsum("tn,tr->nr", dY[t:t + v], V[t:t + v])
        t += v
    return {"dX": dX, "dA": dA, "dB": dB}
