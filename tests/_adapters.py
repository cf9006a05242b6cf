"""Plain 64-bit implementations of the adapter operators and the bounds that the
kernels' arithmetic allows, shared by the adapter tests.

u = eps / 2 of a 16-bit type (bf16 2^-8, f16 2^-11), v = 2^-24 of fp32.
"""

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
V32 = 2.0 ** -24
F16_SUB = 2.0 ** -25  # half the spacing of f16's subnormals
D = torch.float64


def starts_of(lens, first=0):
    at = [first]
    for v in lens:
        at.append(at[-1] + v)
    return torch.tensor(at, dtype=torch.int32)


def make(dtype, k, n, r, na, lens, ids, seed, first=0, tail=0, scale_x=1.0, dev="cuda"):
    """Inputs of one batch: `first` rows before the first request, `tail` behind the last."""
    g = torch.Generator(device=dev).manual_seed(seed)
    m = first + sum(lens) + tail
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    ch = torch.exp(rn(k))
    s = dict(
        X=(rn(m, k) * ch * scale_x).to(dtype), Y=rn(m, n).to(dtype),
        A=(rn(na, r, k) / k ** 0.5).to(dtype), B=(rn(na, n, r) * 0.05).to(dtype),
        scaling=0.5 + torch.rand(na, generator=g, device=dev),
        starts=starts_of(lens, first).to(dev),
        adapter=torch.tensor(ids, dtype=torch.int32, device=dev),
        dY=(rn(m, n) * 0.02).to(dtype), dX=(rn(m, k) * 0.05).to(dtype))
    return s


def spans(s, na):
    """(first row, end, adapter or -1) of every request."""
    st, ad = s["starts"].tolist(), s["adapter"].tolist()
    return [(b, e, a if 0 <= a < na else -1) for b, e, a in zip(st, st[1:], ad)]


def low(S, P, sc, transposed):
    """sc * S P^T (P (r, K)) or sc * S P (transposed: P (K, r)) and its fp32 bound: a sum of K
    exact products in fp32 in any order, counted twice in case an adder truncates, and a few
    roundings for the joins and the scaling."""
    Pd = P.to(D) if transposed else P.to(D).T
    v = sc * (S.to(D) @ Pd)
    mag = abs(sc) * (S.to(D).abs() @ Pd.abs())
    return v, 2 * (S.shape[1] + 24) * V32 * mag


def spread(v, ev, Q, u):
    """v Q^T of a split v = hi + lo (relative error u^2; f16 rows are scaled, what that leaves
    is below 2^-30 of the row's largest) and its bound."""
    q = Q.to(D)
    top = v.abs().amax(1, keepdim=True) if v.shape[1] else v
    e = ev + u * u * v.abs() + 2.0 ** -30 * top
    return v @ q.T, e @ q.abs().T + 2 * (2 * v.shape[1] + 8) * V32 * (v.abs() @ q.abs().T)


def add_ref(s, dtype, with_y=True):
    """(out, bound, V, bound of V, covered rows) in 64 bits."""
    na = s["A"].shape[0]
    u = U[dtype]
    Y = s["Y"].to(D) if with_y else torch.zeros_like(s["Y"], dtype=D)
    out, bo = Y.clone(), torch.zeros_like(Y)
    V = torch.zeros(Y.shape[0], s["A"].shape[1], dtype=D, device=Y.device)
    bv = torch.zeros_like(V)
    cov = torch.zeros(Y.shape[0], dtype=torch.bool, device=Y.device)
    sc = s["scaling"].to(D).tolist()
    for b, e, a in spans(s, na):
        cov[b:e] = True
        if a < 0 or e <= b:
            continue
        v, ev = low(s["X"][b:e], s["A"][a], sc[a], False)
        d, ed = spread(v, ev, s["B"][a], u)
        V[b:e], bv[b:e] = v, ev
        out[b:e] = Y[b:e] + d
        ed = ed + V32 * (Y[b:e].abs() + d.abs())
        bo[b:e] = u * out[b:e].abs() + (1 + u) * ed + F16_SUB
    return out, bo, V, bv, cov


def backward_ref(s, dtype, X, x_rel=0.0, with_dx=True):
    """dict name -> (value, bound): X (m, K) in 64 bits is what the gradient sees."""
    na, r, k = s["A"].shape
    n = s["B"].shape[1]
    u = U[dtype]
    dX = s["dX"].to(D) if with_dx else torch.zeros_like(s["dX"], dtype=D)
    out, bo = dX.clone(), torch.zeros_like(dX)
    dA = torch.zeros(na, r, k, dtype=D, device=dX.device)
    dB = torch.zeros(na, n, r, dtype=D, device=dX.device)
    eA, eB = torch.zeros_like(dA), torch.zeros_like(dB)
    sc = s["scaling"].to(D).tolist()
    V = s["V"].to(D)
    # the gradient kernels split the narrow factor into two bf16 parts (relative error 2^-16,
    # after one fp32 product with the checkpoint's scale), f16 wide rows into two as well
    # (2^-16, and the product of the two low parts is left out: 2^-16 more)
    split = 2.0 ** -16 + (2.0 ** -15 if dtype == torch.float16 else 0.0) + 2 * V32
    count = 0
    for b, e, a in spans(s, na):
        if a < 0 or e <= b:
            continue
        count += e - b
        U_, eU = low(s["dY"][b:e], s["B"][a], sc[a], True)
        d, ed = spread(U_, eU, s["A"][a].T, u)
        out[b:e] = dX[b:e] + d
        ed = ed + V32 * (dX[b:e].abs() + d.abs())
        bo[b:e] = u * out[b:e].abs() + (1 + u) * ed + F16_SUB
        x, y = X[b:e].abs(), s["dY"][b:e].to(D).abs()
        dA[a] += U_.T @ X[b:e]
        dB[a] += s["dY"][b:e].to(D).T @ V[b:e]
        eA[a] += (eU + split * U_.abs()).T @ x
        eB[a] += y.T @ (split * V[b:e].abs())
        # fp32 sums over the tokens (three products per token), counted twice
        eA[a] += 2 * (3 * (e - b) + 64) * V32 * (U_.abs().T @ x)
        eB[a] += 2 * (3 * (e - b) + 64) * V32 * (y.T @ V[b:e].abs())
    fin = lambda w, e: u * w.abs() + (1 + u) * e + F16_SUB  # noqa: E731
    return dict(out=(out, bo), dA=(dA, fin(dA, eA)), dB=(dB, fin(dB, eB)))


def check(got, ref, bound, what=""):
    g = got.to(D)
    assert torch.isfinite(g).all(), what
    err = (g - ref).abs()
    over = err > bound
    if over.any():
        i = over.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} over the bound, first at "
                             f"{i}: {float(g[tuple(i)])} for {float(ref[tuple(i)])}, bound "
                             f"{float(bound[tuple(i)])}")
    return float((err / bound.clamp_min(1e-300)).max()) if err.numel() else 0.0
