"""The gated linear recurrence in float64, its gradients, and bounds on the error of
an fp32 evaluation of both.

Bounds.  u = 2^-24 is half a step of fp32.  exp(g) taken in fp32 is off by at most
(2|g| + 2) u relative: the argument times log2(e) is rounded once and the constant
once (each moves the exponent by |g| u), and the exponential is good to one step
(2 u).  One token's update adds a product a h and a written value beta x (one rounding
each) and one sum, so with H the recurrence of absolute values (which bounds every
partial result, however tokens are grouped),

    err_t <= a err_{t-1} + u ((2|g| + 3) a H_{t-1} + 2 H_t).

Grouped evaluation multiplies decays of several tokens and applies them to a carried
state: a product of n decays carries the sum of their errors, which the recurrence
above counts too, plus one rounding per factor and per joint, at most as many as there
are tokens: one more u a H_{t-1}, and u H_t for the join.  The bound taken is therefore

    err_t = a err_{t-1} + u ((2|g| + 4) a H_{t-1} + 3 H_t) + tiny

with tiny = 2^-120 for values near the smallest fp32.  The adjoint recurrence has the
same form, and products of two bounded values have the product rule's bound.  Rounding
to the output's type adds eps/2 of the value.
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -120


def states_and_bounds(x, g, beta, h0):
    """h [B, T+1, D] (h[:, 0] is the initial state) and the error bound of each, fp64."""
    x, g = x.double(), g.double()
    B, T, D = x.shape
    h = torch.zeros(B, T + 1, D, dtype=torch.float64, device=x.device)
    err, mag = torch.zeros_like(h), torch.zeros_like(h)
    if h0 is not None:
        h[:, 0], mag[:, 0] = h0.double(), h0.double().abs()
    w = x if beta is None else x * beta.double()
    a = g.exp()
    rel = torch.where(a > 0, 2 * g.abs() + 4, torch.zeros_like(g))   # a = 0 is exact
    for t in range(T):
        h[:, t + 1] = a[:, t] * h[:, t] + w[:, t]
        mag[:, t + 1] = a[:, t] * mag[:, t] + w[:, t].abs()
        grow = torch.where(a[:, t] > 0, rel[:, t] * a[:, t] * mag[:, t], torch.zeros_like(mag[:, t]))
        err[:, t + 1] = a[:, t] * err[:, t] + U * (grow + 3 * mag[:, t + 1]) + TINY
    return h, err


def grads_and_bounds(x, g, beta, h0, dO, dhT):
    """{name: (gradient, bound of an fp32 evaluation)} for dx, dg, dbeta and dh0."""
    h, herr = states_and_bounds(x, g, beta, h0)
    x, g, dO = x.double(), g.double(), dO.double()
    b = torch.ones_like(x) if beta is None else beta.double()
    B, T, D = x.shape
    r = torch.zeros(B, D, dtype=torch.float64, device=x.device) if dhT is None else dhT.double()
    rmag, rerr = r.abs(), torch.zeros_like(r)
    out = {n: (torch.zeros_like(x), torch.zeros_like(x)) for n in ("dx", "dg", "dbeta")}
    for t in range(T - 1, -1, -1):
        e, emag = r + dO[:, t], rmag + dO[:, t].abs()
        eerr = rerr + 2 * U * emag
        out["dx"][0][:, t], out["dx"][1][:, t] = b[:, t] * e, b[:, t].abs() * eerr + U * emag * b[:, t].abs()
        out["dbeta"][0][:, t], out["dbeta"][1][:, t] = x[:, t] * e, x[:, t].abs() * eerr + U * emag * x[:, t].abs()
        a = g[:, t].exp()
        rel = torch.where(a > 0, 2 * g[:, t].abs() + 4, torch.zeros_like(a))
        r = a * e
        rerr = a * eerr + U * (rel * a * emag + a * emag) + TINY
        rmag = a * emag
        out["dg"][0][:, t] = r * h[:, t]
        out["dg"][1][:, t] = rerr * h[:, t].abs() + (rmag + rerr) * herr[:, t] + 2 * U * rmag * h[:, t].abs() + TINY
    out["dh0"] = (r, rerr)
    if beta is None:
        del out["dbeta"]
    return out


def check(name, got, ref, bound):
    """Elementwise |got - ref| <= bound + half a step of got's type."""
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    half = torch.finfo(got.dtype).eps / 2
    d = (got.double() - ref).abs()
    tol = bound + half * (ref.abs() + bound) + TINY
    bad = ~(d <= tol)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(got[i])!r}, "
                             f"expected {float(ref[i])!r}, allowed {float(tol[i])!r}")


def inputs(B, T, D, dtype, beta=True, h0=True, scale=1.0, seed=0, device="cuda"):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = rnd(B, T, D).to(dtype).to(device)
    g = (-torch.nn.functional.softplus(rnd(B, T, D)) * scale).to(dtype).to(device)
    b = torch.sigmoid(rnd(B, T, D)).to(dtype).to(device) if beta else None
    s = rnd(B, D).to(device) if h0 else None
    dO = rnd(B, T, D).to(dtype).to(device)
    dhT = rnd(B, D).to(device)
    return x, g, b, s, dO, dhT
