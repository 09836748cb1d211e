"""Cases of the gated linear recurrence and of the pool of recurrent states.

Two families of operators that stand beside the delta-rule memory:

* the gated linear recurrence, a vector state per channel instead of a matrix,
      h_t = exp(g_t) * h_{t-1} + beta_t * x_t,   o_t = h_t,
  over whole sequences ("prefill"), as a training step with its gradients
  ("train") and for one token per sequence ("step");
* the pool of state pages that serving keeps between calls (page i holds the
  fp32 state of one sequence): a delta-rule token step on the pages that a list
  of slots names ("decode"), pages copied, forked and cleared ("copy"), and the
  live pages moved to the front of the pool ("compact").

``run`` computes each in its plain form, elementary torch operations in fp32
rounded once at the end, or (``own``) through the package's entry points.
``exact`` computes the same from the definitions in float64, token by token and
page by page.

Sizes: 16 heads of width 64 or 128 and up to 32768 tokens, as in the package's
other workloads (``recurrent_memory_amd/inputs.py``); the recurrence's width is
16 * 128 = 2048 channels where nothing else is said.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a short prompt of one sequence: latency of the sequence form
        dict(name="prefill_short_bf16", op="prefill", B=1, T=128, D=2048, dtype="bf16", beta=True, h0=False, scale=1.0),
        # a long document of one sequence: few channels, a long axis
        dict(name="prefill_long_bf16", op="prefill", B=1, T=32768, D=2048, dtype="bf16", beta=True, h0=True, scale=0.0625),
        # the training step at the package's headline shape (4 sequences of 4096 tokens)
        dict(name="train_bf16", op="train", B=4, T=4096, D=2048, dtype="bf16", beta=True, h0=False, scale=0.0625),
        # an odd width and length, fp32, no input gate, from a carried state
        dict(name="train_odd_f32", op="train", B=3, T=777, D=1001, dtype="f32", beta=False, h0=True, scale=1.0),
        # one token for a full serving batch, states in a pool, the batch padded to a fixed size
        dict(name="step_batch_bf16", op="step", B=256, live=250, N=512, D=2048, dtype="bf16", beta=True, scale=0.0625),
        # one token for a few sequences: launch latency
        dict(name="step_few_f32", op="step", B=4, live=4, N=16, D=2048, dtype="f32", beta=False, scale=1.0),
        # the delta-rule decode of a full batch, its states spread over a pool
        dict(name="decode_batch_gdn_bf16", op="decode", variant="gdn", B=256, live=256, N=320, H=16, Hk=16, dk=128, dv=128, dtype="bf16"),
        # a few sequences with channel-wise decay, grouped query/key heads and padding rows
        dict(name="decode_few_kda_f32", op="decode", variant="kda", B=8, live=6, N=16, H=16, Hk=8, dk=128, dv=64, dtype="f32"),
        # prompts forked into several continuations: 1 MiB pages, four copies of each, and some cleared
        dict(name="copy_fork", op="copy", N=320, page=16 * 128 * 128, forks=192, clears=16, fan=4),
        # the vector states of new sequences put into their pages from a prefill batch
        dict(name="copy_small_pages", op="copy", N=512, page=2048, forks=48, clears=4, fan=1),
        # a pool after half of its sequences ended
        dict(name="compact_half", op="compact", N=512, page=16 * 128 * 128, live=256, rows=320),
        # many small pages of odd length, a few of which were freed
        dict(name="compact_small_odd", op="compact", N=4096, page=1001, live=3500, rows=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "train", "step", "decode", "copy", "compact"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    scale = rng.choice((1.0, 0.25, 0.0625))
    if op in ("prefill", "train"):
        # at most 2^25 (train, fp32 2^24) values of x
        cap = 25 if (op, dtype) != ("train", "f32") else 24
        T = _log(rng, 1, 32768)
        D = _log(rng, 8, 8192)
        if rng.random() < 0.5:
            D = (D + 63) // 64 * 64
        B = _log(rng, 1, 64)
        while B * T * D > 1 << cap:
            B, T = (B // 2, T) if B > 1 else (B, T // 2)
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, beta=rng.random() < 0.7, h0=rng.random() < 0.5, scale=scale)
    if op == "step":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, live=max(1, B - rng.randrange(8)), N=B + rng.randrange(1, 200), D=_log(rng, 8, 8192), dtype=dtype,
                    beta=rng.random() < 0.5, scale=scale)
    if op == "decode":
        H = rng.choice((2, 4, 6, 8, 16))
        B = _log(rng, 1, 256)
        return dict(op=op, variant=rng.choice(("deltanet", "gdn", "kda", "gdn2", "fg2")), B=B, live=max(1, B - rng.randrange(6)),
                    N=B + rng.randrange(1, 64), H=H, Hk=H // rng.choice((1, 2)), dk=rng.choice((64, 128)), dv=rng.choice((64, 128)), dtype=dtype)
    page = rng.choice((_log(rng, 64, 65536), _log(rng, 16, 16384) * 16, 4 * 64 * 64, 8 * 128 * 64))
    N = min(_log(rng, 16, 8192), (1 << 26) // page)
    if op == "copy":
        fan = rng.choice((1, 1, 2, 4))
        forks = max(1, _log(rng, 1, max(2, N // 2)))
        return dict(op=op, N=N, page=page, forks=min(forks, N // 2), clears=rng.randrange(1, max(2, N // 8)), fan=fan)
    rows = rng.randrange(max(2, N // 2), N + 1)
    return dict(op=op, N=N, page=page, live=rng.randrange(1, rows + 1), rows=rows)


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _neg_softplus(z):
    return -torch.log1p(torch.exp(-z.abs())) - z.clamp(min=0)


def _prepare_rec(c, gen, lead):
    dt = _DT[c["dtype"]]
    x = _randn(gen, *lead, c["D"]).to(dt)
    g = (_neg_softplus(_randn(gen, *lead, c["D"])) * c["scale"]).to(dt)
    beta = torch.sigmoid(_randn(gen, *lead, c["D"])).to(dt) if c["beta"] else None
    return dict(x=x, g=g, beta=beta)


def _unit(z):
    return z / z.square().sum(-1, keepdim=True).sqrt()


def prepare(case, seed):
    c, gen = case, _gen(seed)
    op = c["op"]
    s = dict(case=c)
    if op in ("prefill", "train"):
        s.update(_prepare_rec(c, gen, (c["B"], c["T"])))
        s["h0"] = 0.5 * _randn(gen, c["B"], c["D"]) if c["h0"] else None
        if op == "train":
            s["dO"] = _randn(gen, c["B"], c["T"], c["D"]).to(_DT[c["dtype"]])
            s["dhT"] = _randn(gen, c["B"], c["D"])
            s["leaves"] = [n for n in ("x", "g", "beta", "h0") if s[n] is not None]
            for n in s["leaves"]:
                s[n].requires_grad_(True)
    elif op == "step":
        s.update(_prepare_rec(c, gen, (c["B"],)))
        s["h"] = 0.5 * _randn(gen, c["N"], c["D"])
        s["slots"] = _slots(c, gen)
        s["o"] = torch.zeros(c["B"], c["D"], dtype=_DT[c["dtype"]], device="cuda")
    elif op == "decode":
        dt, lead = _DT[c["dtype"]], (c["B"], c["H"])
        s["q"] = _unit(_randn(gen, c["B"], c["Hk"], c["dk"])).to(dt)
        s["k"] = _unit(_randn(gen, c["B"], c["Hk"], c["dk"])).to(dt)
        s["v"] = _randn(gen, *lead, c["dv"]).to(dt)
        chan = c["variant"] in ("gdn2", "fg2")
        s["beta"] = torch.sigmoid(_randn(gen, *(lead + (c["dk"],) if chan else lead))).to(dt)
        s["wgate"] = torch.sigmoid(_randn(gen, *lead, c["dv"])).to(dt) if c["variant"] == "gdn2" else None
        s["g"] = None
        if c["variant"] != "deltanet":
            z = _neg_softplus(_randn(gen, *(lead if c["variant"] == "gdn" else lead + (c["dk"],))))
            s["g"] = z.clamp(min=-85.0 / 16.0).to(dt)
        s["pool"] = 0.02 * _randn(gen, c["N"], c["H"], c["dv"], c["dk"])
        s["slots"] = _slots(c, gen)
        s["o"] = torch.zeros(c["B"], c["H"], c["dv"], dtype=dt, device="cuda")
    elif op == "copy":
        perm = torch.randperm(c["N"], generator=gen, device="cuda")
        roots = max(1, c["forks"] // c["fan"])
        n = min(c["forks"] + c["clears"], c["N"] - roots)
        src = perm[:roots][torch.arange(n, device="cuda") % roots].to(torch.int32)
        s["src"] = torch.where(torch.arange(n, device="cuda") < c["forks"], src, torch.full_like(src, -1))
        s["dst"] = perm[roots:roots + n].to(torch.int32).contiguous()
        s["pool"] = _randn(gen, c["N"], c["page"])
    else:
        pages = torch.randperm(c["N"], generator=gen, device="cuda")[:c["rows"]].to(torch.int32)
        gone = torch.randperm(c["rows"], generator=gen, device="cuda") >= c["live"]
        s["slots"] = torch.where(gone, torch.full_like(pages, -1), pages)
        s["pool"] = _randn(gen, c["N"], c["page"])
    return s


def _slots(c, gen):
    """A page for each live row, -1 for the rows that pad the batch."""
    slots = torch.full((c["B"],), -1, dtype=torch.int32, device="cuda")
    slots[:c["live"]] = torch.randperm(c["N"], generator=gen, device="cuda")[:c["live"]].to(torch.int32)
    return slots


# ---- the plain forms --------------------------------------------------------

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t with h_0 = b_0 along dim 1, by doubling: after each
    step (a, b) at t stand for the last 2, 4, 8, ... tokens."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat((b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]), 1)
        a = torch.cat((a[:, :n], a[:, n:] * a[:, :-n]), 1)
        n *= 2
    return b


def _plain_rec(x, g, beta, h0):
    """fp32: decays a, written values u, states h and the states before each token."""
    x, a = x.float(), torch.exp(g.float())
    u = x if beta is None else beta.float() * x
    first = u[:, :1] if h0 is None else u[:, :1] + a[:, :1] * h0[:, None]
    h = _scan(a, torch.cat((first, u[:, 1:]), 1))
    return x, a, h


def _plain_train(s):
    x, g, beta, h0 = (None if s[n] is None else s[n].detach() for n in ("x", "g", "beta", "h0"))
    dt = x.dtype
    xf, a, h = _plain_rec(x, g, beta, h0)
    # adjoint states: e_t = dO_t + a_{t+1} e_{t+1}, from the last token backwards
    dO = s["dO"].float()
    last = dO[:, -1:] + s["dhT"][:, None]
    b = torch.cat((last, dO[:, :-1].flip(1)), 1)
    e = _scan(torch.cat((torch.zeros_like(last), a[:, 1:].flip(1)), 1), b).flip(1)
    before = torch.cat((torch.zeros_like(last) if h0 is None else h0[:, None], h[:, :-1]), 1)
    out = dict(o=h.to(dt), h_T=h[:, -1].contiguous())
    out["dx"] = (e if beta is None else beta.float() * e).to(dt)
    out["dg"] = (a * before * e).to(dt)
    if beta is not None:
        out["dbeta"] = (xf * e).to(dt)
    if h0 is not None:
        out["dh0"] = a[:, 0] * e[:, 0]
    return out


def _plain_step(s):
    n = s["case"]["live"]
    at = s["slots"][:n].long()
    u = s["x"][:n].float()
    if s["beta"] is not None:
        u = u * s["beta"][:n].float()
    h = torch.exp(s["g"][:n].float()) * s["h"][at] + u
    s["h"][at] = h
    s["o"][:n] = h.to(s["o"].dtype)
    return s["o"], s["h"]


def _plain_decode(s):
    c = s["case"]
    n, G = c["live"], c["H"] // c["Hk"]
    at = s["slots"][:n].long()
    q = s["q"][:n].float()[:, :, None].expand(n, c["Hk"], G, c["dk"]).reshape(n, c["H"], 1, c["dk"])
    k = s["k"][:n].float()[:, :, None].expand(n, c["Hk"], G, c["dk"]).reshape(n, c["H"], 1, c["dk"])
    v, beta = s["v"][:n].float(), s["beta"][:n].float()
    S = s["pool"][at]
    if s["g"] is not None:
        a = torch.exp(s["g"][:n].float())
        S = S * (a[:, :, None, None] if c["variant"] == "gdn" else a[:, :, None])
    r = (S * k).sum(-1)
    if c["variant"] == "gdn2":
        S = S - r[..., None] * (beta[:, :, None] * k) + (s["wgate"][:n].float() * v)[..., None] * k
    elif c["variant"] == "fg2":
        S = S + (v - r)[..., None] * (beta[:, :, None] * k)
    else:
        S = S + (beta[..., None] * (v - r))[..., None] * k
    s["pool"][at] = S
    s["o"][:n] = (S * q).sum(-1).to(s["o"].dtype)
    return s["o"], s["pool"]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    keep = (src >= 0).to(torch.float32)[:, None]
    s["pool"][dst] = s["pool"][src.clamp(min=0)] * keep
    return s["pool"]


def _plain_compact(s):
    slots, pool = s["slots"].long(), s["pool"]
    N = pool.shape[0]
    used = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    used[torch.where(slots >= 0, slots, N)] = 1
    used = used[:N]
    n = used.sum()
    page = torch.arange(N, device="cuda")
    moves, hole = (used == 1) & (page >= n), (used == 0) & (page < n)
    # the k-th lowest live page behind the front goes to the k-th lowest hole in it
    holes = torch.sort(torch.where(hole, page, N))[0]
    rank = (torch.cumsum(moves.to(torch.int64), 0) - 1).clamp(min=0)
    to = torch.where(moves, holes[rank], page)
    out = torch.where(slots >= 0, to[slots.clamp(min=0)], -1).to(torch.int32)
    # every page fetches its content: its own, or that of the page that moves there
    come = page.clone()
    come = torch.cat((come, come[:1]))
    come[torch.where(moves, to, N)] = page
    pool.copy_(pool[come[:N]])
    return out, n.to(torch.int32).reshape(1), pool


def _plain_prefill(s):
    _, _, h = _plain_rec(s["x"], s["g"], s["beta"], s["h0"])
    return h.to(s["x"].dtype), h[:, -1].contiguous()


_PLAIN = dict(prefill=_plain_prefill, train=_plain_train, step=_plain_step, decode=_plain_decode, copy=_plain_copy, compact=_plain_compact)


# ---- the package's calls ----------------------------------------------------

def _own_prefill(s):
    from recurrent_memory_amd import ops
    o, h_T, _ = ops.linrec_fwd(s["x"], s["g"], beta=s["beta"], h0=s["h0"])
    return o, h_T


def _own_train(s):
    from recurrent_memory_amd.autograd import linear_recurrence
    o, h_T = linear_recurrence(s["x"], s["g"], s["beta"], s["h0"])
    grads = torch.autograd.grad((o, h_T), [s[n] for n in s["leaves"]], (s["dO"], s["dhT"]))
    out = dict(o=o.detach(), h_T=h_T.detach())
    out.update(("d" + n, t) for n, t in zip(s["leaves"], grads))
    return out


def _own_step(s):
    from recurrent_memory_amd import ops
    ops.linrec_step(s["x"], s["g"], s["h"], beta=s["beta"], slots=s["slots"], o=s["o"])
    return s["o"], s["h"]


def _own_decode(s):
    from recurrent_memory_amd import ops
    ops.delta_decode_slots(s["case"]["variant"], s["q"], s["k"], s["v"], s["beta"], s["pool"], s["slots"], wgate=s["wgate"], g=s["g"], o=s["o"])
    return s["o"], s["pool"]


def _own_copy(s):
    from recurrent_memory_amd import ops
    ops.pages_copy(s["pool"], s["dst"], s["src"])
    return s["pool"]


def _own_compact(s):
    from recurrent_memory_amd import ops
    slots, live = ops.pages_compact(s["pool"], s["slots"])
    return slots, live, s["pool"]


_OWN = dict(prefill=_own_prefill, train=_own_train, step=_own_step, decode=_own_decode, copy=_own_copy, compact=_own_compact)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op in ("prefill", "train"):
        e, n, rows = (2 if c["dtype"] == "bf16" else 4), c["B"] * c["T"] * c["D"], c["B"] * c["D"]
        ins = 3 if c["beta"] else 2
        b, f = n * e * (ins + 1) + rows * 4 * (1 + c["h0"]), n * 4
        if op == "train":   # x, g, (beta) and dO read, o and a gradient of each input written
            b, f = n * e * (ins + 1 + 1 + ins) + rows * 4 * (2 + 2 * c["h0"]), n * 12
        return dict(bytes=b, flops=f)
    if op == "step":
        e, n = (2 if c["dtype"] == "bf16" else 4), c["live"] * c["D"]
        return dict(bytes=n * (8 + e * (4 if c["beta"] else 3)) + 4 * c["B"], flops=4 * n)
    if op == "decode":
        e, rows = (2 if c["dtype"] == "bf16" else 4), c["live"] * c["H"]
        state = rows * c["dk"] * c["dv"]
        gates = {"deltanet": 1, "gdn": 2, "kda": 1 + c["dk"], "gdn2": 2 * c["dk"] + c["dv"], "fg2": 2 * c["dk"]}[c["variant"]]
        return dict(bytes=8 * state + e * (2 * c["live"] * c["Hk"] * c["dk"] + rows * (2 * c["dv"] + gates)) + 4 * c["B"], flops=7 * state)
    if op == "copy":
        roots = max(1, c["forks"] // c["fan"])
        n = min(c["forks"] + c["clears"], c["N"] - roots)
        copies = min(c["forks"], n)
        return dict(bytes=4 * c["page"] * (min(roots, copies) + n) + 8 * n, flops=0)
    # live pages behind the front, as many as are expected of a random pool
    moved = c["live"] * (1 - c["live"] / c["N"])
    return dict(bytes=max(8 * c["rows"] + 4, 8 * c["page"] * moved + 8 * c["rows"] + 4), flops=0)


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_rec(s):
    x, g, beta, h0 = (None if s[n] is None else s[n].detach() for n in ("x", "g", "beta", "h0"))
    B, T, D = x.shape
    h = torch.zeros(B, D, dtype=torch.float64, device="cuda") if h0 is None else h0.double()
    states = torch.empty(B, T + 1, D, dtype=torch.float64, device="cuda")
    states[:, 0] = h
    for t in range(T):
        w = x[:, t].double() if beta is None else x[:, t].double() * beta[:, t].double()
        h = torch.addcmul(w, g[:, t].double().exp(), h)
        states[:, t + 1] = h
    return states


def _exact_train(s):
    states = _exact_rec(s)
    x, g, beta, h0 = (None if s[n] is None else s[n].detach() for n in ("x", "g", "beta", "h0"))
    B, T, D = x.shape
    out = dict(o=states[:, 1:], h_T=states[:, T])
    out["dx"], out["dg"] = (torch.empty(B, T, D, dtype=torch.float64, device="cuda") for _ in range(2))
    if beta is not None:
        out["dbeta"] = torch.empty(B, T, D, dtype=torch.float64, device="cuda")
    e = s["dhT"].double()
    for t in range(T - 1, -1, -1):
        e = e + s["dO"][:, t].double()
        out["dx"][:, t] = e if beta is None else e * beta[:, t].double()
        if beta is not None:
            out["dbeta"][:, t] = e * x[:, t].double()
        e = e * g[:, t].double().exp()
        out["dg"][:, t] = e * states[:, t]
    if h0 is not None:
        out["dh0"] = e
    return out


def _exact_step(s):
    h, o = s["h"].double(), s["o"].double()
    for b, page in enumerate(s["slots"].tolist()):
        if page >= 0:
            w = s["x"][b].double() if s["beta"] is None else s["x"][b].double() * s["beta"][b].double()
            h[page] = s["g"][b].double().exp() * h[page] + w
            o[b] = h[page]
    return o, h


def _exact_decode(s):
    c = s["case"]
    pool, o, G = s["pool"].double(), s["o"].double(), c["H"] // c["Hk"]
    for b, page in enumerate(s["slots"].tolist()):
        if page < 0:
            continue
        q, k = (s[n][b].double().repeat_interleave(G, 0) for n in ("q", "k"))      # [H, dk]
        v, beta = s["v"][b].double(), s["beta"][b].double()
        S = pool[page]
        if s["g"] is not None:
            a = s["g"][b].double().exp()
            S = S * a.reshape(c["H"], 1, -1)
        r = torch.matmul(S, k[:, :, None])[:, :, 0]
        if c["variant"] == "gdn2":
            S = S - r[:, :, None] * (beta * k)[:, None] + (s["wgate"][b].double() * v)[:, :, None] * k[:, None]
        elif c["variant"] == "fg2":
            S = S + (v - r)[:, :, None] * (beta * k)[:, None]
        else:
            S = S + ((v - r) * beta[:, None])[:, :, None] * k[:, None]
        pool[page] = S
        o[b] = torch.matmul(S, q[:, :, None])[:, :, 0]
    return o, pool


def _exact_copy(s):
    pool = s["pool"].double()
    for src, dst in zip(s["src"].tolist(), s["dst"].tolist()):
        if src < 0:
            pool[dst] = 0.0
        else:
            pool[dst] = pool[src]
    return pool


def _exact_compact(s):
    slots, pool = s["slots"].tolist(), s["pool"].double()
    used = sorted({p for p in slots if p >= 0})
    free = sorted(set(range(len(used))) - set(used))
    to = dict(zip([p for p in used if p >= len(used)], free))
    for a, b in to.items():
        pool[b] = pool[a]
    out = torch.tensor([to.get(p, p) if p >= 0 else -1 for p in slots], dtype=torch.int32, device="cuda")
    return out, torch.tensor([len(used)], dtype=torch.int32, device="cuda"), pool


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":
        states = _exact_rec(s)
        return states[:, 1:], states[:, case["T"]]
    return dict(train=_exact_train, step=_exact_step, decode=_exact_decode, copy=_exact_copy, compact=_exact_compact)[op](s)
