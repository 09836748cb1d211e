"""Gated linear recurrence on the GPU against the float64 recurrence, with the bounds
of linrecref.py: lengths and widths around the kernels' blocks, resets, long memory,
non-finite values, in-place state, streams, captured replays, outputs' margins."""
import pytest
import torch

import linrecref as R
from gpu_util import announce
from recurrent_memory_amd import ops
from recurrent_memory_amd.autograd import linear_recurrence

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SHAPES = [(1, 1, 1), (2, 1, 7), (3, 2, 64), (1, 15, 3), (2, 16, 130), (2, 17, 65), (1, 31, 128), (3, 33, 63),
          (1, 127, 129), (2, 128, 8), (1, 129, 256), (2, 255, 127), (1, 256, 130), (2, 257, 1), (5, 300, 10),
          (1, 513, 66), (2, 1000, 101), (1, 4099, 48), (70, 40, 2), (3, 777, 1001), (2, 520, 2048), (3, 290, 192)]


def _fwd_check(x, g, b, h0, want_states=True):
    o, hT, st = ops.linrec_fwd(x, g, beta=b, h0=h0, want_states=want_states)
    torch.cuda.synchronize()
    h, err = R.states_and_bounds(x, g, b, h0)
    R.check("o", o, h[:, 1:], err[:, 1:])
    R.check("h_T", hT, h[:, -1], err[:, -1])
    if want_states:
        R.check("states", st, h[:, :-1:16], err[:, :-1:16])
    return o, hT, st


def _bwd_check(x, g, b, h0, dO, dhT, st, names=("dx", "dg", "dbeta", "dh0")):
    gr = ops.linrec_bwd(x, g, st, dO, beta=b, dh_T=dhT)
    torch.cuda.synchronize()
    ref = R.grads_and_bounds(x, g, b, h0, dO, dhT)
    for n in names:
        if n in ref:
            R.check(n, gr[n], *ref[n])
    return gr


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward_and_backward(dtype, B, T, D):
    announce("linrec", dtype, B, T, D)
    # both gates and states in one case, neither in the other
    for beta, h0 in ((True, True), (False, False)):
        x, g, b, s, dO, dhT = R.inputs(B, T, D, DT[dtype], beta, h0, seed=B + T + D)
        _, _, st = _fwd_check(x, g, b, s)
        _bwd_check(x, g, b, s, dO, dhT if h0 else None, st)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,scale", [(1, 20000, 70, 1 / 512), (2, 9000, 256, 1 / 64), (2, 2200, 33, 1 / 16)])
def test_long_sequences(dtype, B, T, D, scale):
    """Slow decays over many tiles: what is carried across them matters."""
    announce("linrec_long", dtype, B, T, D, scale)
    x, g, b, s, dO, dhT = R.inputs(B, T, D, DT[dtype], True, True, scale, seed=T)
    _, _, st = _fwd_check(x, g, b, s)
    _bwd_check(x, g, b, s, dO, dhT, st)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_resets_and_padding(dtype):
    """g = -inf forgets everything before its token, forwards and backwards; tokens
    with g = 0 and x = 0 leave the state as it is."""
    announce("linrec_resets", dtype)
    B, T, D = 2, 700, 96
    x, g, b, s, dO, dhT = R.inputs(B, T, D, DT[dtype], True, True, 0.1, seed=5)
    g[0, 0], g[1, 300], g[0, 256], g[0, 255, :10] = (-float("inf"),) * 4
    g[1, 600:], x[1, 600:] = 0, 0
    o, hT, st = _fwd_check(x, g, b, s)
    gr = _bwd_check(x, g, b, s, dO, dhT, st)
    assert bool((gr["dh0"][0] == 0).all())
    assert bool((gr["dg"][0, 256] == 0).all())
    # the padded tail only carries the state on
    o2, hT2, _ = ops.linrec_fwd(x[1:, :600].contiguous(), g[1:, :600].contiguous(), beta=b[1:, :600].contiguous(), h0=s[1:])
    assert torch.equal(o2[0], o[1, :600])
    h600 = R.states_and_bounds(x[1:, :600], g[1:, :600], b[1:, :600], s[1:])
    R.check("h_T", hT[1:], h600[0][:, -1], 2 * h600[1][:, -1])
    R.check("h_T", hT2, h600[0][:, -1], h600[1][:, -1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_stays_in_its_channel(dtype, value):
    announce("linrec_nonfinite", dtype, value)
    x, g, b, s, dO, dhT = R.inputs(2, 600, 131, DT[dtype], True, True, 0.1, seed=6)
    g = g.clamp(min=-0.125)                     # no decay underflows to zero within 300 tokens
    o0, h0, st0 = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
    x1 = x.clone()
    x1[1, 290, 77] = value
    o1, h1, st1 = ops.linrec_fwd(x1, g, beta=b, h0=s, want_states=True)
    torch.cuda.synchronize()
    rest = torch.ones(2, 131, dtype=torch.bool, device="cuda")
    rest[1, 77] = False
    assert torch.equal(o1.transpose(1, 2)[rest], o0.transpose(1, 2)[rest]) and torch.equal(h1[rest], h0[rest])
    assert torch.equal(o1[1, :290, 77], o0[1, :290, 77])
    assert not bool(torch.isfinite(o1[1, 290:, 77]).any()) and not bool(torch.isfinite(h1[1, 77]))
    dO1 = dO.clone()
    dO1[1, 290, 77] = value
    g0 = ops.linrec_bwd(x, g, st0, dO, beta=b, dh_T=dhT)
    g1 = ops.linrec_bwd(x, g, st0, dO1, beta=b, dh_T=dhT)
    torch.cuda.synchronize()
    for n in ("dx", "dg", "dbeta"):
        assert torch.equal(g1[n].transpose(1, 2)[rest], g0[n].transpose(1, 2)[rest]), n
        assert torch.equal(g1[n][1, 291:, 77], g0[n][1, 291:, 77]), n
        assert not bool(torch.isfinite(g1[n][1, :291, 77]).any()), n
    assert torch.equal(g1["dh0"][rest], g0["dh0"][rest]) and not bool(torch.isfinite(g1["dh0"][1, 77]))


BAD = [float("inf"), -float("inf"), float("nan")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("border,at", [(1, 0), (20, 3), (20, 19), (33, 16), (130, 127), (256, 0), (700, 690), (2200, 5)])
@pytest.mark.parametrize("D", [66, 65])
def test_a_border_stops_what_is_not_finite(D, dtype, border, at):
    """Nothing passes a token that forgets: an infinity or NaN written or handed in before
    it, or arriving as a gradient after it, changes no bit on its other side."""
    announce("linrec_border", D, dtype, border, at)
    B, T = 1, border + 300
    x, g, b, s, dO, dhT = R.inputs(B, T, D, DT[dtype], True, True, 0.1, seed=border)
    g[:, border, ::2] = -float("inf")
    g[:, border, 1::2] = -88.0                               # zero in fp32 too
    want = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
    wgr = ops.linrec_bwd(x, g, want[2], dO, beta=b, dh_T=dhT)
    blocks = -(-border // 16) if border % 16 else border // 16 + 1      # states of tokens behind the border
    for i, bad in enumerate(BAD):
        x1, s1 = x.clone(), s.clone()
        x1[0, at, i::6] = bad
        s1[0, i + 3::6] = bad
        o, hT, st = ops.linrec_fwd(x1, g, beta=b, h0=s1, want_states=True)
        assert torch.equal(o[:, border:], want[0][:, border:]) and torch.equal(hT, want[1])
        assert torch.equal(st[:, blocks:], want[2][:, blocks:])
        assert not bool(torch.isfinite(o[:, at:border, i::6]).any())
        gr = ops.linrec_bwd(x1, g, st, dO, beta=b, dh_T=dhT)
        for n in ("dx", "dg", "dbeta"):
            assert torch.equal(gr[n][:, border:], wgr[n][:, border:]), n
        assert torch.equal(gr["dx"], wgr["dx"]) and torch.equal(gr["dh0"], wgr["dh0"])
        dO1, dhT1 = dO.clone(), dhT.clone()
        dO1[0, border + 1 + at % 200, i::6] = bad
        dhT1[0, i + 3::6] = bad
        gr = ops.linrec_bwd(x, g, want[2], dO1, beta=b, dh_T=dhT1)
        for n in ("dx", "dg", "dbeta"):
            assert torch.equal(gr[n][:, :border], wgr[n][:, :border]), n
        assert torch.equal(gr["dh0"], wgr["dh0"])
        assert not bool(gr["dg"][:, border].any())
        assert not bool(torch.isfinite(gr["dx"][:, border, i::6]).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("g0", [-0.5, -9.0, -80.0])
def test_an_infinity_outlives_small_decays(dtype, g0):
    """However small the product of decays gets, an infinity stays what it is, forwards
    and backwards: only a decay of zero ends it."""
    announce("linrec_inf", dtype, g0)
    x, _, b, s, dO, dhT = R.inputs(1, 2500, 34, DT[dtype], True, True, 1.0, seed=70)
    g = torch.full_like(x, g0)
    x1, s1 = x.clone(), s.clone()
    x1[0, 7, 0], x1[0, 140, 1], s1[0, 2] = float("inf"), -float("inf"), float("inf")
    o, hT, st = ops.linrec_fwd(x1, g, beta=b, h0=s1, want_states=True)
    for c, t, v in ((0, 7, float("inf")), (1, 140, -float("inf")), (2, 0, float("inf"))):
        assert bool((o[0, t:, c] == v).all()) and hT[0, c] == v
        assert bool((st[0, t // 16 + 1:, c] == v).all())
    h, err = R.states_and_bounds(x, g, b, s)
    R.check("o", o[:, :, 3:], h[:, 1:, 3:], err[:, 1:, 3:])
    dO1, dhT1 = dO.clone(), dhT.clone()
    dO1[0, 2490, 0], dO1[0, 2000, 1], dhT1[0, 2] = float("inf"), -float("inf"), float("inf")
    _, _, st = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
    gr = ops.linrec_bwd(x, g, st, dO1, beta=b, dh_T=dhT1)
    for c, t, v in ((0, 2490, float("inf")), (1, 2000, -float("inf")), (2, 2499, float("inf"))):
        assert bool((gr["dx"][0, :t + 1, c] == v).all()) and gr["dh0"][0, c] == v
    ref = R.grads_and_bounds(x, g, b, s, dO, dhT)
    for n in ("dx", "dg", "dbeta"):
        R.check(n, gr[n][:, :, 3:], *(t[:, :, 3:] for t in ref[n]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("with_beta", [True, False])
@pytest.mark.parametrize("D", [64, 71])
def test_sequences_of_documents(D, with_beta, dtype):
    """Borders in every 16 tokens and more seldom, an infinity or NaN in every third document:
    each document is what it is by itself, and the finite ones have finite gradients."""
    announce("linrec_documents", D, with_beta, dtype)
    ends = [0, 3, 4, 11, 16, 30, 33, 64, 200, 201, 330, 700, 900]
    T = ends[-1]
    x, g, b, _, dO, _ = R.inputs(1, T, D, DT[dtype], with_beta, False, 0.2, seed=D)
    for n, lo in enumerate(ends[:-1]):
        g[:, lo] = -float("inf")
        if n % 3 == 1:
            x[:, lo + (ends[n + 1] - lo) // 2] = BAD[n // 3 % 3]
            dO[:, ends[n + 1] - 1] = BAD[n // 3 % 3]
    o, _, st = ops.linrec_fwd(x, g, beta=b, want_states=True)
    gr = ops.linrec_bwd(x, g, st, dO, beta=b)
    for n, (lo, hi) in enumerate(zip(ends, ends[1:])):
        part = [None if v is None else v[:, lo:hi].contiguous() for v in (x, g, b)]
        mid, got = (hi - lo) // 2, o[:, lo:hi]
        if n % 3 == 1:
            assert bool(torch.isfinite(got[:, :mid]).all()) and not bool(torch.isfinite(got[:, mid:]).any()), n
            assert not bool(torch.isfinite(gr["dx"][:, lo:hi]).any()) and not bool(gr["dg"][:, lo].any()), n
            continue
        h, err = R.states_and_bounds(*part, None)
        R.check("o", got, h[:, 1:], err[:, 1:])
        for name, (v, e) in R.grads_and_bounds(*part, None, dO[:, lo:hi], None).items():
            if name != "dh0":
                R.check(name, gr[name][:, lo:hi], v, e)
    assert not bool(gr["dh0"].any())


def test_a_step_forgets_what_is_not_finite():
    announce("linrec_step_border")
    x, g, b, _, _, _ = R.inputs(3, 1, 10, torch.float32, True, False, seed=71)
    x, g, b = x[:, 0], g[:, 0], b[:, 0]
    g[:, :5] = -float("inf")
    for bad in BAD:
        h = torch.full((3, 10), bad, device="cuda")
        o = ops.linrec_step(x, g, h, beta=b)
        assert torch.equal(o[:, :5], (x * b)[:, :5]) and torch.equal(h[:, :5], o[:, :5])
        assert not bool(torch.isfinite(o[:, 5:]).any()) and not bool(torch.isfinite(h[:, 5:]).any())


class Margins:
    """A tensor inside a buffer of NaN patterns, 64 KiB of them on each side."""

    def __init__(self, shape, dtype):
        self.bits = {torch.bfloat16: torch.int16, torch.float32: torch.int32, torch.uint8: torch.uint8}[dtype]
        esz = torch.empty(0, dtype=dtype).element_size()
        self.m, n = 65536 // esz, 1
        for v in shape:
            n *= v
        self.n = n
        self.buf = torch.empty(n + 2 * self.m, dtype=dtype, device="cuda")
        self.buf.view(self.bits).fill_(-1 if dtype != torch.uint8 else 255)
        self.sentinel = self.buf.view(self.bits)[0].item()
        self.t = self.buf[self.m:self.m + n].view(shape)

    def check(self, name, full=True):
        b = self.buf.view(self.bits)
        assert bool((b[:self.m] == self.sentinel).all()), f"{name}: written in front of it"
        assert bool((b[self.m + self.n:] == self.sentinel).all()), f"{name}: written behind it"
        if full:
            assert not bool((b[self.m:self.m + self.n] == self.sentinel).any()), f"{name}: not all written"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 17, 65), (1, 257, 33), (2, 1000, 130), (3, 530, 77)])
def test_writes_only_its_outputs(dtype, B, T, D):
    announce("linrec_margins", dtype, B, T, D)
    x, g, b, s, dO, dhT = R.inputs(B, T, D, DT[dtype], True, True, seed=9)
    d = ops.LinrecDesc(B, T, D, ops.DTYPES[DT[dtype]])
    o, hT = Margins((B, T, D), DT[dtype]), Margins((B, D), torch.float32)
    st = Margins((B, -(-T // 16), D), torch.float32)
    wf, wb = (Margins((max(1, ops.workspace_bytes(e, d)),), torch.uint8) for e in ("linrec_fwd", "linrec_bwd"))
    ops.linrec_fwd(x, g, beta=b, h0=s, o=o.t, h_T=hT.t, states=st.t, workspace=wf.t)
    out = {n: Margins((B, T, D), DT[dtype]) for n in ("dx", "dg", "dbeta")}
    out["dh0"] = Margins((B, D), torch.float32)
    ops.linrec_bwd(x, g, st.t, dO, beta=b, dh_T=dhT, out={n: m.t for n, m in out.items()}, workspace=wb.t)
    torch.cuda.synchronize()
    for n, m in dict(o=o, h_T=hT, states=st, **out).items():
        m.check(n)
    for n, m in (("forward workspace", wf), ("backward workspace", wb)):
        m.check(n, full=False)


def test_in_place_state_and_chunked_prefill():
    """A sequence in two calls, its state updated in place, is the sequence in one."""
    announce("linrec_chunked")
    x, g, b, s, _, _ = R.inputs(2, 600, 130, torch.float32, True, True, 0.1, seed=10)
    h, err = R.states_and_bounds(x, g, b, s)
    st = s.clone()
    for lo, hi in ((0, 1), (1, 290), (290, 600)):
        o, hT, none = ops.linrec_fwd(x[:, lo:hi].contiguous(), g[:, lo:hi].contiguous(), beta=b[:, lo:hi].contiguous(),
                                     h0=st, h_T=st)
        assert hT is st and none is None
        R.check("o", o, h[:, lo + 1:hi + 1], err[:, lo + 1:hi + 1])
    R.check("h_T", st, h[:, -1], err[:, -1])
    o, hT, _ = ops.linrec_fwd(x, g, beta=b, h0=s, want_state=False)
    assert hT is None
    R.check("o", o, h[:, 1:], err[:, 1:])


@pytest.mark.parametrize("B,T,D", [(2, 3000, 300), (4, 100, 64), (1, 16384, 2048)])
def test_same_results_on_every_run(B, T, D):
    """Bitwise, also while another stream runs the same operator."""
    announce("linrec_deterministic", B, T, D)
    x, g, b, s, dO, dhT = R.inputs(B, T, D, torch.bfloat16, True, True, 0.05, seed=11)
    o, hT, st = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
    gr = ops.linrec_bwd(x, g, st, dO, beta=b, dh_T=dhT)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            o1, h1, st1 = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
            gr1 = ops.linrec_bwd(x, g, st1, dO, beta=b, dh_T=dhT)
        o2, h2, st2 = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
        gr2 = ops.linrec_bwd(x, g, st2, dO, beta=b, dh_T=dhT)
        torch.cuda.synchronize()
        for a, c in ((o1, o), (o2, o), (h1, hT), (h2, hT), (st1, st), (st2, st)):
            assert torch.equal(a, c)
        for n in gr:
            assert torch.equal(gr1[n], gr[n]) and torch.equal(gr2[n], gr[n]), n


def test_stream_argument():
    """Results of a call on another stream, while the caller's stream still works on memory
    that was freed before the call."""
    announce("linrec_stream")
    x, g, b, s, dO, _ = R.inputs(2, 700, 200, torch.float32, True, True, 0.1, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.ones(1 << 28, device="cuda")
    total = torch.zeros((), device="cuda")
    for _ in range(20):                                     # a queue of work on the caller's stream
        big.mul_(1.0)
    old = [torch.full_like(x, 7.0) for _ in range(8)]
    for t in old:
        total += t.sum()
    del old, t                                              # free to torch, still to be read
    o, hT, st = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True, stream=side)
    gr = ops.linrec_bwd(x, g, st, dO, beta=b, stream=side)
    step = ops.linrec_step(x[:, 0].contiguous(), g[:, 0].contiguous(), s.clone(), stream=torch.cuda.current_stream())
    side.synchronize()
    h, err = R.states_and_bounds(x, g, b, s)
    R.check("o", o, h[:, 1:], err[:, 1:])
    for n, (v, e) in R.grads_and_bounds(x, g, b, s, dO, None).items():
        R.check(n, gr[n], v, e)
    assert total.item() == 7.0 * 8 * x.numel()
    h1, err1 = R.states_and_bounds(x[:, :1], g[:, :1], None, s)
    R.check("o", step, h1[:, 1], err1[:, 1])


def test_captured_and_replayed():
    """Two graphs of the operator, replayed in turn with new inputs and eager work between."""
    announce("linrec_graph")
    shapes = [(2, 1100, 130), (1, 40, 64)]
    sets, graphs = [], []
    for i, (B, T, D) in enumerate(shapes):
        x, g, b, s, dO, dhT = R.inputs(B, T, D, torch.float32, True, True, 0.1, seed=13 + i)
        ops.linrec_fwd(x, g, beta=b, h0=s)
        torch.cuda.synchronize()
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            o, hT, st = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
            gr = ops.linrec_bwd(x, g, st, dO, beta=b, dh_T=dhT)
        sets.append((x, g, b, s, dO, dhT, o, hT, gr))
        graphs.append(gph)
    for rep in range(3):
        for (x, g, b, s, dO, dhT, o, hT, gr), gph in zip(sets, graphs):
            new = R.inputs(*x.shape, torch.float32, True, True, 0.1, seed=100 + rep)
            for a, c in zip((x, g, b, s, dO, dhT), new):
                a.copy_(c)
            gph.replay()
            torch.cuda.synchronize()
            o2, h2, st2 = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
            gr2 = ops.linrec_bwd(x, g, st2, dO, beta=b, dh_T=dhT)
            torch.cuda.synchronize()
            assert torch.equal(o, o2) and torch.equal(hT, h2), rep
            for n in gr:
                assert torch.equal(gr[n], gr2[n]), (rep, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("with_beta,with_h0", [(True, True), (False, True), (True, False)])
def test_autograd(dtype, with_beta, with_h0):
    announce("linrec_autograd", dtype, with_beta, with_h0)
    x, g, b, s, dO, dhT = R.inputs(2, 300, 70, DT[dtype], with_beta, with_h0, 0.3, seed=20)
    leaves = [t.requires_grad_(True) for t in (x, g, b, s) if t is not None]
    o, hT = linear_recurrence(x, g, b, s)
    grads = torch.autograd.grad((o, hT), leaves, (dO, dhT))
    ref = R.grads_and_bounds(*(None if t is None else t.detach() for t in (x, g, b, s)), dO, dhT)
    names = ["dx", "dg"] + (["dbeta"] if with_beta else []) + (["dh0"] if with_h0 else [])
    for n, got in zip(names, grads):
        R.check(n, got, *ref[n])
    # one of the two outputs used, with a gradient in another layout
    o, hT = linear_recurrence(x, g, b, s)
    w = dO.transpose(0, 1).contiguous().transpose(0, 1)
    (gx,) = torch.autograd.grad(o, [x], w)
    R.check("dx", gx, *R.grads_and_bounds(*(None if t is None else t.detach() for t in (x, g, b, s)), dO, None)["dx"])
    # no gradient wanted: nothing kept
    with torch.no_grad():
        o, _ = linear_recurrence(x, g, b, s)
    assert not o.requires_grad


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("join", [torch.cat, torch.stack])
def test_gradients_at_any_address(dtype, join):
    """Two sequences' outputs joined: the second one's gradients start inside a buffer."""
    announce("linrec_autograd_joined", dtype, join.__name__)
    sets = [R.inputs(3, 7, 5, DT[dtype], True, True, 0.3, seed=60 + i) for i in range(2)]
    leaves, os, hs = [], [], []
    for x, g, b, s, _, _ in sets:
        leaves.append([t.requires_grad_(True) for t in (x, g, b, s)])
        o, hT = linear_recurrence(x, g, b, s)
        os.append(o), hs.append(hT)
    grads = torch.autograd.grad((join(os), join(hs)), sum(leaves, []),
                                (join([v[4] for v in sets]), join([v[5] for v in sets])))
    for i, (x, g, b, s, dO, dhT) in enumerate(sets):
        ref = R.grads_and_bounds(*(t.detach() for t in (x, g, b, s)), dO, dhT)
        for n, got in zip(("dx", "dg", "dbeta", "dh0"), grads[4 * i:]):
            R.check(n, got, *ref[n])


def test_training_step_in_a_graph():
    """Forward and torch.autograd.grad captured together and replayed on new inputs."""
    announce("linrec_autograd_graph")
    x, g, b, s, dO, dhT = R.inputs(2, 300, 66, torch.float32, True, True, 0.2, seed=21)
    leaves = [t.requires_grad_(True) for t in (x, g, b, s)]

    def train():
        o, hT = linear_recurrence(x, g, b, s)
        return torch.autograd.grad((o, hT), leaves, (dO, dhT))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        grads = train()
    for rep in range(3):
        new = R.inputs(2, 300, 66, torch.float32, True, True, 0.2, seed=200 + rep)
        with torch.no_grad():
            for a, c in zip((x, g, b, s, dO, dhT), new):
                a.copy_(c)
        gph.replay()
        torch.cuda.synchronize()
        ref = R.grads_and_bounds(*new)
        for n, got in zip(("dx", "dg", "dbeta", "dh0"), grads):
            R.check(n, got, *ref[n])


def test_whole_numbers_are_exact_over_many_tiles():
    """With g = 0 the states are running sums: of whole numbers, exact however the tiles
    are joined, over thousands of tiles, forwards and backwards."""
    B, T, D = 2, 1000003, 5
    announce("linrec_exact", B, T, D)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randint(-2, 3, (B, T, D), generator=gen, device="cuda").float()
    g = torch.zeros_like(x)
    h0 = torch.randint(-9, 9, (B, D), generator=gen, device="cuda").float()
    o, hT, st = ops.linrec_fwd(x, g, h0=h0, want_states=True)
    h = torch.cumsum(x.double(), 1) + h0.double()[:, None]
    assert torch.equal(o.double(), h) and torch.equal(hT.double(), h[:, -1])
    assert torch.equal(st[:, 0], h0) and torch.equal(st[:, 1:].double(), h[:, 15:-1:16])
    gr = ops.linrec_bwd(x, g, st, x, dh_T=h0)
    e = torch.cumsum(x.double().flip(1), 1).flip(1) + h0.double()[:, None]
    assert torch.equal(gr["dx"].double(), e) and torch.equal(gr["dh0"].double(), e[:, 0])


@pytest.mark.parametrize("B,T,D", [(5, 3, 1000003), (2, 257, 720001)])
def test_more_tiles_than_workgroups(B, T, D):
    """Over 65536 tiles a workgroup takes several, of one tile a sequence and of three."""
    announce("linrec_many_tiles", B, T, D)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randint(-2, 3, (B, T, D), generator=gen, device="cuda").float()
    g = torch.zeros_like(x)
    o, hT, st = ops.linrec_fwd(x, g, want_states=True)
    h = torch.cumsum(x.double(), 1)
    assert torch.equal(o, h.float()) and torch.equal(hT, h[:, -1].float())
    assert torch.equal(st[:, 1:], h[:, 15:-1:16].float()) and not bool(st[:, 0].any())
    gr = ops.linrec_bwd(x, g, st, x)
    e = torch.cumsum(x.double().flip(1), 1).flip(1)
    assert torch.equal(gr["dx"], e.float()) and torch.equal(gr["dh0"], e[:, 0].float())
    assert torch.equal(gr["dg"], (e * torch.cat((torch.zeros_like(h[:, :1]), h[:, :-1]), 1)).float())


def test_workgroups_go_on_after_a_partly_filled_column():
    """40000 columns of three tiles, the last column of 61 lanes: the workgroup that has it in
    its first turn takes another tile after it, and the last tiles have waves without tokens."""
    B, T, D = 1, 257, 40000 * 64 - 3
    announce("linrec_partial_column", B, T, D)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = torch.randint(-2, 3, (B, T, D), generator=gen, device="cuda").float()
    g = torch.zeros_like(x)
    o, hT, st = ops.linrec_fwd(x, g, want_states=True)
    h = torch.cumsum(x, 1)                                   # whole numbers below 2^24: exact
    assert torch.equal(o, h) and torch.equal(hT, h[:, -1])
    assert torch.equal(st[:, 1:], h[:, 15:-1:16]) and not bool(st[:, 0].any())
    gr = ops.linrec_bwd(x, g, st, x)
    e = torch.cumsum(x.flip(1), 1).flip(1)
    assert torch.equal(gr["dx"], e) and torch.equal(gr["dh0"], e[:, 0])


def test_second_derivatives_are_refused():
    x, g, b, s, dO, dhT = R.inputs(1, 20, 4, torch.float32, seed=22)
    x.requires_grad_(True)
    o, _ = linear_recurrence(x, g, b, s)
    (gx,) = torch.autograd.grad(o.square().sum(), [x], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gx.sum(), [x])


def test_more_than_2_to_the_31_elements():
    """Offsets past 32 bits: the last tokens of two sequences of 2^30 + elements each,
    whose states follow from the last reset."""
    B, T, D = 2, 16500, 65600                   # 2.16e9 elements
    announce("linrec_large", B, T, D)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(B, T, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    g = torch.full_like(x, -0.125)
    g[:, T - 300] = -float("inf")
    o, hT, st = ops.linrec_fwd(x, g, want_states=True)
    cols = torch.tensor([0, 1, 64, 127, 128, 65599], device="cuda")
    tail = lambda t: t[:, T - 300:, cols].contiguous()      # noqa: E731
    h, err = R.states_and_bounds(tail(x), tail(g), None, None)
    R.check("o", tail(o), h[:, 1:], err[:, 1:])
    R.check("h_T", hT[:, cols], h[:, -1], err[:, -1])
    gr = ops.linrec_bwd(x, g, st, o)
    ref = R.grads_and_bounds(tail(x), tail(g), None, None, tail(o), None)
    R.check("dx", tail(gr["dx"]), *ref["dx"])
    R.check("dg", tail(gr["dg"]), *ref["dg"])
    del gr, st
    torch.cuda.synchronize()


# ---- one token at a time ----

def _step_ref(x, g, b, pool, slots):
    """fp64 states after the rows' tokens in order, the outputs, and bounds for both."""
    h, err, o, oerr = pool.double().clone(), torch.zeros_like(pool, dtype=torch.float64), {}, {}
    for r, page in enumerate(slots):
        if 0 <= page < pool.shape[0]:
            bb = None if b is None else b[r][None, None]
            st, e = R.states_and_bounds(x[r][None, None], g[r][None, None], bb, h[page][None])
            h[page], err[page] = st[0, 1], e[0, 1] + g[r].double().exp() * err[page]
            o[r], oerr[r] = h[page].clone(), err[page].clone()
    return h, err, o, oerr


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,slots", [
    (3, 3, 1, None), (5, 5, 64, None), (2, 2, 2050, None), (1, 1, 1001, None),
    (4, 9, 130, [8, 0, 3, 5]),
    (6, 4, 260, [-1, 2, 4, 0, -7, 3]),                       # padding and numbers outside the pool
    (7, 3, 65, [1, 1, 2, 1, 0, 2, 1]),                       # pages shared by several rows
    (300, 280, 12, [(7 * i) % 290 - 5 for i in range(300)]),
])
def test_step(dtype, B, N, D, slots):
    announce("linrec_step", dtype, B, N, D)
    for beta in (True, False):
        x, g, b, _, dO, _ = R.inputs(B, 1, D, DT[dtype], beta, False, seed=B + N)
        x, g, b = x[:, 0], g[:, 0], None if b is None else b[:, 0]
        pool = torch.randn(N, D, generator=torch.Generator().manual_seed(3)).cuda()
        st = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        at = list(range(B)) if slots is None else slots
        h, err, o, oerr = _step_ref(x, g, b, pool, at)
        got, out = Margins((N, D), torch.float32), Margins((B, D), DT[dtype])
        got.t.copy_(pool)
        ops.linrec_step(x, g, got.t, beta=b, slots=st, o=out.t)
        torch.cuda.synchronize()
        R.check("h", got.t, h, err)
        for r in range(B):
            if r in o:
                R.check("o", out.t[r], o[r], oerr[r])
            else:
                assert bool((out.t[r].view(out.bits) == out.sentinel).all()), f"row {r} of o was written"
        untouched = [p for p in range(N) if p not in at]
        assert torch.equal(got.t[untouched], pool[untouched])
        got.check("pool")
        out.check("o", full=False)


def test_step_with_many_rows_on_a_page():
    """Lists longer than one scan; pages shared by rows far apart and by runs of rows."""
    announce("linrec_step_shared")
    B, N, D = 700, 500, 9
    slots = [i % 450 for i in range(B)]
    slots[100:140], slots[-1], slots[5] = [499] * 40, 499, -3
    x, g, b, _, _, _ = R.inputs(B, 1, D, torch.float32, True, False, seed=31)
    x, g, b = x[:, 0], g[:, 0], b[:, 0]
    pool = torch.randn(N, D, generator=torch.Generator().manual_seed(4)).cuda()
    h, err, o, oerr = _step_ref(x, g, b, pool, slots)
    out = ops.linrec_step(x, g, pool, beta=b, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    R.check("h", pool, h, err)
    rows = sorted(o)
    R.check("o", out[rows], torch.stack([o[r] for r in rows]), torch.stack([oerr[r] for r in rows]))


def test_step_follows_the_sequence_form():
    announce("linrec_step_sequence")
    x, g, b, s, _, _ = R.inputs(3, 20, 70, torch.float32, True, True, 0.2, seed=30)
    o, hT, _ = ops.linrec_fwd(x, g, beta=b, h0=s)
    h = s.clone()
    for t in range(20):
        ot = ops.linrec_step(x[:, t].contiguous(), g[:, t].contiguous(), h, beta=b[:, t].contiguous())
        R.check("o", ot, *(v[:, t + 1] for v in R.states_and_bounds(x, g, b, s)))
    R.check("h", h, *(v[:, -1] for v in R.states_and_bounds(x, g, b, s)))


def test_refusals():
    x, g, b, s, dO, _ = R.inputs(2, 5, 8, torch.float32, seed=1)
    bad = [
        (lambda: ops.linrec_fwd(x, g[:, :4]), ValueError), (lambda: ops.linrec_fwd(x, g.bfloat16()), ValueError),
        (lambda: ops.linrec_fwd(x.half(), g.half()), ValueError), (lambda: ops.linrec_fwd(x.transpose(0, 1), g), ValueError),
        (lambda: ops.linrec_fwd(x.transpose(0, 1), g.transpose(0, 1)), ValueError),
        (lambda: ops.linrec_fwd(x, g, h0=s.bfloat16()), ValueError), (lambda: ops.linrec_fwd(x, g.cpu()), ValueError),
        (lambda: ops.linrec_fwd(x, g, o=x), ops.DeltaRuleError), (lambda: ops.linrec_fwd(x[:, :0], g[:, :0]), ops.DeltaRuleError),
        (lambda: ops.linrec_bwd(x, g, s, dO), ValueError),
        (lambda: ops.linrec_bwd(x, g, s[:, None], dO, out=dict(dbeta=x)), ValueError),
        (lambda: ops.linrec_step(x[:, 0].contiguous(), g[:, 0].contiguous(), s[:1]), ValueError),
        (lambda: ops.linrec_step(x[:, 0].contiguous(), g[:, 0].contiguous(), s, slots=torch.zeros(2, device="cuda")), ValueError),
        (lambda: ops.linrec_fwd(x, g, stream=5), AttributeError),
    ]
    for i, (call, err) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {i} was taken")
    big = torch.zeros(33, device="cuda")
    with pytest.raises(ops.DeltaRuleError) as e:                       # 4 bytes past a multiple of 16
        ops.linrec_fwd(big[1:].view(1, 4, 8), big[:32].view(1, 4, 8).clone())
    assert e.value.status == 4
