"""The pool of state pages on the GPU: copies, forks, clears and compaction against
page-by-page Python, the delta-rule step on pages against delta_decode, and a serving
run of all of them together against the oracle."""
import random

import numpy as np
import pytest
import torch

from gpu_util import TOL, announce, dev
from oracle import delta_decode as oracle_decode
from oracle import delta_fwd as oracle_fwd
from recurrent_memory_amd import ops
from recurrent_memory_amd.inputs import Workload, draw, make_decode_inputs, make_forward_inputs

pytestmark = pytest.mark.gpu

GAP = 4096          # floats in front of and behind a pool that must stay as they are


def _pool(N, page, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    buf = torch.randn(N * page + 2 * GAP, generator=gen, device="cuda")
    return buf, buf[GAP:GAP + N * page].view(N, page)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _copy_ref(pool, dst, src, src_pool=None):
    out = pool.clone()
    for d, s in zip(dst, src):
        rows = out if src_pool is None else src_pool
        if 0 <= d < out.shape[0] and -1 <= s < rows.shape[0]:
            out[d] = 0.0 if s == -1 else rows[s].clone()
    return out


LISTS = [
    (8, [], []),
    (1, [0], [0]), (1, [0], [-1]),
    (9, [3, 4, 5], [1, 1, 1]),                              # a fork
    (9, [3, 4, 0], [1, -1, 2]),
    (9, [3, -1, 9, 4, 5, 6], [1, 2, 3, 9, -2, 7]),          # numbers outside the pool
    (9, [3, 3, 3], [1, 2, 4]),                              # the last one stays
    (9, [3, 3], [1, -1]),
    (9, [2, 3, 4, 5], [1, 2, 3, 4]),                        # each copies what the one before wrote
    (9, [1, 0], [0, 1]),
    (9, [8, 0, 1, 8], [0, 1, 8, 8]),                        # by way of page 8
    (9, [5, 6], [5, 5]),                                    # onto itself, and a fork of it
    (40, [30, 31, 32, 33, 39], [0, 31, 3, 3, -1]),
]


@pytest.mark.parametrize("page", [1, 3, 4, 64, 127, 512, 516, 1001, 8192, 8196, 70000])
def test_copy_lists(page):
    announce("pages_copy", page)
    for i, (N, dst, src) in enumerate(LISTS):
        buf, pool = _pool(N, page, i)
        before, want = buf.clone(), _copy_ref(pool, dst, src)
        got = ops.pages_copy(pool, _ints(dst), _ints(src))
        torch.cuda.synchronize()
        assert got is pool and torch.equal(pool, want), (page, i)
        assert torch.equal(buf[:GAP], before[:GAP]) and torch.equal(buf[-GAP:], before[-GAP:]), (page, i)


@pytest.mark.parametrize("N,n,page", [(700, 500, 37), (65536, 3000, 4), (33, 4000, 12), (2000, 65536, 1)])
def test_copy_random_lists(N, n, page):
    announce("pages_copy_random", N, n, page)
    rnd = random.Random(N)
    for kind in ("free", "any"):
        if kind == "free":                                  # into pages that nothing else names
            perm = list(range(N))
            rnd.shuffle(perm)
            m = min(n, N // 2)
            dst, src = perm[:m], [rnd.choice(perm[m:] + [-1]) for _ in range(m)]
        else:
            m = min(n, 3000)
            dst, src = [rnd.randrange(-2, N + 2) for _ in range(m)], [rnd.randrange(-2, N + 2) for _ in range(m)]
        _, pool = _pool(N, page, 1)
        want = torch.from_numpy(pool.cpu().numpy().copy())
        for d, s in zip(dst, src):
            if 0 <= d < N and -1 <= s < N:
                want[d] = 0.0 if s == -1 else want[s].clone()
        ops.pages_copy(pool, _ints(dst), _ints(src))
        torch.cuda.synchronize()
        assert torch.equal(pool.cpu(), want), kind


def test_copy_between_pools_and_repeats():
    announce("pages_copy_pools")
    _, pool = _pool(12, 130, 1)
    _, other = _pool(5, 130, 2)
    keep = other.clone()
    dst, src = [3, 7, 0, 3, 9, 1], [4, 0, -1, 2, 5, 4]       # page 3 twice, source 5 is outside
    want = _copy_ref(pool, dst, src, other)
    ops.pages_copy(pool, _ints(dst), _ints(src), src_pool=other)
    torch.cuda.synchronize()
    assert torch.equal(pool, want) and torch.equal(other, keep)
    # shaped pages: [N, H, dv, dk] from a prefill's final states
    p4, s4 = torch.randn(4, 2, 8, 8, device="cuda"), torch.randn(3, 2, 8, 8, device="cuda")
    ops.pages_copy(p4, _ints([2]), _ints([1]), src_pool=s4)
    torch.cuda.synchronize()
    assert torch.equal(p4[2], s4[1])


def test_lists_that_are_parts_of_longer_ones():
    """Lists may start at any int32."""
    announce("pages_list_parts")
    _, pool = _pool(9, 20, 6)
    want = _copy_ref(pool, [3, 4], [1, 0])
    ops.pages_copy(pool, _ints([9, 3, 4])[1:], _ints([7, 7, 7, 1, 0])[3:])
    out, n_live = ops.pages_compact(pool, _ints([5, 8, 0])[1:])
    h = pool.clone()
    x = torch.randn(2, 20, device="cuda")
    ops.linrec_step(x, torch.zeros_like(x), h, slots=_ints([0, 0, 6, 2])[2:])
    torch.cuda.synchronize()
    assert out.tolist() == [1, 0] and n_live.item() == 2
    assert torch.equal(pool[2:], want[2:]) and torch.equal(pool[0], want[0]) and torch.equal(pool[1], want[8])
    assert torch.equal(h[6], pool[6] + x[0]) and torch.equal(h[2], pool[2] + x[1])


def test_decode_slots_streams_large_pools():
    """From 128 MiB of states on the accesses are non-temporal: the same bits, also for
    pages that several rows share."""
    announce("decode_slots_large")
    for variant in ("gdn", "kda"):
        B, H = 130, 16
        t = _step_inputs(variant, "bf16", B, H, 128, 128, seed=9)
        pool = 0.02 * torch.randn(140, H, 128, 128, device="cuda")
        want = pool.clone()
        slots = torch.randperm(140, generator=torch.Generator().manual_seed(3))[:B]
        slots[64], slots[129], slots[128] = slots[0], slots[0], slots[7]
        o = ops.delta_decode_slots(variant, t["q"], t["k"], t["v"], t["beta"], pool, slots.to(torch.int32).cuda(),
                                   g=t["g"])
        turns = [[b for b in range(B) if b not in (64, 128, 129)], [64, 128], [129]]
        for rows in turns:
            at = slots[rows].cuda()
            a = {n: v[rows].contiguous() for n, v in t.items() if v is not None}
            S = want[at].contiguous()
            ow = ops.delta_decode(variant, a["q"], a["k"], a["v"], a["beta"], S, g=a["g"])
            want[at] = S
            assert torch.equal(o[rows], ow)
        assert torch.equal(pool, want)


def test_copy_keeps_bit_patterns():
    """Copies move NaN payloads, infinities and subnormals as they are."""
    announce("pages_copy_bits")
    bits = torch.arange(0, 2 ** 32, 2 ** 32 // 65536 + 1, device="cuda", dtype=torch.int64)
    page = (bits - 2 ** 31).to(torch.int32)[:16384].contiguous()
    pool = torch.zeros(3, 16384, device="cuda")
    pool.view(torch.int32)[1] = page
    ops.pages_copy(pool, _ints([2, 0]), _ints([1, -1]))
    torch.cuda.synchronize()
    assert torch.equal(pool.view(torch.int32)[2], page)


def _compact_ref(N, slots):
    used = sorted({s for s in slots if 0 <= s < N})
    L = len(used)
    free = sorted(set(range(L)) - set(used))
    to = dict(zip([s for s in used if s >= L], free))
    return [to.get(s, s) if 0 <= s < N else -1 for s in slots], L, to


@pytest.mark.parametrize("N,page,slots", [
    (1, 4, [0]), (1, 4, [-1]), (5, 3, []), (5, 1, [4]), (5, 4, [0, 1, 2, 3, 4]), (5, 8, [4, 3, 2, 1, 0]),
    (8, 70000, [7, -1, 2, 5]), (8, 1001, [7, 7, -1, 8, 99, -5, 0, 7, 6]),          # shared, outside
    (32, 130, list(range(16, 32))), (33, 130, [32, 31, 0]), (64, 4, [63]), (65, 4, [64, 0, 63]),
    (300, 20, "half"), (2048, 8, "half"), (65536, 1, "half"), (65535, 4, "few"), (4096, 12, "most"),
])
def test_compact(N, page, slots):
    announce("pages_compact", N, page)
    if isinstance(slots, str):
        rnd = random.Random(N)
        live = rnd.sample(range(N), {"half": N // 2, "few": 40, "most": N - 100}[slots])
        slots = [s if rnd.random() < 0.9 else -1 for s in live] + [-1] * 5
    buf, pool = _pool(N, page, 3)
    before, keep = buf.clone(), pool.clone()
    want, L, to = _compact_ref(N, slots)
    st = _ints(slots)
    out, n_live = ops.pages_compact(pool, st)
    torch.cuda.synchronize()
    assert out.tolist() == want and n_live.tolist() == [L]
    assert st.tolist() == list(slots)
    if L:
        came = torch.arange(L, device="cuda")
        if to:
            came[torch.tensor(list(to.values()), device="cuda")] = torch.tensor(list(to), device="cuda")
        assert torch.equal(pool[:L], keep[came])
    assert torch.equal(buf[:GAP], before[:GAP]) and torch.equal(buf[-GAP:], before[-GAP:])
    # compacting what is compact moves nothing
    again, n2 = ops.pages_compact(pool, out)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and n2.tolist() == [L]


def test_pages_past_32_bit_offsets():
    """A pool of 2.2e9 floats: a fork, a clear and a move at its far end."""
    N, page = 2100, 1 << 20
    announce("pages_large", N, page)
    pool = torch.empty(N, page, device="cuda")
    pool.copy_(torch.arange(N, device="cuda", dtype=torch.float32)[:, None].expand(N, page))
    ops.pages_copy(pool, _ints([2099, 2098, 0]), _ints([2097, -1, 2099]))
    out, n_live = ops.pages_compact(pool, _ints([2099, 2097, 2, 0]))
    torch.cuda.synchronize()
    assert out.tolist() == [3, 1, 2, 0] and n_live.tolist() == [4]
    for p, v in ((2099, 2097.0), (2098, 0.0), (0, 2097.0), (3, 2097.0), (1, 2097.0), (2, 2.0), (2096, 2096.0)):
        assert bool((pool[p] == v).all()), p


def test_lists_captured_and_replayed():
    """A captured call reads the list at each replay."""
    announce("pages_graph")
    _, pool = _pool(20, 1000, 4)
    dst, src, slots = _ints([5, 6]), _ints([1, 1]), _ints([9, 3, -1])
    ops.pages_copy(pool, dst, src)
    torch.cuda.synchronize()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        ops.pages_copy(pool, dst, src)
        out, n_live = ops.pages_compact(pool, slots)
    for d, s, sl in (([5, 6], [1, 2], [9, 3, -1]), ([7, 8], [7, -1], [0, 19, 19]), ([3, 3], [0, 4], [-1, -1, -1])):
        dst.copy_(_ints(d)), src.copy_(_ints(s)), slots.copy_(_ints(sl))
        want = _copy_ref(pool, d, s)
        to, L, moves = _compact_ref(20, sl)
        for a, b in moves.items():
            want[b] = want[a]
        gph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == to and n_live.tolist() == [L] and torch.equal(pool[:L], want[:L])
        if not moves:
            assert torch.equal(pool, want)


# ---- the delta-rule step on pages ----

FORMS = ["deltanet", "gdn", "kda", "gdn2", "fg2"]


def _step_inputs(variant, dtype, B, H, dk, dv, Hk=None, seed=0):
    rng = np.random.Generator(np.random.PCG64(seed))
    d = draw(rng, variant, dtype, (B, H), dk, dv, qk_heads=Hk)
    return {n: dev(t, dtype) for n, t in d.items()}


@pytest.mark.parametrize("variant", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(3, 3, 128, 128), (4, 2, 64, 128), (2, 1, 128, 64), (1, 1, 64, 64)])
def test_decode_slots_is_delta_decode_on_pages(variant, dtype, H, Hk, dk, dv):
    """Bitwise, row by row; rows outside the pool and pages that no row names stay as
    they were, and rows that share a page act one after the other."""
    announce("decode_slots", variant, dtype, H, Hk, dk, dv)
    slots = [4, -1, 0, 4, 9, 6, 2, 4, 7, 0]
    N, B = 7, len(slots)
    t = _step_inputs(variant, dtype, B, H, dk, dv, Hk, seed=7)
    buf, pool = _pool(N, H * dv * dk, 5)
    pool.mul_(0.02)
    before, want = buf.clone(), pool.clone().view(N, H, dv, dk)
    mark = 12345.0
    want_o = torch.full((B, H, dv), mark, dtype=t["v"].dtype, device="cuda")
    for b, s in enumerate(slots):
        if 0 <= s < N:
            row = {n: None if v is None else v[b:b + 1].clone() for n, v in t.items()}   # at aligned addresses
            S = want[s:s + 1].clone()
            want_o[b] = ops.delta_decode(variant, row["q"], row["k"], row["v"], row["beta"], S, wgate=row["wgate"],
                                         g=row["g"])[0]
            want[s] = S[0]
    o = torch.full((B, H, dv), mark, dtype=t["v"].dtype, device="cuda")
    p4 = pool.view(N, H, dv, dk)
    ops.delta_decode_slots(variant, t["q"], t["k"], t["v"], t["beta"], p4, _ints(slots), wgate=t["wgate"], g=t["g"], o=o)
    torch.cuda.synchronize()
    assert torch.equal(p4, want)
    assert torch.equal(o, want_o)
    assert torch.equal(buf[:GAP], before[:GAP]) and torch.equal(buf[-GAP:], before[-GAP:])


def test_decode_slots_many_rows():
    """More rows than one scan of the list covers; two rows far apart share a page."""
    announce("decode_slots_many")
    B, N, H = 1500, 1600, 1
    t = _step_inputs("gdn", "bf16", B, H, 64, 64, seed=8)
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(2))[:B]
    slots[1400] = slots[3]
    pool = 0.02 * torch.randn(N, H, 64, 64, device="cuda")
    want = pool.clone()
    st = slots.to(torch.int32).cuda()
    o = ops.delta_decode_slots("gdn", t["q"], t["k"], t["v"], t["beta"], pool, st, g=t["g"])
    first = torch.ones(B, dtype=torch.bool)
    first[1400] = False
    for rows in (first.nonzero()[:, 0].cuda(), _ints([1400]).long()):
        S = want[st[rows].long()].contiguous()
        a = {n: v[rows].contiguous() for n, v in t.items() if v is not None}
        ow = ops.delta_decode("gdn", a["q"], a["k"], a["v"], a["beta"], S, g=a["g"])
        want[st[rows].long()] = S
        assert torch.equal(o[rows], ow)
    assert torch.equal(pool, want)


def test_token_steps_captured_and_replayed():
    """A captured decode step follows its slots and inputs from replay to replay, with
    eager work in between."""
    announce("decode_slots_graph")
    B, H, N = 4, 2, 9
    t = _step_inputs("gdn", "bf16", B, H, 64, 128, seed=11)
    pool = 0.02 * torch.randn(N, H, 128, 64, device="cuda")
    h, x = torch.randn(N, 40, device="cuda"), torch.randn(B, 40, device="cuda")
    z = torch.zeros_like(x)
    slots = _ints([0, 1, 2, -1])
    o, oh = torch.zeros(B, H, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 40, device="cuda")

    def run(pool, h, o, oh):
        ops.delta_decode_slots("gdn", t["q"], t["k"], t["v"], t["beta"], pool, slots, g=t["g"], o=o)
        ops.linrec_step(x, z, h, slots=slots, o=oh)

    run(pool.clone(), h.clone(), o.clone(), oh.clone())
    torch.cuda.synchronize()
    gph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gph):
        run(pool, h, o, oh)
    for i, rows in enumerate(([0, 1, 2, -1], [8, 8, 3, 8], [-1, -1, 5, 99], [2, 0, 1, 4])):
        new = _step_inputs("gdn", "bf16", B, H, 64, 128, seed=20 + i)
        for n in t:
            if t[n] is not None:
                t[n].copy_(new[n])
        x.copy_(torch.randn(B, 40, device="cuda"))
        slots.copy_(_ints(rows))
        want = [v.clone() for v in (pool, h, o, oh)]
        run(*want)
        gph.replay()
        torch.cuda.synchronize()
        for a, b in zip((pool, h, o, oh), want):
            assert torch.equal(a, b), i


def test_inputs_may_go_after_a_call_on_another_stream():
    """Temporaries given to calls on a busy stream, let go and their memory taken for other
    values at once: the calls still see what they were given."""
    import linrecref as R
    announce("stream_inputs")
    B, D, T, H, N = 4, 130, 300, 2, 9
    x, g, b, s, dO, dhT = R.inputs(B, T, D, torch.float32, True, True, 0.1, seed=80)
    _, _, st = ops.linrec_fwd(x, g, beta=b, h0=s, want_states=True)
    rx, rg, rb = (v[:, 0].contiguous() for v in (x, g, b))
    t = _step_inputs("gdn", "bf16", B, H, 64, 128, seed=81)
    pool, other = (0.02 * torch.randn(N, H, 128, 64, device="cuda") for _ in range(2))
    h = torch.randn(N, D, device="cuda")
    slots, dst, src, live = _ints([3, 0, 8, 3]), _ints([1, 2]), _ints([3, -1]), _ints([8, -1, 0])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def calls(take, stream):
        """Every call that takes a stream, its inputs by way of ``take``."""
        p, q = pool.clone(), h.clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        res = list(ops.linrec_fwd(take(x), take(g), beta=take(b), h0=take(s), want_states=True, workspace=take(ws), stream=stream))
        res += ops.linrec_bwd(take(x), take(g), take(st), take(dO), beta=take(b), dh_T=take(dhT), stream=stream).values()
        res.append(ops.linrec_step(take(rx), take(rg), q, beta=take(rb), slots=take(slots), stream=stream))
        res.append(ops.delta_decode_slots("gdn", take(t["q"]), take(t["k"]), take(t["v"]), take(t["beta"]), p, take(slots),
                                          g=take(t["g"]), stream=stream))
        ops.pages_copy(p, take(dst), take(src), src_pool=take(other), stream=stream)
        res += ops.pages_compact(q, take(live), stream=stream)
        return res + [p, q[:2]]

    want = calls(lambda v: v, None)
    side, taken = torch.cuda.Stream(), []
    big = torch.ones(1 << 28, device="cuda")

    def take(v):
        c = v.clone()
        side.wait_stream(torch.cuda.current_stream())
        taken.append(v)
        return c

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):                                 # 80 ms and more
            big.mul_(1.0)
    got = calls(take, side)
    junk = [torch.full_like(v, 7) for v in 3 * taken]
    torch.cuda.synchronize()
    del junk
    for i, (a, c) in enumerate(zip(got, want)):
        assert torch.equal(a, c), i


def test_refusals():
    pool = torch.zeros(4, 8, device="cuda")
    i = _ints([0, 1])
    p4 = torch.zeros(4, 1, 64, 64, device="cuda")
    t = _step_inputs("gdn", "f32", 2, 1, 64, 64)
    a = (t["q"], t["k"], t["v"], t["beta"])
    bad = [
        lambda: ops.pages_copy(pool, i, i[:1]), lambda: ops.pages_copy(pool, i.long(), i), lambda: ops.pages_copy(pool.half(), i, i),
        lambda: ops.pages_copy(pool, i, i, src_pool=torch.zeros(4, 9, device="cuda")), lambda: ops.pages_copy(pool, i.cpu(), i),
        lambda: ops.pages_copy(pool.t(), i, i), lambda: ops.pages_copy(pool[0], i, i), lambda: ops.pages_compact(pool, i.float()),
        lambda: ops.pages_compact(pool, i, slots_out=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: ops.delta_decode_slots("gdn", *a, p4, i), lambda: ops.delta_decode_slots("gdn", *a, p4, i.long(), g=t["g"]),
        lambda: ops.delta_decode_slots("deltanet", *a, p4, i, g=t["g"]),
        lambda: ops.delta_decode_slots("gdn", *a, p4[:, :, :32], i, g=t["g"]),
        lambda: ops.delta_decode_slots("gdn", *a, p4, _ints([0]), g=t["g"]),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"case {n} was taken")
    for call, status in ((lambda: ops.pages_compact(pool, i, slots_out=i), 7), (lambda: ops.pages_copy(pool[:0], i, i), 2),
                         (lambda: ops.pages_copy(pool, i, i, src_pool=pool[:2]), 2),
                         (lambda: ops.pages_copy(pool[:2], i, i, src_pool=pool[1:3]), 7)):
        with pytest.raises(ops.DeltaRuleError) as e:
            call()
        assert e.value.status == status


# ---- all of it together ----

@pytest.mark.parametrize("variant,dtype", [("gdn", "bf16"), ("kda", "f32")])
def test_serving_run(variant, dtype):
    """Prompts are prefilled and put into pages, decoded, forked, some end, the pool is
    compacted, and decoding goes on: every output against the oracle's own sequences."""
    announce("serving_run", variant, dtype)
    H, dk, dv, N, B = 2, 64, 64, 10, 6                       # the decode batch is always 6 rows, padded
    pool = torch.full((N, H, dv, dk), float("nan"), device="cuda")
    w = Workload("t", variant, dtype, B=3, H=H, T=70, dk=dk, dv=dv, random_s0=True, seed=40)
    x = make_forward_inputs(w)
    _, S_T = ops.delta_fwd(variant, dev(x["q"], dtype), dev(x["k"], dtype), dev(x["v"], dtype), dev(x["beta"], dtype),
                           g=dev(x["g"], dtype), S0=dev(x["S0"], "f32"))
    _, S = oracle_fwd(variant, **x)
    ref = {i: S[i] for i in range(3)}                        # sequence -> oracle state
    where = {0: 7, 1: 2, 2: 9}                               # sequence -> page
    ops.pages_copy(pool, _ints([where[0], where[1], where[2]]), _ints([0, 1, 2]), src_pool=S_T)
    ref[3], where[3] = np.zeros((H, dv, dk)), 4              # a sequence without a prompt
    ops.pages_copy(pool, _ints([4]), _ints([-1]))
    steps = make_decode_inputs(Workload("t", variant, dtype, B=B, H=H, T=1, dk=dk, dv=dv, seed=41), 6)["steps"]

    def decode(n):
        st = steps[n]
        rows = sorted(where)
        slots = _ints([where[s] for s in rows] + [-1] * (B - len(rows)))
        o = ops.delta_decode_slots(variant, dev(st["q"], dtype), dev(st["k"], dtype), dev(st["v"], dtype),
                                   dev(st["beta"], dtype), pool, slots, g=dev(st["g"], dtype))
        torch.cuda.synchronize()
        for b, s in enumerate(rows):
            a = {m: None if t is None else t[b:b + 1] for m, t in st.items()}
            ow, Sw = oracle_decode(variant, **a, S=ref[s][None])
            ref[s] = Sw[0]
            got = o[b].float().cpu().numpy()
            for h in range(H):
                assert np.abs(got[h] - ow[0, h]).max() <= TOL[dtype] * np.abs(ow[0, h]).max(), (n, s, h)

    decode(0)
    decode(1)
    ops.pages_copy(pool, _ints([0, 5]), _ints([where[1], where[1]]))     # two more continuations of sequence 1
    ref[4], where[4], ref[5], where[5] = ref[1].copy(), 0, ref[1].copy(), 5
    decode(2)
    for s in (0, 3):                                         # two sequences end
        del where[s], ref[s]
    rows = sorted(where)
    out, n_live = ops.pages_compact(pool, _ints([where[s] for s in rows]))
    where = dict(zip(rows, out.tolist()))
    assert n_live.item() == 4 and sorted(where.values()) == [0, 1, 2, 3]
    decode(3)
    ref[6], where[6] = np.zeros((H, dv, dk)), 4              # a new one in the first free page
    ops.pages_copy(pool, _ints([4]), _ints([-1]))
    decode(4)
    decode(5)
    for s in where:
        got = pool[where[s]].cpu().numpy()
        for h in range(H):
            assert np.abs(got[h] - ref[s][h]).max() <= TOL[dtype] * np.abs(ref[s][h]).max(), (s, h)


def test_serving_run_of_the_recurrence():
    """The same with vector states: prefill, pages, steps, a fork, compaction, steps."""
    announce("serving_run_linrec")
    import linrecref as R
    D, N = 70, 8
    x, g, b, s, _, _ = R.inputs(3, 90, D, torch.float32, True, True, 0.2, seed=50)
    pool = torch.full((N, D), float("nan"), device="cuda")
    _, hT, _ = ops.linrec_fwd(x[:, :60].contiguous(), g[:, :60].contiguous(), beta=b[:, :60].contiguous(), h0=s)
    ops.pages_copy(pool, _ints([6, 3, 5]), _ints([0, 1, 2]), src_pool=hT)
    h, err = R.states_and_bounds(x, g, b, s)
    slots = _ints([6, 3, 5, -1])
    pad = lambda v, t: torch.cat((v[:, t], torch.zeros(1, D, device="cuda")))    # noqa: E731
    for t in range(60, 90):
        if t == 70:                                          # sequence 1 goes on from a copy of its page
            ops.pages_copy(pool, _ints([0]), _ints([3]))
            slots = _ints([6, 0, 5, -1])
        if t == 80:
            slots, n_live = ops.pages_compact(pool, slots)
            assert slots.tolist() == [2, 0, 1, -1] and n_live.item() == 3
        o = ops.linrec_step(pad(x, t), pad(g, t), pool, beta=pad(b, t), slots=slots)
        R.check("o", o[:3], h[:, t + 1], err[:, t + 1])
