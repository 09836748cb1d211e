"""Contract of include/deltarule_ext.h on the CPU: exports, and every refusal before
any HIP call (the pointers are fake, so nothing that passes may be dereferenced)."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from recurrent_memory_amd import autograd, ops

lib = ops.load_library()

(DR_OK, DR_E_NULLPTR, DR_E_SHAPE, DR_E_UNSUPPORTED, DR_E_ALIGN, DR_E_DEVICE, DR_E_LAUNCH, DR_E_ALIAS,
 DR_E_WORKSPACE) = range(9)
FAKE = [0x7f0000000000 + (i << 36) for i in range(14)]
WS, WS_BYTES = FAKE[13], 1 << 31
GPU = torch.cuda.is_available()


def test_exports_every_header_symbol():
    names = ops.header_functions(ops.EXT_HEADER)
    assert set(names) == {"dr_ext_version", "delta_linrec_fwd_workspace_bytes", "delta_linrec_fwd",
                          "delta_linrec_bwd_workspace_bytes", "delta_linrec_bwd", "delta_linrec_step",
                          "delta_decode_slots", "delta_pages_copy", "delta_pages_compact"}
    for n in names:
        assert hasattr(lib, n), n
    text = open(ops.EXT_HEADER).read()
    assert lib.dr_ext_version() == ops.EXT_VERSION
    for line in (f"DR_EXT_VERSION {ops.EXT_VERSION}", f"DR_LINREC_BLOCK {ops.LINREC_BLOCK}",
                 f"DR_MAX_PAGES {ops.MAX_PAGES}"):
        assert "#define " + line in text


def ld(**kw):
    return ops.LinrecDesc(**{**dict(B=2, T=100, D=48, dtype=1), **kw})


def ref(d):
    return ctypes.byref(d) if d is not None else None


def fwd(d, x=FAKE[0], g=FAKE[1], beta=FAKE[2], h0=FAKE[3], o=FAKE[4], hT=FAKE[5], states=FAKE[6], ws=WS, wn=WS_BYTES):
    return lib.delta_linrec_fwd(ref(d), x, g, beta, h0, o, hT, states, ws, wn, None)


def bwd(d, x=FAKE[0], g=FAKE[1], beta=FAKE[2], states=FAKE[3], dO=FAKE[4], dhT=FAKE[5], dx=FAKE[6], dg=FAKE[7],
        dbeta=FAKE[8], dh0=FAKE[9], ws=WS, wn=WS_BYTES):
    return lib.delta_linrec_bwd(ref(d), x, g, beta, states, dO, dhT, dx, dg, dbeta, dh0, ws, wn, None)


def step(d, x=FAKE[0], g=FAKE[1], beta=FAKE[2], h=FAKE[3], n=16, slots=FAKE[4], o=FAKE[5]):
    return lib.delta_linrec_step(ref(d), x, g, beta, h, n, slots, o, None)


def dec(d, q=FAKE[0], k=FAKE[1], v=FAKE[2], beta=FAKE[3], wgate=None, g=FAKE[5], pool=FAKE[6], n=16, slots=FAKE[7],
        o=FAKE[8]):
    return lib.delta_decode_slots(ref(d), q, k, v, beta, wgate, g, pool, n, slots, o, None)


def pd(**kw):
    return ops.PagesDesc(**{**dict(page=1024, n_pages=8, n=4), **kw})


def copy(d, pool=FAKE[0], dst=FAKE[1], src_pool=FAKE[0], src_pages=8, src=FAKE[2]):
    return lib.delta_pages_copy(ref(d), pool, dst, src_pool, src_pages, src, None)


def compact(d, pool=FAKE[0], slots=FAKE[1], out=FAKE[2], n_live=FAKE[3]):
    return lib.delta_pages_compact(ref(d), pool, slots, out, n_live, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), DR_E_UNSUPPORTED), (dict(dtype=-1), DR_E_UNSUPPORTED), (dict(B=0), DR_E_SHAPE),
    (dict(T=0), DR_E_SHAPE), (dict(D=0), DR_E_SHAPE), (dict(T=-5), DR_E_SHAPE), (dict(B=(1 << 20) + 1), DR_E_SHAPE),
    (dict(D=(1 << 24) + 1, B=1), DR_E_SHAPE), (dict(B=1 << 10, D=1 << 22), DR_E_SHAPE),
    (dict(B=1 << 10, D=1 << 20, T=(1 << 10) + 1), DR_E_SHAPE),
])
def test_linrec_descriptor(kw, status):
    assert fwd(ld(**kw)) == status
    assert bwd(ld(**kw)) == status
    n = ctypes.c_size_t(0)
    for q in (lib.delta_linrec_fwd_workspace_bytes, lib.delta_linrec_bwd_workspace_bytes):
        assert q(ref(ld(**kw)), ctypes.byref(n)) == status


def test_linrec_null_and_unsupported_pointers():
    assert fwd(None) == bwd(None) == step(None) == DR_E_NULLPTR
    for name in ("x", "g", "o"):
        assert fwd(ld(), **{name: None}) == DR_E_NULLPTR, name
    for name in ("x", "g", "states", "dO", "dx", "dg", "dbeta"):
        assert bwd(ld(), **{name: None}) == DR_E_NULLPTR, name
    assert bwd(ld(), beta=None) == DR_E_UNSUPPORTED          # a gradient of the gate that is not there
    for name in ("x", "g", "h", "o"):
        assert step(ld(T=1), **{name: None}) == DR_E_NULLPTR, name
    n = ctypes.c_size_t(0)
    assert lib.delta_linrec_fwd_workspace_bytes(None, ctypes.byref(n)) == DR_E_NULLPTR
    assert lib.delta_linrec_bwd_workspace_bytes(ref(ld()), None) == DR_E_NULLPTR


def test_linrec_alignment_and_aliasing():
    assert fwd(ld(), x=FAKE[0] + 8) == DR_E_ALIGN
    assert fwd(ld(), states=FAKE[6] + 4) == DR_E_ALIGN
    assert bwd(ld(), dh0=FAKE[9] + 4) == DR_E_ALIGN
    assert step(ld(T=1), slots=FAKE[4] + 2) == DR_E_ALIGN          # lists of int32: 4 bytes
    for name in ("x", "g", "beta", "h0"):
        i = ("x", "g", "beta", "h0").index(name)
        assert fwd(ld(), o=FAKE[i]) == DR_E_ALIAS, name
    assert fwd(ld(), o=FAKE[0] + 2 * 100 * 48 * 2 - 16) == DR_E_ALIAS     # over the end of x
    assert fwd(ld(), hT=FAKE[3] + 16) == DR_E_ALIAS                       # shifted onto h0
    assert fwd(ld(), states=FAKE[4]) == DR_E_ALIAS
    # states are ceil(100 / 16) = 7 rows of each sequence
    assert fwd(ld(), hT=FAKE[6] + 2 * 7 * 48 * 4 - 16) == DR_E_ALIAS
    assert bwd(ld(), dx=FAKE[4]) == DR_E_ALIAS                            # over dO
    assert bwd(ld(), dg=FAKE[6]) == DR_E_ALIAS                            # over dx
    assert bwd(ld(), dh0=FAKE[5]) == DR_E_ALIAS                           # over dh_T
    assert step(ld(T=1), o=FAKE[3] + 15 * 48 * 4) == DR_E_ALIAS           # over the last page
    assert step(ld(T=1), h=FAKE[0]) == DR_E_ALIAS
    if not GPU:
        assert fwd(ld(), hT=FAKE[3]) == DR_E_DEVICE                       # in place
        assert fwd(ld(), o=FAKE[0] + 2 * 100 * 48 * 2) == DR_E_DEVICE     # right behind x
        assert fwd(ld(), beta=None, h0=None, hT=None, states=None) == DR_E_DEVICE
        assert bwd(ld()) == DR_E_DEVICE
        assert bwd(ld(), beta=None, dbeta=None, dhT=None, dh0=None) == DR_E_DEVICE


@pytest.mark.parametrize("D", [2048, 1001])
def test_linrec_workspace(D):
    d = ld(B=3, T=5000, D=D)
    for entry, call in (("fwd", fwd), ("bwd", bwd)):
        n = ctypes.c_size_t(0)
        assert getattr(lib, f"delta_linrec_{entry}_workspace_bytes")(ref(d), ctypes.byref(n)) == DR_OK
        if n.value:
            assert call(d, ws=None, wn=0) == DR_E_WORKSPACE
            assert call(d, wn=n.value - 1) == DR_E_WORKSPACE
            assert call(d, ws=WS + 16) == DR_E_ALIGN
            assert call(d, ws=FAKE[1]) == DR_E_ALIAS
        elif not GPU:
            assert call(d, ws=None, wn=0) == DR_E_DEVICE


def test_step_and_slots():
    assert step(ld(T=2)) == DR_E_SHAPE                        # one token only
    assert step(ld(T=1), n=0) == DR_E_SHAPE
    assert step(ld(T=1), n=ops.MAX_PAGES + 1) == DR_E_SHAPE
    assert step(ld(T=1), slots=None, n=3) == DR_E_SHAPE       # without slots the pool is the batch
    assert step(ld(T=1, B=ops.MAX_PAGES + 1, D=4)) == DR_E_SHAPE
    d = ops.DrDesc(B=2, T=1, H=3, d_k=128, d_v=128, chunk=64, variant=1, dtype=1)
    assert dec(None) == DR_E_NULLPTR
    for name in ("q", "k", "v", "beta", "g", "pool", "slots", "o"):
        assert dec(d, **{name: None}) == DR_E_NULLPTR, name
    assert dec(d, wgate=FAKE[9]) == DR_E_UNSUPPORTED
    assert dec(d, n=0) == dec(d, n=ops.MAX_PAGES + 1) == DR_E_SHAPE
    assert dec(ops.DrDesc(B=ops.MAX_PAGES + 1, T=1, H=1, d_k=64, d_v=64, chunk=64, variant=1, dtype=1)) == DR_E_SHAPE
    assert dec(d, pool=FAKE[6] + 8) == DR_E_ALIGN
    assert dec(d, o=FAKE[6] + 15 * 3 * 128 * 128 * 4) == DR_E_ALIAS       # over the pool's last page
    assert dec(d, pool=FAKE[7]) == DR_E_ALIAS                             # over the slots
    assert dec(ops.DrDesc(B=2, T=2, H=3, d_k=128, d_v=128, chunk=64, variant=1, dtype=1)) == DR_E_SHAPE
    if not GPU:
        assert step(ld(T=1), slots=None, n=2) == DR_E_DEVICE
        assert step(ld(T=1, B=ops.MAX_PAGES + 1, D=4), slots=None, n=ops.MAX_PAGES + 1) == DR_E_DEVICE
        assert step(ld(T=1)) == dec(d) == DR_E_DEVICE


def test_pages():
    for call in (copy, compact):
        assert call(None) == DR_E_NULLPTR
        assert call(pd(), pool=None) == DR_E_NULLPTR
        for kw in (dict(page=0), dict(n_pages=0), dict(n_pages=ops.MAX_PAGES + 1), dict(n=-1),
                   dict(n=ops.MAX_PAGES + 1), dict(page=(1 << 37) + 1)):
            assert call(pd(**kw)) == DR_E_SHAPE, kw
    for name in ("dst", "src", "src_pool"):
        assert copy(pd(), **{name: None}) == DR_E_NULLPTR, name
    for name in ("slots", "out", "n_live"):
        assert compact(pd(), **{name: None}) == DR_E_NULLPTR, name
    assert copy(pd(), src_pages=7) == DR_E_SHAPE              # the same pool, another size
    assert copy(pd(), src_pool=FAKE[5], src_pages=0) == DR_E_SHAPE
    assert copy(pd(), src_pool=FAKE[0] + 4096) == DR_E_ALIAS  # a shifted view of the pool
    assert copy(pd(), dst=FAKE[0]) == DR_E_ALIAS
    assert copy(pd(), src=FAKE[2] + 2) == copy(pd(), pool=FAKE[0] + 4, src_pool=FAKE[5]) == DR_E_ALIGN
    assert compact(pd(), out=FAKE[1]) == DR_E_ALIAS           # slots are read while slots_out is written
    assert compact(pd(), n_live=FAKE[2]) == DR_E_ALIAS
    assert compact(pd(), n_live=FAKE[3] + 2) == DR_E_ALIGN
    assert copy(pd(n=0), dst=None, src=None) == DR_OK         # nothing to do
    if not GPU:
        assert copy(pd()) == copy(pd(), src_pool=FAKE[5], src_pages=3) == DR_E_DEVICE
        assert compact(pd(n=0), slots=None, out=None) == DR_E_DEVICE
        assert copy(pd(), dst=FAKE[1] + 4) == compact(pd(), slots=FAKE[1] + 4) == DR_E_DEVICE   # part of a list


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 4, 8)
    for call in (lambda: ops.linrec_fwd(x, x), lambda: ops.linrec_bwd(x, x, x, x), lambda: ops.linrec_step(x[0], x[0], x[0]),
                 lambda: ops.pages_copy(x, x, x), lambda: ops.pages_compact(x, x),
                 lambda: ops.delta_decode_slots("gdn", x, x, x, x, x, x), lambda: autograd.linear_recurrence(x, x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32, 2 ** 32 + 2, 2 ** 33 + 3])
def test_binding_refuses_sizes_past_32_bits(past):
    """Descriptors hold 32-bit sizes, and ctypes masks what does not fit: 2^32 + 2 tokens
    must not be taken as 2.  Tensors without storage, so that nothing is allocated."""
    with FakeTensorMode():
        def f32(*shape):
            return torch.empty(shape, device="cuda")

        def i32(n):
            return torch.empty(n, dtype=torch.int32, device="cuda")

        row, pool = f32(2, 1), f32(4, 8)
        calls = []
        for shape in ((past, 1, 1), (1, past, 1), (1, 1, past)):
            y = f32(*shape)
            st = f32(shape[0], -(-shape[1] // ops.LINREC_BLOCK), shape[2])
            calls += [lambda y=y: ops.linrec_fwd(y, y, o=y, want_state=False), lambda y=y, st=st: ops.linrec_bwd(
                y, y, st, y, want_dh0=False, out=dict(dx=y, dg=y))]
        for y in (f32(past, 1), f32(1, past)):
            calls.append(lambda y=y: ops.linrec_step(y, y, y, o=y))
        calls += [lambda: ops.linrec_step(row, row, f32(past, 1), slots=i32(2), o=row),
                  lambda: ops.pages_copy(f32(past, 8), i32(2), i32(2)), lambda: ops.pages_copy(pool, i32(past), i32(past)),
                  lambda: ops.pages_copy(pool, i32(2), i32(2), src_pool=f32(past, 8)),
                  lambda: ops.pages_compact(f32(past, 8), i32(2), slots_out=i32(2), n_live=i32(1)),
                  lambda: ops.pages_compact(pool, i32(past), slots_out=i32(past), n_live=i32(1))]
        for n, call in enumerate(calls):
            with pytest.raises(ops.DeltaRuleError) as e:
                call()
            assert e.value.status == DR_E_SHAPE, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("join", [torch.cat, torch.stack])
def test_gradients_are_taken_at_any_address(join, dtype):
    """The gradients that torch hands to the outputs of a joined tensor are contiguous parts
    of one buffer; the library takes them at multiples of 16 bytes."""
    parts = [torch.zeros(3, 7, 5, dtype=dtype, requires_grad=True) for _ in range(4)]
    seen = []

    class Same(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            return t.clone()

        @staticmethod
        def backward(ctx, grad):
            seen.append((grad, autograd._gradient(grad, dtype)))
            return grad

    whole = join([Same.apply(p) for p in parts])
    whole.backward(torch.arange(whole.numel(), dtype=dtype).view_as(whole))
    assert any(given.is_contiguous() and given.data_ptr() % 16 for given, _ in seen)
    for given, taken in seen:
        assert torch.equal(given, taken) and taken.is_contiguous() and taken.data_ptr() % 16 == 0
    even = torch.zeros(4, 4, dtype=dtype)
    assert autograd._gradient(even, dtype) is even                        # nothing copied without need
