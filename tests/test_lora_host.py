"""Host-side checks of the low-rank adapter and clipping calls that need no GPU: sizes, and
arguments refused before the device is touched (the pointers below are never dereferenced)."""
import copy
import ctypes
import pickle

import pytest
import torch

P = ctypes.c_void_p
W = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from unstructured_sparse_linear_gb300 import _lib, build
    build.build()
    return _lib.load()


def test_sizes(lib):
    assert lib.spops_lora_plan_size(-1, 1) == 0 and lib.spops_lora_plan_size(5, 0) == 0
    small = lib.spops_lora_plan_size(1, 1)
    assert 0 < small < lib.spops_lora_plan_size(1000, 1) < lib.spops_lora_plan_size(1000, 50)
    assert lib.spops_lora_grad_workspace_size(0, 8) >= 16
    assert lib.spops_lora_grad_workspace_size(100, 8) >= 2 * 100 * 8 * 4
    assert lib.spops_grad_set_size(-1) == 0 and lib.spops_grad_set_size(10) > lib.spops_grad_set_size(1) > 0
    assert lib.spops_grad_norm_workspace_size() >= 8


def add(lib, **kw):
    a = dict(X=P(0x100000), ldx=64, A=P(0x200000), B=P(0x300000), scale=None, scale_all=1.0, dtype=2, tokens=8, k=64,
             n=32, rank=4, na=2, base=P(0x400000), ldb=32, Y=P(0x500000), ldy=32, h=None, plan=P(0x600000))
    a.update(kw)
    return lib.spops_lora_add(a["X"], a["ldx"], a["A"], a["B"], a["scale"], a["scale_all"], a["dtype"], a["tokens"],
                              a["k"], a["n"], a["rank"], a["na"], a["base"], a["ldb"], a["Y"], a["ldy"], a["h"],
                              a["plan"], None)


def test_lora_add_refusals(lib):
    assert add(lib, tokens=0) == 0  # nothing to do
    for bad in (dict(dtype=7), dict(tokens=-1), dict(k=0), dict(n=0), dict(rank=0), dict(na=0), dict(A=None),
                dict(X=None), dict(X=P(0x100001)), dict(ldx=63), dict(ldy=31), dict(ldb=31), dict(plan=None),
                dict(plan=P(0x600004)), dict(scale=P(0x700002)), dict(scale_all=float("inf")), dict(Y=None),
                dict(h=P(0x800002)), dict(Y=P(0x100000)), dict(Y=P(0x200000)), dict(Y=P(0x400002)),
                dict(h=P(0x500000)), dict(h=P(0x100000)), dict(base=P(0x500000), ldb=40)):
        assert add(lib, **bad) == 1, bad
    assert add(lib, rank=129) == 2 and b"129" in lib.spops_last_error()


def grad(lib, **kw):
    a = dict(dY=P(0x100000), lddy=32, X=P(0x200000), ldx=64, A=P(0x300000), B=P(0x400000), scale=None, scale_all=1.0,
             dtype=2, tokens=8, k=64, n=32, rank=4, na=2, h=None, base=None, ldb=64, dX=P(0x500000), lddx=64,
             dA=P(0x600000), dB=P(0x700000), plan=P(0x800000), ws=P(0x900000), size=W)
    a.update(kw)
    return lib.spops_lora_grad(a["dY"], a["lddy"], a["X"], a["ldx"], a["A"], a["B"], a["scale"], a["scale_all"],
                               a["dtype"], a["tokens"], a["k"], a["n"], a["rank"], a["na"], a["h"], a["base"], a["ldb"],
                               a["dX"], a["lddx"], a["dA"], a["dB"], a["plan"], a["ws"], a["size"], None)


def test_lora_grad_refusals(lib):
    assert grad(lib, dX=None, dA=None, dB=None) == 0  # nothing asked for
    for bad in (dict(dtype=-1), dict(rank=0), dict(dY=None), dict(X=None), dict(lddy=31), dict(lddx=63),
                dict(h=P(0x900002)), dict(dX=P(0x200000)), dict(dX=P(0x100000)), dict(dA=P(0x300000)),
                dict(dA=P(0x700000)), dict(dB=P(0x200000)), dict(base=P(0x500002)), dict(base=P(0x600000)),
                dict(dA=P(0x600001))):
        assert grad(lib, **bad) == 1, bad
    assert grad(lib, rank=200) == 2
    assert grad(lib, size=16) == 3 and grad(lib, ws=None) == 3 and grad(lib, ws=P(0x900008)) == 3


def test_lora_plan_refusals(lib):
    f = lib.spops_lora_plan_build
    assert f(P(0x1000), -1, 1, P(0x2000), W, None) == 1 and f(P(0x1000), 4, 0, P(0x2000), W, None) == 1
    assert f(P(0x1002), 4, 1, P(0x2000), W, None) == 1
    assert f(P(0x1000), 4, 1, P(0x2004), W, None) == 3 and f(P(0x1000), 4, 1, P(0x2000), 16, None) == 3
    assert f(P(0x1000), 0, 1, None, 0, None) == 0


def build_set(lib, grads, outs, counts, dtypes, set_=P(0x10000), size=W):
    n = len(grads)
    chunks, in_place = ctypes.c_int64(-1), ctypes.c_int32(-1)
    return lib.spops_grad_set_build((P * n)(*grads), (P * n)(*outs) if outs is not None else None,
                                    (ctypes.c_int64 * n)(*counts), (ctypes.c_int32 * n)(*dtypes), n, set_, size,
                                    ctypes.byref(chunks), ctypes.byref(in_place), None)


def test_grad_set_refusals(lib):
    assert build_set(lib, [0x1000], None, [-1], [0]) == 1
    assert build_set(lib, [0x1000], None, [4], [3]) == 1
    assert build_set(lib, [0x1002], None, [4], [0]) == 1
    assert build_set(lib, [0], None, [4], [0]) == 1
    assert build_set(lib, [0x1000, 0x1008], None, [4, 4], [0, 0]) == 1         # two gradients overlap
    assert build_set(lib, [0x1000, 0x3000], [0x2000, 0x2004], [4, 4], [0, 0]) == 1  # two outputs do
    assert build_set(lib, [0x1000, 0x3000], [0x2000, 0x1000], [4, 4], [0, 0]) == 1  # an output over a gradient
    assert b"overlaps" in lib.spops_last_error()
    assert build_set(lib, [0x1000], None, [4], [0], size=8) == 3
    assert build_set(lib, [0x1000], None, [4], [0], set_=P(0x10008)) == 3


def test_clip_refusals(lib):
    f = lib.spops_clip_grads
    assert f(P(0x1000), 1, 1, 1, -1.0, P(0x2000), P(0x3000), W, None) == 1
    assert f(P(0x1000), 1, 1, 1, float("nan"), P(0x2000), P(0x3000), W, None) == 1
    assert f(None, 1, 1, 1, 1.0, P(0x2000), P(0x3000), W, None) == 1
    assert f(P(0x1000), 1, 1, 1, 1.0, P(0x2002), P(0x3000), W, None) == 1
    assert f(P(0x1000), 1, 1, 1, 1.0, P(0x2000), P(0x3000), 8, None) == 3
    assert lib.spops_grad_norm(P(0x1000), -1, 1, P(0x2000), P(0x3000), W, None) == 1


def test_argument_blocks(lib):
    """The calls that take their arguments in a block see the same ones: each refusal names the value."""
    from unstructured_sparse_linear_gb300 import lora

    def add_block(x=0x100000, ldx=64, ldb=32, ldy=32, h=0, plan=0x600000, scale_all=1.0, dtype=2, tokens=8, k=64, n=32,
                  rank=4, na=2):
        return lib.spops_lora_add_block(lora._ADD_ARGS(x, ldx, 0x200000, 0x300000, 0, 0x400000, ldb, 0x500000, ldy, h,
                                                       plan, 0, scale_all, dtype, tokens, k, n, rank, na))

    def grad_block(dy=0x100000, lddy=32, ldx=64, h=0, ldb=64, lddx=64, da=0x600000, db=0x700000, plan=0x800000,
                   ws=0x900000, size=W, scale_all=1.0, dtype=2, tokens=8, k=64, n=32, rank=4, na=2):
        return lib.spops_lora_grad_block(lora._GRAD_ARGS(dy, lddy, 0x200000, ldx, 0x300000, 0x400000, 0, h, 0xa00000,
                                                         ldb, 0x500000, lddx, da, db, plan, ws, size, 0, scale_all,
                                                         dtype, tokens, k, n, rank, na))

    assert lib.spops_lora_add_block(None) == 1 and lib.spops_lora_grad_block(None) == 1
    assert add_block(tokens=0) == 0 and grad_block(tokens=0, da=0, db=0) == 0
    for call in (add_block, grad_block):
        assert call(dtype=7) == 1 and b"7" in lib.spops_last_error()
        assert call(tokens=-11) == 1 and b"-11" in lib.spops_last_error()
        assert call(k=-12) == 1 and b"-12" in lib.spops_last_error()
        assert call(n=-13) == 1 and b"-13" in lib.spops_last_error()
        assert call(na=-14) == 1 and b"-14" in lib.spops_last_error()
        assert call(rank=129) == 2 and b"129" in lib.spops_last_error()
        assert call(scale_all=float("nan")) == 1 and b"scale_all" in lib.spops_last_error()
        assert call(plan=0x600004) == 1 and b"plan" in lib.spops_last_error()
        assert call(ldx=61) == 1 and b"X" in lib.spops_last_error()
        assert call(h=0x800002) == 1 and b"h is not" in lib.spops_last_error()
    assert add_block(x=0) == 1 and add_block(ldb=31) == 1 and add_block(ldy=31) == 1
    assert grad_block(dy=0) == 1 and grad_block(lddy=31) == 1 and grad_block(ldb=63) == 1 and grad_block(lddx=63) == 1
    assert grad_block(da=0x600001) == 1 and grad_block(db=0x700001) == 1
    assert grad_block(ws=0x900008) == 3 and grad_block(size=16) == 3


def test_plan_sizes_beyond_32_bits():
    import unstructured_sparse_linear_gb300 as sp
    for tokens, n in ((2 ** 31, 1), (2 ** 32 + 5, 1), (-1, 1), (5, 2 ** 31), (5, 2 ** 32 + 1), (5, 0)):
        with pytest.raises(ValueError, match="tokens >= 0"):
            sp.lora_plan(None, n, tokens=tokens, device="cuda:0")


def test_copies_hold_no_plan_of_the_original():
    import unstructured_sparse_linear_gb300 as sp
    from unstructured_sparse_linear_gb300.lora import Built
    for cls in (sp.LoraPlan, sp.GradSet):
        table = cls.__new__(cls)
        assert isinstance(table, Built)
        for copier in (copy.copy, copy.deepcopy, pickle.dumps):
            with pytest.raises(TypeError, match=cls.__name__):
                copier(table)
    layer = sp.RosaLinear(torch.randn(6, 4), 2)
    plan = layer._plans[3] = sp.LoraPlan.__new__(sp.LoraPlan)
    for twin in (copy.copy(layer), copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        assert twin._plans == {} and torch.equal(twin.A, layer.A) and torch.equal(twin.weight, layer.weight)
    assert layer._plans == {3: plan}
