"""What the layer operators (quantised rows, integer products with scales, MoE sort / dispatch / combine)
refuse, without a GPU: the binding's checks on stand-ins for device tensors, and the C entry points' own
checks, which come before the context is looked at."""

import ctypes as C

import pytest

ARG, SHAPE = -1, -2


@pytest.fixture(scope="module")
def fp():
    from sum_check_prover_b200 import build
    build.build()
    import sum_check_prover_b200 as m
    m.lib()
    return m


class Dev:
    type = "cuda"

    def __init__(self, index=0):
        self.index = index

    def __str__(self):
        return f"cuda:{self.index}"


class T:
    """A stand-in for a device tensor: shape, strides and type, with an address that nothing reads."""

    def __init__(self, *shape, dtype="float32", stride=None, device=0, ptr=1 << 20):
        self.shape, self.dtype, self.device, self._ptr = shape, "torch." + dtype, Dev(device), ptr
        dense, n = [], 1
        for s in reversed(shape):
            dense.insert(0, n)
            n *= s
        self._dense, self._stride, self._n = tuple(dense), tuple(stride or dense), n

    def get_device(self):
        return self.device.index

    def stride(self):
        return self._stride

    def is_contiguous(self):
        return all(s == d for s, d, n in zip(self._stride, self._dense, self.shape) if n > 1)

    def numel(self):
        return self._n

    def element_size(self):
        return {"float32": 4, "int32": 4, "int8": 1}.get(self.dtype[6:], 2)

    def data_ptr(self):
        return self._ptr


@pytest.fixture()
def ctx(fp):
    c = object.__new__(fp.Context)
    c._L, c.h, c.device = fp.lib(), None, 0
    yield c


def refused(call, text):
    with pytest.raises(ValueError, match=text):
        call()


def test_binding_checks_types_shapes_and_devices(ctx):
    i8 = dict(dtype="int8")
    i32 = dict(dtype="int32")
    good = T(4, 8)
    refused(lambda: ctx.quantize_rows(T(4, 8, dtype="int8"), T(4, 8, **i8), T(4), stream=0), "x must be float32")
    refused(lambda: ctx.quantize_rows(good, T(4, 7, **i8), T(4), stream=0), "q must be")
    refused(lambda: ctx.quantize_rows(good, T(4, 8), T(4), stream=0), "q must be int8")
    refused(lambda: ctx.quantize_rows(good, T(4, 8, **i8), T(5), stream=0), "scale must be")
    refused(lambda: ctx.quantize_rows(good, T(4, 8, **i8), T(4), pos=T(3, 1, **i32), stream=0), "pos must be")
    refused(lambda: ctx.quantize_rows(T(4, 8, device=1), T(4, 8, **i8), T(4), stream=0), "x must be on cuda:0")
    refused(lambda: ctx.quantize_rows(T(4, 8, stride=(1, 4)), T(4, 8, **i8), T(4), stream=0), "rows must be contiguous")
    refused(lambda: ctx.quantize_rows(T(4, 8, stride=(0, 1)), T(4, 8, **i8), T(4), stream=0), "rows must be contiguous")
    refused(lambda: ctx.matmul_i8(T(6, 8, **i8), T(4, 9, **i8), T(4, 6), T(6), T(4), stream=0), "x must be")
    refused(lambda: ctx.matmul_i8(T(6, 8, **i8), T(4, 8, **i8), T(4, 6), T(5), T(4), stream=0), "w_scale must be")
    refused(lambda: ctx.matmul_i8(T(6, 8, **i8), T(4, 8, **i8), T(4, 6, dtype="int32"), T(6), T(4), stream=0), "y must be")
    refused(lambda: ctx.matmul_i8(T(2, 6, 8, **i8), T(4, 8, **i8), T(4, 6), T(2, 6), T(4), stream=0), "w must be")
    refused(lambda: ctx.matmul_i8(T(2, 6, 8, **i8), T(4, 8, **i8), T(4, 6), T(2, 6), T(4), offsets=T(2, **i32), stream=0),
            "offsets must be")
    refused(lambda: ctx.moe_sort(T(4, 2, **i32), 3, T(3, **i32), T(4, 2, **i32), stream=0), "offsets must be")
    refused(lambda: ctx.moe_sort(T(4, 2, dtype="int64"), 3, T(4, **i32), T(4, 2, **i32), stream=0), "e must be int32")
    refused(lambda: ctx.moe_sort(T(4, 2, stride=(1, 4), **i32), 3, T(4, **i32), T(4, 2, **i32), stream=0), "contiguous")
    refused(lambda: ctx.moe_dispatch(good, T(4, 1, **i32), T(4, 8, dtype="float16"), stream=0), "rows must be float32")
    refused(lambda: ctx.moe_dispatch(good, T(4, 1, **i32), T(4, 9), stream=0), "rows must be")
    refused(lambda: ctx.moe_combine(good, T(4, 1, **i32), T(4, 8, dtype="int8"), stream=0), "out must be")
    refused(lambda: ctx.moe_combine(good, T(4, 2, **i32), T(4, 8), weights=T(4, 1), stream=0), "weights must be")
    refused(lambda: ctx.moe_combine(good, T(4, 1, **i32), T(4, 8), base=T(4, 8, dtype="float16"), stream=0), "base must be")
    refused(lambda: ctx.moe_combine_grad(T(4, 8), T(4, 9), T(4, 1, **i32), drows=T(4, 8), stream=0), "rows must be")
    refused(lambda: ctx.moe_combine_grad(T(4, 8), T(4, 8), T(4, 1, **i32), drows=T(4, 8, dtype="float16"), stream=0), "drows")
    refused(lambda: ctx.moe_combine_grad(T(4, 8), T(4, 8), T(4, 1, **i32), dweights=T(4, 2), stream=0), "dweights")


P = 1 << 20  # an address: aligned, never read


def test_quantize_checks(fp):
    f = fp.lib().fp_quantize_rows

    def rc(x=P, t=2, T=4, K=8, ldx=8, pos=None, k=0, R=4, q=P, ldq=8, s=P):
        return f(None, x, t, T, K, ldx, pos, k, R, q, ldq, s, None)

    assert rc() == ARG  # nothing wrong but the context
    for bad in (dict(t=3), dict(t=-1), dict(x=None), dict(q=None), dict(s=None), dict(x=P + 1), dict(s=P + 2),
                dict(pos=P + 1, k=1)):
        assert rc(**bad) == ARG, bad
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(K=0), dict(K=(1 << 20) + 1), dict(R=3), dict(ldx=7), dict(ldq=7),
                dict(pos=P, k=0), dict(pos=P, k=-1), dict(pos=P, T=1 << 24, k=128), dict(R=-1), dict(R=1 << 31)):
        assert rc(**bad) == SHAPE, bad


def test_matmul_checks(fp):
    f = fp.lib().fp_matmul_i8

    def rc(w=P, ldw=8, ws=P, E=1, M=6, K=8, x=P, ldx=8, xs=P, N=4, off=None, y=P, t=2, ldy=6):
        return f(None, w, ldw, ws, E, M, K, x, ldx, xs, N, off, y, t, ldy, None)

    assert rc() == ARG
    for bad in (dict(t=3), dict(w=None), dict(ws=None), dict(x=None), dict(xs=None), dict(y=None), dict(E=2),
                dict(y=P + 1), dict(ws=P + 1), dict(xs=P + 3), dict(off=P + 2)):
        assert rc(**bad) == ARG, bad
    for bad in (dict(M=0), dict(M=(1 << 24) + 1), dict(N=-1), dict(N=(1 << 24) + 1), dict(K=0), dict(K=1 << 17, ldw=1 << 17, ldx=1 << 17),
                dict(E=0), dict(E=4097, off=P), dict(E=4096, M=1 << 20, ldy=1 << 20, off=P), dict(ldw=7), dict(ldx=7), dict(ldy=5)):
        assert rc(**bad) == SHAPE, bad


def test_moe_checks(fp):
    L = fp.lib()

    def sort(e=P, n=8, E=4, off=P, pos=P):
        return L.fp_moe_sort(None, e, n, E, off, pos, None)

    assert sort() == ARG and sort(e=None) == ARG and sort(off=None) == ARG and sort(pos=None) == ARG
    assert sort(e=P + 1) == ARG and sort(off=P + 2) == ARG
    assert sort(n=-1) == SHAPE and sort(n=1 << 31) == SHAPE and sort(E=0) == SHAPE and sort(E=4097) == SHAPE

    def disp(x=P, T=4, b=8, ldx=8, pos=P, k=2, R=8, rows=P, ldr=8):
        return L.fp_moe_dispatch(None, x, T, b, ldx, pos, k, R, rows, ldr, None)

    assert disp() == ARG and disp(x=None) == ARG and disp(pos=None) == ARG and disp(rows=None) == ARG and disp(pos=P + 1) == ARG
    for bad in (dict(T=-1), dict(k=0), dict(b=0), dict(b=(1 << 24) + 1), dict(ldx=7), dict(ldr=7), dict(R=-1),
                dict(T=1 << 24, k=128)):
        assert disp(**bad) == SHAPE, bad

    def comb(rows=P, rt=2, R=8, ldr=8, pos=P, w=None, base=None, ldb=0, T=4, k=2, M=8, out=P, ot=2, ldo=8):
        return L.fp_moe_combine(None, rows, rt, R, ldr, pos, w, base, ldb, T, k, M, out, ot, ldo, None)

    assert comb() == ARG
    for bad in (dict(rt=3), dict(ot=-1), dict(rows=None), dict(pos=None), dict(out=None), dict(rows=P + 1), dict(out=P + 1),
                dict(base=P + 1, ldb=8), dict(w=P + 2)):
        assert comb(**bad) == ARG, bad
    for bad in (dict(T=-1), dict(k=0), dict(M=0), dict(ldr=7), dict(ldo=7), dict(base=P, ldb=7), dict(R=1 << 31)):
        assert comb(**bad) == SHAPE, bad

    def grad(dout=P, ot=2, ldd=8, rows=P, rt=2, R=8, ldr=8, pos=P, w=None, T=4, k=2, M=8, dr=P, lddr=8, dw=P):
        return L.fp_moe_combine_grad(None, dout, ot, ldd, rows, rt, R, ldr, pos, w, T, k, M, dr, lddr, dw, None)

    assert grad() == ARG
    for bad in (dict(rt=3), dict(ot=3), dict(dr=None, dw=None), dict(dout=None), dict(pos=None), dict(rows=None), dict(dr=P + 1),
                dict(dout=P + 1), dict(dw=P + 2)):
        assert grad(**bad) == ARG, bad
    for bad in (dict(T=-1), dict(k=0), dict(M=0), dict(ldd=7), dict(ldr=7), dict(lddr=7), dict(R=-1)):
        assert grad(**bad) == SHAPE, bad


def test_kernels_have_names(fp):
    names = fp.kernel_names()
    for n in ("quant_rows", "matmul_i8", "realign_rows", "moe_sort", "moe_dispatch", "moe_combine", "moe_grad"):
        assert n in names
    assert len(set(names)) == len(names)


def test_binding_leaves_what_it_does_not_know(fp):
    # the compiled binding makes no call for tensors of the CPU, stand-ins, wrong counts of arguments or what
    # is no number, and raises nothing: the methods' checks say what is wrong
    import torch
    short = fp._load_binding()
    f, i, q = torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int8)
    s = torch.zeros(2)
    for h in (None, 1 << 20, "h", 1 << 80):
        for stream in (0, 1 << 80, "s", object()):
            assert short.quantize_rows(h, 0, f, q, s, i, stream) is None
            assert short.matmul_i8(h, 0, q, q, f, s, s, None, stream) is None
            assert short.moe_sort(h, 0, i, 4, i, i, stream) is None
            assert short.moe_sort(h, 0, i, 1 << 80, i, i, stream) is None
            assert short.moe_dispatch(h, 0, f, i, f, stream) is None
            assert short.moe_combine(h, 0, f, i, f, None, None, stream) is None
            assert short.moe_combine_grad(h, 0, f, f, i, None, None, None, stream) is None
    t = T(2, 4)
    assert short.moe_combine(1 << 20, 0, t, t, t, None, None, 0) is None
    assert short.moe_dispatch() is None and short.moe_sort(1, 2, 3) is None


def test_counts_past_an_int(ctx):
    big = 1 << 32
    refused(lambda: ctx.moe_sort(T(4, 1, dtype="int32"), big + 3, T(big + 4, dtype="int32"), T(4, 1, dtype="int32"), stream=0), "E must be below")
    refused(lambda: ctx.moe_dispatch(T(1, 8), T(1, big + 1, dtype="int32"), T(4, 8), stream=0), "pos' choices")
    refused(lambda: ctx.matmul_i8(T(big + 1, 1, 1, dtype="int8"), T(4, 1, dtype="int8"), T(4, 1), T(big + 1, 1), T(4),
                                  offsets=T(big + 2, dtype="int32"), stream=0), "experts must be below")


def test_status_without_a_context(fp):
    assert fp.lib().fp_ops_status(None) == ARG and fp.lib().fp_ops_selftest(None, None) == ARG


def test_choices_past_what_the_kernels_step_over(fp):
    # a single token with more than 2^30 choices: steps of several at a time would pass 2^31
    L = fp.lib()
    for k, code in (((1 << 31) - 1, SHAPE), ((1 << 30) + 1, SHAPE), (1 << 30, ARG)):  # ARG: nothing wrong but the context
        assert L.fp_moe_dispatch(None, P, 1, 8, 8, P, k, 8, P, 8, None) == code
        assert L.fp_moe_combine(None, P, 2, 8, 8, P, None, None, 0, 1, k, 8, P, 2, 8, None) == code
        assert L.fp_moe_combine_grad(None, P, 2, 8, P, 2, 8, 8, P, None, 1, k, 8, P, 8, P, None) == code


def test_values_still_to_be_conjugated_or_negated(ctx):
    # such a view has another tensor's values at its address
    class Conj(T):
        def is_conj(self):
            return True

    class Neg(T):
        def is_neg(self):
            return True

    pos = T(4, 1, dtype="int32")
    refused(lambda: ctx.moe_dispatch(Conj(4, 8), pos, T(4, 8), stream=0), "x must be resolved")
    refused(lambda: ctx.moe_dispatch(T(4, 8), pos, Conj(4, 8), stream=0), "rows must be resolved")
    refused(lambda: ctx.quantize_rows(Neg(4, 8), T(4, 8, dtype="int8"), T(4), stream=0), "x must be resolved")
    refused(lambda: ctx.quantize_rows(T(4, 8), T(4, 8, dtype="int8"), Neg(4), stream=0), "scale must be resolved")


def test_trim_without_a_context(fp):
    assert fp.lib().fp_ops_trim(None) == ARG
