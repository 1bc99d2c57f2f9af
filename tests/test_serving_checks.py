"""Refusals of the serving operators, without a GPU: the binding's size checks
(host tensors stop at "must be a CUDA tensor") and the library's own checks
(no device pointer is touched before a failed one)."""
import ctypes as C

import pytest
import torch

import integer_only_quantized_int8_b200 as ivit
from integer_only_quantized_int8_b200 import build as ivit_build


@pytest.fixture(scope="module", autouse=True)
def built():
    ivit_build.build()


def i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def refused(fn, *a, **k):
    with pytest.raises(ValueError, match="holds|shape"):
        fn(*a, **k)


def past_checks(fn, *a, **k):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fn(*a, **k)


P = 0x100000
D = ivit.Dyadic(1, 0)
NONE = ivit.Residual(0, 0, 0)


def test_linear_lora_sizes():
    M, K, N, R, n = 32, 64, 48, 16, 3
    ws = torch.zeros(M * R, dtype=torch.uint8)

    def call(X=i8(M, K), W=i8(N, K), b=i32(N), A=i8(n, R, K), bt=i32(n, R), ct=i8(n, R), B=i8(n, N, R), idx=i32(4),
             rows=8, Y=i8(M, N), skip=None):
        return (ivit.ivit_linear_lora, X, W, None, b, i8(N), (A, bt, ct, B), idx, rows, Y, ws, 8, skip, (1, 1, 1))

    past_checks(*call())
    past_checks(*call(skip=i8(M, N)))
    for bad in (dict(W=i8(N, K + 16)), dict(b=i32(N - 1)), dict(A=i8(n, R, K - 16)), dict(bt=i32(n * R - 1)),
                dict(ct=i8(n, R - 1)), dict(B=i8(n - 1, N, R)), dict(B=i8(n, N - 16, R)), dict(idx=i32(3)),
                dict(rows=5), dict(rows=0), dict(rows=-8), dict(Y=i8(M, N - 16)), dict(skip=i8(M - 1, N))):
        refused(*call(**bad))
    X, W, t, ad = i8(M, K), i8(N, K), (i32(N), i32(N), i8(N)), (i8(n, R, K), i32(n, R), i8(n, R), i8(n, N, R))
    past_checks(ivit.ivit_linear_lora_shiftgelu, X, W, *t, ad, i32(4), 8, 4, 30, 8, (1, 0), i8(M, N), ws)
    refused(ivit.ivit_linear_lora_shiftgelu, X, W, *t, ad, i32(4), 7, 4, 30, 8, (1, 0), i8(M, N), ws)


def test_linear_lora_library_checks():
    L = ivit.lib()

    def call(M=32, K=64, N=48, n=3, R=16, rows=8, idx=P, ws=P, wb=32 * 16, gelu=False, rounding=0, out_bits=8, **ptr):
        l = ivit.Lora(n, R, ptr.get("A", P), ptr.get("b_t", P), ptr.get("c_t", P), ptr.get("B", P))
        lp = None if ptr.get("null") else C.byref(l)
        if gelu:
            return L.ivit_linear_lora_shiftgelu(P, M, K, P, N, None, P, P, rounding, lp, idx, rows, 4, 30, 8, D, P, ws, wb,
                                                None)
        return L.ivit_linear_lora(P, M, K, P, N, None, P, P, out_bits, rounding, lp, idx, rows, None, NONE, P, ws, wb,
                                  None)

    assert ivit.ivit_linear_lora_workspace_bytes(32, 16) == 512
    assert ivit.ivit_linear_lora_workspace_bytes(33, 16) == 768
    assert ivit.ivit_linear_lora_workspace_bytes(-1, 16) == 0
    for gelu in (False, True):
        for bad in (dict(R=8), dict(R=24), dict(R=144, wb=1 << 20), dict(n=0), dict(rows=0), dict(rows=5), dict(idx=None),
                    dict(ws=None), dict(ws=P + 16), dict(wb=511), dict(A=None), dict(b_t=None), dict(c_t=None),
                    dict(B=None), dict(A=P + 1), dict(B=P + 8), dict(idx=P + 4), dict(null=True), dict(rounding=2),
                    dict(K=72), dict(N=40), dict(M=0)):
            assert call(gelu=gelu, **bad) == 1, bad
    assert call(out_bits=9) == 1
    assert call(K=16400) == 2
    assert L.ivit_linear_lora_shiftgelu(P, 32, 64, P, 48, None, P, P, 0, C.byref(ivit.Lora(3, 16, P, P, P, P)), P, 8, 0, 30,
                                        8, D, P, P, 512, None) == 1


def test_residual_norm_sizes():
    r, c = 12, 64
    n = (i8(c), i32(c), 7, 23, (1, 0))

    def call(x=i8(r, c), o=i8(r, c), s=i32(c), y=i8(r, c), **k):
        return (ivit.ivit_residual_norm, x, o, s, 1, 0, y), k

    def run(check, **k):
        a, kk = call(**k)
        check(*a, **kk)

    run(past_checks)
    run(past_checks, post=n, pre=n, z=i8(r, c), gate=i8(3, c), gate_rows=5)
    for bad in (dict(o=i8(r - 1, c)), dict(s=i32(c - 1)), dict(y=i8(r, c - 16)), dict(pre=n), dict(z=i8(r, c)),
                dict(pre=n, z=i8(r, c + 16)), dict(gate=i8(2, c), gate_rows=5), dict(gate=i8(3, c), gate_rows=0),
                dict(post=(i8(c - 1), i32(c), 7, 23, (1, 0))), dict(pre=(i8(c), i32(c + 1), 7, 23, (1, 0)), z=i8(r, c))):
        run(refused, **bad)


def test_residual_norm_library_checks():
    L = ivit.lib()
    X, O, G, Y, Z, S = (P + i * 0x10000 for i in range(6))

    def call(skip=X, branch=O, rows=4, cols=32, post=True, gate=G, T=2, scale=S, b=1, c=0, pre=True, y=Y, z=Z, **n):
        nm = ivit.Norm(n.get("gamma", P), n.get("beta", P), n.get("F", 7), n.get("M", 23), n.get("out", D))
        p = C.byref(nm)
        return L.ivit_residual_norm(skip, branch, rows, cols, p if post else None, gate, T, scale, b, c,
                                    p if pre else None, y, z, None)

    for bad in (dict(cols=24), dict(cols=0), dict(cols=2064), dict(rows=-1), dict(b=-1), dict(c=32), dict(c=-1),
                dict(T=0), dict(skip=None), dict(branch=None), dict(scale=None), dict(y=None), dict(z=None),
                dict(skip=X + 1), dict(branch=O + 8), dict(scale=S + 4), dict(y=Y + 2), dict(z=Z + 4), dict(gate=G + 1),
                dict(gamma=None), dict(beta=None), dict(gamma=P + 1), dict(F=15), dict(F=-1), dict(M=24), dict(M=6),
                dict(out=ivit.Dyadic(1, 32)), dict(out=ivit.Dyadic(-1, 3)),
                # overlaps other than an output in an input's exact place
                dict(y=X + 32), dict(z=O + 16), dict(y=G), dict(z=G + 32), dict(y=Z), dict(y=Z + 64), dict(y=X - 112)):
        assert call(**bad) == 1, bad
    assert call(rows=0, skip=None, branch=None, y=None, z=None, scale=None) == 0
    assert call(rows=0, c=40) == 1


def test_attention_diff_checks():
    args = ((1, 0), 8, 4, 30, 8)
    past_checks(ivit.ivit_attention_diff, i8(18, 768), 2, 9, 2, *args, i32(2), (1, 0), i8(18, 256))
    for qkv, lam, ctx in ((i8(18, 384), i32(2), i8(18, 256)), (i8(17, 768), i32(2), i8(18, 256)),
                          (i8(18, 768), i32(1), i8(18, 256)), (i8(18, 768), i32(2), i8(18, 128))):
        refused(ivit.ivit_attention_diff, qkv, 2, 9, 2, *args, lam, (1, 0), ctx)
    L = ivit.lib()

    def call(qkv=P, B=2, N=9, H=2, logit=D, k_s=8, I0=4, M=30, k_out=8, lam=P, out=D, ctx=P):
        return L.ivit_attention_diff(qkv, B, N, H, logit, k_s, I0, M, k_out, lam, out, ctx, None)

    for bad in (dict(qkv=None), dict(lam=None), dict(ctx=None), dict(qkv=P + 1), dict(lam=P + 4), dict(ctx=P + 8),
                dict(B=-1), dict(N=-1), dict(H=0), dict(k_s=1), dict(k_s=9), dict(I0=0), dict(I0=(1 << 22) + 1), dict(M=31),
                dict(M=6), dict(k_out=0), dict(k_out=9), dict(logit=ivit.Dyadic(1, 32)), dict(out=ivit.Dyadic(-1, 0))):
        assert call(**bad) == 1, bad
    assert call(N=641) == 2
    assert call(H=2049) == 2
    assert call(B=0) == 0 and call(N=0) == 0


def test_residual_norm_refuses_outputs_over_its_tables():
    """scale and the norms' gamma and beta are read by every block while others write: no output may lie in them."""
    L = ivit.lib()
    X, O, Y, Z, S, PG, PB, NG, NB = (P + i * 0x10000 for i in range(9))
    cols = 32

    def call(post=True, pre=True, y=Y, z=Z):
        po, nx = ivit.Norm(PG, PB, 7, 23, D), ivit.Norm(NG, NB, 7, 23, D)
        return L.ivit_residual_norm(X, O, 4, cols, C.byref(po) if post else None, None, 1, S, 1, 0,
                                    C.byref(nx) if pre else None, y, z, None)

    out = 4 * cols   # bytes of y and of z
    for table, size in ((S, 4 * cols), (PG, cols), (PB, 4 * cols), (NG, cols), (NB, 4 * cols)):
        for at in (table, table + size - 16, table - out + 16):
            assert call(y=at) == 1, (hex(table), at - table)
            assert call(z=at) == 1, (hex(table), at - table)
    assert call(pre=False, y=S, z=None) == 1 and call(pre=False, y=PB, z=None) == 1
    assert call(post=False, y=NG) == 1 and call(post=False, z=S) == 1
    if not torch.cuda.is_available():   # beside a table, or where a norm that is not there would lie: past the checks
        for ok in (dict(y=S + 4 * cols), dict(y=S - out), dict(z=NB + 4 * cols), dict(z=PG - out),
                   dict(post=False, y=PG), dict(pre=False, y=NB, z=None)):
            assert call(**ok) in (2, 3), ok


@pytest.mark.parametrize("gate_rows", [(1 << 63) - 1, (1 << 63) - 12])
def test_residual_norm_gate_of_all_rows(gate_rows):
    """A gate_rows near the largest integer is one gate for every row: the gate still has to hold that row."""
    r, c = 12, 64

    def call(gate, rows=r):
        ivit.ivit_residual_norm(i8(rows, c), i8(rows, c), i32(c), 1, 0, i8(rows, c), gate=gate, gate_rows=gate_rows)

    refused(call, i8(0, c))
    refused(call, i8(c - 1))
    past_checks(call, i8(1, c))
    past_checks(call, i8(0, c), rows=0)


class Fields:
    def __init__(self, b, c):
        self.b, self.c = b, c


class Raw:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


def test_bad_plain_arguments_raise():
    """Numbers, dyadics and streams that do not convert raise before anything is passed on; none is cut to 32 bits."""
    r, c = 12, 64

    def diff(B=2, N=9, H=2, logit=(1, 0), k_s=8, I0=4, M=30, k_out=8, out=(1, 0), stream=None):
        ivit.ivit_attention_diff(i8(18, 768), B, N, H, logit, k_s, I0, M, k_out, i32(2), out, i8(18, 256), stream=stream)

    def norm(b_skip=1, shift=0, n=None, stream=None):
        ivit.ivit_residual_norm(i8(r, c), i8(r, c), i32(c), b_skip, shift, i8(r, c), post=n, stream=stream)

    def tables(F=7, M=23, out=(1, 0)):
        return dict(n=(i8(c), i32(c), F, M, out))

    def lora(bits=8, res=(1, 1, 1), stream=None, rounding=0):
        ad = (i8(3, 16, 64), i32(3, 16), i8(3, 16), i8(3, 48, 16))
        ivit.ivit_linear_lora(i8(32, 64), i8(48, 64), None, i32(48), i8(48), ad, i32(4), 8, i8(32, 48),
                              torch.zeros(512, dtype=torch.uint8), bits, i8(32, 48), res, stream, rounding)

    def gelu(I0=4, M=30, k_out=8, out=(1, 0), stream=None, rounding=0):
        ad = (i8(3, 16, 64), i32(3, 16), i8(3, 16), i8(3, 48, 16))
        ivit.ivit_linear_lora_shiftgelu(i8(32, 64), i8(48, 64), None, i32(48), i8(48), ad, i32(4), 8, I0, M, k_out, out,
                                        i8(32, 48), torch.zeros(512, dtype=torch.uint8), stream, rounding)

    def raises(error, fn, **k):
        with pytest.raises(error):
            fn(**k)

    for fn in (diff, norm, lora, gelu):
        past_checks(fn)
        for ok in (0, Raw(0), Raw(1 << 40)):
            past_checks(fn, stream=ok)
        raises(AttributeError, fn, stream=object())
        raises(TypeError, fn, stream=Raw("0"))
        raises(OverflowError, fn, stream=1 << 70)
        raises(OverflowError, fn, stream=Raw(1 << 70))
    for bad, error in ((Fields("1", 0), TypeError), (Fields(1, None), TypeError), (Fields(1.5, 0), TypeError),
                       (Fields(1 << 32, 0), OverflowError), (Fields(1, 1 << 80), OverflowError), (object(), AttributeError),
                       ((1, "0"), TypeError), ((1 << 32, 0), OverflowError), ((1,), ValueError), ((1, 0, 0), ValueError)):
        raises(error, diff, logit=bad)
        raises(error, diff, out=bad)
        raises(error, gelu, out=bad)
        raises(error, norm, **tables(out=bad))
    past_checks(diff, logit=ivit.Dyadic(1, 0), out=Fields(1, 0))
    past_checks(norm, **tables(out=ivit.Dyadic(1, 0)))
    for v, error in ((None, TypeError), (1.5, TypeError), (1 << 31, OverflowError), (1 << 64, OverflowError)):
        for k in ("B", "N", "H", "k_s", "I0", "M", "k_out"):
            raises(error, diff, **{k: v})
        for k in ("b_skip", "shift"):
            raises(error, norm, **{k: v})
        raises(error, norm, **tables(F=v))
        raises(error, norm, **tables(M=v))
        for k in ("bits", "rounding"):
            raises(error, lora, **{k: v})
        raises(error, lora, res=(1, v, 1))
        for k in ("I0", "M", "k_out", "rounding"):
            raises(error, gelu, **{k: v})


def test_a_sequence_that_shrinks_while_it_is_read():
    """A list emptied by the conversion of its first element is not read past its end."""
    pair = []

    class Empties:
        def __index__(self):
            pair.clear()
            return 1

    pair += [Empties(), 0]
    with pytest.raises(ValueError):
        ivit.ivit_attention_diff(i8(18, 768), 2, 9, 2, pair, 8, 4, 30, 8, i32(2), (1, 0), i8(18, 256))
