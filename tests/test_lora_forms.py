"""Every kernel that a linear layer with adapters can take, with several tiles per
CTA where its form allows that.  The form of each shape is looked up without a
GPU, so a changed rule shows which of them lost its shape; on the GPU each is
compared with the plain 64-bit form, bit for bit."""
import numpy as np
import pytest

import integer_only_quantized_int8_b200 as ivit
from integer_only_quantized_int8_b200 import build as ivit_build
from oracle import serving

from test_gpu_serving import GELU, LoraCase, dev, guarded, host, workspace

ONE, MMA, DP4A, LONG = 1, 2, 3, 4
REQUEST, ADAPTER = 0, 1
SHARED, OWN = 0, 1
SMS = 148

# (requests, rows, K, N, R, n): the form, and whether a CTA takes more than one tile
SHAPES = [
    ((1, 2, 48, 400, 128, 64), (ONE, 64, REQUEST, 0), False),
    ((4, 1, 272, 304, 128, 1), (ONE, 64, ADAPTER, 0), False),
    ((41, 33, 784, 2384, 80, 57), (MMA, 128, REQUEST, SHARED), True),
    ((220, 7, 784, 2096, 112, 9), (MMA, 128, ADAPTER, SHARED), True),
    ((38, 65, 784, 1888, 64, 64), (MMA, 160, REQUEST, SHARED), True),
    ((363, 7, 784, 1808, 64, 20), (MMA, 160, ADAPTER, SHARED), True),
    ((45, 33, 784, 1840, 128, 64), (MMA, 176, REQUEST, SHARED), False),
    ((21, 130, 784, 2080, 32, 64), (MMA, 176, REQUEST, SHARED), True),
    ((2841, 1, 784, 2096, 48, 2), (MMA, 176, ADAPTER, SHARED), True),
    ((85, 33, 784, 2336, 32, 6), (MMA, 192, REQUEST, SHARED), True),
    ((177, 7, 784, 2400, 32, 5), (MMA, 192, ADAPTER, SHARED), False),
    ((2750, 1, 784, 2336, 32, 1), (MMA, 192, ADAPTER, SHARED), True),
    ((7, 333, 208, 1184, 48, 57), (MMA, 128, REQUEST, OWN), True),
    ((474, 5, 400, 1184, 128, 6), (MMA, 128, ADAPTER, OWN), True),
    ((515, 3, 144, 1440, 32, 70), (MMA, 144, REQUEST, OWN), False),
    ((16, 130, 512, 2192, 48, 3), (MMA, 144, REQUEST, OWN), True),
    ((2868, 1, 272, 1600, 128, 2), (MMA, 144, ADAPTER, OWN), True),
    ((81, 33, 400, 2000, 128, 20), (MMA, 160, REQUEST, OWN), True),
    ((2787, 1, 144, 1808, 112, 4), (MMA, 160, ADAPTER, OWN), True),
    ((14, 1, 128, 400, 32, 20), (DP4A, 16, 0, 0), False),
    ((173, 5, 144, 272, 16, 20), (DP4A, 48, 0, 0), False),
    ((396, 1, 272, 2368, 32, 57), (DP4A, 128, 0, 0), False),
    ((2236, 1, 144, 1168, 16, 57), (DP4A, 128, 0, 0), True),
    # ranks above 32: a row of B by four lanes (to 64) or eight, some of them idle
    ((40, 1, 128, 272, 80, 37), (LONG, 16, 0, 0), False),
    ((39, 1, 784, 144, 48, 64), (LONG, 16, 0, 0), False),
    ((482, 5, 16, 112, 64, 20), (LONG, 48, 0, 0), False),
    ((130, 3, 256, 1040, 96, 61), (LONG, 48, 0, 0), False),
    ((512, 1, 1024, 2048, 128, 64), (LONG, 128, 0, 0), False),
    ((762, 2, 272, 1808, 48, 64), (LONG, 128, 0, 0), True),
    ((1500, 1, 144, 1744, 64, 60), (LONG, 128, 0, 0), True),
    ((1574, 1, 400, 1424, 128, 64), (LONG, 128, 0, 0), True),
    ((577, 1, 144, 1584, 96, 57), (LONG, 128, 0, 0), False),
    ((1400, 1, 208, 2064, 112, 70), (LONG, 128, 0, 0), True),
    ((1300, 1, 48, 2064, 80, 128), (LONG, 128, 0, 0), True),
]


@pytest.fixture(scope="module", autouse=True)
def built():
    ivit_build.build()


def tiles(shape, form):
    req, rows, _, N = shape[:4]
    return -(-N // 128) * -(-req * rows // form[1])


@pytest.mark.parametrize("shape,form,several", SHAPES)
def test_form_of_each_shape(shape, form, several):
    req, rows, K, N, R, n = shape
    for gelu in (False, True):
        assert ivit.ivit_selftest_lora_form(req * rows, K, N, n, R, rows, gelu, SMS) == form
    assert (tiles(shape, form) > SMS) == several


def test_every_form_has_a_shape():
    """Those that a random walk over sizes meets are all listed, with several tiles per CTA where it meets that."""
    have = {(form, tiles(shape, form) > SMS) for shape, form, _ in SHAPES}
    r = np.random.default_rng(1)
    for _ in range(20000):
        rows = int(r.choice([1, 1, 2, 3, 5, 7, 9, 17, 33, 65, 130, 197, 333, 577]))
        req = max(1, int(2 ** r.uniform(0, 14) / rows))
        K, N, R = 16 * int(2 ** r.uniform(0, 8)), 16 * int(2 ** r.uniform(0, 8)), 16 * int(r.integers(1, 9))
        n = int(2 ** r.uniform(0, 8))
        form = ivit.ivit_selftest_lora_form(req * rows, K, N, n, R, rows, bool(r.integers(2)), SMS)
        several = -(-N // 128) * -(-req * rows // form[1]) > SMS
        assert (form, True) in have or (form, several) in have, (req, rows, K, N, R, n, form)
        if several:
            assert (form, True) in have, (req, rows, K, N, R, n, form)


def test_form_refusals():
    import ctypes as C
    L, form = ivit.lib(), (C.c_int32 * 4)()
    ok = dict(M=64, K=64, N=64, n=1, R=16, rows=8, gelu=0, sms=148)
    assert L.ivit_selftest_lora_form(*ok.values(), form) == 0
    for bad in (dict(M=0), dict(M=63), dict(K=8), dict(K=24), dict(K=16400), dict(N=0), dict(N=40), dict(n=0), dict(R=0),
                dict(R=24), dict(R=144), dict(rows=0), dict(rows=5), dict(sms=0)):
        assert L.ivit_selftest_lora_form(*{**ok, **bad}.values(), form) == 1, bad
    assert L.ivit_selftest_lora_form(*ok.values(), None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("shape,form,several", SHAPES)
@pytest.mark.parametrize("epi", ["plain", "residual", "gelu"])
def test_lora_form_parity(shape, form, several, epi):
    req, rows, K, N, R, n = shape
    q = LoraCase(req, rows, K, N, R, n, seed=req + rows + K + N + R)
    d, res = q.device(), (1 << 29, (1 << 28) + 77, 30)
    for rounding in (0, 1):
        y, untouched = guarded((q.M, N))
        if epi == "gelu":
            ivit.ivit_linear_lora_shiftgelu(*d, *GELU, y, workspace(q.M, R), rounding=rounding)
            want = serving.linear_lora(*q.host(), rounding=rounding, gelu=GELU)
        else:
            skip = q.skip if epi == "residual" else None
            bits = 8 - 2 * rounding
            ivit.ivit_linear_lora(*d, y, workspace(q.M, R), bits, dev(skip), res if epi == "residual" else None,
                                  rounding=rounding)
            want = serving.linear_lora(*q.host(), bits, skip, res if epi == "residual" else None, rounding)
        np.testing.assert_array_equal(host(y), want)
        assert untouched()
    assert ivit.ivit_stream_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("req,K,N,R,n", [(60, 768, 784, 16, 60), (512, 272, 2048, 128, 64), (512, 1024, 1024, 32, 64),
                                         (12, 272, 400, 16, 3), (3000, 784, 784, 48, 2)])
def test_calls_in_a_row_on_one_workspace(req, K, N, R, n):
    """The same rows of t are written and read by call after call, each with other rows and adapters: none may see what
    the one before left there."""
    q = [LoraCase(req, 1, K, N, R, n, seed=60 + i) for i in range(3)]
    for t in q[1:]:
        t.W, t.bias, t.b, t.c, t.adapters = q[0].W, q[0].bias, q[0].b, q[0].c, q[0].adapters
    d, ws = [t.device() for t in q], workspace(req, R)
    ys = [dev(np.zeros((req, N), np.int8)) for _ in range(60)]
    for i, y in enumerate(ys):
        ivit.ivit_linear_lora(*d[i % 3], y, ws)
    want = [serving.linear_lora(*t.host()) for t in q]
    for i, y in enumerate(ys):
        np.testing.assert_array_equal(host(y), want[i % 3])
    assert ivit.ivit_stream_status() == 0
