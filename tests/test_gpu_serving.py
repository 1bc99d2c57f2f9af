"""GPU parity of the serving operators against their plain 64-bit forms, bit
for bit (every quantity is an integer): linear layers with a low-rank adapter
per request, the end of a residual branch, differential attention, and a block
of all three.  Outputs sit between canary bytes."""
import numpy as np
import pytest
import torch

import integer_only_quantized_int8_b200 as ivit
from integer_only_quantized_int8_b200 import build as ivit_build
from oracle import serving

pytestmark = pytest.mark.gpu

GUARD = 4096
CANARY = 0x5A


@pytest.fixture(scope="module", autouse=True)
def built():
    ivit_build.build()
    yield
    assert ivit.ivit_stream_status() == 0


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def guarded(shape):
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), CANARY, dtype=torch.uint8, device="cuda")
    view = buf[GUARD:GUARD + n].view(torch.int8).view(shape)

    def untouched():
        h = host(buf)
        return bool((h[:GUARD] == CANARY).all() and (h[GUARD + n:] == CANARY).all())

    return view, untouched


def rng_i8(r, *shape):
    return r.integers(-128, 128, shape, dtype=np.int8)


def workspace(M, R):
    """A workspace full of stale bytes."""
    return torch.full((ivit.ivit_linear_lora_workspace_bytes(M, R),), CANARY, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- adapters

class LoraCase:
    """Inputs whose accumulators spread over the output range; wild: multipliers over their whole range."""

    def __init__(self, req, rows, K, N, R, n, seed, wild=False, idx=None):
        r = np.random.default_rng(seed)
        self.M, self.rows, self.R = req * rows, rows, R
        self.X, self.W = rng_i8(r, self.M, K), rng_i8(r, N, K)
        A, B = rng_i8(r, n, R, K), rng_i8(r, n, N, R)
        acc = 74.0 * 74.0 * np.sqrt(K)
        self.bias = (r.standard_normal(N) * acc / 4).astype(np.int32)
        if wild:
            self.b, self.c = r.integers(0, 1 << 31, N).astype(np.int32), r.integers(0, 32, N).astype(np.int8)
            b_t, c_t = r.integers(0, 1 << 31, (n, R)).astype(np.int32), r.integers(0, 32, (n, R)).astype(np.int8)
        else:
            c = int(min(31, 30 + np.log2(acc / 60)))
            self.b = (r.uniform(0.5, 1.0, N) * 60 / acc * 2.0 ** c).astype(np.int32)
            self.c = np.full(N, c, np.int8)
            b_t = (r.uniform(0.5, 1.0, (n, R)) * 60 / acc * 2.0 ** c).astype(np.int32)
            c_t = np.full((n, R), c, np.int8)
        self.adapters = (A, b_t, c_t, B)
        self.idx = r.integers(-1, n + 1, req).astype(np.int32) if idx is None else np.asarray(idx, np.int32)
        self.skip = rng_i8(r, self.M, N)

    def device(self):
        return [dev(t) for t in (self.X, self.W, self.bias, self.b, self.c)] + [tuple(dev(t) for t in self.adapters),
                                                                              dev(self.idx), self.rows]

    def host(self):
        return [self.X, self.W, self.bias, self.b, self.c, self.adapters, self.idx, self.rows]


GELU = (27, 30, 8, (1476395008, 27))

LORA_SHAPES = [
    (1, 1, 16, 16, 16, 1), (3, 1, 144, 48, 16, 2), (130, 1, 96, 144, 16, 7), (300, 1, 768, 80, 48, 40),
    (5, 7, 48, 80, 32, 3), (33, 9, 640, 272, 128, 5), (2, 197, 192, 576, 16, 4), (3, 130, 768, 144, 48, 2),
    (1, 300, 384, 128, 112, 3), (2, 128, 128, 256, 64, 2), (7, 64, 1040, 1008, 16, 9), (2, 640, 2048, 192, 80, 2),
]


@pytest.mark.parametrize("req,rows,K,N,R,n", LORA_SHAPES)
@pytest.mark.parametrize("epi", ["plain", "residual", "gelu"])
def test_linear_lora_parity(req, rows, K, N, R, n, epi):
    q = LoraCase(req, rows, K, N, R, n, seed=req + rows + K + N + R)
    for rounding in (0, 1):
        y, untouched = guarded((q.M, N))
        if epi == "gelu":
            ivit.ivit_linear_lora_shiftgelu(*q.device(), *GELU, y, workspace(q.M, R), rounding=rounding)
            want = serving.linear_lora(*q.host(), rounding=rounding, gelu=GELU)
        else:
            res = (1 << 29, (1 << 28) + 77, 30) if epi == "residual" else None
            skip = q.skip if epi == "residual" else None
            bits = 8 - 2 * rounding
            ivit.ivit_linear_lora(*q.device(), y, workspace(q.M, R), bits, dev(skip), res, rounding=rounding)
            want = serving.linear_lora(*q.host(), bits, skip, res, rounding)
        np.testing.assert_array_equal(host(y), want)
        assert untouched()


@pytest.mark.parametrize("req,rows,K,N,R,n", [(40, 1, 96, 272, 32, 5), (4, 70, 208, 144, 48, 3), (2, 200, 784, 160, 16, 2)])
@pytest.mark.parametrize("rounding", [0, 1])
def test_linear_lora_multipliers_of_every_size(req, rows, K, N, R, n, rounding):
    q = LoraCase(req, rows, K, N, R, n, seed=7, wild=True)
    q.bias[::3] = np.where(np.arange(len(q.bias[::3])) % 2, -(1 << 30), 1 << 30)
    y, untouched = guarded((q.M, N))
    ivit.ivit_linear_lora(*q.device(), y, workspace(q.M, R), rounding=rounding)
    np.testing.assert_array_equal(host(y), serving.linear_lora(*q.host(), rounding=rounding))
    assert untouched()


@pytest.mark.parametrize("rows", [1, 37])
@pytest.mark.parametrize("x,a", [(-128, -128), (-128, 127)])
def test_linear_lora_largest_sums(rows, x, a):
    """Every product of one sign: |t| saturates, the accumulator takes 2^14 (K + R)."""
    q = LoraCase(3, rows, 2048, 64, 128, 2, seed=8, idx=[1, 0, 1])
    q.X[:], q.W[:] = x, a
    A, b_t, c_t, B = q.adapters
    A[:], b_t[:], c_t[:], B[:] = a, (1 << 31) - 1, 0, a
    q.b[:], q.c[:] = 5, 21
    y, _ = guarded((q.M, 64))
    ivit.ivit_linear_lora(*q.device(), y, workspace(q.M, 128))
    np.testing.assert_array_equal(host(y), serving.linear_lora(*q.host()))


@pytest.mark.parametrize("idx", [[-1, -1, -1, -1], [2, 2, 2, 2], [3, -(1 << 31), (1 << 31) - 1, 0]])
@pytest.mark.parametrize("rows", [1, 65])
def test_linear_lora_indexes(idx, rows):
    """No adapter anywhere, one adapter for all, indexes far outside."""
    q = LoraCase(4, rows, 160, 96, 16, 3, seed=9, idx=idx)
    y, _ = guarded((q.M, 96))
    ivit.ivit_linear_lora(*q.device(), y, workspace(q.M, 16))
    np.testing.assert_array_equal(host(y), serving.linear_lora(*q.host()))


def test_linear_lora_without_bias_and_without_rank():
    """bias NULL; an adapter whose down projections are zero rows adds nothing."""
    q = LoraCase(3, 50, 96, 112, 32, 2, seed=10, idx=[0, 1, 0])
    q.bias = None
    q.adapters[0][1] = 0
    d = q.device()
    y, _ = guarded((q.M, 112))
    ivit.ivit_linear_lora(*d, y, workspace(q.M, 32))
    np.testing.assert_array_equal(host(y), serving.linear_lora(*q.host()))
    base = torch.empty_like(y)
    ivit.ivit_linear_requant(*d[:5], base)
    np.testing.assert_array_equal(host(y)[50:100], host(base)[50:100])


def test_linear_lora_workspace_use():
    """Only t's bytes are written, and only those of requests with an adapter."""
    q = LoraCase(3, 20, 96, 112, 16, 2, seed=11, idx=[0, -1, 1])
    ws = workspace(q.M + 64, 16)
    y, _ = guarded((q.M, 112))
    ivit.ivit_linear_lora(*q.device(), y, ws)
    h = host(ws)
    assert (h[20 * 16:40 * 16] == CANARY).all() and (h[60 * 16:] == CANARY).all()


def test_linear_lora_capture_and_streams():
    """A captured call replays on new inputs; two streams with a workspace each do not disturb one another."""
    qs = [LoraCase(6, 33, 384, 256, 32, 4, seed=s) for s in (12, 13)]
    want = [serving.linear_lora(*q.host()) for q in qs]
    d = [q.device() for q in qs]
    ys, wss = [guarded((qs[0].M, 256))[0] for _ in qs], [workspace(qs[0].M, 32) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            ivit.ivit_linear_lora(*d[i], ys[i], wss[i], stream=s)
    for y, w in zip(ys, want):
        np.testing.assert_array_equal(host(y), w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ivit.ivit_linear_lora(*d[0], ys[0], wss[0])
    d[0][0].copy_(d[1][0])
    d[0][6].copy_(d[1][6])
    qs[0].X, qs[0].idx = qs[1].X, qs[1].idx
    for _ in range(2):
        ys[0].zero_()
        g.replay()
        np.testing.assert_array_equal(host(ys[0]), serving.linear_lora(*qs[0].host()))


# ---------------------------------------------------------------- the end of a branch

def norm_params(r, cols, wild=False):
    g = rng_i8(r, cols)
    be = r.integers(-(1 << 30), (1 << 30) + 1, cols, dtype=np.int32) if wild else \
        r.integers(-3000, 3000, cols, dtype=np.int32)
    if wild:
        F = int(r.integers(0, 15))
        return g, be, F, int(r.integers(F, 24)), (int(r.integers(0, 1 << 31)), int(r.integers(0, 32)))
    return g, be, 7, 23, (1466015503, 38 - 7)


def dev_norm(n):
    return None if n is None else (dev(n[0]), dev(n[1])) + tuple(n[2:])


def branch_end(rows, cols, T, post, gate, pre, seed, wild=False, inplace=False):
    r = np.random.default_rng(seed)
    x, o = rng_i8(r, rows, cols), rng_i8(r, rows, cols)
    o[0] = 17                                            # a row without variance
    pp, np_ = (norm_params(r, cols, wild) if f else None for f in (post, pre))
    g = rng_i8(r, -(-rows // T), cols) if gate else None
    if wild:
        scale = r.integers(-(1 << 31), 1 << 31, cols).astype(np.int32)
        scale[:2] = -(1 << 31), (1 << 31) - 1
        b_skip, c = int(r.integers(0, 1 << 31)), int(r.integers(0, 32))
    else:
        scale = (r.standard_normal(cols) * (4e6 if gate else 2.5e8)).astype(np.int32)
        b_skip, c = 939524096, 30
    want = serving.residual_norm(x, o, scale, b_skip, c, pp, g, T, np_)
    y, ok_y = guarded((rows, cols))
    z, ok_z = guarded((rows, cols)) if pre else (None, lambda: True)
    dx, do = dev(x), dev(o)
    if inplace:
        y, z = dx, (do if pre else None)
    got = ivit.ivit_residual_norm(dx, do, dev(scale), b_skip, c, y, dev_norm(pp), dev(g), T, dev_norm(np_), z)
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        if a is not None:
            np.testing.assert_array_equal(host(a), b)
    assert ok_y() and ok_z()


@pytest.mark.parametrize("rows,cols,T", [(1, 16, 1), (5, 48, 2), (197, 192, 197), (394, 768, 197), (130, 1024, 7),
                                         (9, 2048, 9), (2500, 320, 50), (3, 528, 1), (64, 1296, 16), (33, 784, 40)])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_residual_norm_parity(rows, cols, T, post, gate, pre):
    branch_end(rows, cols, T, post, gate, pre, seed=rows + cols)


@pytest.mark.parametrize("seed", range(24))
def test_residual_norm_parameters_of_every_size(seed):
    r = np.random.default_rng(seed)
    branch_end(int(r.integers(1, 90)), 16 * int(r.integers(1, 129)), int(r.integers(1, 20)), seed % 2 == 0, seed % 3 != 0,
               seed % 5 != 0, seed=100 + seed, wild=True)


@pytest.mark.parametrize("pre", [True, False])
def test_residual_norm_in_place(pre):
    branch_end(300, 384, 100, True, True, pre, seed=5, inplace=True)


def test_residual_norm_capture_and_empty():
    r = np.random.default_rng(6)
    x, o = rng_i8(r, 40, 96), rng_i8(r, 40, 96)
    scale, pre = r.integers(-(1 << 28), 1 << 28, 96).astype(np.int32), norm_params(r, 96)
    dx, do, ds, dp = dev(x), dev(o), dev(scale), dev_norm(pre)
    y, z = torch.empty_like(dx), torch.empty_like(dx)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ivit.ivit_residual_norm(dx, do, ds, 1 << 29, 30, y, pre=dp, z=z)
    dx.copy_(do)
    g.replay()
    want = serving.residual_norm(o, o, scale, 1 << 29, 30, pre=pre)
    np.testing.assert_array_equal(host(y), want[0])
    np.testing.assert_array_equal(host(z), want[1])
    ivit.ivit_residual_norm(dx[:0], do[:0], ds, 1, 0, y[:0], pre=dp, z=z[:0])


# ---------------------------------------------------------------- differential attention

DIFF_ARGS = ((1 << 20, 28), 8, 20, 30, 8)   # logits of std ~56 at |q|, |k| ~ 30


def diff_inputs(B, N, H, seed, spread=30):
    r = np.random.default_rng(seed)
    qkv = np.clip(np.round(r.standard_normal((B * N, 384 * H)) * spread), -128, 127).astype(np.int8)
    return qkv, r.integers(0, (1 << 30) + 1, H).astype(np.int32)


def diff_check(qkv, B, N, H, args, lam, out):
    ctx, untouched = guarded((B * N, 128 * H))
    ivit.ivit_attention_diff(dev(qkv), B, N, H, *args, dev(lam), out, ctx)
    np.testing.assert_array_equal(host(ctx), serving.attention_diff(qkv, B, N, H, *args, lam, out))
    assert untouched()


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 96, 97, 112, 127, 128, 129, 144, 160, 161, 192, 193,
                               197, 224, 225, 255, 256, 257, 288, 320, 321, 383, 384, 385, 448, 449, 511, 512, 513, 576, 577,
                               608, 609, 639, 640])
def test_attention_diff_parity(N):
    qkv, lam = diff_inputs(2, N, 2, seed=N)
    diff_check(qkv, 2, N, 2, DIFF_ARGS, lam, (1 << 20, 25))


@pytest.mark.parametrize("B,N,H", [(1, 197, 3), (40, 197, 6), (9, 130, 9), (200, 5, 3), (6, 577, 6), (33, 64, 5), (3, 260, 20)])
def test_attention_diff_many_items(B, N, H):
    """More work items than SMs: every ring and phase wraps."""
    qkv, lam = diff_inputs(B, N, H, seed=B + N)
    diff_check(qkv, B, N, H, DIFF_ARGS, lam, (1 << 20, 25))


@pytest.mark.parametrize("k_s,I0,M,k_out", [(8, 1, 30, 8), (2, 3, 30, 8), (4, 5, 12, 4), (6, 97, 7, 8), (8, 1 << 22, 30, 8),
                                            (8, 20, 30, 1), (8, 20, 0, 1), (3, 1000, 30, 8), (8, 7, 20, 6)])
@pytest.mark.parametrize("N", [37, 197, 470])
def test_attention_diff_constants(k_s, I0, M, k_out, N):
    qkv, _ = diff_inputs(2, N, 2, seed=k_s)
    lam = np.array([(1 << M) // 3, 1 << M], np.int32)
    diff_check(qkv, 2, N, 2, ((1 << 20, 26), k_s, I0, M, k_out), lam, (3, 2))


@pytest.mark.parametrize("logit", [(0, 5), (1, 0), ((1 << 31) - 1, 0), ((1 << 31) - 1, 31), (3, 1), (1 << 30, 31), (1, 31)])
@pytest.mark.parametrize("out", [(0, 0), (1, 0), ((1 << 31) - 1, 0), (7, 4), ((1 << 31) - 1, 31)])
def test_attention_diff_multipliers_of_every_size(logit, out):
    qkv, lam = diff_inputs(2, 70, 2, seed=3, spread=80)
    diff_check(qkv, 2, 70, 2, (logit, 8, 20, 30, 8), lam, out)


@pytest.mark.parametrize("lam", [[0, 0], [1 << 30, 1 << 30], [-5, (1 << 31) - 1], [-(1 << 31), 1]])
def test_attention_diff_weights(lam):
    """lam is clamped to [0, 2^M]; 0 leaves the first map alone."""
    qkv, _ = diff_inputs(2, 150, 2, seed=4)
    diff_check(qkv, 2, 150, 2, DIFF_ARGS, np.array(lam, np.int32), (1 << 20, 25))


@pytest.mark.parametrize("N", [40, 200, 600])
def test_attention_diff_extreme_values(N):
    """Every product of one sign; one key that takes a whole row; keys of the next image that would win every maximum."""
    qkv, lam = diff_inputs(2, N, 1, seed=5)
    qkv[:] = -128
    diff_check(qkv, 2, N, 1, ((1, 0), 8, 1, 30, 8), lam, (1, 7))
    qkv, _ = diff_inputs(2, N, 1, seed=6)
    qkv[N - 1, 128:256] = 127
    qkv[:, :128] = np.abs(qkv[:, :128].astype(np.int32)).clip(0, 127)
    qkv[N:, 128:256] = 127
    diff_check(qkv, 2, N, 1, DIFF_ARGS, lam, (1 << 20, 25))


def test_attention_diff_capture_streams_and_empty():
    qkv, lam = diff_inputs(8, 197, 3, seed=7)
    other, _ = diff_inputs(8, 197, 3, seed=8)
    out = (1 << 20, 25)
    want = [serving.attention_diff(t, 8, 197, 3, *DIFF_ARGS, lam, out) for t in (qkv, other)]
    d, dl = [dev(qkv), dev(other)], dev(lam)
    ctx = [torch.empty(8 * 197, 384, dtype=torch.int8, device="cuda") for _ in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            ivit.ivit_attention_diff(d[i], 8, 197, 3, *DIFF_ARGS, dl, out, ctx[i], stream=s)
    for c, w in zip(ctx, want):
        np.testing.assert_array_equal(host(c), w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ivit.ivit_attention_diff(d[0], 8, 197, 3, *DIFF_ARGS, dl, out, ctx[0])
    d[0].copy_(d[1])
    for _ in range(2):
        ctx[0].zero_()
        g.replay()
        np.testing.assert_array_equal(host(ctx[0]), want[1])
    ivit.ivit_attention_diff(d[0][:0], 0, 197, 3, *DIFF_ARGS, dl, out, ctx[0][:0])


# ---------------------------------------------------------------- together

def test_adapted_block():
    """An encoder block of these operators alone, as a server runs it: adapters on all four linear layers, differential
    attention between them, the branch ends with post-norm, gate, residual scale and the next norm; then once more
    from a graph on other inputs."""
    B, N, H = 5, 197, 2
    Dm, D = 512, 128 * H
    r = np.random.default_rng(9)
    layers = [LoraCase(B, N, K, n, 16, 3, seed=s, idx=[0, -1, 2, 1, 0])
              for s, (K, n) in enumerate([(D, 3 * D), (D, D), (D, Dm), (Dm, D)], 20)]
    pre, post, nxt = (norm_params(r, D) for _ in range(3))
    gate, lam = rng_i8(r, B, D), r.integers(0, 1 << 30, H).astype(np.int32)
    scale = (r.standard_normal(D) * 4e6).astype(np.int32)
    out = (1 << 20, 25)

    def host_block(x, z):
        def lin(i, t, gelu=None):
            q = layers[i]
            return serving.linear_lora(t, q.W, q.bias, q.b, q.c, q.adapters, q.idx, N, gelu=gelu)
        ctx = serving.attention_diff(lin(0, z), B, N, H, *DIFF_ARGS, lam, out)
        x, z = serving.residual_norm(x, lin(1, ctx), scale, 939524096, 30, post, gate, N, pre)
        return serving.residual_norm(x, lin(3, lin(2, z, GELU)), scale, 939524096, 30, post, gate, N, nxt)

    d = [q.device() for q in layers]
    dpre, dpost, dnxt = dev_norm(pre), dev_norm(post), dev_norm(nxt)
    dg, dl, ds = dev(gate), dev(lam), dev(scale)
    buf = [torch.empty(B * N, w, dtype=torch.int8, device="cuda") for w in (3 * D, D, D, Dm, D)]
    x, z = rng_i8(r, B * N, D), rng_i8(r, B * N, D)
    dx, dz, ws = dev(x), dev(z), workspace(B * N, 16)

    def block():
        ivit.ivit_linear_lora(dz, *d[0][1:], buf[0], ws)
        ivit.ivit_attention_diff(buf[0], B, N, H, *DIFF_ARGS, dl, out, buf[1])
        ivit.ivit_linear_lora(buf[1], *d[1][1:], buf[2], ws)
        ivit.ivit_residual_norm(dx, buf[2], ds, 939524096, 30, dx, dpost, dg, N, dpre, dz)
        ivit.ivit_linear_lora_shiftgelu(dz, *d[2][1:], *GELU, buf[3], ws)
        ivit.ivit_linear_lora(buf[3], *d[3][1:], buf[4], ws)
        ivit.ivit_residual_norm(dx, buf[4], ds, 939524096, 30, dx, dpost, dg, N, dnxt, dz)

    for _ in range(3):    # the block's outputs are its next inputs
        block()
        x, z = host_block(x, z)
    np.testing.assert_array_equal(host(dx), x)
    np.testing.assert_array_equal(host(dz), z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block()
    x, z = rng_i8(r, B * N, D), rng_i8(r, B * N, D)
    dx.copy_(dev(x))
    dz.copy_(dev(z))
    for _ in range(2):
        g.replay()
        x, z = host_block(x, z)
    np.testing.assert_array_equal(host(dx), x)
    np.testing.assert_array_equal(host(dz), z)


# ---------------------------------------------------------------- the ways adapters join

@pytest.mark.parametrize("req,rows,K,N,R,n", [
    (700, 2, 64, 2304, 16, 64),      # dp4a on wide tiles: many one- and two-token requests, many adapters
    (130, 3, 256, 1040, 48, 61),     # dp4a on narrow tiles
    (40, 1, 128, 272, 128, 37),
    (900, 1, 144, 1168, 32, 8),      # an axis by adapter: more requests than adapters in a tile
    (500, 3, 640, 576, 112, 3), (90, 7, 1040, 528, 16, 5),
    (3, 333, 528, 2064, 96, 2), (12, 21, 96, 4096, 64, 50),   # an axis by request, several slices long
    (2, 1100, 48, 64, 16, 3),        # a request of several tiles and one that shares its last
    (20, 197, 768, 2304, 16, 5), (20, 197, 384, 1152, 16, 3), (64, 60, 1040, 1536, 32, 9), (9, 577, 192, 1600, 112, 4),
    (4, 16, 2064, 256, 32, 3), (1, 3, 4096, 1008, 128, 2), (16, 8, 320, 4096, 16, 20), (5, 130, 2048, 64, 16, 2),  # one kernel
    (300, 1, 768, 304, 16, 8), (64, 1, 320, 1008, 32, 4), (77, 3, 144, 528, 128, 1), (45, 7, 208, 640, 48, 2),
])
@pytest.mark.parametrize("epi", ["plain", "residual", "gelu"])
def test_linear_lora_ways(req, rows, K, N, R, n, epi):
    q = LoraCase(req, rows, K, N, R, n, seed=req + rows + K)
    y, untouched = guarded((q.M, N))
    if epi == "gelu":
        ivit.ivit_linear_lora_shiftgelu(*q.device(), *GELU, y, workspace(q.M, R))
        want = serving.linear_lora(*q.host(), gelu=GELU)
    else:
        res = (1 << 29, (1 << 28) + 77, 30) if epi == "residual" else None
        skip = q.skip if epi == "residual" else None
        ivit.ivit_linear_lora(*q.device(), y, workspace(q.M, R), 5, dev(skip), res, rounding=1)
        want = serving.linear_lora(*q.host(), 5, skip, res, 1)
    np.testing.assert_array_equal(host(y), want)
    assert untouched()


def test_linear_lora_back_to_back():
    """Layers in a row on one workspace, each reading what the one before wrote: the GEMM that starts while its down
    projection runs must see neither's inputs early nor its t late."""
    r = np.random.default_rng(30)
    dims = [192, 256, 1024, 192, 768, 192]
    layers = [LoraCase(9, 50, K, N, 32, 4, seed=40 + i) for i, (K, N) in enumerate(zip(dims, dims[1:]))]
    x = rng_i8(r, 450, 192)
    bufs = [dev(x)] + [torch.zeros(450, N, dtype=torch.int8, device="cuda") for N in dims[1:]]
    ws = workspace(450, 32)
    d = [q.device() for q in layers]
    for _ in range(10):
        for i in range(len(layers)):
            ivit.ivit_linear_lora(bufs[i], *d[i][1:], bufs[i + 1], ws)
        bufs[0].copy_(bufs[-1])
    t = x
    for _ in range(10):
        for q in layers:
            t = serving.linear_lora(t, q.W, q.bias, q.b, q.c, q.adapters, q.idx, q.rows)
    np.testing.assert_array_equal(host(bufs[-1]), t)


# ---------------------------------------------------------------- bounded waits

def times_out_then_exact(run, want):
    assert ivit.ivit_stream_status() == 0
    run(True)
    assert ivit.ivit_status_string(ivit.ivit_stream_status()) == "IVIT_ERR_TIMEOUT"
    got = run(False)
    assert ivit.ivit_stream_status() == 0
    np.testing.assert_array_equal(got, want)


# K = 1024 takes the shared-tile GEMM kernel, K = 384 the own-tile one, 60 one-token requests of 60 adapters the dp4a way,
# 5 requests the one-kernel form
@pytest.mark.parametrize("K,req,rows,n", [(1024, 40, 197, 4), (384, 40, 197, 4), (1024, 60, 1, 60), (1024, 5, 197, 4)])
def test_linear_lora_producer_stops_and_reports_timeout(K, req, rows, n):
    q = LoraCase(req, rows, K, 512, 32, n, seed=50)
    d, y, ws = q.device(), torch.zeros(q.M, 512, dtype=torch.int8, device="cuda"), workspace(q.M, 32)

    def run(stop):
        if stop:
            ivit.ivit_selftest_withhold(ivit.SELFTEST_GEMM, 2)
        ivit.ivit_linear_lora(*d, y, ws)
        return host(y)

    times_out_then_exact(run, serving.linear_lora(*q.host()))


@pytest.mark.parametrize("N", [197, 500])
def test_attention_diff_producer_stops_and_reports_timeout(N):
    qkv, lam = diff_inputs(30, N, 3, seed=51)
    d, dl = dev(qkv), dev(lam)
    ctx = torch.zeros(30 * N, 384, dtype=torch.int8, device="cuda")

    def run(stop):
        if stop:
            ivit.ivit_selftest_withhold(ivit.SELFTEST_ATTENTION, 1)
        ivit.ivit_attention_diff(d, 30, N, 3, *DIFF_ARGS, dl, (1 << 20, 25), ctx)
        return host(ctx)

    times_out_then_exact(run, serving.attention_diff(qkv, 30, N, 3, *DIFF_ARGS, lam, (1 << 20, 25)))
