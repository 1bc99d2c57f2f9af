"""Tables that the call just before writes, on the same stream: a kernel that starts
while its predecessor finishes must not read them early.  The predecessor is a call
of this library (an exact copy of a large tensor that holds the tables), since
its kernels let the next one start before they end."""
import numpy as np
import pytest
import torch

import integer_only_quantized_int8_b200 as ivit
import oracle
import synthetic
from integer_only_quantized_int8_b200 import build as ivit_build
from integer_only_quantized_int8_b200 import params as ivit_params
from oracle import serving

pytestmark = pytest.mark.gpu

CALLS = 40
OUT = (400000000, 30)


@pytest.fixture(scope="module", autouse=True)
def built():
    ivit_build.build()
    yield
    assert ivit.ivit_stream_status() == 0


class Tables:
    """Two sets of tables, each somewhere in a large tensor of its own, and a tensor that takes the one or the other."""
    ROWS, COLS = 4096, 768

    def __init__(self, sets, place):
        self.at, n = {}, 0
        for name, t in sets[0].items():
            self.at[name] = (n, t.dtype, t.size)
            n += -(-t.nbytes // 256) * 256
        first = {"first": 0, "last": (self.ROWS * self.COLS - n) // 256 * 256}[place]
        self.src = []
        for s in sets:
            h = np.random.default_rng(1).integers(-128, 128, self.ROWS * self.COLS, dtype=np.int8)
            for name, t in s.items():
                o = first + self.at[name][0]
                h[o:o + t.nbytes] = t.view(np.int8)
            self.src.append(torch.from_numpy(h.reshape(self.ROWS, self.COLS)).cuda())
        self.dst = torch.zeros(self.ROWS, self.COLS, dtype=torch.int8, device="cuda")
        self.zero = torch.zeros(self.COLS, dtype=torch.int32, device="cuda")
        self.first = first

    def view(self, name):
        o, dtype, size = self.at[name]
        o += self.first
        t = self.dst.view(-1)[o:o + size * dtype.itemsize]
        return t if dtype == np.int8 else t.view(torch.int32)

    def write(self, i):
        """dst = src[i], by a call of the library."""
        ivit.ivit_residual_norm(self.src[i], self.src[i], self.zero, 1, 0, self.dst)


def norm_tables(r, cols, name):
    return {name + "_gamma": r.integers(-128, 128, cols, dtype=np.int8),
            name + "_beta": r.integers(-3000, 3000, cols, dtype=np.int32)}


def run(tables, call, outputs, graph):
    """CALLS calls, the tables changed before each one; outputs[k]: what call k writes."""
    def all_calls():
        for k in range(CALLS):
            tables.write(k & 1)
            call(k)

    if graph:
        tables.write(0)
        call(0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_calls()
        for o in outputs:
            for t in o:
                t.zero_()
        g.replay()
    else:
        torch.cuda.synchronize()
        all_calls()
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,cols", [(1, 192), (394, 768), (3000, 1024)])
@pytest.mark.parametrize("place", ["first", "last"])
@pytest.mark.parametrize("graph", [False, True])
def test_branch_end_tables_of_the_call_before(rows, cols, place, graph):
    r = np.random.default_rng(rows + cols)
    sets = [{"scale": r.integers(-(1 << 28), 1 << 28, cols).astype(np.int32), **norm_tables(r, cols, "post"),
             **norm_tables(r, cols, "pre")} for _ in range(2)]
    t = Tables(sets, place)
    x, o = (r.integers(-128, 128, (rows, cols), dtype=np.int8) for _ in range(2))
    dx, do = torch.from_numpy(x).cuda(), torch.from_numpy(o).cuda()
    outs = [(torch.zeros_like(dx), torch.zeros_like(dx)) for _ in range(CALLS)]

    def norm(n):
        return t.view(n + "_gamma"), t.view(n + "_beta"), 7, 23, OUT

    def call(k):
        ivit.ivit_residual_norm(dx, do, t.view("scale"), 1 << 29, 30, outs[k][0], post=norm("post"), pre=norm("pre"),
                                z=outs[k][1])

    run(t, call, outs, graph)
    want = [serving.residual_norm(x, o, s["scale"], 1 << 29, 30, (s["post_gamma"], s["post_beta"], 7, 23, OUT),
                                  pre=(s["pre_gamma"], s["pre_beta"], 7, 23, OUT)) for s in sets]
    assert (want[0][0] != want[1][0]).any() and (want[0][1] != want[1][1]).any()
    for k in range(CALLS):
        for got, w in zip(outs[k], want[k & 1]):
            np.testing.assert_array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("rows,cols", [(1, 192), (394, 768), (3000, 1024)])
@pytest.mark.parametrize("place", ["first", "last"])
@pytest.mark.parametrize("graph", [False, True])
def test_layernorm_tables_of_the_call_before(rows, cols, place, graph):
    r = np.random.default_rng(rows + cols)
    sets = [norm_tables(r, cols, "ln") for _ in range(2)]
    t = Tables(sets, place)
    x = r.integers(-128, 128, (rows, cols), dtype=np.int8)
    dx = torch.from_numpy(x).cuda()
    outs = [(torch.zeros_like(dx),) for _ in range(CALLS)]
    run(t, lambda k: ivit.ivit_layernorm(dx, t.view("ln_gamma"), t.view("ln_beta"), 7, 23, OUT, outs[k][0]), outs, graph)
    want = [oracle.layernorm(x, s["ln_gamma"], s["ln_beta"], 7, 23, OUT) for s in sets]
    assert (want[0] != want[1]).any()
    for k in range(CALLS):
        np.testing.assert_array_equal(outs[k][0].cpu().numpy(), want[k & 1])


@pytest.mark.parametrize("place", ["first", "last"])
def test_block_tables_of_the_call_before(place):
    """Both norms' tables of an encoder block; the block's later kernels take them for granted."""
    B, N, D = 2, 65, 192
    wl = synthetic.make_workload(B=B, N=N, D=D, H=3, Dm=768, seed=21, n_cal=2)
    p = ivit_params.integer_params(wl.blocks[0])
    names = ("ln1_gamma", "ln1_beta", "ln2_gamma", "ln2_beta")
    dtypes = (np.int8, np.int32) * 2
    one = {n: np.ascontiguousarray(p[n]).astype(d) for n, d in zip(names, dtypes)}
    two = {n: np.ascontiguousarray(t[::-1]) for n, t in one.items()}
    t = Tables([one, two], place)
    dp = ivit_params.to_device(p, torch.device("cuda"))
    for n in names:
        setattr(dp.c, n, t.view(n).data_ptr())
    x = torch.from_numpy(wl.x).cuda()
    outs = [(torch.zeros_like(x),) for _ in range(CALLS)]
    ws = torch.empty(ivit.ivit_block_workspace_bytes(B, N, D, 768), dtype=torch.uint8, device="cuda")
    run(t, lambda k: ivit.ivit_block_forward(dp, x, outs[k][0], ws, B, N), outs, False)
    q = oracle.block_params(wl.blocks[0])
    want = [oracle.block_forward({**q, **s}, wl.x, B, N) for s in (one, two)]
    assert (want[0] != want[1]).any()
    for k in range(CALLS):
        np.testing.assert_array_equal(outs[k][0].cpu().numpy(), want[k & 1])


GELU = (27, 30, 8, (1476395008, 27))
# one kernel; a down projection, then k-slices of the shared-tile and own-tile GEMM; then dp4a of short and long ranks
LAYERS = [(4, 50, 256, 512, 16, 4), (24, 33, 784, 528, 64, 8), (24, 65, 256, 1040, 16, 3), (90, 1, 256, 528, 16, 40),
          (60, 1, 272, 400, 64, 20)]


@pytest.mark.parametrize("layer,form", list(zip(LAYERS, [(1, 64), (2, 128), (2, 128), (3, 16), (4, 16)])))
@pytest.mark.parametrize("place", ["first", "last"])
@pytest.mark.parametrize("gelu", [False, True])
def test_adapter_tables_of_the_call_before(layer, form, place, gelu):
    """Everything that a layer with adapters reads, its own weights and input among it."""
    from test_gpu_serving import LoraCase
    req, rows, K, N, R, n = layer
    assert ivit.ivit_selftest_lora_form(req * rows, K, N, n, R, rows, gelu)[:2] == form
    qs = [LoraCase(req, rows, K, N, R, n, seed=i) for i in (1, 2)]
    shapes = {"X": (req * rows, K), "W": (N, K), "A": (n, R, K), "b_t": (n, R), "c_t": (n, R), "B": (n, N, R)}
    sets = [dict(X=q.X, W=q.W, bias=q.bias, b=q.b, c=q.c, A=q.adapters[0], b_t=q.adapters[1], c_t=q.adapters[2],
                 B=q.adapters[3], idx=q.idx) for q in qs]
    t = Tables([{k: np.ascontiguousarray(v).reshape(-1) for k, v in s.items()} for s in sets], place)
    v = {k: t.view(k).view(shapes[k]) if k in shapes else t.view(k) for k in sets[0]}
    outs = [(torch.zeros(req * rows, N, dtype=torch.int8, device="cuda"),) for _ in range(CALLS)]
    ws = torch.zeros(ivit.ivit_linear_lora_workspace_bytes(req * rows, R), dtype=torch.uint8, device="cuda")
    args = (v["X"], v["W"], v["bias"], v["b"], v["c"], (v["A"], v["b_t"], v["c_t"], v["B"]), v["idx"], rows)

    def call(k):
        if gelu:
            ivit.ivit_linear_lora_shiftgelu(*args, *GELU, outs[k][0], ws)
        else:
            ivit.ivit_linear_lora(*args, outs[k][0], ws, skip=outs[0][0], res=(0, 1 << 20, 20))

    run(t, call, outs, False)
    want = [serving.linear_lora(*q.host(), gelu=GELU if gelu else None) for q in qs]
    assert (want[0] != want[1]).any()
    for k in range(CALLS):
        np.testing.assert_array_equal(outs[k][0].cpu().numpy(), want[k & 1])


@pytest.mark.parametrize("N", [65, 300])
@pytest.mark.parametrize("place", ["first", "last"])
def test_attention_diff_inputs_of_the_call_before(N, place):
    B, H, args = 2, 2, ((1 << 20, 28), 8, 20, 30, 8)
    r = np.random.default_rng(N)
    sets = [{"qkv": np.clip(np.round(r.standard_normal(B * N * 384 * H) * 30), -128, 127).astype(np.int8),
             "lam": r.integers(0, (1 << 30) + 1, H).astype(np.int32)} for _ in range(2)]
    t = Tables(sets, place)
    qkv, lam = t.view("qkv").view(B * N, 384 * H), t.view("lam")
    outs = [(torch.zeros(B * N, 128 * H, dtype=torch.int8, device="cuda"),) for _ in range(CALLS)]
    run(t, lambda k: ivit.ivit_attention_diff(qkv, B, N, H, *args, lam, (1 << 20, 25), outs[k][0]), outs, False)
    want = [serving.attention_diff(s["qkv"].reshape(B * N, 384 * H), B, N, H, *args, s["lam"], (1 << 20, 25)) for s in sets]
    assert (want[0] != want[1]).any()
    for k in range(CALLS):
        np.testing.assert_array_equal(outs[k][0].cpu().numpy(), want[k & 1])
