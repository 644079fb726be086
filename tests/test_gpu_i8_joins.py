"""Products whose tiles fill more than a wave: whole tiles, and the rest cut into parts of k that
meet in the workspace; and codes, weights and rows past 2^31 values.
"""
import pytest
import torch

from tests.gpu_helpers import binding, require_gpu
from tests.test_gpu_i8 import TYPES, U

pytestmark = pytest.mark.gpu

COUNTERS = 262144  # bytes at the front of a workspace, zeros between calls


@pytest.fixture(scope="module")
def B():
    require_gpu()
    return binding()


def _padded(codes):
    rows, k = codes.shape
    out = torch.zeros((rows, -(-k // 16) * 16), dtype=torch.int8, device="cuda")
    out[:, :k] = codes
    return out


class Case:
    """A product of codes -128 .. 127, with rows whose sums pass 2^24 on the way and rows that cancel."""

    def __init__(self, B, m, n, k):
        gen = torch.Generator(device="cuda").manual_seed(m * n + k)
        a = torch.randint(-128, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
        w = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
        a[m - 1], a[1, ::2], a[1, 1::2] = 127, 127, -128
        w[5], w[n - 1], w[n // 2, ::2], w[n // 2, 1::2] = 127, -128, -128, 127
        self.B, self.m, self.n, self.k = B, m, n, k
        self.want = (a.double() @ w.double().T).float()
        self.a, self.one = _padded(a), torch.ones(max(m, n), device="cuda")
        self.packed = torch.empty(B.llama_q8_i8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
        B.llama_q8_i8_pack(_padded(w), self.one, n, k, self.packed)
        self.y = torch.full((m + 1, n + 3), 3.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.size = B.llama_q8_i8_matmul_workspace_bytes(n, k, m)

    def run(self, ws, stream=0):
        self.B.llama_q8_i8_matmul(self.packed, self.n, self.k, self.a, self.one, self.m, 0, self.y, self.n + 3, ws,
                                  ws.numel(), self.err, stream)

    def check(self, ws):
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        assert torch.equal(self.y[:self.m, :self.n], self.want)
        assert (self.y[self.m] == 3.0).all() and (self.y[:, self.n:] == 3.0).all()
        assert not ws[:COUNTERS].any()
        self.y[:self.m, :self.n] = 7.0


# tokens, channels, k: 157 to 344 tiles on 152 SMs, the ones past whole waves in 2 to 4 parts (the plan's choice), tokens
# widened by the CTAs (up to 64) and by a kernel before
SIZES = [(17, 20483, 2500), (20, 25001, 2333), (40, 39001, 1700), (48, 28672, 4096), (64, 20001, 2050), (64, 28672, 4096),
         (100, 20001, 2333), (100, 28672, 4096), (128, 28601, 4001), (130, 22000, 3000), (256, 22016, 14336),
         (777, 11008, 4096)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_parts_beside_whole_tiles(B, m, n, k):
    case = Case(B, m, n, k)
    ws = torch.zeros(case.size, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        case.run(ws)
        case.check(ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.run(ws, torch.cuda.current_stream().cuda_stream)
    for _ in range(2):
        graph.replay()
        case.check(ws)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(48, 25001, 2333), (100, 20001, 2333)])
def test_parts_beside_whole_tiles_16_bit(B, kind, m, n, k):
    case = Case(B, m, n, k)
    ws = torch.zeros(case.size, dtype=torch.uint8, device="cuda")
    scale = torch.full((m,), 2.0 ** -12, device="cuda")
    y = torch.full((m, n), 3.0, dtype=TYPES[kind][1], device="cuda")
    B.llama_q8_i8_matmul(case.packed, n, k, case.a, scale, m, TYPES[kind][0], y, n, ws, case.size, case.err)
    assert torch.equal(y, (case.want * 2.0 ** -12).to(TYPES[kind][1]))  # a power of two: the one rounding is the type's
    assert int(case.err.item()) == 0 and not ws[:COUNTERS].any()


def test_one_workspace_for_parts_of_many_sizes(B):
    """Sizes with parts in the workspace, parts in clusters and none, in turn and without a wait between, on one workspace."""
    cases = [Case(B, *size) for size in ((64, 20001, 2050), (100, 20001, 2333), (40, 4096, 4500), (17, 20483, 2500),
                                         (300, 4096, 300), (130, 22000, 3000), (20, 25001, 2333))]
    ws = torch.zeros(max(c.size for c in cases), dtype=torch.uint8, device="cuda")
    for order in (cases, cases[::-1], cases):
        for c in order:
            c.run(ws)
        for c in order:
            c.check(ws)


# ---- past 2^31

@pytest.mark.parametrize("m", [1, 5, 40, 70])
def test_weights_past_2_31_codes(B, m):
    n, k = 160001, 14336
    gen = torch.Generator(device="cuda").manual_seed(m)
    a = torch.randint(-128, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    one = torch.ones(n, device="cuda")
    packed = torch.empty(B.llama_q8_i8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
    B.llama_q8_i8_pack(w, one, n, k, packed)
    size = B.llama_q8_i8_matmul_workspace_bytes(n, k, m)
    ws = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((m, n), 3.0, device="cuda")
    B.llama_q8_i8_matmul(packed, n, k, a, one, m, 0, y, n, ws, size, err)
    for at in (slice(0, 300), slice(149700, 150100), slice(n - 300, n)):
        assert torch.equal(y[:, at], (a.double() @ w[at].double().T).float())
    assert int(err.item()) == 0


def test_tokens_past_2_31_codes(B):
    m, n, k = 150001, 300, 14336
    gen = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randint(-128, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    one = torch.ones(m, device="cuda")
    packed = torch.empty(B.llama_q8_i8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
    B.llama_q8_i8_pack(w, one, n, k, packed)
    size = B.llama_q8_i8_matmul_workspace_bytes(n, k, m)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((m, n), 3.0, device="cuda")
    B.llama_q8_i8_matmul(packed, n, k, a, one, m, 0, y, n, ws, size, err)
    for at in (slice(0, 300), slice(149700, 149900), slice(m - 300, m)):
        assert torch.equal(y[at], (a[at].double() @ w.double().T).float())
    assert int(err.item()) == 0


@pytest.mark.parametrize("k", [14336, 14329])
@pytest.mark.parametrize("op", ["rows", "norm", "silu"])
def test_quantisers_past_2_31_values(B, op, k):
    """The last rows of a long call are those of a call on them alone."""
    rows, few = 150001, 40
    gen = torch.Generator(device="cuda").manual_seed(k)
    x = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    out = [[torch.full((n, -(-k // 16) * 16), 77, dtype=torch.int8, device="cuda"), torch.full((n,), 5.5, device="cuda")]
           for n in (rows, few)]
    g = torch.ones(k, device="cuda")
    tail = x[rows - few:].clone()
    for v, n, (codes, scale) in ((x, rows, out[0]), (tail, few, out[1])):
        if op == "rows":
            B.llama_q8_rows_quant(30, v, k, n, k, codes, scale)
        elif op == "norm":
            B.llama_q8_norm_quant(30, v, k, None, 0, v, k, g, 1e-5, n, k, codes, scale)
        else:
            B.llama_q8_silu_quant(30, v, v, k, n, k, codes, scale)
    torch.cuda.synchronize()
    assert torch.equal(x[rows - few:], tail)
    for long, short in zip(*out):
        assert torch.equal(long[rows - few:], short)
    want = out[1][0][:, :k].float() * out[1][1][:, None]  # and the few are near what they stand for
    v = tail.float()
    if op == "norm":
        v = v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt()
    elif op == "silu":
        v = v / (1 + torch.exp(-v)) * v
    assert ((want - v).abs() <= out[1][1][:, None] * 0.5001 + 100 * U * v.abs()).all()
