"""The 8-bit quantisers and their product on the GPU against the CPU definitions.

Codes are equal to those of exact arithmetic. Scales: rows f32(M / 127) exactly; silu two
roundings (M to f32, the quotient): 2 * 2^-24; norm: M, the quotient, 127 *, the root, the mean
and eps under the root (half each): 5 * 2^-24, and the f32 sum of squares, at most 30 additions
deep, under the root: 15 * 2^-24; together 20 * 2^-24. Product: f32 of the exact sum and two
products by scales: 3 * 2^-24, and half a step of a 16-bit type.
"""
import numpy as np
import pytest
import torch

from oracle import i8_oracle as I
from tests.gpu_helpers import binding, require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"f32": (0, torch.float32), "f16": (1, torch.float16), "bf16": (30, torch.bfloat16)}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    require_gpu()
    return binding()


def _rand(seed, *shape, scale=1.0):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32))


def _host(t):
    return t.detach().double().cpu().numpy()


def _outputs(rows, k, extra=2):
    """Codes and scales with guard rows behind the last."""
    codes = torch.full((rows + extra, I.row_bytes(k)), 77, dtype=torch.int8, device="cuda")
    return codes, torch.full((rows + extra,), 5.5, device="cuda")


def _check(codes, scale, rows, want, tol):
    torch.cuda.synchronize()
    wc, ws = want
    assert (codes[rows:] == 77).all() and (scale[rows:] == 5.5).all()
    got = codes[:rows].cpu().numpy()
    assert np.array_equal(got, wc), f"{(got != wc).sum()} codes differ, first at {np.argwhere(got != wc)[:4].tolist()}"
    s = scale[:rows].double().cpu().numpy()
    ws = np.asarray(ws, np.float64)
    assert np.array_equal(np.isnan(s), np.isnan(ws))
    fine = ~np.isnan(ws)
    assert (np.abs(s - ws)[fine] <= tol * np.abs(ws)[fine]).all()


def _strided(x, stride, dtype, shift=0):
    """x as rows `stride` apart in a buffer of its own, `shift` elements in; the rest is NaN."""
    rows, k = x.shape
    flat = torch.full((shift + rows * stride + 8,), float("nan"), dtype=dtype, device="cuda")
    view = flat[shift:shift + rows * stride].view(rows, stride)
    view[:, :k] = x.to(dtype).cuda()
    return flat, view


# row lengths at the borders of what a warp, each size of CTA and the registers hold
LENGTHS = [1, 3, 16, 31, 100, 512, 513, 576, 1001, 2048, 2052, 4096, 4097, 8192, 14336, 16384, 16388, 40001]


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("k", LENGTHS)
def test_rows_quant(B, kind, k):
    t, dtype = TYPES[kind]
    rows = 7 if k < 5000 else 3
    for stride, shift in ((k, 0), (k + 5, 1), (-(-k // 8) * 8, 0)):
        _, x = _strided(_rand(k, rows, k), stride, dtype, shift)
        codes, scale = _outputs(rows, k)
        B.llama_q8_rows_quant(t, x, stride, rows, k, codes, scale)
        _check(codes, scale, rows, I.rows_quant(_host(x[:, :k])), 0.0)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("k", LENGTHS)
def test_norm_quant(B, kind, k):
    t, dtype = TYPES[kind]
    rows = 6 if k < 5000 else 3
    g = (1.0 + 0.2 * _rand(1, k)).cuda()
    for stride, shift, eps in ((k, 0, 1e-5), (k + 3, 1, 0.0), (-(-k // 8) * 8, 0, 0.5)):
        base = _rand(k + 1, rows, k, scale=3.0)
        base[:, k // 3] *= 40.0
        _, x = _strided(base, stride, dtype, shift)
        _, d = _strided(_rand(k + 2, rows, k), stride, dtype, shift)
        h = (x[:, :k].float() + d[:, :k].float()).to(dtype)
        want = I.norm_quant(_host(h), _host(g), float(np.float32(eps)))
        flat, out = _strided(torch.zeros(rows, k), stride, dtype, shift)
        before = flat.clone()
        codes, scale = _outputs(rows, k)
        B.llama_q8_norm_quant(t, x, stride, d, stride, out, stride, g, eps, rows, k, codes, scale)
        _check(codes, scale, rows, want, 20 * U)
        assert torch.equal(out[:, :k], h)
        out[:, :k] = 0
        assert torch.equal(flat.nan_to_num(3.25), before.nan_to_num(3.25))  # nothing beside the rows
        # without the stored sum; then no addition; then the sum in the place of delta, and of x
        B.llama_q8_norm_quant(t, x, stride, d, stride, None, 0, g, eps, rows, k, codes, scale)
        _check(codes, scale, rows, want, 20 * U)
        B.llama_q8_norm_quant(t, x, stride, None, 0, None, 0, g, eps, rows, k, codes, scale)
        _check(codes, scale, rows, I.norm_quant(_host(x[:, :k]), _host(g), float(np.float32(eps))), 20 * U)
        into = d.clone()
        B.llama_q8_norm_quant(t, x, stride, into, stride, into, stride, g, eps, rows, k, codes, scale)
        _check(codes, scale, rows, want, 20 * U)
        assert torch.equal(into[:, :k], h)
        B.llama_q8_norm_quant(t, x, stride, d, stride, x, stride, g, eps, rows, k, codes, scale)
        _check(codes, scale, rows, want, 20 * U)
        assert torch.equal(x[:, :k], h)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("k", LENGTHS)
def test_silu_quant(B, kind, k):
    t, dtype = TYPES[kind]
    rows = 5 if k < 5000 else 2
    for stride, shift in ((2 * k, 0), (2 * k + 3, 1), (-(-2 * k // 8) * 8, 0)):
        _, both = _strided(_rand(k + 3, rows, 2 * k, scale=2.5), stride, dtype, shift)
        gate, up = both[:, :k], both[:, k:2 * k]
        codes, scale = _outputs(rows, k)
        B.llama_q8_silu_quant(t, gate, up, stride, rows, k, codes, scale)
        _check(codes, scale, rows, I.silu_quant(_host(gate), _host(up)), 2 * U)


def test_many_rows(B):
    x = _rand(9, 5000, 40).cuda()
    codes, scale = _outputs(5000, 40)
    B.llama_q8_rows_quant(0, x, 40, 5000, 40, codes, scale)
    _check(codes, scale, 5000, I.rows_quant(_host(x)), 0.0)


@pytest.mark.parametrize("k", [32, 96, 576, 4096, 16416])
def test_rows_quant_blocks(B, k):
    """Q8_0 blocks as the library makes them, rows further apart than their blocks."""
    rows, stride = 5, k + 32
    blocks = torch.zeros((rows, stride // 32 * 34), dtype=torch.uint8, device="cuda")
    w = _rand(k, rows, k, scale=0.02).cuda()
    packed = torch.empty((rows, k // 32 * 34), dtype=torch.uint8, device="cuda")
    B.llama_q8_quantize(w, rows, k, packed)
    blocks[:, :k // 32 * 34] = packed
    codes, scale = _outputs(rows, k)
    B.llama_q8_rows_quant(8, blocks, stride, rows, k, codes, scale)
    _check(codes, scale, rows, I.rows_quant(I.q8_0_values(packed.cpu().numpy(), k)), 0.0)
    # the same blocks, two bytes on: 2-byte boundaries are enough
    flat = torch.zeros(rows * (stride // 32 * 34) + 2, dtype=torch.uint8, device="cuda")
    flat[2:] = blocks.flatten()
    codes, scale = _outputs(rows, k)
    B.llama_q8_rows_quant(8, flat[2:], stride, rows, k, codes, scale)
    _check(codes, scale, rows, I.rows_quant(I.q8_0_values(packed.cpu().numpy(), k)), 0.0)


# more rows than the GPU takes at once, in every form for them, with rows among them that leave the usual way
@pytest.mark.parametrize("op", ["rows", "norm", "silu"])
@pytest.mark.parametrize("kind,rows,k", [("bf16", 1300, 4096), ("f16", 400, 10000), ("bf16", 5000, 520), ("f32", 2500, 2080),
                                         ("f32", 200, 14336), ("f16", 1301, 2049)])
def test_many_long_rows(B, op, kind, rows, k):
    t, dtype = TYPES[kind]
    tiny = 2.0 ** -110 if kind != "f16" else 2.0 ** -20
    x, y = _rand(rows, rows, k, scale=2.0), _rand(k, rows, k)
    for at in (3, min(307, rows - 4), rows // 2, rows - 1):
        x[at], x[at - 1, k // 2], x[at - 2] = 0.0, float("nan"), x[at - 2] * tiny
        y[at], y[at - 2] = 0.0, y[at - 2] * tiny
    x[rows // 3, 5] = float("inf")
    x, y = x.to(dtype).cuda(), y.to(dtype).cuda()
    codes, scale = _outputs(rows, k)
    if op == "rows":
        B.llama_q8_rows_quant(t, x, k, rows, k, codes, scale)
        return _check(codes, scale, rows, I.rows_quant(_host(x)), 0.0)
    if op == "silu":
        B.llama_q8_silu_quant(t, x, y, k, rows, k, codes, scale)
        want = I.silu_quant(_host(x), _host(y))
        # A gate of a 16-bit type comes twice in a row, and its ups may have the ratio (2 q + 1) / 254: 127 v / M is then
        # q + 1/2 in fact, in double q + 1/2 off by three roundings of 2^-53 of at most 127, and the code follows it: q or
        # q + 1. Everything else is settled (numbers that are no halves lie further off than 1e-12 but for 1e-12 of them).
        v = _host(x) / (1.0 + np.exp(-_host(x))) * _host(y)
        with np.errstate(all="ignore"):
            a = 127.0 * np.abs(v) / np.abs(v).max(1, keepdims=True)
            half = np.abs(a - np.floor(a) - 0.5) < 1e-12
        got = codes[:rows, :k].cpu().numpy()
        assert half.sum() < 1e-4 * half.size and (np.abs(np.abs(got[half]) - np.floor(a[half]) - 0.5) == 0.5).all()
        want[0][:, :k][half] = got[half]
        # a scale of 2^-220 is 0 in f32: the wanted one is rounded too, by U at most
        return _check(codes, scale, rows, (want[0], want[1].astype(np.float32)), 3 * U)
    g = (1.0 + 0.2 * _rand(1, k)).cuda()
    h = (x.float() + y.float()).to(dtype)
    B.llama_q8_norm_quant(t, x, k, y, k, x, k, g, 1e-5, rows, k, codes, scale)
    _check(codes, scale, rows, I.norm_quant(_host(h), _host(g), float(np.float32(1e-5))), 20 * U)
    assert torch.equal(x.nan_to_num(9.0), h.nan_to_num(9.0))


@pytest.mark.parametrize("rows,k", [(700, 4096), (1300, 2080)])
def test_many_rows_of_blocks(B, rows, k):
    blocks = torch.empty((rows, k // 32 * 34), dtype=torch.uint8, device="cuda")
    w = _rand(k, rows, k, scale=0.02)
    w[3] = 0.0
    B.llama_q8_quantize(w.cuda(), rows, k, blocks)
    codes, scale = _outputs(rows, k)
    B.llama_q8_rows_quant(8, blocks, k, rows, k, codes, scale)
    _check(codes, scale, rows, I.rows_quant(I.q8_0_values(blocks.cpu().numpy(), k)), 0.0)


# ---- values next to the border between two codes

def test_rows_quant_ties(B):
    """Every half, and the f32 numbers on both sides of it, for several maxima."""
    half = np.arange(127) + 0.5
    rows = []
    for m in (254.0, 127.0, 1.0, 3.0, 1e-20, 1.7e30):
        v = np.float32(m) * half / 127.0
        f = v.astype(np.float32)
        rows.append(np.concatenate([[np.float32(m)], f, np.nextafter(f, np.float32(0)),
                                    np.nextafter(f, np.float32(np.inf)), -f]).astype(np.float32))
    x = np.stack(rows)
    codes, scale = _outputs(*x.shape)
    B.llama_q8_rows_quant(0, torch.from_numpy(x).cuda(), x.shape[1], x.shape[0], x.shape[1], codes, scale)
    _check(codes, scale, x.shape[0], I.rows_quant(x), 0.0)


@pytest.mark.parametrize("k", [300, 3000, 17000])
def test_norm_quant_near_halves(B, k):
    """Products h g within one rounding of every border: only the exact product tells the code."""
    rng = np.random.default_rng(k)
    g = (0.5 + rng.random(k)).astype(np.float32)
    q = rng.integers(0, 127, (4, k)) + 0.5
    h = (2.0 * q / g * np.where(rng.random((4, k)) < 0.5, -1, 1)).astype(np.float32)
    g[7], h[:, 7] = 1.0, 254.0
    codes, scale = _outputs(4, k)
    B.llama_q8_norm_quant(0, torch.from_numpy(h).cuda(), k, None, 0, None, 0, torch.from_numpy(g).cuda(), 1e-5, 4, k,
                          codes, scale)
    _check(codes, scale, 4, I.norm_quant(h, g, float(np.float32(1e-5))), 20 * U)


@pytest.mark.parametrize("k", [300, 3000])
def test_norm_quant_maximum_among_equals(B, k):
    """Many products that are equal in f32 and not in fact: the largest is the unit."""
    rng = np.random.default_rng(k)
    g = (1.0 + rng.random(k)).astype(np.float32)
    h = (200.0 / g).astype(np.float32)[None].repeat(3, 0)
    h[1:] *= np.where(rng.random((2, k)) < 0.5, np.float32(1.0), np.float32(0.25 + 2.0 ** -8))
    codes, scale = _outputs(3, k)
    B.llama_q8_norm_quant(0, torch.from_numpy(h).cuda(), k, None, 0, None, 0, torch.from_numpy(g).cuda(), 0.0, 3, k,
                          codes, scale)
    _check(codes, scale, 3, I.norm_quant(h, g, 0.0), 20 * U)


@pytest.mark.parametrize("k", [300, 3000, 17000])
def test_silu_quant_near_halves(B, k):
    rng = np.random.default_rng(k)
    gate = (rng.standard_normal((3, k)) * 4.0).astype(np.float32)
    gate[:, 7] = 30.0
    silu = gate.astype(np.longdouble) / (1 + np.exp(-gate.astype(np.longdouble)))
    unit = 254.0 / 127.0
    up = ((rng.integers(0, 60, (3, k)) + 0.5) * unit / np.where(np.abs(silu) < 1e-3, 1e6, silu)).astype(np.float32)
    up[:, 7] = 254.0 / 30.0
    top = np.abs(silu[:, 7] * up[:, 7].astype(np.longdouble)).max()
    up = np.where(np.abs(silu * up) > top, 0, up).astype(np.float32)
    codes, scale = _outputs(3, k)
    B.llama_q8_silu_quant(0, torch.from_numpy(gate).cuda(), torch.from_numpy(up).cuda(), k, 3, k, codes, scale)
    _check(codes, scale, 3, I.silu_quant(gate, up), 2 * U)


def test_silu_quant_halves_of_one_gate(B):
    """One gate and ups whose ratios are exact halves: either neighbour is as near; every other code is the nearest."""
    rng = np.random.default_rng(5)
    rows, k = 40, 300
    gate = np.repeat((rng.standard_normal((rows, 1)) * 4.0).astype(np.float32), k, 1)
    up = (rng.integers(-127, 127, (rows, k)) + 0.5).astype(np.float32)
    up[:, 9] = 127.0
    codes, scale = _outputs(rows, k)
    B.llama_q8_silu_quant(0, torch.from_numpy(gate).cuda(), torch.from_numpy(up).cuda(), k, rows, k, codes, scale)
    torch.cuda.synchronize()
    got = codes[:rows, :k].cpu().numpy() * np.sign(gate)
    assert (np.abs(got - up)[:, np.arange(k) != 9] == 0.5).all() and (got[:, 9] == 127).all()
    off = np.nextafter(up, np.float32(np.inf))  # just past the halves: no choice is left
    off[:, 9] = 127.0
    B.llama_q8_silu_quant(0, torch.from_numpy(gate).cuda(), torch.from_numpy(off).cuda(), k, rows, k, codes, scale)
    torch.cuda.synchronize()
    assert np.array_equal(codes[:rows, :k].cpu().numpy() * np.sign(gate), np.where(off == 127, 127, np.floor(off + 0.5)))


# ---- rows that f32 does not hold, zeros, NaN and infinities

@pytest.mark.parametrize("k", [20, 576, 5000, 17000])
def test_far_magnitudes(B, k):
    base = np.random.default_rng(k).standard_normal((12, k))
    size = np.array([1e-44, 1e-40, 1e-36, 1e-30, 1e-25, 1e-12, 1.0, 1e12, 1e19, 1e30, 5e36, 6e37])[:, None]
    x = (base * size).astype(np.float32)
    dx = torch.from_numpy(x).cuda()
    codes, scale = _outputs(12, k)
    B.llama_q8_rows_quant(0, dx, k, 12, k, codes, scale)
    _check(codes, scale, 12, I.rows_quant(x), 0.0)
    g = (1.0 + 0.1 * np.random.default_rng(1).standard_normal(k)).astype(np.float32)
    for factor, eps in ((1.0, 0.0), (1e-20, 1e-5), (1e20, 0.0)):
        gf = (g * np.float32(factor)).astype(np.float32)
        codes, s = I.norm_quant(x, gf, float(np.float32(eps)))
        got, scale = _outputs(12, k)
        B.llama_q8_norm_quant(0, dx, k, None, 0, None, 0, torch.from_numpy(gf).cuda(), eps, 12, k, got, scale)
        # a scale below the normal range keeps what f32 keeps there
        torch.cuda.synchronize()
        assert np.array_equal(got[:12].cpu().numpy(), codes)
        assert (np.abs(_host(scale[:12]) - s) <= 20 * U * s + 2.0 ** -149).all()


def test_silu_far_gates(B):
    """Gates whose exponentials leave the range, beside and without larger products."""
    gate = np.array([[-200, -90, -88, -85, -81, -80, -79, -20, 0.0, 5.0, 60.0, 90.0, 200.0, 1e30, -1e30, 3e-39],
                     [-200, -110, -100, -90, -150, -88.5, -95, -101, -102, -103, -104, -105, -106, -88, -500, -1e4],
                     [-88, -87, -86, -85, -84, -83, -82, -81, -80, -79, -78, -77, -76, -75, -74, -73]], np.float32)
    up = np.array([[3e38, 1e38, 1e37, 2.0, 1e36, 1.0, 1e33, 1e6, 3.0, 1.0, 1.0, -1.0, 1.0, 1e-30, 1.0, 1.0],
                   [1.0] * 16, [1e30, -2e30, 3e29, 1e30, 1e30, 1e30, 1e29, 1e29, 1e28, 1e28, 1e28, 1e27, 1e27, 1e27,
                                1e26, 1e26]], np.float32)
    codes, scale = _outputs(3, 16)
    B.llama_q8_silu_quant(0, torch.from_numpy(gate).cuda(), torch.from_numpy(up).cuda(), 16, 3, 16, codes, scale)
    wc, ws = I.silu_quant(gate, up)
    torch.cuda.synchronize()
    assert np.array_equal(codes[:3].cpu().numpy(), wc)
    assert (np.abs(_host(scale[:3]) - ws) <= 2 * U * ws + 2.0 ** -149).all()


@pytest.mark.parametrize("k", [24, 576, 17000])
def test_rows_that_are_not_finite_spoil_themselves_alone(B, k):
    for op in ("rows", "norm", "norm_g", "silu"):
        x = np.random.default_rng(k).standard_normal((7, k)).astype(np.float32)
        y = np.random.default_rng(k + 1).standard_normal((7, k)).astype(np.float32)
        g = np.ones(k, np.float32)
        x[1], x[2, k - 1], x[3, 0], x[4, k // 2] = 0.0, np.nan, np.inf, -np.inf
        if op == "norm":  # a sum past the range of f32
            x[5, 3], y[5, 3] = 3e38, 3e38
        elif op == "norm_g":
            g[k - 2] = np.nan
        elif op == "silu":
            y[5, 1] = np.inf
        dx, dy, dg = (torch.from_numpy(v).cuda() for v in (x, y, g))
        codes, scale = _outputs(7, k)
        if op == "rows":
            B.llama_q8_rows_quant(0, dx, k, 7, k, codes, scale)
            want, tol = I.rows_quant(x), 0.0
        elif op == "silu":
            B.llama_q8_silu_quant(0, dx, dy, k, 7, k, codes, scale)
            want, tol = I.silu_quant(x, y), 2 * U
        else:
            B.llama_q8_norm_quant(0, dx, k, dy, k, None, 0, dg, 1e-5, 7, k, codes, scale)
            with np.errstate(all="ignore"):
                h = (x + y).astype(np.float32)
            want, tol = I.norm_quant(h, g, float(np.float32(1e-5))), 20 * U
        _check(codes, scale, 7, want, tol)
        assert np.isnan(want[1]).sum() >= 3


def test_a_zero_norm_row_with_a_gain_of_zero(B):
    x = torch.tensor([[1.0, 2.0, 0.0, 3.0], [0.0, 0.0, 5.0, 0.0]], device="cuda")
    g = torch.tensor([0.0, 0.0, 7.0, 0.0], device="cuda")
    codes, scale = _outputs(2, 4)
    B.llama_q8_norm_quant(0, x, 4, None, 0, None, 0, g, 0.0, 2, 4, codes, scale)
    _check(codes, scale, 2, I.norm_quant(_host(x), _host(g), 0.0), 20 * U)


# ---- the product

def _codes(seed, rows, k, low=-127, high=127):
    c = np.zeros((rows, I.row_bytes(k)), np.int8)
    c[:, :k] = np.random.default_rng(seed).integers(low, high + 1, (rows, k))
    return c, (0.01 + np.random.default_rng(seed + 1).random(rows)).astype(np.float32)


class Product:
    def __init__(self, B, w, sw, k, m_max):
        self.B, self.n, self.k = B, w.shape[0], k
        self.packed = torch.full((B.llama_q8_i8_packed_bytes(self.n, k),), 0x55, dtype=torch.uint8, device="cuda")
        dw, ds = torch.from_numpy(w).cuda(), torch.from_numpy(sw).cuda()
        B.llama_q8_i8_pack(dw, ds, self.n, k, self.packed)
        self.ws_bytes = B.llama_q8_i8_matmul_workspace_bytes(self.n, k, m_max)
        self.ws = torch.zeros(max(16, self.ws_bytes), dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def __call__(self, a, sa, kind, stride, y, stream=0):
        self.B.llama_q8_i8_matmul(self.packed, self.n, self.k, a, sa, sa.numel(), TYPES[kind][0], y, stride, self.ws,
                                  self.ws_bytes, self.err, stream)


def _product(B, a, sa, w, sw, k, kind="f32", pad=0, want=None):
    m, n = a.shape[0], w.shape[0]
    p = Product(B, w, sw, k, m)
    y = torch.full((m + 1, n + pad), 3.0, dtype=TYPES[kind][1], device="cuda")
    p(torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda(), kind, n + pad, y)
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    assert (y[m] == 3.0).all() and (y[:, n:] == 3.0).all()
    want = I.matmul(a, sa, w, sw, k) if want is None else want
    got = _host(y[:m, :n])
    step = 0.0 if kind == "f32" else torch.finfo(TYPES[kind][1]).eps / 2
    tiny = 0.0 if kind == "f32" else torch.finfo(TYPES[kind][1]).smallest_normal * step * 2
    off = np.abs(got - want)
    assert (off <= (3 * U * (1 + step) + step) * np.abs(want) + tiny).all(), (off.max(), np.argwhere(
        off > (3 * U * (1 + step) + step) * np.abs(want) + tiny)[:5].tolist())
    return y


TOKENS = [1, 2, 3, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 520]


@pytest.mark.parametrize("m", TOKENS)
@pytest.mark.parametrize("n,k", [(1, 1), (32, 16), (33, 17), (100, 200), (127, 64), (129, 65), (576, 576), (960, 130),
                                 (300, 1024), (257, 1100), (64, 4100), (4096, 512)])
def test_matmul(B, m, n, k):
    a, sa = _codes(m, m, k)
    w, sw = _codes(n + 7, n, k)
    _product(B, a, sa, w, sw, k, pad=(m + n) % 4)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 100, 300), (7, 33, 64), (40, 200, 576), (130, 259, 1100), (300, 513, 96)])
def test_matmul_16_bit(B, kind, m, n, k):
    a, sa = _codes(m, m, k)
    w, sw = _codes(n + 7, n, k)
    _product(B, a, sa * np.float32(1e-3), w, sw * np.float32(1e-2), k, kind, pad=m % 3)


@pytest.mark.parametrize("m", [1, 4, 8, 12, 40, 70, 150, 270])
@pytest.mark.parametrize("n,k", [(40, 1024), (136, 4096), (200, 14336), (40, 131056)])
def test_matmul_sums_are_exact(B, m, n, k):
    """Sums far past 2^24, and the largest there are: equal to the integers, whatever cancels on the way."""
    rng = np.random.default_rng(m + k)
    one = np.ones(1, np.float32)
    a = np.zeros((m, I.row_bytes(k)), np.int8)
    w = np.zeros((n, I.row_bytes(k)), np.int8)
    a[:, :k], w[:, :k] = 127, 127
    a[0, :k] = -128
    w[1, :k] = -128
    w[2, :k] = np.where(np.arange(k) % 2 == 0, 127, -127)
    w[3, :k] = np.where(np.arange(k) < k // 2, 127, -127)
    w[4, :k] = np.where(np.arange(k) < k - 1, 0, 1)
    w[5, :k] = np.where(np.arange(k) < k - 1, 127, -126)
    w[6:20, :k] = rng.integers(100, 128, (14, k))
    if m > 2:
        a[2, :k] = np.where(np.arange(k) % 3 == 0, 1, 127)
        a[m - 1, :k] = rng.integers(-128, 128, k)
    y = _product(B, a, one.repeat(m), w, one.repeat(n), k)
    # f32 of the exact integers, to the last bit
    sums = a[:, :k].astype(np.int64) @ w[:, :k].astype(np.int64).T
    assert np.array_equal(y[:m, :n].cpu().numpy(), sums.astype(np.float32))


@pytest.mark.parametrize("m", [1, 5, 40, 300])
def test_matmul_rows_that_are_not_finite_spoil_themselves_alone(B, m):
    n, k = 130, 100
    a, sa = _codes(3, m, k)
    w, sw = _codes(4, n, k)
    clean = _product(B, a, sa, w, sw, k)
    sa2, sw2 = sa.copy(), sw.copy()
    sa2[m // 2], sw2[17] = np.nan, np.inf
    p = Product(B, w, sw2, k, m)
    y = torch.zeros((m, n), device="cuda")
    p(torch.from_numpy(a).cuda(), torch.from_numpy(sa2).cuda(), "f32", n, y)
    torch.cuda.synchronize()
    assert torch.isnan(y[m // 2]).all() and not torch.isfinite(y[:, 17]).any()
    rest = [t for t in range(m) if t != m // 2]
    keep = [i for i in range(n) if i != 17]
    assert torch.equal(y[rest][:, keep], clean[:m, :n][rest][:, keep])


# sizes at which the matrix kernel takes few tokens, too: whole and cut tiles, an odd last block of k, the last tile's
# channels, several reads of the sums of a long k, a last group of tokens
@pytest.mark.parametrize("m", [17, 31, 33, 48, 50, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("n,k", [(9000, 2000), (20001, 1025), (8200, 4111), (1301, 14336), (2600, 7000)])
def test_matmul_of_few_tokens_on_the_matrix_kernel(B, m, n, k):
    gen = torch.Generator(device="cuda").manual_seed(m * n)
    a = torch.randint(-128, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    # rows whose sums pass 2^24 on the way, and cancel
    w[5], w[n - 1], a[m - 1] = 127, -128, 127
    a[1, ::2], a[1, 1::2] = 127, -128
    pad = torch.zeros((m, I.row_bytes(k)), dtype=torch.int8, device="cuda")
    wpad = torch.zeros((n, I.row_bytes(k)), dtype=torch.int8, device="cuda")
    pad[:, :k], wpad[:, :k] = a, w
    one = torch.ones(max(m, n), device="cuda")
    p = Product(B, wpad.cpu().numpy(), one[:n].cpu().numpy(), k, m)
    y = torch.full((m + 1, n + 3), 3.0, device="cuda")
    p(pad, one[:m], "f32", n + 3, y)
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    assert torch.equal(y[:m, :n], (a.double() @ w.double().T).float())
    assert (y[m] == 3.0).all() and (y[:, n:] == 3.0).all()


@pytest.mark.parametrize("m,n,k", [(1, 4096, 14336), (6, 28672, 576), (16, 49152, 576), (48, 4096, 14336),
                                   (512, 6144, 4096), (203, 1536, 576), (1000, 4096, 4096), (2049, 640, 1536)])
def test_matmul_model_shapes(B, m, n, k):
    """Larger products, against f64 on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    a = torch.randint(-127, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(m, generator=gen, device="cuda") + 0.1, torch.rand(n, generator=gen, device="cuda") + 0.1
    want = (a.double() @ w.double().T) * sa.double()[:, None] * sw.double()[None, :]
    _product(B, a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), k, want=want.cpu().numpy())


def test_matmul_offsets_past_32_bits(B):
    """Outputs and codes beyond 2^31 elements: the first and last rows of what the GPU holds."""
    m, n, k = 70001, 32768, 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(-127, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    one = torch.ones(m, device="cuda")
    p = Product(B, w.cpu().numpy(), np.ones(n, np.float32), k, m)
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    p(a, one, "bf16", n, y)
    for at in (slice(0, 40), slice(65520, 65560), slice(m - 40, m)):
        assert torch.equal(y[at], (a[at].double() @ w.double().T).bfloat16())
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("more", [1, 20, 70, 300])
def test_matmul_of_two_launches(B, more):
    """The tokens behind the first launch's 65536 go by a plan of their own."""
    m, n, k = 65536 + more, 300, 600
    gen = torch.Generator(device="cuda").manual_seed(more)
    pad = torch.zeros((m, I.row_bytes(k)), dtype=torch.int8, device="cuda")
    pad[:, :k] = torch.randint(-128, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.zeros((n, I.row_bytes(k)), dtype=torch.int8, device="cuda")
    w[:, :k] = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    p = Product(B, w.cpu().numpy(), np.ones(n, np.float32), k, m)
    y = torch.full((m + 1, n), 3.0, device="cuda")
    p(pad, torch.ones(m, device="cuda"), "f32", n, y)
    torch.cuda.synchronize()
    assert int(p.err.item()) == 0
    assert torch.equal(y[:m], (pad.double() @ w.double().T).float())
    assert (y[m] == 3.0).all()


# ---- a run of them together, streams, graphs, workspaces

def _mlp(B, rows, h, f, seed):
    """norm_quant -> gate | up -> silu_quant -> down, as a layer's second half makes it."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(x=torch.randn((rows, h), generator=gen, device="cuda") * 2,
              d=torch.randn((rows, h), generator=gen, device="cuda"), g=1 + 0.1 * torch.randn(h, generator=gen, device="cuda"))
    for name, n, k in (("gu", 2 * f, h), ("down", h, f)):
        w = torch.randn((n, k), generator=gen, device="cuda") * 0.05
        codes, scale = torch.zeros((n, I.row_bytes(k)), dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda")
        B.llama_q8_rows_quant(0, w, k, n, k, codes, scale)
        st[name] = torch.zeros(B.llama_q8_i8_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
        B.llama_q8_i8_pack(codes, scale, n, k, st[name])
        st[name + "_host"] = (codes.cpu().numpy(), scale.cpu().numpy())
    n_ws = max(B.llama_q8_i8_matmul_workspace_bytes(2 * f, h, rows), B.llama_q8_i8_matmul_workspace_bytes(h, f, rows))
    st.update(ws=torch.zeros(max(16, n_ws), dtype=torch.uint8, device="cuda"), n_ws=n_ws,
              err=torch.zeros(1, dtype=torch.int32, device="cuda"), out=torch.zeros((rows, h), device="cuda"),
              h=torch.zeros((rows, h), device="cuda"), gu_y=torch.zeros((rows, 2 * f), device="cuda"),
              a=torch.zeros((rows, I.row_bytes(h)), dtype=torch.int8, device="cuda"), sa=torch.zeros(rows, device="cuda"),
              b=torch.zeros((rows, I.row_bytes(f)), dtype=torch.int8, device="cuda"), sb=torch.zeros(rows, device="cuda"))

    def run(stream=0):
        B.llama_q8_norm_quant(0, st["x"], h, st["d"], h, st["h"], h, st["g"], 1e-5, rows, h, st["a"], st["sa"], stream)
        B.llama_q8_i8_matmul(st["gu"], 2 * f, h, st["a"], st["sa"], rows, 0, st["gu_y"], 2 * f, st["ws"], st["n_ws"],
                             st["err"], stream)
        B.llama_q8_silu_quant(0, st["gu_y"], st["gu_y"][:, f:], 2 * f, rows, f, st["b"], st["sb"], stream)
        B.llama_q8_i8_matmul(st["down"], h, f, st["b"], st["sb"], rows, 0, st["out"], h, st["ws"], st["n_ws"],
                             st["err"], stream)
    return st, run


def _mlp_check(st, rows, h, f):
    """Every step against the oracle on the step's own inputs."""
    hh = _host(st["h"])
    codes, scale = I.norm_quant(hh, _host(st["g"]), float(np.float32(1e-5)))
    assert np.array_equal(st["a"].cpu().numpy(), codes)
    assert np.allclose(_host(st["sa"]), scale, rtol=20 * U, atol=0)
    gu = I.matmul(codes, _host(st["sa"]), *st["gu_host"], h)
    assert (np.abs(_host(st["gu_y"]) - gu) <= 3 * U * np.abs(gu)).all()
    y = _host(st["gu_y"])
    codes, scale = I.silu_quant(y[:, :f], y[:, f:])
    assert np.array_equal(st["b"].cpu().numpy(), codes)
    out = I.matmul(codes, _host(st["sb"]), *st["down_host"], f)
    assert (np.abs(_host(st["out"]) - out) <= 3 * U * np.abs(out)).all()
    assert int(st["err"].item()) == 0


@pytest.mark.parametrize("rows,h,f", [(1, 576, 1536), (5, 576, 1536), (40, 576, 1536), (203, 576, 1536), (33, 130, 200)])
def test_mlp_of_a_layer(B, rows, h, f):
    st, run = _mlp(B, rows, h, f, rows)
    run()
    torch.cuda.synchronize()
    _mlp_check(st, rows, h, f)


@pytest.mark.parametrize("rows", [1, 40, 203])
def test_mlp_captured_and_replayed_on_a_stream(B, rows):
    h, f = 576, 1536
    st, run = _mlp(B, rows, h, f, 50 + rows)
    run()
    torch.cuda.synchronize()
    first = st["out"].clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(torch.cuda.current_stream().cuda_stream)
    st["out"].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(st["out"], first)  # the same bits, call or graph
    st["x"].mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    _mlp_check(st, rows, h, f)
    run(side.cuda_stream)
    side.synchronize()
    _mlp_check(st, rows, h, f)


@pytest.mark.parametrize("kind,rows,k", [("f32", 1, 576), ("bf16", 1, 4096), ("f32", 8, 1000), ("f16", 24, 576),
                                         ("f32", 48, 4160), ("bf16", 90, 4160)])
def test_a_chain_of_calls_on_a_stream_equals_single_steps(B, kind, rows, k):
    """Each kernel reads what the one before it wrote, and its launch may overlap that one's end."""
    t, dtype = TYPES[kind]
    gen = torch.Generator(device="cuda").manual_seed(k)
    w = torch.randn((k, k), generator=gen, device="cuda")
    wc, ws = torch.zeros((k, I.row_bytes(k)), dtype=torch.int8, device="cuda"), torch.zeros(k, device="cuda")
    B.llama_q8_rows_quant(0, w, k, k, k, wc, ws)
    packed = torch.zeros(B.llama_q8_i8_packed_bytes(k, k), dtype=torch.uint8, device="cuda")
    B.llama_q8_i8_pack(wc, ws, k, k, packed)
    n_ws = B.llama_q8_i8_matmul_workspace_bytes(k, k, rows)
    work = torch.zeros(max(16, n_ws), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.full((k,), 0.01, device="cuda")
    start = torch.randn((rows, k), generator=gen, device="cuda").to(dtype)

    def run(wait):
        x, y = start.clone(), torch.zeros((rows, k), dtype=dtype, device="cuda")
        codes, scale = _outputs(rows, k, 0)
        for _ in range(40):
            B.llama_q8_norm_quant(t, x, k, y, k, x, k, g, 1e-5, rows, k, codes, scale)
            wait()
            B.llama_q8_i8_matmul(packed, k, k, codes, scale, rows, t, y, k, work, n_ws, err)
            wait()
            B.llama_q8_silu_quant(t, y, x, k, rows, k, codes, scale)
            wait()
            B.llama_q8_i8_matmul(packed, k, k, codes, scale, rows, t, y, k, work, n_ws, err)
            wait()
            B.llama_q8_rows_quant(t, y, k, rows, k, codes, scale)
            wait()
            B.llama_q8_i8_matmul(packed, k, k, codes, scale, rows, t, y, k, work, n_ws, err)
            wait()
            y.mul_(1e-4)
            wait()
        torch.cuda.synchronize()
        return x.clone(), y.clone(), codes.clone()

    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(v.float()).all() for v in want)
    for _ in range(5):
        for got, w_ in zip(run(lambda: None), want):
            assert torch.equal(got, w_)
    assert int(err.item()) == 0


def test_one_workspace_for_products_of_many_sizes(B):
    shapes = [(40, 960, 576), (300, 4096, 300), (9, 576, 4100), (64, 96, 1536), (130, 2048, 2048), (33, 33, 33),
              (40, 4096, 4500), (200, 700, 3000)]
    size = max(B.llama_q8_i8_matmul_workspace_bytes(n, k, m) for m, n, k in shapes)
    ws = torch.zeros(max(16, size), dtype=torch.uint8, device="cuda")
    for seed in (0, 1):
        for m, n, k in shapes[::-1] if seed else shapes:
            a, sa = _codes(seed + m, m, k)
            w, sw = _codes(seed + n, n, k)
            p = Product(B, w, sw, k, m)
            p.ws, p.ws_bytes = ws, size
            y = torch.zeros((m, n), device="cuda")
            p(torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda(), "f32", n, y)
            want = I.matmul(a, sa, w, sw, k)
            assert (np.abs(_host(y) - want) <= 3 * U * np.abs(want)).all() and int(p.err.item()) == 0


def test_two_products_at_once_on_streams_of_their_own(B):
    a, sa = _codes(1, 100, 2048)
    runs = []
    for i in range(2):
        w, sw = _codes(20 + i, 1500, 2048)
        runs.append((Product(B, w, sw, 2048, 100), torch.cuda.Stream(), torch.zeros((100, 1500), device="cuda"),
                     I.matmul(a, sa, w, sw, 2048)))
    da, dsa = torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda()
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s, y, _ in runs:
            p(da, dsa, "f32", 1500, y, s.cuda_stream)
    torch.cuda.synchronize()
    for p, _, y, want in runs:
        assert (np.abs(_host(y) - want) <= 3 * U * np.abs(want)).all() and int(p.err.item()) == 0


def test_no_rows(B):
    codes, scale = _outputs(0, 64)
    x = torch.zeros((1, 64), device="cuda")
    B.llama_q8_rows_quant(0, x, 64, 0, 64, codes, scale)
    B.llama_q8_norm_quant(0, x, 64, None, 0, None, 0, x, 1e-5, 0, 64, codes, scale)
    B.llama_q8_silu_quant(0, x, x, 64, 0, 64, codes, scale)
    torch.cuda.synchronize()
    assert (codes == 77).all() and (scale == 5.5).all()
