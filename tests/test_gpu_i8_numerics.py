"""The 8-bit quantisers against the CPU definitions where f32 reaches its ends, and to the last bit of their scales."""
import numpy as np
import pytest
import torch

from oracle import i8_oracle as I
from tests.gpu_helpers import binding, require_gpu
from tests.test_gpu_i8 import TYPES, U, _check, _host, _outputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    require_gpu()
    return binding()


def _silu(gate):
    gate = gate.astype(np.longdouble)
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate))


def _near_halves(rng, gate, at, top, kind):
    """(gate, up) of a row in a type: the product at `at` is the largest, about `top`, the others lie as near to halves of its
    127th as the type's ups allow. None is closer than 1e-11 to one, so that the definition in f64 knows every code."""
    dtype = TYPES[kind][1]
    gate = torch.from_numpy(gate.astype(np.float32)).to(dtype).double().numpy()
    silu = _silu(gate)
    q = rng.integers(0, 127, gate.size) + 0.5
    q[at] = 127.0
    with np.errstate(all="ignore"):
        up = torch.from_numpy((q * top / 127.0 / silu).astype(np.float64)).to(dtype).double().numpy()
        up[~np.isfinite(up)] = 0.0
        v = np.abs(silu * up.astype(np.longdouble))
        t = 127.0 * v / v[at]
        t[at] = 0.0
        up[(t > 127.0) | (np.abs(t - np.floor(t) - 0.5) < 1e-11)] = 0.0
    assert up[at] != 0.0
    return gate, up


def _check_silu(B, kind, rows):
    gate, up = (np.stack(x) for x in zip(*rows))
    n, k = gate.shape
    dtype = TYPES[kind][1]
    codes, scale = _outputs(n, k)
    B.llama_q8_silu_quant(TYPES[kind][0], torch.from_numpy(gate).to(dtype).cuda(), torch.from_numpy(up).to(dtype).cuda(), k,
                          n, k, codes, scale)
    _check(codes, scale, n, I.silu_quant(gate, up), 2 * U)


# the row's largest product has a gate below -80, and others next to a half have one
FAR = [(-80.5, 1e-3), (-82, 2e-4), (-85, 1e-10), (-88, 5e-5), (-88.5, 3e-7), (-90, 7e-8), (-90, 0.07), (-96, 1e-9),
       (-100, 4e-6), (-104, 2e-7)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("k", [40, 600, 4096, 17000])
def test_silu_largest_product_of_a_far_gate(B, kind, k):
    rng = np.random.default_rng(k)
    rows = []
    for far, top in FAR:
        gate = rng.standard_normal(k) * 4.0
        gate = np.where(rng.random(k) < 0.3, rng.choice([-82.0, -84.5, -88.0, -88.5, -90.0, -97.0], k), gate)
        at = int(rng.integers(k))
        gate[at] = far
        rows.append(_near_halves(rng, gate, at, top, kind))
    _check_silu(B, kind, rows)


# gates in or next to the subnormal range with ups that bring the products back, and the reverse
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("k", [40, 600, 4096, 9000, 17000])
def test_silu_gates_and_ups_at_the_ends_of_f32(B, kind, k):
    rng = np.random.default_rng(k + 1)
    rows = []
    for low, high, top in ((-44.5, -38.5, 1e-7), (-43, -42, 1e-20), (-42, -37, 1e-20), (-39, -34, 1e-3), (-38.2, -37.7, 1.0),
                           (-33, -28, 1e6), (28, 34, 1e-7), (30, 31, 1e-12 if kind == "f32" else 1e-8)):
        least = 1.5e-45 if kind == "f32" else 1e-40
        gate = np.maximum(10.0 ** rng.uniform(low, high, k), least) * rng.choice([-1.0, 1.0] if low < 0 else [1.0], k)
        gate = np.where(rng.random(k) < 0.2, rng.standard_normal(k) * 3.0, gate)
        at = int(rng.integers(k))
        gate[at] = max(10.0 ** ((low + high) / 2), least)
        rows.append(_near_halves(rng, gate, at, top, kind))
    _check_silu(B, kind, rows)


# h g a step of 2^-46 below q + 1/2 in 127ths of the largest product, which f32 alone takes for the half itself. Of a product of
# about 2^-107 the part below f32 is under the smallest f32 number. The last rows are 2^6, 2^8 and 2^30 times as large.
@pytest.mark.parametrize("k", [30, 900, 9000, 17000])
def test_norm_products_whose_second_part_is_below_f32(B, k):
    pairs = [(8388607, 8388609, 46), (4783982, 14709241, 46), (4374971, 16084391, 46), (13911026, 15175461, 46),
             (13140607, 13387651, 45), (12582911, 12582913, 44), (12653911, 15292825, 44)]  # odd 2^bits - 1 to 6
    h, g = np.zeros(k), np.zeros(k)
    h[3], g[3] = 254.0 * 2.0 ** -40, 2.0 ** -67
    for i, (a, b, bits) in enumerate(pairs):
        odd = round(a * b / 2.0 ** bits)
        assert odd % 2 == 1 and 0 < odd * 2 ** bits - a * b < 8
        at = (7 + i * (k // 8)) % k
        h[at], g[at] = a * 2.0 ** -60, b * 2.0 ** (-47 - bits)
        h[(at + 1) % k], g[(at + 1) % k] = -h[at], g[at]
    rows = np.stack([h, h * 0.5, h * 2.0 ** 6, h * 2.0 ** 8, h * 2.0 ** 30]).astype(np.float32)
    g = g.astype(np.float32)
    codes, scale = _outputs(5, k)
    B.llama_q8_norm_quant(0, torch.from_numpy(rows).cuda(), k, None, 0, None, 0, torch.from_numpy(g).cuda(), 0.0, 5, k,
                          codes, scale)
    _check(codes, scale, 5, I.norm_quant(rows, g, 0.0), 20 * U)


def test_norm_scale_of_a_sum_that_loses_every_small_square(B):
    """One thread has a large square and then small ones, each a little under half a step of the sum, which an addition to it
    drops; so do the additions of lanes and of warps. 30 additions deep a scale is off by 20 * 2^-24 at most."""
    k, tiny = 13952, 2.0 ** -12 * (1 - 2.0 ** -10)
    x = np.zeros((8, 448, 4), np.float32)  # pieces of four values, dealt over 448 threads
    x[:, 0, :] = tiny
    x[0, 0, 0] = 1.0
    x[0, [1, 2, 4, 8, 16], 0] = tiny
    x[0, [32, 64, 128, 256], 0] = tiny
    x = x.reshape(1, -1)[:, :k]
    g = np.ones(k, np.float32)
    g[0] = 1.25
    codes, scale = _outputs(1, k)
    B.llama_q8_norm_quant(0, torch.from_numpy(x).cuda(), k, None, 0, None, 0, torch.from_numpy(g).cuda(), 0.0, 1, k, codes,
                          scale)
    _check(codes, scale, 1, I.norm_quant(x, g, 0.0), 20 * U)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("k", [9, 700, 17000])
def test_silu_scale_is_rounded_once(B, kind, k):
    """M / 127, M known to 2^-40, rounded to f32: off by half a step, and by that 2^-40 where it decides."""
    dtype = TYPES[kind][1]
    gen = torch.Generator(device="cuda").manual_seed(k)
    rows = 400 if k < 1000 else 30
    gate = (torch.randn((rows, k), generator=gen, device="cuda") * 3).to(dtype)
    up = torch.randn((rows, k), generator=gen, device="cuda").to(dtype)
    codes, scale = _outputs(rows, k)
    B.llama_q8_silu_quant(TYPES[kind][0], gate, up, k, rows, k, codes, scale)
    torch.cuda.synchronize()
    want = np.abs(_silu(_host(gate)) * _host(up)).max(1) / 127
    got = _host(scale[:rows])
    step = np.spacing(want.astype(np.float32)).astype(np.float64)  # of the binade: a half step is at most U of the value
    assert (np.abs(got - want) <= step * (0.5 + 2.0 ** -15)).all()


def test_silu_products_below_any_scale(B):
    """Gates so far down that no f32 scale holds their products: zeros, alone in a row or beside others."""
    k = 40
    gate, up = np.full((2, k), -1000.0, np.float32), np.full((2, k), 3e38, np.float32)
    gate[0, ::3], gate[1, 5], up[1, 5] = -1e30, 2.0, 1.0
    codes, scale = _outputs(2, k)
    B.llama_q8_silu_quant(0, torch.from_numpy(gate).cuda(), torch.from_numpy(up).cuda(), k, 2, k, codes, scale)
    torch.cuda.synchronize()
    assert not codes[0].any() and float(scale[0]) == 0.0
    assert int(codes[1, 5]) == 127 and int(codes[1].count_nonzero()) == 1
    assert abs(float(scale[1]) * 127 / float(_silu(np.float32([2.0]))[0]) - 1) <= 1.001 * U
