"""The 8-bit products without a GPU: the refusals of every entry point, the sizes the
queries give, the binding's checks of tensors, and properties that pin the oracle."""
import ctypes as C
from fractions import Fraction

import numpy as np
import pytest

from oracle import i8_oracle as I
from tests.gpu_helpers import built_lib
from tests.test_paged_binding import Library, Tensor

X, Y, Z, G, CODES, SCALE, PACKED, WS, ERR = (C.c_void_p(i << 20) for i in range(1, 10))  # stand-in addresses


def _off(p, n):
    return C.c_void_p(p.value + n)


@pytest.fixture(scope="module")
def B():
    built_lib()
    from q8_quantized_llama_gb300 import binding
    binding.lib()
    return binding


def _status(B, name):
    return {"ARG": B.LQ8_ERR_ARG, "UNSUPPORTED": B.LQ8_ERR_UNSUPPORTED, "OK": B.LQ8_OK}[name]


MAX_K = 131056

COMMON = [(dict(rows=-1), "ARG"), (dict(k=0), "ARG"), (dict(k=-4), "ARG"), (dict(codes=None), "ARG"),
          (dict(scale=None), "ARG"), (dict(codes=_off(CODES, 8)), "ARG"), (dict(scale=_off(SCALE, 2)), "ARG"),
          (dict(type=2), "UNSUPPORTED"), (dict(type=12), "UNSUPPORTED"), (dict(type=-1), "UNSUPPORTED"),
          (dict(k=MAX_K + 1, stride=1 << 20), "UNSUPPORTED"), (dict(stride=575), "ARG"), (dict(rows=0), "OK"),
          (dict(x=_off(X, 2)), "ARG"), (dict(x=_off(X, 1), type=1), "ARG"), (dict(x=None), "ARG")]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(type=8, k=560), "ARG"), (dict(type=8, stride=592), "ARG"), (dict(type=8, x=_off(X, 1)), "ARG"),
    (dict(type=8, rows=0), "OK"), (dict(type=1, x=_off(X, 2), rows=0), "OK")])
def test_rows_quant_refusals(B, kw, status):
    f = dict(type=0, x=X, stride=576, rows=3, k=576, codes=CODES, scale=SCALE)
    f.update(kw)
    assert B.lib().llama_q8_rows_quant(f["type"], f["x"], f["stride"], f["rows"], f["k"], f["codes"], f["scale"],
                                       None) == _status(B, status)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(type=8), "UNSUPPORTED"), (dict(g=None), "ARG"), (dict(g=_off(G, 1)), "ARG"), (dict(eps=-1e-5), "ARG"),
    (dict(eps=float("nan")), "ARG"), (dict(eps=float("inf")), "ARG"), (dict(ds=575), "ARG"), (dict(os=575), "ARG"),
    (dict(delta=_off(Y, 1)), "ARG"), (dict(out=_off(Z, 2)), "ARG"), (dict(out=X, os=580), "ARG"),
    (dict(out=Y, os=580), "ARG"), (dict(delta=None, out=None, ds=0, os=0, rows=0), "OK")])
def test_norm_quant_refusals(B, kw, status):
    f = dict(type=0, x=X, stride=576, delta=Y, ds=576, out=Z, os=576, g=G, eps=1e-5, rows=3, k=576, codes=CODES,
             scale=SCALE)
    f.update(kw)
    if f["k"] > 576:
        f["ds"] = f["os"] = f["stride"]
    assert B.lib().llama_q8_norm_quant(f["type"], f["x"], f["stride"], f["delta"], f["ds"], f["out"], f["os"], f["g"],
                                       f["eps"], f["rows"], f["k"], f["codes"], f["scale"],
                                       None) == _status(B, status)


@pytest.mark.parametrize("kw,status", COMMON + [(dict(type=8), "UNSUPPORTED"), (dict(up=None), "ARG"),
                                                (dict(up=_off(Y, 2)), "ARG")])
def test_silu_quant_refusals(B, kw, status):
    f = dict(type=0, x=X, up=Y, stride=576, rows=3, k=576, codes=CODES, scale=SCALE)
    f.update(kw)
    assert B.lib().llama_q8_silu_quant(f["type"], f["x"], f["up"], f["stride"], f["rows"], f["k"], f["codes"],
                                       f["scale"], None) == _status(B, status)


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), "ARG"), (dict(scale=None), "ARG"), (dict(packed=None), "ARG"), (dict(rows=-1), "ARG"),
    (dict(k=0), "ARG"), (dict(codes=_off(CODES, 4)), "ARG"), (dict(packed=_off(PACKED, 8)), "ARG"),
    (dict(scale=_off(SCALE, 1)), "ARG"), (dict(rows=(1 << 30) + 1), "UNSUPPORTED"), (dict(k=MAX_K + 1), "UNSUPPORTED"),
    (dict(rows=0), "OK")])
def test_pack_refusals(B, kw, status):
    f = dict(codes=CODES, scale=SCALE, rows=33, k=100, packed=PACKED)
    f.update(kw)
    assert B.lib().llama_q8_i8_pack(f["codes"], f["scale"], f["rows"], f["k"], f["packed"], None) == _status(B, status)


@pytest.mark.parametrize("kw,status", [
    (dict(packed=None), "ARG"), (dict(codes=None), "ARG"), (dict(scale=None), "ARG"), (dict(y=None), "ARG"),
    (dict(rows=0), "ARG"), (dict(k=0), "ARG"), (dict(m=-1), "ARG"), (dict(stride=99), "ARG"),
    (dict(type=8), "UNSUPPORTED"), (dict(packed=_off(PACKED, 4)), "ARG"), (dict(codes=_off(CODES, 8)), "ARG"),
    (dict(ws=_off(WS, 8)), "ARG"), (dict(scale=_off(SCALE, 2)), "ARG"), (dict(err=_off(ERR, 2)), "ARG"),
    (dict(y=_off(Y, 2)), "ARG"), (dict(y=_off(Y, 1), type=1), "ARG"), (dict(m=(1 << 30) + 1), "UNSUPPORTED"),
    (dict(rows=(1 << 30) + 1, stride=1 << 31), "UNSUPPORTED"), (dict(k=MAX_K + 1), "UNSUPPORTED"),
    (dict(m=0, ws=None), "OK")])
def test_matmul_refusals(B, kw, status):
    f = dict(packed=PACKED, rows=100, k=200, codes=CODES, scale=SCALE, m=40, type=0, y=Y, stride=100, ws=WS,
             ws_bytes=1 << 40, err=ERR)
    f.update(kw)
    assert B.lib().llama_q8_i8_matmul(f["packed"], f["rows"], f["k"], f["codes"], f["scale"], f["m"], f["type"], f["y"],
                                      f["stride"], f["ws"], f["ws_bytes"], f["err"], None) == _status(B, status)


# one workspace, of the largest matrix and the most tokens, serves all
def test_matmul_workspace_never_falls(B):
    sizes = B.llama_q8_i8_matmul_workspace_bytes
    ms = [1, 16, 17, 32, 33, 64, 65, 100, 128, 129, 255, 256, 257, 300, 512, 777, 1024, 2048, 4096, 65536, 65537, 200000]
    rows, ks = [1, 33, 576, 4096, 28672, 128256], [1, 16, 576, 4096, 14336, 131056]
    for n in rows:
        for k in ks:
            found = [sizes(n, k, m) for m in ms]
            assert found == sorted(found)
    for m in ms:
        for k in ks:
            found = [sizes(n, k, m) for n in rows]
            assert found == sorted(found)
        for n in rows:
            found = [sizes(n, k, m) for k in ks]
            assert found == sorted(found)


@pytest.mark.parametrize("rows,k,m", [(100, 200, 140), (4096, 14336, 48), (28672, 4096, 512), (28672, 4096, 17), (4096, 4096, 32)])
def test_matmul_refuses_a_short_workspace(B, rows, k, m):
    need = B.llama_q8_i8_matmul_workspace_bytes(rows, k, m)
    assert need > 0
    for ws, n in ((WS, need - 1), (WS, 0), (None, need)):
        assert B.lib().llama_q8_i8_matmul(PACKED, rows, k, CODES, SCALE, m, 0, Y, rows, ws, n, None,
                                          None) == B.LQ8_ERR_ARG


def test_sizes(B):
    assert [B.llama_q8_i8_row_bytes(k) for k in (-1, 0, 1, 16, 17, 4096)] == [0, 0, 16, 16, 32, 4096]
    assert B.llama_q8_i8_packed_bytes(32, 16) == 512 + 132
    for rows, k in ((1, 1), (70, 70), (96, 4096), (28672, 4096), (100, 14336)):
        assert B._packed_bytes(rows, k) == B.llama_q8_i8_packed_bytes(rows, k)
    assert B.llama_q8_i8_packed_bytes(33, 17) == 64 * 32 + 66 * 4
    for rows, k in ((0, 16), (16, 0), (1 << 31, 16), (16, MAX_K + 1)):
        assert B.llama_q8_i8_packed_bytes(rows, k) == 0
        assert B.llama_q8_i8_matmul_workspace_bytes(rows, k, 64) == 0


# ---- the binding's checks, on stand-in tensors and a stand-in library

ROWS, K, WIDTH = 5, 70, 90


@pytest.fixture
def S(B, monkeypatch):
    stub = Library()
    monkeypatch.setattr(B, "lib", lambda: stub)
    monkeypatch.setattr(B, "stub", stub, raising=False)
    return B


def _tensors(**kw):
    f32 = lambda *s, **o: Tensor("float32", *s, **o)  # noqa: E731
    t = dict(x=f32(ROWS, WIDTH), delta=f32(ROWS, WIDTH), out=f32(ROWS, WIDTH), g=f32(K), codes=Tensor("int8", ROWS, 80),
             scale=f32(ROWS), packed=Tensor("uint8", 8076), y=f32(ROWS, WIDTH), ws=Tensor("uint8", 64),
             err=Tensor("int32", 1))
    t.update(kw)
    return t


CALLS = {
    "rows": lambda B, t: B.llama_q8_rows_quant(0, t["x"], WIDTH, ROWS, K, t["codes"], t["scale"]),
    "norm": lambda B, t: B.llama_q8_norm_quant(0, t["x"], WIDTH, t["delta"], WIDTH, t["out"], WIDTH, t["g"], 1e-5, ROWS,
                                               K, t["codes"], t["scale"]),
    "silu": lambda B, t: B.llama_q8_silu_quant(0, t["x"], t["delta"], WIDTH, ROWS, K, t["codes"], t["scale"]),
    "pack": lambda B, t: B.llama_q8_i8_pack(t["codes"], t["scale"], ROWS, K, t["packed"]),
    "matmul": lambda B, t: B.llama_q8_i8_matmul(t["packed"], K, K, t["codes"], t["scale"], ROWS, 0, t["y"], WIDTH,
                                                t["ws"], 64, t["err"]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_accepts(S, name):
    CALLS[name](S, _tensors())
    assert len(S.stub.calls) == 1


BAD_CODES = [("codes", Tensor("int8", ROWS, 79)), ("codes", Tensor("uint8", ROWS, 80)),
             ("codes", Tensor("int8", ROWS, 80, row_stride=96)), ("scale", Tensor("float32", ROWS - 1)),
             ("scale", Tensor("float16", ROWS))]
BAD_X = [("x", Tensor("float16", ROWS, WIDTH)), ("x", Tensor("float32", ROWS * WIDTH - 21)),
         ("x", Tensor("float32", ROWS, K, row_stride=WIDTH + 1)), ("x", Tensor("float32", ROWS, K - 1, row_stride=WIDTH)),
         ("x", Tensor("float32", ROWS - 1, K, row_stride=WIDTH))]


@pytest.mark.parametrize("name,key,bad", [("rows", *b) for b in BAD_X + BAD_CODES] + [
    ("norm", *b) for b in BAD_X + BAD_CODES] + [("silu", *b) for b in BAD_X + BAD_CODES] + [
    ("norm", "delta", Tensor("float32", ROWS, WIDTH - 10)), ("norm", "out", Tensor("bfloat16", ROWS, WIDTH)),
    ("norm", "g", Tensor("float32", K - 1)), ("silu", "delta", Tensor("float32", ROWS, WIDTH - 10)),
    ("pack", "codes", Tensor("int8", ROWS, 79)), ("pack", "packed", Tensor("uint8", 2691)),
    ("matmul", "y", Tensor("float32", ROWS, WIDTH - 10)), ("matmul", "y", Tensor("float16", ROWS, WIDTH)),
    ("matmul", "codes", Tensor("int8", ROWS, 79)), ("matmul", "packed", Tensor("uint8", 8075)),
    ("matmul", "scale", Tensor("float32", ROWS - 1)), ("matmul", "err", Tensor("float32", 1))])
def test_binding_refuses(S, name, key, bad):
    with pytest.raises((TypeError, ValueError)):
        CALLS[name](S, _tensors(**{key: bad}))
    assert not S.stub.calls


def test_binding_refuses_short_blocks(S):
    blocks = Tensor("uint8", 3, 68)  # 64 values a row
    S.llama_q8_rows_quant(8, blocks, 64, 3, 64, Tensor("int8", 3, 64), Tensor("float32", 3))
    with pytest.raises(ValueError):
        S.llama_q8_rows_quant(8, blocks, 64, 4, 64, Tensor("int8", 4, 64), Tensor("float32", 4))
    assert len(S.stub.calls) == 1


# ---- the oracle

def test_oracle_hand_row():
    x = np.array([[-254.0, 1.0, -1.0, 0.99999, 2.0, 3.0, 0.0, 127.0, 253.0, -252.99]], np.float64)
    codes, scale = I.rows_quant(x)
    # halves: 1/2, 3/2 (3 of 254), 127/2, 253/2 go away from zero
    assert codes[0].tolist() == [-127, 1, -1, 0, 1, 2, 0, 64, 127, -126] + [0] * 6
    assert scale[0] == 2.0


def test_oracle_codes_are_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 50))
    codes, scale = I.rows_quant(x)
    unit = np.abs(x).max(1, keepdims=True) / 127
    assert (np.abs(codes[:, :50] * unit - x) <= unit / 2 * (1 + 1e-12)).all()
    assert (np.abs(codes).max(1) == 127).all()


def test_oracle_product_ties_are_rational():
    # 3 * (1 / 3 in f64) is not 1: the product of the factors decides, not its f64 rounding
    third = 1.0 / 3.0
    assert Fraction(third) * 3 < 1
    f, g = np.array([[254.0, 3.0]]), np.array([[1.0, third]])
    assert I.quantise(f, g)[0][0, :2].tolist() == [127, 0]
    assert I.quantise(f, np.array([[1.0, np.nextafter(third, 1)]]))[0][0, :2].tolist() == [127, 1]


def test_oracle_norm_codes_do_not_depend_on_the_row_factor():
    rng = np.random.default_rng(2)
    h, g = rng.standard_normal((3, 40)), rng.standard_normal(40)
    a, s = I.norm_quant(h, g, 1e-5)
    b, t = I.norm_quant(h * 8.0, g, 64e-5)
    assert (a == b).all() and np.allclose(s, t, rtol=1e-12)


def test_oracle_odd_rows():
    nan, inf = np.nan, np.inf
    codes, scale = I.rows_quant(np.array([[0.0, 0.0], [1.0, nan], [inf, 1.0]]))
    assert (codes == 0).all() and scale[0] == 0 and np.isnan(scale[1:]).all()
