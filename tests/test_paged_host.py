"""Paged-cache operators without a GPU: the refusals of every entry point, the
rotation's frequencies against their formulas, and properties that pin the
oracle's bookkeeping."""
import ctypes as C
import math

import numpy as np
import pytest

from oracle import paged_oracle as P
from tests.gpu_helpers import built_lib

K, V, A, B4, C4, D4, E4, F4, G4, W = (C.c_void_p(i << 20) for i in range(1, 11))  # stand-in addresses


@pytest.fixture(scope="module")
def B():
    built_lib()
    from q8_quantized_llama_gb300 import binding
    binding.lib()
    return binding


def _pool(B, **kw):
    f = dict(k=K, v=V, type=B.GGUF_F32, n_layer=2, n_pages=10, page=16, n_head_kv=3, head_dim=64)
    f.update(kw)
    return B.llama_q8_pages(*(f[n] for n, _ in B.llama_q8_pages._fields_))


BAD_POOLS = [(dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(k=C.c_void_p((1 << 20) + 8)), "ARG"),
             (dict(n_layer=0), "ARG"), (dict(n_pages=0), "ARG"), (dict(n_pages=-4), "ARG"), (dict(n_head_kv=0), "ARG"),
             (dict(type=8), "UNSUPPORTED"), (dict(page=24), "UNSUPPORTED"), (dict(page=4), "UNSUPPORTED"),
             (dict(page=512), "UNSUPPORTED"), (dict(page=0), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED")]


def _status(B, name):
    return {"ARG": B.LQ8_ERR_ARG, "UNSUPPORTED": B.LQ8_ERR_UNSUPPORTED, "OK": B.LQ8_OK}[name]


def _rope_call(B, **kw):
    r = dict(freq=A, rot_dim=64, style=0, magnitude=1.0)
    r.update({k: kw.pop(k) for k in list(kw) if k in r})
    rope = B.llama_q8_rope(r["freq"], r["rot_dim"], r["style"], r["magnitude"])
    f = dict(pages=_pool(B, **kw.pop("pool", {})), layer=0, qkv=B4, stride=15 * 64, rows=4, pos=C4, seq=D4, n_head=9,
             rope=rope, table=E4, n_seq=4, width=8, q_out=F4, err=G4)
    f.update(kw)
    ref = lambda s: None if s is None else C.addressof(s)  # noqa: E731
    return B.lib().llama_q8_rope_append(ref(f["pages"]), f["layer"], f["qkv"], f["stride"], f["rows"], f["pos"],
                                        f["seq"], f["n_head"], ref(f["rope"]), f["table"], f["n_seq"], f["width"],
                                        f["q_out"], f["err"], None)


def _off(p, n):
    return C.c_void_p(p.value + n)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), "ARG"), (dict(layer=2), "ARG"), (dict(layer=-1), "ARG"), (dict(qkv=None), "ARG"),
    (dict(pos=None), "ARG"), (dict(table=None), "ARG"), (dict(q_out=None), "ARG"), (dict(rope=None), "ARG"),
    (dict(freq=None), "ARG"), (dict(rows=-1), "ARG"), (dict(n_head=0), "ARG"), (dict(n_head=10), "ARG"),
    (dict(n_seq=0), "ARG"), (dict(width=0), "ARG"), (dict(stride=14 * 64), "ARG"), (dict(stride=15 * 64 + 2), "ARG"),
    (dict(style=2), "ARG"), (dict(magnitude=math.inf), "ARG"), (dict(magnitude=math.nan), "ARG"),
    (dict(rot_dim=0), "UNSUPPORTED"), (dict(rot_dim=12), "UNSUPPORTED"), (dict(rot_dim=72), "UNSUPPORTED"),
    (dict(seq=None, rows=5), "ARG"), (dict(qkv=_off(B4, 8)), "ARG"), (dict(q_out=_off(F4, 4)), "ARG"),
    (dict(pos=_off(C4, 2)), "ARG"), (dict(freq=_off(A, 4)), "ARG"), (dict(rows=0), "OK")]
    + [(dict(pool=p), s) for p, s in BAD_POOLS])
def test_rope_append_refuses(B, kw, status):
    assert _rope_call(B, **kw) == _status(B, status)


def _attn_call(B, **kw):
    f = dict(pages=_pool(B, **kw.pop("pool", {})), layer=0, q=A, rows=4, pos=B4, seq=C4, n_head=9, scale=0.0, window=0,
             table=D4, n_seq=4, width=8, out=E4, lse=F4, ws=W, ws_bytes=None, err=G4)
    f.update(kw)
    if f["ws_bytes"] is None:
        f["ws_bytes"] = B.llama_q8_attention_paged_workspace_bytes(max(f["rows"], 0), 9, 3, 64)
    return B.lib().llama_q8_attention_paged(None if f["pages"] is None else C.addressof(f["pages"]), f["layer"],
                                            f["q"], f["rows"], f["pos"], f["seq"], f["n_head"], f["scale"],
                                            f["window"], f["table"], f["n_seq"], f["width"], f["out"], f["lse"],
                                            f["ws"], f["ws_bytes"], f["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), "ARG"), (dict(layer=2), "ARG"), (dict(q=None), "ARG"), (dict(pos=None), "ARG"),
    (dict(table=None), "ARG"), (dict(out=None), "ARG"), (dict(ws=None), "ARG"), (dict(ws_bytes=16), "ARG"),
    (dict(rows=-1), "ARG"), (dict(n_head=8), "ARG"), (dict(window=-1), "ARG"), (dict(scale=-1.0), "ARG"),
    (dict(scale=math.nan), "ARG"), (dict(scale=math.inf), "ARG"), (dict(n_head=27), "UNSUPPORTED"),
    (dict(seq=None, rows=5), "ARG"), (dict(q=_off(A, 4)), "ARG"), (dict(out=_off(E4, 8)), "ARG"),
    (dict(ws=_off(W, 4)), "ARG"), (dict(lse=_off(F4, 2)), "ARG"), (dict(rows=(1 << 24)), "UNSUPPORTED"),
    (dict(pool=dict(n_head_kv=64), n_head=64, width=1 << 28), "UNSUPPORTED"),
    (dict(rows=0), "OK")] + [(dict(pool=p), s) for p, s in BAD_POOLS])
def test_attention_paged_refuses(B, kw, status):
    assert _attn_call(B, **kw) == _status(B, status)


def _fork_call(B, **kw):
    f = dict(pages=_pool(B, **kw.pop("pool", {})), rows_in=4, len_in=A, table_in=B4, width=8, refs_in=C4, rows_out=4,
             parent=D4, reserve=1, len_out=E4, table_out=F4, refs_out=G4, ws=W, ws_bytes=None, err=_off(W, 1 << 19))
    f.update(kw)
    if f["ws_bytes"] is None:
        f["ws_bytes"] = 1 << 60
    return B.lib().llama_q8_pages_fork(None if f["pages"] is None else C.addressof(f["pages"]), f["rows_in"],
                                       f["len_in"], f["table_in"], f["width"], f["refs_in"], f["rows_out"],
                                       f["parent"], f["reserve"], f["len_out"], f["table_out"], f["refs_out"],
                                       f["ws"], f["ws_bytes"], f["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), "ARG"), (dict(rows_in=0), "ARG"), (dict(rows_out=0), "ARG"), (dict(width=0), "ARG"),
    (dict(reserve=-1), "ARG"), (dict(len_in=None), "ARG"), (dict(table_in=None), "ARG"), (dict(refs_in=None), "ARG"),
    (dict(parent=None), "ARG"), (dict(len_out=None), "ARG"), (dict(table_out=None), "ARG"),
    (dict(refs_out=None), "ARG"), (dict(ws=None), "ARG"), (dict(err=None), "ARG"), (dict(ws_bytes=100), "ARG"),
    (dict(len_out=A), "ARG"), (dict(table_out=B4), "ARG"), (dict(refs_out=C4), "ARG"),
    (dict(parent=_off(D4, 2)), "ARG"), (dict(ws=_off(W, 8)), "ARG"), (dict(rows_in=65537), "UNSUPPORTED"),
    (dict(rows_out=65537), "UNSUPPORTED"), (dict(rows_out=65536, width=40000), "UNSUPPORTED")]
    + [(dict(pool=p), s) for p, s in BAD_POOLS])
def test_pages_fork_refuses(B, kw, status):
    assert _fork_call(B, **kw) == _status(B, status)


def _compact_call(B, **kw):
    f = dict(pages=_pool(B, **kw.pop("pool", {})), rows=4, table_in=A, width=8, refs_in=B4, table_out=C4, refs_out=D4,
             n_used=E4, ws=W, ws_bytes=1 << 40, err=F4)
    f.update(kw)
    return B.lib().llama_q8_pages_compact(None if f["pages"] is None else C.addressof(f["pages"]), f["rows"],
                                          f["table_in"], f["width"], f["refs_in"], f["table_out"], f["refs_out"],
                                          f["n_used"], f["ws"], f["ws_bytes"], f["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=None), "ARG"), (dict(rows=-1), "ARG"), (dict(width=0), "ARG"), (dict(table_in=None), "ARG"),
    (dict(table_out=None), "ARG"), (dict(refs_in=None), "ARG"), (dict(refs_out=None), "ARG"),
    (dict(n_used=None), "ARG"), (dict(ws=None), "ARG"), (dict(err=None), "ARG"), (dict(ws_bytes=100), "ARG"),
    (dict(table_out=A), "ARG"), (dict(refs_out=B4), "ARG"), (dict(n_used=_off(E4, 1)), "ARG"),
    (dict(ws=_off(W, 4)), "ARG")] + [(dict(pool=p), s) for p, s in BAD_POOLS])
def test_pages_compact_refuses(B, kw, status):
    assert _compact_call(B, **kw) == _status(B, status)


def _beam_call(B, **kw):
    f = dict(logits=A, stride=1000, groups=2, beams=4, vocab=1000, scores=B4, n_out=8, o1=C4, o2=D4, o3=E4, ws=W,
             ws_bytes=None)
    f.update(kw)
    if f["ws_bytes"] is None:
        f["ws_bytes"] = B.llama_q8_beam_select_workspace_bytes(f["groups"], f["beams"], f["vocab"], f["n_out"])
    return B.lib().llama_q8_beam_select(f["logits"], f["stride"], f["groups"], f["beams"], f["vocab"], f["scores"],
                                        f["n_out"], f["o1"], f["o2"], f["o3"], f["ws"], f["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), "ARG"), (dict(scores=None), "ARG"), (dict(o1=None), "ARG"), (dict(o2=None), "ARG"),
    (dict(o3=None), "ARG"), (dict(ws=None), "ARG"), (dict(stride=999), "ARG"), (dict(groups=-1), "ARG"),
    (dict(beams=0), "ARG"), (dict(vocab=0), "ARG"), (dict(n_out=0), "ARG"), (dict(vocab=1, n_out=5), "ARG"),
    (dict(ws_bytes=10), "ARG"), (dict(ws=_off(W, 8)), "ARG"), (dict(logits=_off(A, 2)), "ARG"),
    (dict(beams=65), "UNSUPPORTED"), (dict(n_out=65), "UNSUPPORTED"), (dict(groups=20000), "UNSUPPORTED"),
    (dict(vocab=(1 << 24) + 1, stride=1 << 30), "UNSUPPORTED"),
    (dict(groups=0), "OK")])
def test_beam_select_refuses(B, kw, status):
    assert _beam_call(B, **kw) == _status(B, status)


def test_workspace_queries(B):
    assert B.llama_q8_attention_paged_workspace_bytes(4, 9, 3, 64) > 0
    assert B.llama_q8_attention_paged_workspace_bytes(4, 9, 4, 64) == 0
    assert B.llama_q8_pages_fork_workspace_bytes(0, 4, 8) == 0
    assert B.llama_q8_pages_compact_workspace_bytes(0) == 0
    assert B.llama_q8_pages_compact_workspace_bytes(1) > 0
    assert B.llama_q8_beam_select_workspace_bytes(1, 4, 1000, 8) > 0
    assert B.llama_q8_beam_select_workspace_bytes(1, 65, 1000, 8) == 0


# ------------------------------------------------------------------ frequencies

@pytest.mark.parametrize("dim", [2, 64, 128, 80])
def test_frequencies_plain_and_linear(B, dim):
    want = 10000.0 ** (-2.0 * np.arange(dim // 2) / dim)
    f, m = B.llama_q8_rope_frequencies(dim, 10000.0)
    np.testing.assert_allclose(f, want, rtol=1e-15)
    assert m == 1.0
    f, m = B.llama_q8_rope_frequencies(dim, 10000.0, B.LQ8_ROPE_LINEAR, 8.0)
    np.testing.assert_allclose(f, want / 8, rtol=1e-15)
    assert m == 1.0


def test_frequencies_base_reaches_the_linear_factor_at_the_slowest_pair(B):
    dim, s = 128, 4.0
    f0, _ = B.llama_q8_rope_frequencies(dim, 10000.0)
    f, m = B.llama_q8_rope_frequencies(dim, 10000.0, B.LQ8_ROPE_BASE, s)
    assert f[0] == 1.0 and m == 1.0
    np.testing.assert_allclose(f[-1], f0[-1] / s, rtol=1e-13)   # (theta s^(d/(d-2)))^(-(d-2)/d) = theta^.. / s
    assert np.all(np.diff(np.log(f0 / f)) > 0)


@pytest.mark.parametrize("low,high,ctx,s", [(1.0, 32.0, 4096, 16.0), (1.0, 4.0, 8192, 8.0), (0.0, 1.0, 2048, 1.0)])
def test_frequencies_ramp(B, low, high, ctx, s):
    dim = 128
    f0, _ = B.llama_q8_rope_frequencies(dim, 500000.0)
    turns = ctx * f0 / (2 * np.pi)
    w = np.clip((turns - low) / (high - low), 0, 1)
    for kind, mag in ((B.LQ8_ROPE_RAMP, 1.0), (B.LQ8_ROPE_RAMP_M, 0.1 * math.log(s) + 1)):
        f, m = B.llama_q8_rope_frequencies(dim, 500000.0, kind, s, ctx, low, high)
        np.testing.assert_allclose(f, w * f0 + (1 - w) * f0 / s, rtol=1e-14)
        np.testing.assert_allclose(f[turns >= high], f0[turns >= high], rtol=1e-15)
        np.testing.assert_allclose(f[turns <= low], f0[turns <= low] / s, rtol=1e-15)
        assert abs(m - mag) < 1e-6


@pytest.mark.parametrize("args", [(0, 1e4), (3, 1e4), (64, 0.0), (64, -1.0), (64, math.inf), (64, math.nan),
                                  (64, 1e4, 5, 2.0), (64, 1e4, -1, 2.0), (64, 1e4, 1, 0.5), (64, 1e4, 1, math.nan),
                                  (2, 1e4, 2, 2.0), (64, 1e4, 3, 2.0, 0, 1.0, 4.0), (64, 1e4, 3, 2.0, 4096, 4.0, 4.0),
                                  (64, 1e4, 4, 2.0, 4096, -1.0, 4.0), (64, 1e4, 4, 2.0, 4096, 1.0, math.inf)])
def test_frequencies_refuse(B, args):
    with pytest.raises(B.Q8Error) as e:
        B.llama_q8_rope_frequencies(*args)
    assert e.value.status == B.LQ8_ERR_ARG


def test_frequencies_refuse_null(B):
    sc = B.llama_q8_rope_scaling(0, 0, 1.0, 0.0, 0.0)
    f, m = np.zeros(32), C.c_float()
    g = B.lib().llama_q8_rope_frequencies
    assert g(64, 1e4, None, B.ptr(f), C.addressof(m)) == B.LQ8_ERR_ARG
    assert g(64, 1e4, C.addressof(sc), None, C.addressof(m)) == B.LQ8_ERR_ARG
    assert g(64, 1e4, C.addressof(sc), B.ptr(f), None) == B.LQ8_ERR_ARG


# ------------------------------------------------------------------ the oracle

def _counts(table, n):
    c = np.zeros(n, int)
    for p in np.asarray(table).ravel():
        if p >= 0:
            c[p] += 1
    return c


def test_oracle_fork_keeps_counts_and_contents():
    """Random trees of forks: every page's count stays the number of entries
    that name it, no writable block is shared, and what a child reads at each
    position is what its parent read."""
    rng = np.random.default_rng(3)
    page, width, n_pages, rows = 8, 6, 90, 5
    lens = np.array([13, 8, 1, 0, 21])
    table = np.full((rows, width), -1)
    ids = iter(rng.permutation(n_pages))
    for r, n in enumerate(lens):
        for b in range(-(-n // page)):
            table[r, b] = next(ids)
    refs = _counts(table, n_pages)
    data = rng.integers(0, 1 << 30, (n_pages, page))
    for step in range(20):
        parent = rng.integers(-1, rows, rows)
        if lens.max() + 2 > width * page:
            break
        before = [[data[table[p, j // page], j % page] for j in range(lens[p])] if p >= 0 else [] for p in parent]
        lens, table, refs, copies = P.fork(lens, table, refs, parent, 2, page)
        for src, dst, n in copies:
            data[dst, :n] = data[src, :n]
        np.testing.assert_array_equal(refs, _counts(table, n_pages))
        for i in range(rows):
            assert [data[table[i, j // page], j % page] for j in range(lens[i])] == before[i]
            if parent[i] >= 0:
                for j in (lens[i], lens[i] + 1):
                    assert refs[table[i, j // page]] == 1
                    data[table[i, j // page], j % page] = rng.integers(0, 1 << 30)
                lens[i] += 1


def test_oracle_compact_keeps_contents():
    rng = np.random.default_rng(4)
    refs = np.where(rng.random(40) < 0.4, rng.integers(1, 4, 40), 0)
    table = rng.permutation(np.flatnonzero(refs)).reshape(-1, 1)
    data = rng.integers(0, 1000, 40)
    out, refs2, used, moves = P.compact(table, refs)
    new = data.copy()
    for s, d in moves:
        new[d] = data[s]
    assert used == (refs > 0).sum() and (refs2[:used] > 0).all() and not refs2[used:].any()
    np.testing.assert_array_equal(new[out], data[table])
    np.testing.assert_array_equal(refs2[out], refs[table])


def test_oracle_beam_select_is_the_probability_order():
    rng = np.random.default_rng(5)
    x, s = rng.normal(size=(4, 7)), rng.normal(size=4)
    got, parent, token = P.beam_select(x, s, 2, 5)
    for g in range(2):
        p = np.exp(x[2 * g:2 * g + 2])
        full = np.log(p / p.sum(1, keepdims=True)) + s[2 * g:2 * g + 2, None]
        np.testing.assert_allclose(got[g], np.sort(full.ravel())[::-1][:5])
        np.testing.assert_allclose(full[parent[g] - 2 * g, token[g]], got[g])
