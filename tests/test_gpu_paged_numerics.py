"""Paged attention and beam selection where their arithmetic can go wrong:
scores far from zero, long sums, parts that are joined, parts of split numbers.
What is checked has a closed form, so that the bounds are a few roundings."""
import numpy as np
import pytest

from tests.gpu_helpers import binding, require_gpu, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of f32, relative
LOG2E = 1.4426950408889634
KINDS = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dt(kind):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def attend(B, k, v, q, pos, table, window=0, seq=None, scale=0.0):
    """(out, lse) of rows over the pages k, v [pages][kv][page][dim]."""
    rows, heads, dim = q.shape
    n = B.llama_q8_attention_paged_workspace_bytes(rows, heads, k.shape[1], dim)
    out, lse, err = torch.empty_like(q), torch.empty((rows, heads), device="cuda"), i32([0])
    B.llama_q8_attention_paged(B.make_pages(k[None], v[None]), 0, q, rows, i32(pos), None if seq is None else i32(seq),
                               heads, scale, window, i32(table), len(table), len(table[0]), out, lse,
                               torch.zeros(n, dtype=torch.uint8, device="cuda"), n, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    return out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("m", [2.0 ** 20, 2.0 ** 24 + 64, 2.0 ** 25 + 64, 2.0 ** 27 + 64, 2.0 ** 29, 2.0 ** 100])
def test_attention_paged_scores_far_from_zero(kind, sign, m):
    """One key far above all others, its score (in units of log2) anywhere: its value is the answer."""
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(7)
    for n, heads, kv, dim, page in [(8, 1, 1, 64, 8), (700, 6, 2, 128, 16), (9000, 8, 1, 64, 64)]:
        blocks, best = -(-n // page), n * 2 // 3
        k = torch.zeros((blocks, kv, page, dim), device="cuda", dtype=_dt(kind))
        v = torch.randn(k.shape, generator=g, device="cuda").to(_dt(kind))
        k[..., 0] = 1.0 if sign > 0 else -2.0
        k[best // page, :, best % page, 0] = 2.0 if sign > 0 else -1.0
        q = torch.zeros((1, heads, dim), device="cuda")
        q[0, :, 0] = m / 2 / LOG2E if sign > 0 else m / LOG2E
        out, lse = attend(B, k, v, q, [n - 1], [list(range(blocks))], scale=1.0)
        # the others' probabilities are 2^-(2^19) at most: 0; the one is 1, and no sum rounds
        want = v[best // page, :, best % page].float().repeat_interleave(heads // kv, 0)
        assert torch.equal(out[0], want), (n, heads)
        # lse: log2 e, q times it, ln 2 and the product with it round; f16: the second part of q ends 2^-23 below q,
        # and the two parts' sum rounds
        score = f64(q)[..., 0] * (2.0 if sign > 0 else -1.0)
        assert (np.abs(f64(lse) - score) <= (7 if kind == "f16" else 4) * U * np.abs(score)).all(), (n, heads)


def chain_bounds(kind, dim, n):
    """Relative bounds, in half steps of f32, of the sum of a row's weighted values and of the sum of its weights, for
    n positions that one CTA's four warps take: tiles of 4 KB of keys, 16 (f32) or 32 tiles per partial sum. The i-th of
    N additions of terms of about one size errs by at most half a step of i / N of the sum: N / 2 half steps in all."""
    size = 4 if kind == "f32" else 2
    tile = 4096 // (dim * size)
    fold = 16 if kind == "f32" else 32
    tiles = -(-n // (4 * tile))
    weights = (fold + tiles / fold) / 2
    # f32: a multiply-add per position. 16-bit: four products per tile at most in the tensor cores, which cut what lies
    # below a step of the sum (2 half steps each), and the probabilities to 22 bits (4 half steps)
    values = (fold * tile + tiles / fold) / 2 if kind == "f32" else weights + 4 * 2 + 4
    # a tile's own tree or the parts' sum, the joins of lanes and warps, the factors as the maximum grows
    return values + 32, weights + 32


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim", [(2, 64), (2, 128), (10, 64), (16, 128)])
def test_attention_paged_long_sums(kind, heads, dim):
    """Rows enough that a CTA has whole rows, 131071 positions each, and values that are all 1: the answer is 1. With
    random keys, and with equal keys but one, where every addition to a sum rounds the same way."""
    B = binding()
    n, kv, rows, page = 131071, 2, 256, 64
    blocks = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(heads + dim)
    k = torch.randn((blocks, kv, page, dim), generator=g, device="cuda").to(_dt(kind))
    v = torch.ones_like(k)
    q = 0.5 * torch.randn((rows, heads, dim), generator=g, device="cuda")
    values, weights = chain_bounds(kind, dim, n)
    table, pos, seq = [list(range(blocks))], [n - 1] * rows, [0] * rows
    out, _ = attend(B, k, v, q, pos, table, seq=seq)
    err = f64(out) - 1.0
    assert np.abs(err).max() <= (values + weights) * U
    k.zero_()
    k[0, :, 0] = 1.0
    q = 0.02 * torch.rand((rows, heads, dim), generator=g, device="cuda")
    out, lse = attend(B, k, v, q, pos, table, seq=seq)
    assert np.abs(f64(out) - 1.0).max() <= (values + weights) * U
    s = f64(q).sum(-1) * dim ** -0.5
    # and the score's products and sums, and the logarithm of about 11.8 (a step and its own rounding)
    tol = (weights + (dim + 8) * s + 4 * 12) * U
    assert (np.abs(f64(lse) - np.log(np.exp(s) + n - 1)) <= tol).all()


@pytest.mark.parametrize("vocab", [100003, 1 << 20, (1 << 22) + 5, 1 << 24])
def test_beam_select_long_vocabulary_sums(vocab):
    """Log sums of up to 2^24 logits: rows of two values, whose block sums are all equal, and rising rows, whose maximum
    grows with every block."""
    B = binding()
    i = torch.arange(vocab, device="cuda", dtype=torch.float64)
    rows = [torch.where(i % 2 == 0, -a, 0.0 * i) for a in (0.3, 0.7, 1.1, 1.9, 2.3, 3.1)] + [i * (8.0 / vocab), i * (1.0 / vocab)]
    x = torch.stack([r.float() for r in rows])
    n, g = B.llama_q8_beam_select_workspace_bytes(len(rows), 1, vocab, 1), len(rows)
    s, p, t = torch.empty(g, device="cuda"), i32([0] * g), i32([0] * g)
    B.llama_q8_beam_select(x, vocab, g, 1, vocab, torch.zeros(g, device="cuda"), 1, s, p, t,
                           torch.zeros(n, dtype=torch.uint8, device="cuda"), n)
    y = x.double()
    top = y.max(1).values
    want = f64(-torch.log(torch.exp(y - top[:, None]).sum(1)))  # top - lse
    # In half steps of f32: a block's sum 10 (eight additions of growing sums: 4; the lanes' six), ex2 4 and its argument
    # of 1.9 on average, times ln 2, 3; a block's factor 2 and product 1, the sums of eight 3, the row's none; a change of
    # the reference, for a lane's blocks and for the row, 3 each; the logarithm 2. And the rounding of the total.
    np.testing.assert_allclose(f64(s), want, rtol=U, atol=31 * U)
