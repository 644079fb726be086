"""Paged attention and beam selection where their arithmetic can go wrong:
scores far from zero, long sums, parts that are joined, parts of split numbers.
What is checked has a closed form, so that the bounds are a few roundings."""
import numpy as np
import pytest

from tests import test_gpu_paged
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


# lens, heads, kv, dim, page, window, share of holes among the pages, rows of one sequence
JOINED = [([131071], 7, 1, 128, 16, 0, 0.0, False), ([131071], 8, 1, 64, 64, 0, 0.1, False),
          ([70000, 1, 40000], 3, 1, 64, 8, 0, 0.0, False), ([50000, 50000], 9, 3, 64, 32, 20001, 0.0, False),
          ([30000, 0, 63, 64, 65, 29999], 32, 8, 128, 256, 0, 0.2, False), ([9000] * 5, 4, 2, 64, 16, 0, 0.0, True),
          ([0, 1, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257], 6, 3, 128, 8, 0, 0.0, False),
          ([int(300 ** (i / 400)) for i in range(400)], 8, 8, 64, 16, 0, 0.1, False),
          ([1 + 37 * i % 2500 for i in range(101)], 10, 2, 64, 16, 333, 0.0, True)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,heads,kv,dim,page,window,holes,shared", JOINED)
@pytest.mark.parametrize("steps", [0, 3])
def test_attention_paged_counts_every_position_once(kind, lens, heads, kv, dim, page, window, holes, shared, steps):
    """Values that are 1 in one dimension, drawn per position: the answer counts the positions of each dimension, so one
    that is lost or counted twice shows, wherever it lies among units, pages, warps, CTAs and joined parts. All scores
    0, or (steps) scores that fall and rise by powers of two along the sequence and differ between the heads."""
    B = binding()
    rng = np.random.default_rng(len(lens) * 7 + dim + heads + steps)
    n_seq = 1 if shared else len(lens)
    longest = [max(lens)] if shared else lens
    blocks = [-(-n // page) for n in longest]
    table, at, ids = np.full((n_seq, max(blocks) + 1), -1), 0, rng.permutation(sum(blocks) + 2)
    for r, b in enumerate(blocks):
        table[r, :b] = ids[at:at + b]
        at += b
    where = rng.integers(0, dim, (len(ids), kv, page))      # of a slot: its value's dimension,
    level = rng.integers(0, 3, (len(ids), kv, page))        # its score in units of log2, with the steps below
    for r in range(n_seq):
        for b in range(blocks[r]):
            level[table[r, b]] += 3 * (abs(b * 8 // blocks[r] - 3) % 4)
    v = torch.zeros((len(ids), kv, page, dim), device="cuda", dtype=_dt(kind))
    v.scatter_(3, torch.as_tensor(where, device="cuda")[..., None], 1.0)
    k = torch.zeros_like(v)
    k[..., 5] = torch.as_tensor(level, device="cuda").to(_dt(kind))
    table[rng.random(table.shape) < holes] = -1
    group = heads // kv
    size = np.array([[0.0, 1.0, -1.0, 0.5, 0.25, -0.5, 0.75, 2.0][g % group] for g in range(heads)]) * (steps > 0)
    q = torch.zeros((len(lens), heads, dim), device="cuda")
    q[:, :, 5] = torch.as_tensor(size / LOG2E, device="cuda").float()
    pos, seq = np.array(lens) - 1, [0] * len(lens) if shared else list(range(len(lens)))
    out, lse = (f64(x) for x in attend(B, k, v, q, pos, table.tolist(), window, seq, scale=1.0))
    step = f64(q)[0, :, 5]
    for r, p in enumerate(pos):
        j = np.arange(max(0, p + 1 - window) if window else 0, p + 1)
        pg = table[seq[r], j // page] if len(j) else j
        j, pg = j[pg >= 0], pg[pg >= 0]
        if not len(j):
            assert (out[r] == 0).all() and (lse[r] == -np.inf).all()
            continue
        values, weights = chain_bounds(kind, dim, len(j))
        for h in range(heads):
            s = step[h] * level[pg, h // group, j % page]
            top = s.max()
            w = np.exp(s - top)
            want = np.bincount(where[pg, h // group, j % page], w, dim) / w.sum()
            # scores 0: whole numbers up to 2^17, times 2^15 for f16, which no sum rounds: the reciprocal and the product
            # do. Steps: a weight's exponent of 22 at most rounds four times (log2 e, q times it, the score, less the
            # maximum), f16's parts of q twice, times ln 2: 92; the exponential 4; in the weights and in their sum.
            tol = 2 if steps == 0 else values + weights + 2 * (92 + 4)
            assert (np.abs(out[r, h] - want) <= tol * U * want).all(), (r, h)
            # the logarithm is off by a step at most and rounded
            wl = top + np.log(w.sum())
            tol = 4 * abs(wl) if steps == 0 else 4 * (abs(top) + np.log(w.sum())) + weights + 92 + 4
            assert abs(lse[r, h] - wl) <= tol * U, (r, h)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim", [(4, 64), (8, 64), (3, 128), (7, 128)])
def test_attention_paged_keeps_the_digits_of_probabilities(kind, heads, dim):
    """Two keys: the second's weight c against 1 is c / (1 + c), for weights with all their 24 bits."""
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(heads * dim)
    q = torch.zeros((500, heads, dim), device="cuda")
    q[..., 0] = -0.05 - 0.95 * torch.rand((500, heads), generator=g, device="cuda")
    k = torch.zeros((1, 1, 8, dim), device="cuda", dtype=_dt(kind))
    v = torch.zeros_like(k)
    k[0, 0, 1, 0] = v[0, 0, 1, 1] = v[0, 0, 0, 2] = 1.0
    out, _ = attend(B, k, v, q, [1] * 500, [[0]], seq=[0] * 500, scale=1.0)
    c = np.exp(f64(q)[..., 0])
    # half steps: the exponent (1.45 at most) by log2 e, the product, f16's parts of q (2) and the parts' sum, times ln 2:
    # 5; the exponential 4; f16's parts of the weight 2; the sum, its reciprocal and the product 3
    want = np.stack([c / (1 + c), 1 / (1 + c)], -1)
    assert (np.abs(f64(out)[..., 1:3] - want) <= 14 * U * want).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim", [(4, 64), (8, 64), (3, 128), (7, 128)])
def test_attention_paged_keeps_the_digits_of_queries(kind, heads, dim):
    """Scores 128 (q0 + q1) with q1 the negative of q0 rounded to the digits that the parts of q but the last hold: only
    the last part is left of them."""
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(heads + dim)
    q0 = 1.0 + torch.rand((500, heads), generator=g, device="cuda")
    bits = {"f32": 12, "f16": 11, "bf16": 16}[kind]
    q = torch.zeros((500, heads, dim), device="cuda")
    q[..., 0], q[..., dim // 2 + 1] = q0, -torch.round(q0 * 2.0 ** (bits - 1)) / 2.0 ** (bits - 1)
    k = torch.zeros((1, 1, 8, dim), device="cuda", dtype=_dt(kind))
    v = torch.zeros_like(k)
    k[0, 0, 1, 0] = k[0, 0, 1, dim // 2 + 1] = 128.0
    v[0, 0, 1, 1] = 1.0
    out, _ = attend(B, k, v, q, [1] * 500, [[0]], seq=[0] * 500, scale=1.0)
    s = 128.0 * f64(q).sum(-1)
    # a score's two products of at most 370 (in units of log2): each q rounds as it is multiplied (1), f16 drops 2 of its
    # parts, the sums of up to four products round or cut (2 each) and the sums' sums round (2): 2 (1 + 2) + 10 half steps
    # of 370, times ln 2: 4110; a weight's derivative is 1 / 4 at most
    assert np.abs(f64(out)[..., 1] - 1 / (1 + np.exp(-s))).max() <= (4110 / 4 + 14) * U


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [5, 90, 20000])
def test_attention_paged_nan_query_spoils_its_head_alone(kind, n):
    """NaN in one head's query: that head's out and lse are NaN (not an empty row's), all others as without it."""
    B = binding()
    heads, kv, dim, page = 12, 2, 64, 16
    blocks = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn((blocks, kv, page, dim), generator=g, device="cuda").to(_dt(kind)) for _ in range(2))
    q = torch.randn((3, heads, dim), generator=g, device="cuda")
    args = [n - 1] * 3, [list(range(blocks))]
    want, wl = attend(B, k, v, q, *args, seq=[0] * 3)
    q[1, 7, 3] = float("nan")
    out, lse = attend(B, k, v, q, *args, seq=[0] * 3)
    assert out[1, 7].isnan().all() and lse[1, 7].isnan()
    out[1, 7], lse[1, 7] = want[1, 7], wl[1, 7]
    assert torch.equal(out, want) and torch.equal(lse, wl)


# rows, heads, kv, dim, rot, style, page, kind: the sizes at which narrow rows go eight to a CTA (from 19456 rows of more
# than 64 and at most 128 items of 8 values, twice as many for heads of 128), on both sides of each border
@pytest.mark.parametrize("rows,heads,kv,dim,rot,style,page,kind", [
    (19455, 9, 3, 64, 64, 0, 16, "f32"), (19459, 9, 3, 64, 32, 1, 16, "f16"), (19457, 6, 1, 64, 64, 0, 32, "bf16"),
    (19461, 7, 1, 64, 64, 1, 64, "bf16"), (19463, 14, 1, 64, 64, 0, 16, "bf16"),
    (19470, 15, 1, 64, 48, 0, 16, "f16"), (38911, 3, 1, 128, 96, 1, 64, "f32"),
    (38917, 3, 1, 128, 128, 0, 64, "f16"), (38913, 2, 1, 128, 64, 1, 16, "f32")])
def test_rope_append_long_prompts_of_narrow_rows(rows, heads, kv, dim, rot, style, page, kind):
    test_gpu_paged.test_rope_append(rows, heads, kv, dim, rot, style, page, kind, 50, True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim", [(2, 64), (8, 128), (16, 64)])
@pytest.mark.parametrize("rise", [0.1, 1.0, 10.0])
def test_attention_paged_rising_scores(kind, heads, dim, rise):
    """Scores that rise along 131071 positions of one CTA's share, so that every tile has a new maximum."""
    B = binding()
    n, kv, rows, page = 131071, 2, 256, 64
    blocks = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(heads)
    k = torch.zeros((blocks, kv, page, dim), device="cuda", dtype=_dt(kind))
    left = torch.arange(blocks * page, device="cuda", dtype=torch.float64) / n
    for c in range(3):  # position / n in as many values of the pages' type as hold it
        k[..., c] = left.to(_dt(kind)).view(blocks, 1, page)
        left = left - k[:, 0, :, c].reshape(-1).double()
    v = (1 + torch.randn(k.shape, generator=g, device="cuda")).to(_dt(kind))
    q = torch.zeros((rows, heads, dim), device="cuda")
    q[..., :3] = rise * (1 - 0.1 * torch.rand((rows, heads, 1), generator=g, device="cuda"))
    out, lse = attend(B, k, v, q, [n - 1] * rows, [list(range(blocks))], seq=[0] * rows, scale=1.0)
    values, weights = chain_bounds(kind, dim, n)
    # half steps: a score's log2 e, its product, sums, f16's parts: 8 of it; the exponential 4; changes of the reference,
    # of which each rounds (5) what counts half after the next: 10
    weight = 8 * rise + 4 + 10
    at = k[:, 0, :, :3].double().sum(-1).view(-1)[:n]
    for r in (0, 100, 255):
        s = q[r, :, 0].double()[:, None] * at
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None]).view(kv, heads // kv, n)
        w = v.double().transpose(0, 1).reshape(kv, -1, dim)[:, :n]
        err, size = (out[r].double() - (p @ w).view(heads, dim)).abs(), (p @ w.abs()).view(heads, dim)
        assert (err <= (values + weights + 2 * weight) * U * size).all()
        # and the logarithm of up to 11.8 and the reference, a step and a rounding each
        assert ((lse[r].double() - z).abs() <= (weights + weight + 4 * (12 + 2 * rise)) * U).all()
