"""Paged-cache operators on the GPU against their definitions in f64: rotary
append, paged attention, forking and compacting pages, beam selection, and a
decode loop of all of them."""
import numpy as np
import pytest

from oracle import paged_oracle as P
from tests.gpu_helpers import binding, require_gpu, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # f32 unit roundoff
STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step of a type, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dt(kind):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(t):
    return t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def pool(layers, pages, kv, page, dim, kind, seed, fill=None):
    """K and V pages; fill: what stands in every slot (a test writes the ones it uses)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pages, kv, page, dim)
    if fill is not None:
        return [torch.full(shape, fill, dtype=_dt(kind), device="cuda") for _ in range(2)]
    return [torch.randn(shape, generator=g, device="cuda").to(_dt(kind)) for _ in range(2)]


def zeros(n):
    return torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ rotary append

ROPE = [  # rows, heads, kv, dim, rot, style, page, kind, far, pad
    (1, 9, 3, 64, 64, 0, 16, "f32", 0, False), (4, 9, 3, 64, 64, 1, 16, "f16", 330, False),
    (37, 32, 8, 128, 128, 0, 64, "bf16", 1000, True), (5, 32, 8, 128, 64, 1, 8, "f16", 100000, True),
    (3, 5, 5, 64, 8, 0, 256, "f32", 1 << 20, False), (2, 7, 1, 128, 24, 1, 32, "bf16", 77, False),
    (3, 71, 71, 64, 40, 1, 16, "f32", 12345, False), (129, 8, 1, 64, 32, 0, 8, "f16", 3, True),
    (5003, 9, 3, 64, 64, 0, 16, "f32", 40, True), (6001, 4, 1, 128, 96, 1, 32, "bf16", 9, True)]


@pytest.mark.parametrize("rows,heads,kv,dim,rot,style,page,kind,far,pad", ROPE)
def test_rope_append(rows, heads, kv, dim, rot, style, page, kind, far, pad):
    B = binding()
    rng = np.random.default_rng(rows * 131 + dim + rot)
    n_seq = 3
    seq = rng.integers(0, n_seq, rows)
    pos = np.empty(rows, int)
    for s in range(n_seq):
        at = np.flatnonzero(seq == s)
        pos[at] = far + rng.permutation(len(at))
    if pad:
        pos[::5] = -1
    width = (far + rows) // page + 1
    lo = far // page
    used = width - lo
    table = np.full((n_seq, width), -1)
    table[:, lo:] = rng.permutation(n_seq * used + 2)[:n_seq * used].reshape(n_seq, used)
    stride = (heads + 2 * kv) * dim + 12
    qkv = torch.randn((rows, stride), device="cuda")
    k, v = pool(2, n_seq * used + 2, kv, page, dim, kind, 1)
    k0, v0 = k.clone(), v.clone()
    freq, mag = B.llama_q8_rope_frequencies(rot, 10000.0, B.LQ8_ROPE_RAMP_M, 4.0, 4096, 1.0, 32.0)
    q_out = torch.full((rows, heads, dim), 7.0, device="cuda")
    err = i32([0])
    rope = B.make_rope(torch.from_numpy(freq).cuda(), style, mag)
    rows_of = qkv[:, :(heads + 2 * kv) * dim]   # a view whose rows lie `stride` apart
    B.llama_q8_rope_append(B.make_pages(k, v), 1, rows_of, stride, rows, i32(pos), i32(seq), heads, rope,
                           i32(table), n_seq, width, q_out, err)
    torch.cuda.synchronize()
    assert int(err[0]) == 0
    x = host(qkv)[:, :(heads + 2 * kv) * dim].reshape(rows, -1, dim)
    want = x.copy()
    want[:, :heads + kv] = P.rope(x[:, :heads + kv], pos, freq, style, mag)
    # |error| of a rotated value: the fraction of a turn is rounded to f32 (2^-26 turns: 2^-23.3 in the angle), cos and
    # sin are within one step (2^-23), the products and their sum round three times, the factor once: below 2^-21
    # (|x| + |y|) mag; then half a step of the cache's type (f16: at least half its smallest step, 2^-25)
    pair = np.zeros_like(x)
    h = rot // 2
    a = np.abs(x[:, :heads + kv])
    if style == 0:
        pair[:, :heads + kv, 0:rot:2] = pair[:, :heads + kv, 1:rot:2] = a[..., 0:rot:2] + a[..., 1:rot:2]
    else:
        pair[:, :heads + kv, :h] = pair[:, :heads + kv, h:rot] = a[..., :h] + a[..., h:rot]
    tol = 2.0 ** -21 * mag * pair
    live = pos >= 0
    got = host(q_out)
    assert (np.abs(got - want[:, :heads])[live] <= tol[:, :heads][live]).all()
    assert (got[~live] == 7.0).all()
    kk, vv = host(k0), host(v0)
    kt = np.zeros_like(kk)
    for r in np.flatnonzero(live):
        p, s = table[seq[r], pos[r] // page], pos[r] % page
        kk[1, p, :, s], vv[1, p, :, s] = want[r, heads:heads + kv], x[r, heads + kv:]
        kt[1, p, :, s] = tol[r, heads:heads + kv] + STEP[kind] * (np.abs(want[r, heads:heads + kv]) +
                                                                  tol[r, heads:heads + kv]) + 2.0 ** -25
    if kind == "f32":
        kt[kt > 0] -= 2.0 ** -25  # f32 pages take the rotated value as it is
    assert (np.abs(host(k) - kk) <= kt).all()
    np.testing.assert_array_equal(host(v), host(torch.from_numpy(vv).to(_dt(kind))))


def test_rope_append_reports_and_skips_what_is_out_of_range():
    B = binding()
    k, v = pool(1, 4, 1, 8, 64, "f32", 2)
    k0 = k.clone()
    qkv = torch.randn((1, 3 * 64), device="cuda")
    rope = B.make_rope(torch.from_numpy(B.llama_q8_rope_frequencies(64, 1e4)[0]).cuda())
    table = i32([[0, -1, 4, 1 << 30]])
    for pos, seq, status in [(8, 0, B.LQ8_ERR_ARG), (16, 0, B.LQ8_ERR_ARG), (24, 0, B.LQ8_ERR_ARG),
                             (32, 0, B.LQ8_ERR_CTX), (2 ** 31 - 1, 0, B.LQ8_ERR_CTX), (0, 1, B.LQ8_ERR_ARG),
                             (0, -1, B.LQ8_ERR_ARG)]:
        err, q = i32([0]), torch.zeros((1, 1, 64), device="cuda")
        B.llama_q8_rope_append(B.make_pages(k, v), 0, qkv, 192, 1, i32([pos]), i32([seq]), 1, rope, table, 1, 4, q, err)
        assert int(err[0]) == status, (pos, seq)
        assert torch.equal(k, k0)
        np.testing.assert_allclose(host(q)[0], P.rope(host(qkv)[:, :64].reshape(1, 1, 64), [pos], 1e4 ** (
            -np.arange(32) / 32), 0)[0], atol=2.0 ** -20 * 8)
        B.llama_q8_rope_append(B.make_pages(k, v), 0, qkv, 192, 1, i32([pos]), i32([seq]), 1, rope, table, 1, 4, q)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ attention

ATTN = [  # lens, heads, kv, dim, page, kind, window
    ([1], 9, 3, 64, 16, "f32", 0), ([1], 32, 8, 128, 8, "bf16", 0), ([0], 8, 1, 64, 16, "f16", 0),
    ([331], 9, 3, 64, 16, "f32", 0), ([0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129], 6, 3, 64, 16, "f16", 0),
    ([5, 0, 300, 0, 1, 0], 32, 8, 128, 64, "bf16", 0), ([1000, 77, 513], 8, 8, 128, 32, "f16", 0),
    ([1000, 77, 513], 7, 1, 128, 256, "bf16", 0), ([700, 31, 33], 5, 5, 64, 8, "bf16", 0),
    ([900, 12, 3], 16, 2, 128, 8, "f32", 0), ([640, 100, 9], 32, 8, 128, 16, "f32", 100),
    ([640, 100, 9], 14, 2, 64, 16, "bf16", 33), ([640, 100, 0, 9], 12, 4, 128, 64, "f16", 1),
    ([70000], 7, 1, 128, 16, "bf16", 0), ([40000, 30000], 3, 1, 64, 8, "f16", 0), ([50000, 5], 8, 1, 64, 32, "f32", 0),
    ([33] * 40, 8, 8, 64, 8, "bf16", 0), ([40, 0, 9] * 30, 32, 8, 128, 8, "f16", 0), ([31, 260] * 30, 16, 8, 64, 16, "f16", 20),
    ([5000], 2, 1, 64, 64, "f16", 0), ([4097], 9, 3, 64, 32, "f32", 4096), ([3, 9000], 4, 1, 128, 128, "bf16", 0)]


def attention_tolerance(kind, dim, mag, reach, count, v_mag=1.0):
    """|out error| / sum p |v|. Scores: dim products and sums in f32, and for 16-bit pages q kept to 22 bits or more:
    ds = (dim + 8) 2^-24 + 2^-22, times the largest scale sum |q k|. Each weight then is off by 2 ds (its own and the
    sum's), by 2^-19 for the exponential of a rounded argument and for joining, by the rounding of the probabilities
    (16-bit pages, in parts: 2^-21), and the sums run over `count` terms in f32."""
    ds = ((dim + 8) * U + 2.0 ** -22) * reach
    p = 0.0 if kind == "f32" else 2.0 ** -21
    return 2 * ds + 2.0 ** -19 + p + count[:, None] * U


def run_attention(B, k, v, q, pos, table, window=0, seq=None, scale=0.0, layer=0, lse=True, stream=0, ws=None):
    rows, heads, dim = q.shape
    n = B.llama_q8_attention_paged_workspace_bytes(rows, heads, k.shape[2], dim)
    ws = zeros(n) if ws is None else ws
    out = torch.full((rows + 1, heads, dim), 5.0, device="cuda")
    ls = torch.full((rows + 1, heads), 5.0, device="cuda")
    err = i32([0])
    B.llama_q8_attention_paged(B.make_pages(k, v), layer, q, rows, i32(pos), None if seq is None else i32(seq), heads,
                               scale, window, i32(table), len(table), np.shape(table)[1], out, ls if lse else None,
                               ws, n, err, stream)
    torch.cuda.synchronize()
    assert (out[rows] == 5.0).all() and (ls[rows] == 5.0).all()  # rows behind the last one are left alone
    return out[:rows], ls[:rows], int(err[0])


def check_attention(B, kind, k, v, q, pos, table, window=0, seq=None, scale=0.0, layer=0, status=0):
    out, lse, err = run_attention(B, k, v, q, pos, table, window, seq, scale, layer)
    assert err == status
    dim = q.shape[2]
    want, wl, mag, reach, count = P.attention(host(q), host(k[layer]), host(v[layer]), pos, seq, np.asarray(table),
                                              scale or dim ** -0.5, window)
    tol = attention_tolerance(kind, dim, mag, reach, count)
    bad = ~(np.abs(host(out) - want) <= tol[..., None] * mag)
    worst = np.nanmax(np.abs(host(out) - want) / np.maximum(tol[..., None] * mag, 1e-300))
    assert not bad.any(), (bad.sum(), worst)
    empty = ~np.isfinite(wl)
    assert (host(lse)[empty] == -np.inf).all() and (host(out)[empty] == 0).all()
    assert (np.abs(host(lse) - wl)[~empty] <= (tol + 2.0 ** -22 * np.abs(wl))[~empty]).all()
    return out


def paged_case(lens, heads, kv, dim, page, kind, seed, extra=2):
    """Pages whose unused slots hold NaN and infinities, rows with tables of their own."""
    rng = np.random.default_rng(seed)
    blocks = [-(-n // page) for n in lens]
    total = sum(blocks) + 3
    ids = rng.permutation(total)
    table, at = np.full((len(lens), max(blocks) + extra), -1), 0
    k, v = (pool(1, total, kv, page, dim, kind, seed, fill=f)[0] for f in (float("nan"), float("inf")))
    g = torch.Generator(device="cuda").manual_seed(seed)
    for r, n in enumerate(lens):
        table[r, :blocks[r]] = ids[at:at + blocks[r]]
        at += blocks[r]
        for b in range(blocks[r]):
            m = min(page, n - b * page)
            for x in (k, v):
                x[0, int(table[r, b]), :, :m] = torch.randn((kv, m, dim), generator=g, device="cuda").to(_dt(kind))
    q = 1.5 * torch.randn((len(lens), heads, dim), generator=g, device="cuda")
    return k, v, q, np.array(lens) - 1, table


@pytest.mark.parametrize("lens,heads,kv,dim,page,kind,window", ATTN)
def test_attention_paged(lens, heads, kv, dim, page, kind, window):
    B = binding()
    k, v, q, pos, table = paged_case(lens, heads, kv, dim, page, kind, sum(lens) + heads)
    check_attention(B, kind, k, v, q, pos, table, window)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,kv,dim,heads", [(150, 3, 64, 9), (70, 8, 128, 32), (400, 1, 64, 8)])
def test_attention_paged_many_ragged_rows(kind, rows, kv, dim, heads):
    B = binding()
    rng = np.random.default_rng(rows)
    lens = np.where(rng.random(rows) < 0.2, 0, (300 ** rng.random(rows)).astype(int))
    k, v, q, pos, table = paged_case(list(lens), heads, kv, dim, 16, kind, rows)
    check_attention(B, kind, k, v, q, pos, table)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_attention_paged_rows_of_one_sequence(kind):
    """A prompt's chunk: several tokens of one sequence, each seeing what is before it."""
    B = binding()
    k, v, q, _, table = paged_case([200, 90], 9, 3, 64, 16, kind, 8)
    pos = np.array([i for i in range(180, 200)] + [89, 0, -1])
    seq = np.array([0] * 20 + [1, 1, 0])
    q = 1.5 * torch.randn((len(pos), 9, 64), device="cuda")
    check_attention(B, kind, k, v, q, pos, table, seq=seq, scale=0.3)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_attention_paged_holes_and_bad_pages_are_masked(kind):
    B = binding()
    k, v, q, pos, table = paged_case([200, 64, 40], 8, 2, 64, 16, kind, 9)
    table[0, 3] = -1          # a hole: masked, not an error
    table[1, :] = -7          # nothing left
    check_attention(B, kind, k, v, q, pos, table)
    table[2, 1] = 1 << 30     # out of range: masked and reported
    check_attention(B, kind, k, v, q, pos, table, status=B.LQ8_ERR_ARG)
    for x in (k, v):          # the last page's slots 200 .. 207 become visible
        x[0, int(table[0, 12]), :, 8:] = 0.5
    pos[0] = 2 ** 31 - 1      # past the table: what is inside counts (the entries behind the sequence are holes)
    table[2, 1] = -1
    check_attention(B, kind, k, v, q, pos, table, status=B.LQ8_ERR_CTX)
    check_attention(B, kind, k, v, q, np.array([5, 5, 5]), table, seq=np.array([0, 3, -1]), status=B.LQ8_ERR_ARG)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", [1e-6, 30.0])
def test_attention_paged_flat_and_peaked(kind, size):
    """Nearly uniform weights over many positions, and weights all on a few: scores up to +-1000."""
    B = binding()
    k, v, q, pos, table = paged_case([3000], 8, 1, 128, 64, kind, 10)
    check_attention(B, kind, k, v, (q * size).contiguous(), pos, table)


def test_attention_paged_extreme_queries():
    """Queries whose values span the f32 range and zero queries against 16-bit keys."""
    B = binding()
    for kind in ("f16", "bf16"):
        k, v, q, pos, table = paged_case([50, 50, 50, 50], 4, 2, 64, 16, kind, 11)
        q[0] = 0.0
        q[1] *= 1e-30
        q[2, :, ::2] *= 1e-12
        q[3, :, 0] = 2000.0
        check_attention(B, kind, k, v, q, pos, table)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_attention_paged_equal_calls_give_equal_bits(kind):
    B = binding()
    k, v, q, pos, table = paged_case([2000, 5, 700, 0, 90], 32, 8, 128, 16, kind, 12)
    ws = zeros(B.llama_q8_attention_paged_workspace_bytes(5, 32, 8, 128))
    c = paged_case([60000], 8, 1, 64, 16, kind, 13)   # parts joined in groups
    a = run_attention(B, *c[:3], c[3], c[4], ws=ws)[0]
    for _ in range(3):
        assert torch.equal(a, run_attention(B, *c[:3], c[3], c[4], ws=ws)[0])
    a = run_attention(B, k, v, q, pos, table, ws=ws)[0]
    for _ in range(3):
        assert torch.equal(a, run_attention(B, k, v, q, pos, table, ws=ws)[0])
    assert torch.equal(a, run_attention(B, k, v, q, pos, table, ws=ws, lse=False)[0])


def test_attention_paged_workspace_serves_other_sizes_next():
    """One workspace, calls of different rows and lengths in a row."""
    B = binding()
    ws = zeros(B.llama_q8_attention_paged_workspace_bytes(64, 32, 8, 128))
    for lens, kind in [([900] * 3, "bf16"), ([5], "f32"), (list(range(0, 640, 10)), "f16"), ([900] * 3, "bf16")]:
        k, v, q, pos, table = paged_case(lens, 32, 8, 128, 32, kind, 13)
        out, lse, err = run_attention(B, k, v, q, pos, table, ws=ws)
        want = run_attention(B, k, v, q, pos, table)[0]
        assert torch.equal(out, want) and err == 0


def test_attention_paged_parts_join_by_lse():
    """Attention over the two parts of a cache joined by lse equals attention over all of it."""
    B = binding()
    k, v, q, pos, table = paged_case([500], 9, 3, 64, 16, "f32", 14)
    full, fl, _ = run_attention(B, k, v, q, pos, table)
    a, la, _ = run_attention(B, k, v, q, np.array([255]), table)
    b, lb, _ = run_attention(B, k, v, q, pos, table, window=500 - 256)
    w = torch.exp(la - torch.logaddexp(la, lb))[..., None]
    np.testing.assert_allclose(host(a * w + b * (1 - w)), host(full), atol=1e-5)
    np.testing.assert_allclose(host(torch.logaddexp(la, lb)), host(fl), atol=1e-5)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attention_paged_agrees_with_the_contiguous_kernels(kind):
    """Pages in order are the contiguous cache of llama_q8_attention_decode (f32)."""
    B = binding()
    n, kv, dim, page = 777, 3, 64, 16
    k, v, q, pos, table = paged_case([n], 9, kv, dim, page, kind, 15)
    idx = torch.as_tensor(table[0, :-(-n // page)].astype(np.int64), device="cuda")
    flat = [x[0][idx].float().transpose(0, 1).reshape(kv, -1, dim).contiguous() for x in (k, v)]
    out = torch.empty((9, dim), device="cuda")
    B.llama_q8_attention_decode(q[0].contiguous(), flat[0], flat[1], n, 9, kv, dim, flat[0].shape[1], out)
    got = run_attention(B, k, v, q, pos, table)[0]
    np.testing.assert_allclose(host(got[0]), host(out), atol=4e-5 if kind == "bf16" else 4e-6)


def test_attention_paged_offsets_past_32_bits():
    """A layer far inside a pool whose offsets pass 2^31 elements."""
    B = binding()
    kv, page, dim, pages, layers = 8, 256, 128, 2100, 5    # 5 x 2100 x 8 x 256 x 128: 2.75e9 values
    k, v = (torch.empty((layers, pages, kv, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small_k, small_v, q, pos, table = paged_case([700], 8, kv, dim, page, "bf16", 16)
    far = np.array([pages - 1, 0, pages - 2])
    for b in range(3):
        k[layers - 1, int(far[b])] = small_k[0, int(table[0, b])]
        v[layers - 1, int(far[b])] = small_v[0, int(table[0, b])]
    want = run_attention(B, small_k, small_v, q, pos, table)[0]
    table2 = np.full((1, 4), -1)
    table2[0, :3] = far
    assert torch.equal(run_attention(B, k, v, q, pos, table2, layer=layers - 1)[0], want)


# ------------------------------------------------------------------ pages

def run_fork(B, k, v, lens, table, refs, parent, reserve, rows_out=None, stream=0):
    rows_in, width = np.shape(table)
    rows_out = len(parent)
    n = B.llama_q8_pages_fork_workspace_bytes(rows_in, rows_out, width)
    o_len, o_tab, o_refs = i32([9] * rows_out), i32(np.full((rows_out, width), 9)), i32([9] * len(refs))
    err = i32([0])
    B.llama_q8_pages_fork(B.make_pages(k, v), rows_in, i32(lens), i32(table), width, i32(refs), rows_out, i32(parent),
                          reserve, o_len, o_tab, o_refs, zeros(n), n, err, stream)
    torch.cuda.synchronize()
    return host(o_len), host(o_tab), host(o_refs), int(err[0])


def held(lens, page, n_pages, width, seed, shared=0):
    """Tables of rows of the given lengths; the first `shared` blocks of all rows are the same pages."""
    rng = np.random.default_rng(seed)
    ids = iter(rng.permutation(n_pages))
    common = [next(ids) for _ in range(shared)]
    table, refs = np.full((len(lens), width), -1), np.zeros(n_pages, int)
    for r, n in enumerate(lens):
        for b in range(-(-n // page)):
            table[r, b] = common[b] if b < min(shared, n // page) else next(ids)
    for p in table.ravel():
        if p >= 0:
            refs[p] += 1
    return table, refs


FORK = [  # lens, parents, page, layers, kv, dim, kind, reserve, pages, width, shared
    ([5], [0], 8, 1, 1, 64, "f32", 0, 4, 3, 0), ([5], [0, 0, 0], 8, 3, 2, 64, "bf16", 1, 8, 3, 0),
    ([16, 16], [0, 0, 1, 1], 16, 2, 3, 64, "f32", 1, 12, 4, 0), ([0, 33], [1, 0, 0, 1, 1], 16, 2, 1, 128, "f16", 3, 40, 6, 0),
    ([40, 40, 41, 47], [3, 3, 0, -1, 2, 2, 2], 8, 4, 3, 64, "f32", 20, 60, 12, 4),
    ([100, 90, 80], [-1, -1], 32, 1, 8, 128, "bf16", 1, 30, 8, 2), ([511] * 6, [0, 0, 0, 5, 5, 5], 64, 3, 8, 128, "bf16", 1, 70, 9, 3),
    ([255, 256, 257], [2, 1, 0, 0, 1, 2], 256, 2, 1, 64, "f16", 2, 20, 3, 0)]


@pytest.mark.parametrize("lens,parent,page,layers,kv,dim,kind,reserve,pages,width,shared", FORK)
def test_pages_fork(lens, parent, page, layers, kv, dim, kind, reserve, pages, width, shared):
    B = binding()
    table, refs = held(lens, page, pages, width, 1, shared)
    k, v = pool(layers, pages, kv, page, dim, kind, 2)
    want = P.fork(np.array(lens), table, refs, parent, reserve, page)
    assert not isinstance(want, str)
    wk, wv = k.clone(), v.clone()
    for src, dst, n in want[3]:
        wk[:, dst, :, :n], wv[:, dst, :, :n] = wk[:, src, :, :n].clone(), wv[:, src, :, :n].clone()
    got = run_fork(B, k, v, lens, table, refs, parent, reserve)
    assert got[3] == 0
    for g, w in zip(got[:3], want[:3]):
        np.testing.assert_array_equal(g, w)
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_pages_fork_many_rows_and_a_large_pool():
    """More rows than the plan's threads, a pool of several ranking passes, wide tables."""
    B = binding()
    rng = np.random.default_rng(7)
    rows, page, width, pages = 1500, 8, 300, 150000
    lens = rng.integers(0, 120, rows)
    lens[::100] = 2000
    table, refs = held(lens, page, pages, width, 3)
    parent = rng.integers(-1, rows, 2100)
    k, v = pool(1, pages, 1, page, 64, "f16", 4)
    wk = k.clone()
    want = P.fork(lens, table, refs, parent, 9, page)
    for src, dst, n in want[3]:
        wk[:, dst, :, :n] = wk[:, src, :, :n]
    got = run_fork(B, k, v, lens, table, refs, parent, 9)
    assert got[3] == 0
    for g, w in zip(got[:3], want[:3]):
        np.testing.assert_array_equal(g, w)
    assert torch.equal(k, wk)


def test_pages_fork_pages_held_elsewhere_and_shared_tails():
    """A partly filled page with another holder is copied for every child; reserved pages nobody shares stay with
    the first child; a count the caller holds keeps a page."""
    B = binding()
    page, width = 8, 5
    table = np.array([[0, 1, 2, 3, -1], [0, 1, -1, -1, -1]])   # both end inside page 1; row 0 has two spare pages
    refs = np.array([3, 2, 1, 1, 0, 0, 0, 0, 0, 0])            # page 0: and the caller
    k, v = pool(2, 10, 2, page, 64, "f32", 5)
    lens = [12, 12]
    for parent, reserve in [([0, 0, 1], 1), ([1, 1], 9), ([0], 0), ([-1], 4), ([0, 1], 13)]:
        want = P.fork(np.array(lens), table, refs, parent, reserve, page)
        got = run_fork(B, k, v, lens, table, refs, parent, reserve)
        assert got[3] == 0
        for g, w in zip(got[:3], want[:3]):
            np.testing.assert_array_equal(g, w)
        for src, dst, n in want[3]:
            assert torch.equal(k[:, dst, :, :n], k[:, src, :, :n]) and torch.equal(v[:, dst, :, :n], v[:, src, :, :n])


def test_pages_fork_reports_what_cannot_be_done():
    B = binding()
    page, width = 8, 3
    table, refs = held([12, 9], page, 5, width, 6)
    k, v = pool(1, 5, 1, page, 64, "f32", 7)
    k0 = k.clone()
    lens = np.array([12, 9])
    for parent, reserve, n, status in [([0, 0, 0], 1, lens, "OOM"), ([0, 1], 16, lens, "CTX"), ([2], 0, lens, "ARG"),
                                       ([-2], 0, lens, "ARG"), ([0], 0, np.array([-1, 0]), "CTX"),
                                       ([0], 0, np.array([25, 0]), "CTX"), ([0], 2 ** 31 - 1, lens, "CTX")]:
        assert P.fork(n, table, refs, parent, reserve, page) == status
        got = run_fork(B, k, v, n, table, refs, parent, reserve)
        assert got[3] == {"OOM": B.LQ8_ERR_OOM, "CTX": B.LQ8_ERR_CTX, "ARG": B.LQ8_ERR_ARG}[status]
        assert torch.equal(k, k0)
    bad = table.copy()
    bad[0, 2] = 77  # a page number out of range: a hole, reported
    got = run_fork(B, k, v, lens, bad, refs, [0, -1], 0)
    assert got[3] == B.LQ8_ERR_ARG
    np.testing.assert_array_equal(got[1], P.fork(lens, bad, refs, [0, -1], 0, page)[1])


def run_compact(B, k, v, table, refs):
    rows, width = (0, 0) if table is None else np.shape(table)
    n = B.llama_q8_pages_compact_workspace_bytes(len(refs))
    o_tab, o_refs, used, err = i32(np.full((max(rows, 1), max(width, 1)), 9)), i32([9] * len(refs)), i32([9]), i32([0])
    B.llama_q8_pages_compact(B.make_pages(k, v), rows, None if table is None else i32(table), width, i32(refs),
                             None if table is None else o_tab, o_refs, used, zeros(n), n, err)
    torch.cuda.synchronize()
    return host(o_tab), host(o_refs), int(used[0]), int(err[0])


@pytest.mark.parametrize("pages,share,layers,kv,page,dim,kind", [
    (1, 0.0, 1, 1, 8, 64, "f32"), (1, 1.0, 1, 1, 8, 64, "f32"), (17, 0.5, 3, 3, 16, 64, "f32"),
    (100, 0.3, 2, 8, 64, 128, "bf16"), (64, 1.0, 1, 1, 8, 64, "f16"), (64, 0.0, 1, 1, 8, 64, "f16"),
    (40000, 0.5, 1, 1, 8, 64, "bf16"), (70001, 0.9, 1, 1, 8, 64, "f16"), (33, 0.6, 2, 5, 256, 128, "f32")])
def test_pages_compact(pages, share, layers, kv, page, dim, kind):
    B = binding()
    rng = np.random.default_rng(pages)
    refs = np.where(rng.random(pages) < share, rng.integers(1, 3, pages), 0)
    names = np.repeat(np.arange(pages), refs)
    table = np.full((3, len(names) // 3 + 2), -1)
    table.ravel()[rng.permutation(table.size)[:len(names)]] = rng.permutation(names)
    k, v = pool(layers, pages, kv, page, dim, kind, 8)
    wk, wv = k.clone(), v.clone()
    wt, wr, used, moves = P.compact(table, refs)
    if moves:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        wk[:, dst], wv[:, dst] = wk[:, src], wv[:, src]
    got = run_compact(B, k, v, table, refs)
    np.testing.assert_array_equal(got[0], wt)
    np.testing.assert_array_equal(got[1], wr)
    assert got[2:] == (used, 0)
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_pages_compact_reports_unknown_pages_and_works_without_tables():
    B = binding()
    k, v = pool(1, 4, 1, 8, 64, "f32", 9)
    got = run_compact(B, k, v, np.array([[3, 0, -1, 7]]), np.array([0, 0, 0, 1]))
    np.testing.assert_array_equal(got[0], [[0, -1, -1, -1]])
    assert got[3] == B.LQ8_ERR_ARG and got[2] == 1
    got = run_compact(B, k, v, None, np.array([0, 2, 0, 1]))
    np.testing.assert_array_equal(got[1], [1, 2, 0, 0])
    assert got[3] == 0


# ------------------------------------------------------------------ beams

def run_beam(B, logits, scores, beams, n_out, vocab=None, stride=None, ws=None):
    rows, width = logits.shape
    vocab, stride, groups = vocab or width, stride or width, rows // beams
    n = B.llama_q8_beam_select_workspace_bytes(groups, beams, vocab, n_out)
    s, p, t = torch.full((groups, n_out), 9.0, device="cuda"), i32(np.full((groups, n_out), 9)), i32(np.full((groups, n_out), 9))
    B.llama_q8_beam_select(logits, stride, groups, beams, vocab, scores, n_out, s, p, t, zeros(n) if ws is None else ws, n)
    torch.cuda.synchronize()
    return host(s), host(p), host(t)


def check_beam(B, logits, scores, beams, n_out):
    got = run_beam(B, logits, scores, beams, n_out)
    want = P.beam_select(host(logits), host(scores), beams, n_out)
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[2], want[2])
    # lse: exponentials and chunk sums in f32 (2^-21 relative), joined in f64; one rounding of the result
    fin = np.isfinite(want[0])
    np.testing.assert_array_equal(got[0][~fin], want[0][~fin])
    assert (np.abs(got[0] - want[0])[fin] <= 2.0 ** -20 + U * np.abs(want[0][fin])).all()


@pytest.mark.parametrize("groups,beams,vocab,n_out", [
    (1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 2, 6), (1, 4, 49152, 8), (3, 5, 100003, 10), (7, 1, 2048, 64), (2, 64, 4097, 64),
    (64, 4, 20000, 4), (1, 64, 3, 64), (5, 7, 8191, 33), (2, 2, 255, 64), (70, 8, 9000, 16), (1, 1, 300000, 3)])
def test_beam_select(groups, beams, vocab, n_out):
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(vocab + beams)
    logits = 3.0 * torch.randn((groups * beams, vocab), generator=g, device="cuda")
    scores = -5.0 * torch.rand(groups * beams, generator=g, device="cuda")
    check_beam(B, logits, scores, beams, n_out)


@pytest.mark.parametrize("vocab", [40, 5000, 90000])
def test_beam_select_ties_take_the_lowest_beam_and_token(vocab):
    B = binding()
    for groups in (1, 30):
        logits = torch.zeros((groups * 4, vocab), device="cuda")
        logits[:, 7::11] = -0.0
        scores = torch.zeros(groups * 4, device="cuda")
        check_beam(B, logits, scores, 4, 20)
        logits[1::4, ::3] = 1.0
        check_beam(B, logits, scores, 4, 64)


def test_beam_select_forbidden_inactive_and_broken_rows():
    B = binding()
    inf, nan = float("inf"), float("nan")
    g = torch.Generator(device="cuda").manual_seed(3)
    for vocab in (6, 3000, 70000):
        x = torch.randn((12, vocab), generator=g, device="cuda")
        s = -torch.rand(12, generator=g, device="cuda")
        x[0, 2:] = -inf          # two tokens left
        x[1] = -inf              # nothing left
        x[2, 1] = nan
        x[3, vocab - 1] = inf
        s[4], s[5], s[6] = -inf, nan, inf
        x[7, 1:] = -inf
        x[8], x[9], x[10], s[11] = nan, -inf, inf, -inf    # a group with nothing to choose
        for beams in (1, 2, 4):
            for n_out in (1, 4, min(64, beams * vocab)):
                check_beam(B, x, s, beams, n_out)


def test_beam_select_one_large_value_per_thread_stripe():
    """All of a row's largest values in the values one thread reads (every 256th)."""
    B = binding()
    x = torch.randn((4, 65536), device="cuda")
    x[:, 5::256] += 20.0
    check_beam(B, x, torch.zeros(4, device="cuda"), 2, 64)
    check_beam(B, x.repeat(80, 1), torch.zeros(320, device="cuda"), 4, 64)


@pytest.mark.parametrize("groups,beams", [(2, 2), (300, 2), (700, 1)])
def test_beam_select_sorted_rows(groups, beams):
    """Rising rows, where every block holds larger values than all before it, falling ones, and steps of equal values."""
    B = binding()
    x = torch.arange(100001, device="cuda", dtype=torch.float32)
    for row in (x * 1e-3, -x * 1e-3, torch.floor(x / 3000)):
        check_beam(B, row[None].repeat(groups * beams, 1).contiguous(), torch.zeros(groups * beams, device="cuda"), beams, 7)


@pytest.mark.parametrize("groups,beams,vocab", [(1, 4, 5001), (3, 5, 70001), (40, 6, 30002), (130, 5, 8200), (7, 3, 100000)])
def test_beam_select_equal_rows_tie(groups, beams, vocab):
    """Beams with equal rows and scores have equal totals, wherever in memory their rows lie: the lowest beam first."""
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = 3.0 * torch.randn((groups, 1, vocab), generator=g, device="cuda").expand(groups, beams, vocab)
    check_beam(B, x.reshape(groups * beams, vocab).contiguous(), torch.zeros(groups * beams, device="cuda"), beams, 2 * beams + 1)


@pytest.mark.parametrize("shift", [1e3, -1e4, 3e4, 1e6])
def test_beam_select_logits_far_from_zero(shift):
    """Log sums far larger than the totals: what the f32 number nearest to score - lse leaves out decides."""
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(int(abs(shift)))
    for vocab, rows in ((3001, 8), (40009, 240)):
        x = (4.0 * torch.randn((rows, vocab), generator=g, device="cuda")).round() + shift   # many equal logits
        s = -3.0 * torch.rand(rows, generator=g, device="cuda")
        got = run_beam(B, x, s, 4, 12)
        want = P.beam_select(host(x), host(s), 4, 12)
        np.testing.assert_array_equal(got[1], want[1])
        np.testing.assert_array_equal(got[2], want[2])
        # lse is off by 2^-20 of its own scale at most; one rounding
        assert (np.abs(got[0] - want[0]) <= 2.0 ** -20 + U * np.abs(want[0])).all()


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("vocab,rows", [(1, 4), (3, 4), (6, 4), (4099, 8), (70001, 8), (9001, 640)])
def test_beam_select_unaligned_rows(offset, vocab, rows):
    """Rows that start 0 to 12 bytes behind a 16-byte boundary, the best values and ties at both ends."""
    B = binding()
    g = torch.Generator(device="cuda").manual_seed(vocab)
    big = torch.randn(rows * (vocab + 2) + 8, generator=g, device="cuda")
    x = big[offset:offset + rows * (vocab + 2)].view(rows, vocab + 2)
    x[:, 0], x[:, vocab - 1] = 9.0, 9.0
    x[1::2, min(1, vocab - 1)] = 9.0
    x[:, vocab:] = 1e30   # behind the row: not looked at
    s = torch.zeros(rows, device="cuda")
    n_out = min(5, 4 * vocab)
    got = run_beam(B, x, s, 4, n_out, vocab=vocab, stride=vocab + 2)
    want = P.beam_select(host(x)[:, :vocab], host(s), 4, n_out)
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[2], want[2])


def test_beam_select_strided_rows_and_repeated_calls():
    B = binding()
    x = torch.randn((8, 1003), device="cuda")
    s = -torch.rand(8, device="cuda")
    n = B.llama_q8_beam_select_workspace_bytes(2, 4, 997, 8)
    ws = zeros(n)
    want = P.beam_select(host(x)[:, :997], host(s), 4, 8)
    for _ in range(3):
        got = run_beam(B, x, s, 4, 8, vocab=997, stride=1003, ws=ws)
        np.testing.assert_array_equal(got[1], want[1])
        np.testing.assert_array_equal(got[2], want[2])


# ------------------------------------------------------------------ together

class Loop:
    """Beam search with a small random model of one attention layer: the buffers a program keeps, and one step."""

    def __init__(self, B, groups=2, beams=3, kind="bf16", seed=0):
        self.B, self.groups, self.beams = B, groups, beams
        self.h, self.kv, self.d, self.page, self.width, self.pages_n, self.vocab = 4, 2, 64, 8, 5, 80, 199
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = self.rows = groups * beams
        self.embed = torch.randn((self.vocab, 96), generator=g, device="cuda")
        self.wqkv = torch.randn((96, (self.h + 2 * self.kv) * self.d), generator=g, device="cuda") * 0.1
        self.head = torch.randn((self.h * self.d, self.vocab), generator=g, device="cuda") * 0.15
        self.k, self.v = pool(1, self.pages_n, self.kv, self.page, self.d, kind, seed, fill=float("nan"))
        self.pages = B.make_pages(self.k, self.v)
        self.freq = B.llama_q8_rope_frequencies(self.d, 1e4)[0]
        self.rope = B.make_rope(torch.from_numpy(self.freq).cuda(), 1)
        self.len = [i32([0] * rows), i32([0] * rows)]
        self.table = [i32(np.arange(rows)[:, None].repeat(self.width, 1) * 0 - 1) for _ in range(2)]
        self.refs = [i32([0] * self.pages_n), i32([0] * self.pages_n)]
        self.token = i32([1 + 7 * (r // beams) for r in range(rows)])
        self.scores = torch.full((rows,), float("-inf"), device="cuda")
        self.scores[::beams] = 0.0   # the beams of a group start as one
        self.parent = i32(list(range(rows)))
        self.qkv = torch.empty((rows, (self.h + 2 * self.kv) * self.d), device="cuda")
        self.q = torch.empty((rows, self.h, self.d), device="cuda")
        self.out = torch.empty((rows, self.h * self.d), device="cuda")
        self.logits = torch.empty((rows, self.vocab), device="cuda")
        self.err = i32([0])
        sizes = (B.llama_q8_attention_paged_workspace_bytes(rows, self.h, self.kv, self.d),
                 B.llama_q8_pages_fork_workspace_bytes(rows, rows, self.width),
                 B.llama_q8_beam_select_workspace_bytes(groups, beams, self.vocab, beams))
        self.ws = [(zeros(n), n) for n in sizes]

    def step(self, i, stream=0):
        """Fork to the chosen parents (room for one token), append, attend, choose. i: which buffers are the old ones."""
        B, a, b = self.B, i % 2, 1 - i % 2
        B.llama_q8_pages_fork(self.pages, self.rows, self.len[a], self.table[a], self.width, self.refs[a], self.rows,
                              self.parent, 1, self.len[b], self.table[b], self.refs[b], *self.ws[1], self.err, stream)
        torch.mm(self.embed[self.token.long()], self.wqkv, out=self.qkv)
        B.llama_q8_rope_append(self.pages, 0, self.qkv, self.qkv.shape[1], self.rows, self.len[b], None, self.h,
                               self.rope, self.table[b], self.rows, self.width, self.q, self.err, stream)
        B.llama_q8_attention_paged(self.pages, 0, self.q, self.rows, self.len[b], None, self.h, 0.0, 0, self.table[b],
                                   self.rows, self.width, self.out, None, *self.ws[0], self.err, stream)
        torch.mm(self.out, self.head, out=self.logits)
        B.llama_q8_beam_select(self.logits, self.vocab, self.groups, self.beams, self.vocab, self.scores, self.beams,
                               self.scores, self.parent, self.token, *self.ws[2], stream)
        self.len[b] += 1


def _reference_loop(lp, steps):
    """The same search without pages: every beam recomputes its whole sequence in f64."""
    e, w, hd = host(lp.embed), host(lp.wqkv), host(lp.head)
    seqs = [[int(lp.token[r])] for r in range(lp.rows)]
    scores = host(lp.scores)
    rnd = lambda x: host(torch.from_numpy(x).to(lp.k.dtype))  # noqa: E731
    for _ in range(steps):
        logits = np.zeros((lp.rows, lp.vocab))
        for r, s in enumerate(seqs):
            x = (e[s] @ w).reshape(len(s), -1, lp.d)
            qk = P.rope(x[:, :lp.h + lp.kv], np.arange(len(s)), lp.freq, 1)
            kk, vv = rnd(qk[:, lp.h:])[None].transpose(0, 2, 1, 3), rnd(x[:, lp.h + lp.kv:])[None].transpose(0, 2, 1, 3)
            o = P.attention(qk[-1:, :lp.h], kk, vv, [len(s) - 1], [0], np.array([[0]]), lp.d ** -0.5)[0]
            logits[r] = o.reshape(-1) @ hd
        scores, parent, token = P.beam_select(logits, scores, lp.beams, lp.beams)
        scores, parent, token = scores.ravel(), parent.ravel(), token.ravel()
        seqs = [seqs[p] + [int(t)] for p, t in zip(parent, token)]
    return seqs, scores


def _sequences(first, history):
    seqs = [[t] for t in first]
    for parent, token in history:
        seqs = [seqs[p] + [int(t)] for p, t in zip(parent, token)]
    return seqs


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("groups,beams", [(1, 1), (2, 3), (1, 5)])
def test_beam_search_over_pages(kind, groups, beams):
    B = binding()
    torch.backends.cuda.matmul.allow_tf32 = False
    lp = Loop(B, groups, beams, kind, seed=groups * 10 + beams)
    first = host(lp.token)
    steps, history = 22, []
    want, ws = _reference_loop(lp, steps)
    for i in range(steps):
        lp.step(i)
        history.append((host(lp.parent), host(lp.token)))
    assert int(lp.err[0]) == 0
    got = _sequences(first, history)
    assert got == want
    np.testing.assert_allclose(host(lp.scores), ws, atol=2e-2 if kind == "bf16" else 1e-3)
    # every page's count is the number of entries that name it; compaction keeps what is read
    cur = steps % 2
    table, refs = host(lp.table[cur]), host(lp.refs[cur])
    np.testing.assert_array_equal(np.bincount(table[table >= 0], minlength=lp.pages_n), refs)
    before, _, _ = run_attention(B, lp.k, lp.v, lp.q, host(lp.len[cur]) - 1, table)
    t2, r2, used, err = run_compact(B, lp.k, lp.v, table, refs)
    assert err == 0 and used == (refs > 0).sum()
    after, _, _ = run_attention(B, lp.k, lp.v, lp.q, host(lp.len[cur]) - 1, t2)
    assert torch.equal(before, after)


def test_beam_search_captured_in_a_graph():
    """Two steps (the buffers swap) captured once and replayed give what the eager loop gives."""
    B = binding()
    eager, lp = Loop(B, 2, 3, "f16", 5), Loop(B, 2, 3, "f16", 5)
    hist = []
    for i in range(12):
        eager.step(i)
        hist.append((host(eager.parent), host(eager.token)))
    side = torch.cuda.Stream()
    saved = [t.clone() for t in (lp.scores, lp.parent, lp.token, *lp.len, *lp.table, *lp.refs)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # warm-up outside the capture
        lp.step(0, side.cuda_stream)
        lp.step(1, side.cuda_stream)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st = torch.cuda.current_stream().cuda_stream
        lp.step(0, st)
        lp.step(1, st)
    for t, s in zip((lp.scores, lp.parent, lp.token, *lp.len, *lp.table, *lp.refs), saved):
        t.copy_(s)
    lp.k.fill_(float("nan"))
    lp.v.fill_(float("nan"))
    for i in range(6):
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(host(lp.parent), hist[2 * i + 1][0])
        np.testing.assert_array_equal(host(lp.token), hist[2 * i + 1][1])
    assert torch.equal(lp.scores, eager.scores) and torch.equal(lp.table[0], eager.table[0])
    assert int(lp.err[0]) == 0


def test_one_workspace_for_all_operators_in_turn():
    """Calls of every operator and of other sizes leave the counters of the next call alone."""
    B = binding()
    attn = [paged_case([900] * 3, 32, 8, 128, 32, "bf16", 31), paged_case([4000], 7, 1, 128, 8, "f32", 32)]
    want = [run_attention(B, *c[:3], c[3], c[4])[0] for c in attn]
    ws = zeros(64 << 20)
    table, refs = held([40, 41], 8, 40, 8, 1)
    for groups, beams in [(1, 2), (300, 4), (5, 64), (9000, 1)]:
        x = torch.randn((groups * beams, 500), device="cuda")
        s = torch.zeros(groups * beams, device="cuda")
        first = run_beam(B, x, s, beams, 5)
        for c, w in zip(attn, want):
            assert torch.equal(run_attention(B, *c[:3], c[3], c[4], ws=ws)[0], w)
            got = run_beam(B, x, s, beams, 5, ws=ws)
            for a, b in zip(first, got):
                np.testing.assert_array_equal(a, b)
            k, v = pool(1, 40, 1, 8, 64, "f32", 1)
            out = [i32([0] * 3), i32(np.zeros((3, 8))), i32([0] * 40), i32([0])]
            B.llama_q8_pages_fork(B.make_pages(k, v), 2, i32([40, 41]), i32(table), 8, i32(refs), 3, i32([0, 1, 1]), 1,
                                  out[0], out[1], out[2], ws, ws.numel(), out[3])
            wl, wt, wr, _ = P.fork(np.array([40, 41]), table, refs, [0, 1, 1], 1, 8)
            np.testing.assert_array_equal(host(out[1]), wt)
            np.testing.assert_array_equal(host(out[2]), wr)
            used = i32([0])
            B.llama_q8_pages_compact(B.make_pages(k, v), 3, out[1], 8, out[2], i32(np.zeros((3, 8))), i32([0] * 40),
                                     used, ws, ws.numel(), out[3])
            assert int(used[0]) == (wr > 0).sum() and int(out[3][0]) == 0


def test_calls_on_two_streams_with_their_own_workspaces():
    B = binding()
    cases = [paged_case([1500, 3, 800], 32, 8, 128, 16, "bf16", 21), paged_case([40, 2500], 9, 3, 64, 32, "f32", 22)]
    want = [run_attention(B, *c[:3], c[3], c[4])[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    held_, outs = [], []
    for c in cases:
        k, v, q, pos, table = c
        n = B.llama_q8_attention_paged_workspace_bytes(q.shape[0], q.shape[1], k.shape[2], q.shape[2])
        held_.append((i32(pos), i32(table), zeros(n), n, torch.empty_like(q), B.make_pages(k, v)))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, hd, s in zip(cases, held_, streams):
            q, (pos, table, ws, n, out, pages) = c[2], hd
            B.llama_q8_attention_paged(pages, 0, q, q.shape[0], pos, None, q.shape[1], 0.0, 0, table, table.shape[0],
                                       table.shape[1], out, None, ws, n, None, s.cuda_stream)
    torch.cuda.synchronize()
    for hd, w in zip(held_, want):
        assert torch.equal(hd[4], w)


def test_binding_refuses_other_types_and_layouts():
    B = binding()
    k, v, q, pos, table = paged_case([20], 9, 3, 64, 16, "f32", 23)
    args = lambda **kw: dict(dict(q=q, pos=i32(pos), table=i32(table)), **kw)  # noqa: E731

    def call(a):
        B.llama_q8_attention_paged(B.make_pages(k, v), 0, a["q"], 1, a["pos"], None, 9, 0.0, 0, a["table"], 1,
                                   table.shape[1], torch.empty_like(q), None, zeros(1 << 20), 1 << 20)
    with pytest.raises(TypeError):
        call(args(pos=torch.zeros(1, dtype=torch.int64, device="cuda")))
    with pytest.raises(TypeError):
        call(args(q=q.half()))
    with pytest.raises(ValueError):
        call(args(q=q.transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(ValueError):
        call(args(table=torch.zeros((1, table.shape[1]), dtype=torch.int32)))   # on the host
    with pytest.raises(TypeError):
        call(args(q=q.cpu().numpy()))
    with pytest.raises(TypeError):
        B.make_pages(k.double(), v.double())
    with pytest.raises(ValueError):
        B.make_pages(k, v[:, :1])
    torch.cuda.synchronize()
