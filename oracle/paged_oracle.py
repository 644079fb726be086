"""Plain definitions of the paged-cache operators in numpy f64 (test
infrastructure: only tests import it). Bookkeeping is written as loops over
rows and blocks, arithmetic as the formula says."""
import numpy as np


def rope(x, pos, freq, style, magnitude=1.0):
    """x[rows][heads][dim] rotated at pos[rows] (rows with pos < 0 unchanged)."""
    x = np.array(x, np.float64)
    half = len(freq)
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)[None, :]
    c, s = magnitude * np.cos(ang)[:, None, :], magnitude * np.sin(ang)[:, None, :]
    y = x.copy()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if style == 0 else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * c - b * s, a * s + b * c
    if style == 0:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ra, rb
    else:
        y[..., :half], y[..., half:2 * half] = ra, rb
    pad = np.asarray(pos) < 0
    y[pad] = x[pad]
    return y


def visible(pos, window, table_row, page, n_pages):
    """Positions a token at pos attends to, with their pages."""
    if pos < 0:
        return []
    lo = max(0, pos - window + 1) if window else 0
    out = []
    for j in range(lo, min(pos + 1, len(table_row) * page)):
        p = int(table_row[j // page])
        if 0 <= p < n_pages:
            out.append((j, p))
    return out


def attention(q, k, v, pos, seq, table, scale, window=0):
    """q[rows][heads][dim] over k, v [pages][kv][page][dim]: out, lse, and what
    the error bounds need: sum p |v| and the largest scale * sum |q k|."""
    rows, heads, dim = q.shape
    n_pages, kv, page = k.shape[:3]
    g = heads // kv
    out, mag = np.zeros((rows, heads, dim)), np.zeros((rows, heads, dim))
    lse, reach = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    count = np.zeros(rows, int)
    for r in range(rows):
        s = r if seq is None else int(seq[r])
        if not 0 <= s < len(table):
            continue
        see = visible(int(pos[r]), window, table[s], page, n_pages)
        count[r] = len(see)
        if not see:
            continue
        pg, sl = np.array([p for _, p in see]), np.array([j % page for j, _ in see])
        for h in range(heads):
            kk, vv = np.float64(k[pg, h // g, sl]), np.float64(v[pg, h // g, sl])
            qq = np.float64(q[r, h])
            sc = scale * (kk @ qq)
            m = sc.max()
            e = np.exp(sc - m)
            p = e / e.sum()
            out[r, h], mag[r, h] = p @ vv, p @ np.abs(vv)
            lse[r, h] = m + np.log(e.sum())
            reach[r, h] = scale * (np.abs(kk) @ np.abs(qq)).max()
    return out, lse, mag, reach, count


def fork(len_in, table_in, refs_in, parent, reserve, page):
    """(len_out, table_out, refs_out, copies [(src, dst, positions)]), or the
    name of the status the call reports."""
    n_pages, width = len(refs_in), table_in.shape[1]
    if any(p < -1 or p >= len(len_in) for p in parent):
        return "ARG"
    refs = [int(x) for x in refs_in]
    free = [i for i in range(n_pages) if refs_in[i] == 0]
    in_row = lambda p, b: int(table_in[p, b]) if 0 <= table_in[p, b] < n_pages else -1  # noqa: E731
    for p in range(len(len_in)):
        for b in range(width):
            if in_row(p, b) >= 0:
                refs[in_row(p, b)] -= 1
    seen, lens, rows, copies, wanted = set(), [], [], [], 0
    for p in map(int, parent):
        row = [-1] * width
        n = 0
        if p >= 0:
            n = int(len_in[p])
            if n < 0 or n + reserve > width * page:
                return "CTX"
            need = -(-(n + reserve) // page)
            for b in range(width):
                old = in_row(p, b)
                if b < n // page or (p not in seen and old >= 0 and refs_in[old] == 1):
                    row[b] = old
                elif b < need:
                    wanted += 1
                    row[b] = free.pop(0) if free else -2
                    if b == n // page and n % page and old >= 0:
                        copies.append((old, row[b], n % page))
            seen.add(p)
        lens.append(n)
        rows.append(row)
    if any(x == -2 for r in rows for x in r):
        return "OOM"
    for r in rows:
        for x in r:
            if x >= 0:
                refs[x] += 1
    return np.array(lens), np.array(rows), np.array(refs), copies


def compact(table_in, refs_in):
    """(table_out, refs_out, used, moves [(src, dst)])."""
    used = sum(int(r) > 0 for r in refs_in)
    holes = [p for p in range(used) if refs_in[p] <= 0]
    to, moves = {}, []
    refs = np.zeros(len(refs_in), np.int64)
    for p, r in enumerate(refs_in):
        if r > 0:
            to[p] = p if p < used else holes.pop(0)
            if to[p] != p:
                moves.append((p, to[p]))
            refs[to[p]] = r
    table = np.array([[to.get(int(p), -1) for p in row] for row in table_in]).reshape(np.shape(table_in))
    return table, refs, used, moves


def beam_select(logits, scores, beams, n_out):
    """(scores, parent, token), each [groups][n_out]."""
    rows, vocab = logits.shape
    total = np.full((rows, vocab), -np.inf)
    for r in range(rows):
        x = logits[r].astype(np.float64)
        top = x.max() if not np.isnan(x).any() else np.nan
        if np.isfinite(scores[r]) and np.isfinite(top):
            total[r] = np.float64(scores[r]) + (x - (top + np.log(np.exp(x - top).sum())))
    out = []
    for g in range(rows // beams):
        t = total[g * beams:(g + 1) * beams].ravel()
        order = np.lexsort((np.arange(t.size), -t))[:n_out]
        out.append((t[order], g * beams + order // vocab, order % vocab))
    return tuple(np.array([o[i] for o in out]) for i in range(3))
