"""64-bit CPU restatements of the serving-side operators: page tables and slot maps, the 4-bit
cache's element format, attention over cached rows, and projections with low-rank adapters.
Plain loops over the definitions in the C header; nothing here is shared with the CUDA path."""

from __future__ import annotations

import numpy as np

E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3_VALUES = np.array([(m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
                        for e in range(16) for m in range(8)][:127])  # 0x7f is NaN


# ---- pages ---------------------------------------------------------------------------------

def _pages_for(rows, page_size):
    return -(-rows // page_size)


def pages_extend(table, held, free, count, length, rows, max_rows, page_size, num_pages):
    """Mutates table [b][max_blocks], held [b], free [num_pages]; returns (count, slots per
    sequence, flags) with flags a set of "pool", "rows", "page"."""
    flags, slots, out = set(), [], False
    avail = count if 0 <= count <= num_pages else 0
    if avail != count:
        flags.add("pool")
    taken = 0
    for b in range(len(held)):
        n, ln, h = int(rows[b]), int(length[b]), int(held[b])
        if not 0 <= n <= max_rows or ln < 0 or not 0 <= h <= table.shape[1] or ln + n > table.shape[1] * page_size:
            flags.add("rows")
            slots.append([])
            continue
        need = max(0, _pages_for(ln + n, page_size) - h)
        if need and (out or taken + need > avail):
            out = True
            flags.add("pool")
            slots.append([-1] * n)
            continue
        for j in range(need):
            table[b, h + j] = free[avail - 1 - taken - j]
        taken += need
        held[b] += need
        mine = []
        for i in range(n):
            page = int(table[b, (ln + i) // page_size])
            if not 0 <= page < num_pages:
                flags.add("page")
                mine.append(-1)
            else:
                mine.append(page * page_size + (ln + i) % page_size)
        slots.append(mine)
    return (count - taken if avail == count else count), slots, flags


def pages_trim(table, held, free, count, length, page_size, num_pages):
    """The pages behind ceil(length / page_size) go back; returns (count, flags)."""
    flags, back = set(), []
    for b in range(len(held)):
        ln, h = int(length[b]), int(held[b])
        if ln < 0 or not 0 <= h <= table.shape[1]:
            flags.add("rows")
            back.append([])
            continue
        keep = min(h, _pages_for(ln, page_size))
        back.append([(b, j) for j in range(keep, h)])
    order = [x for s in back for x in s]
    if count < 0 or count + len(order) > num_pages:
        return count, flags | {"pool"}
    real = [(b, j) for b, j in order if 0 <= table[b, j] < num_pages]
    if len(real) < len(order):  # ids that name no page are dropped
        flags.add("page")
    for at, (b, j) in enumerate(real):  # the first one ends up on top of the stack
        free[count + len(real) - 1 - at] = table[b, j]
    for b, j in order:
        table[b, j] = -1
        held[b] -= 1
    return count + len(real), flags


# ---- the 4-bit format -----------------------------------------------------------------------

def _nearest(x, values):
    """Index of the value nearest to each x >= 0; a tie goes to the even index."""
    x = np.minimum(x, values[-1])
    hi = np.searchsorted(values, x, side="left")
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, len(values) - 1)
    dlo, dhi = x - values[lo], values[hi] - x
    return np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)


def kv4_encode(x):
    """(codes uint8 [..., D/2], scales uint8 [..., D/16]) of float64 rows x [..., D]. The quotient
    max|x| / 6 is taken in float32, as the format is defined on it."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    top = np.abs(g).max(-1)
    bad = ~np.isfinite(g).all(-1)
    q = (np.where(bad, 0, top).astype(np.float32) / np.float32(6)).astype(np.float64)
    scale = _nearest(q, E4M3_VALUES)
    s = E4M3_VALUES[scale][..., None]
    y = np.where(s > 0, np.where(bad[..., None], 0, g) / np.where(s > 0, s, 1), 0)
    code = _nearest(np.abs(y), E2M1_VALUES).astype(np.uint8) | ((np.signbit(y) & (s > 0)).astype(np.uint8) << 3)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(bad, 0x7f, scale).astype(np.uint8)


def kv4_decode(codes, scales):
    """Float64 rows of codes [..., D/2] and scales [..., D/16]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = E2M1_VALUES[c & 7] * np.where(c & 8, -1.0, 1.0)
    table = np.concatenate([E4M3_VALUES, [np.nan]])
    s = np.where(scales & 0x80, -1.0, 1.0) * table[scales & 0x7f]
    return v * np.repeat(s, 16, -1)


def kv4_sections(page, head, page_size, dim):
    """(K codes, V codes, K scales, V scales) views of one page's bytes for one KV head."""
    n = page_size * dim * 9 // 8
    blk = page[head * n:(head + 1) * n]
    c, s = page_size * dim // 2, page_size * dim // 16
    return (blk[:c].reshape(page_size, -1), blk[c:2 * c].reshape(page_size, -1),
            blk[2 * c:2 * c + s].reshape(page_size, -1), blk[2 * c + s:].reshape(page_size, -1))


def kv4_row(cache, slot, head, page_size, dim):
    """(key, value) of one head's row at a slot; cache uint8 [pages][bytes]."""
    kc, vc, ks, vs = kv4_sections(cache[slot // page_size], head, page_size, dim)
    o = slot % page_size
    return kv4_decode(kc[o], ks[o]), kv4_decode(vc[o], vs[o])


# ---- attention --------------------------------------------------------------------------------

def attend_rows(q, k, v, first, scale):
    """q [n][Hq][D] at positions first, first + 1, ...; k, v [t][Hkv][D]. Returns (out, absolute
    weighted sum of |v|, largest |logit| terms) per [n][Hq][D] / [n][Hq]."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, mass, terms = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n, hq))
    for i in range(n):
        t = min(max(first + i + 1, 0), k.shape[0])
        if t == 0:
            continue
        for h in range(hq):
            kk, vv = k[:t, h // group], v[:t, h // group]
            x = scale * (kk @ q[i, h])
            w = np.exp(x - x.max())
            w /= w.sum()
            out[i, h] = w @ vv
            mass[i, h] = w @ np.abs(vv)
            terms[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, mass, terms


# ---- projections with adapters ------------------------------------------------------------------

def project_lora(w, x, adapters, a, b, scale):
    """w [L][N][H], x [b][L][rows][H], adapters [b], a [n][L][r][H], b [n][L][N][r], scale [n].
    Returns (y, sum |w x|, sum over the rank of scale |B| sum_k |A x|, magnitudes) [b][L][rows][N]."""
    y = np.einsum("lnh,blih->blin", w, x)
    mag = np.einsum("lnh,blih->blin", np.abs(w), np.abs(x))
    low_mag = np.zeros_like(y)
    for s, ad in enumerate(adapters):
        if ad < 0 or ad >= len(scale):
            continue
        for l in range(w.shape[0]):
            h = x[s, l] @ a[ad, l].T
            y[s, l] += scale[ad] * (h @ b[ad, l].T)
            low_mag[s, l] = abs(scale[ad]) * ((np.abs(x[s, l]) @ np.abs(a[ad, l]).T) @ np.abs(b[ad, l]).T)
    return y, mag, low_mag
