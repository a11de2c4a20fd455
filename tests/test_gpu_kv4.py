"""The 4-bit cache (ls_kv4_append, ls_kv4_read_rows, ls_verify_attend_kv4) against the 64-bit
oracle. Rows are compared bit for bit. The attention's bound per output element:

    |gpu - ref| <= e_out |ref| + (2^-10 + 2 e_x + 2 (t + 256) 2^-24) sum_t w_t |v_t| + t 2^-33 max|v|

e_out is the output's rounding (2^-8 in bf16, 2^-24 in fp32). 2^-10: a softmax weight rounded
to 11 bits (2^-11), in the numerator only, against a sum of the weights before rounding, plus
2^-11 for everything of the size of an fp32 rounding (exp2, the divide). e_x: the
error of a logit in natural units, D fp32 additions plus the queries' rounding (to 11 bits at
most, exact but for elements below 2^-14 of their row's largest: 2^-25 of it): bounded by
(D + 8) 2^-24 scale sum_d |q_d k_d| + D 2^-25 scale max|q| max|k|. t 2^-24: fp32 sums of t weights or
weighted values. The last term: weights below fp16's normal range, off by 2^-25 of 2^-8."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fixed_cost_drafter_b200 as F
    import oracle as O
    from tests.serving_side import Cache4, Lib, refused


def _f64(t):
    return t.double().cpu().numpy()


# ---- rows ------------------------------------------------------------------------------------

def _rows(n, heads, dim, stride, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, stride, generator=g, device="cuda") * 10.0 ** torch.randint(-3, 3, (n, 1), generator=g, device="cuda")
    x[::3, 5] *= 40
    if n > 4:
        x[1, :16] = 0
        x[2, 3] = float("inf")
        x[3, 20] = float("nan")
        x[4, :heads * dim] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0.5],
                                          device="cuda").repeat(heads * dim // 16)
        x[0] = x[0] * 0 + 3e38
        x[n - 1] = 1e-30
    return x.to(dtype)


@pytest.mark.parametrize("dtype,dim,heads,ps,n,extra", [
    ("bf16", 128, 8, 16, 37, 0), ("bf16", 128, 2, 256, 300, 64), ("bf16", 64, 3, 32, 1, 8), ("f32", 64, 2, 16, 77, 40),
    ("f32", 128, 1, 128, 9, 0), ("bf16", 128, 8, 64, 3000, 5120)])
def test_rows_written_and_read_back(dtype, dim, heads, ps, n, extra):
    lib = Lib(kv_heads=heads, q_heads=2 * heads, dim=dim, dtype=dtype)
    stride = heads * dim + extra
    k, v = (_rows(n, heads, dim, stride, lib.tdtype, s) for s in (1, 2))
    pages = -(-n // ps) + 2
    rng = np.random.default_rng(n)
    slots = rng.permutation(pages * ps)[:n].astype(np.int64)
    if n > 8:
        slots[7] = -1
    per = F.ls_kv4_page_bytes(lib.cfg, ps)
    cache = torch.full((pages, per + 32), 0xA5, dtype=torch.uint8, device="cuda")
    kv = F.make_paged_kv4([cache], per + 32, None, 1, ps, pages)
    d_slots = torch.from_numpy(slots).cuda()
    F.ls_kv4_append(lib.st, kv, 0, k, v, stride, d_slots, n)
    want = np.full((pages, per + 32), 0xA5, np.uint8)
    got = [torch.full((n, stride), 7.0, dtype=lib.tdtype, device="cuda") for _ in range(2)]
    ref = [np.full((n, stride), 7.0) for _ in range(2)]
    for which, x in enumerate((k, v)):
        c, s = O.kv4_encode(_f64(x)[:, :heads * dim].reshape(n, heads, dim))
        vals = O.kv4_decode(c, s)
        for i in range(n):
            if slots[i] < 0:
                continue
            for h in range(heads):
                sec = O.kv4_sections(want[slots[i] // ps], h, ps, dim)
                sec[which][slots[i] % ps] = c[i, h]
                sec[2 + which][slots[i] % ps] = s[i, h]
            ref[which][i, :heads * dim] = vals[i].reshape(-1)
    have = cache.cpu().numpy()
    # codes of a NaN group mean nothing; everything else is equal byte for byte
    nan_rows = {int(slots[i]) for i in (2, 3) if n > 4}
    for p in range(pages):
        for h in range(heads):
            for x, y in zip(O.kv4_sections(have[p], h, ps, dim), O.kv4_sections(want[p], h, ps, dim)):
                rows = [o for o in range(ps) if p * ps + o not in nan_rows]
                assert np.array_equal(x[rows], y[rows]), (p, h)
    assert np.array_equal(have[:, per:], want[:, per:])
    F.ls_kv4_read_rows(lib.st, kv, 0, d_slots, n, got[0], got[1], stride)
    for a, b in zip(got, ref):
        assert np.array_equal(_f64(a), b, equal_nan=True)
    assert lib.error() == (F.LS_OK, 0)


def test_rows_of_every_pair_of_values():
    """Every bf16 of several binades against every group maximum of one binade: all borders."""
    lib = Lib(kv_heads=1, q_heads=1, dim=64)
    m = torch.arange(0x3f80, 0x4000, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)  # 1 .. 2
    x = torch.arange(0x3c00, 0x4000, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)  # 2^-7 .. 2
    n = m.numel() * x.numel() // 64
    rows = torch.zeros(n * 4, 16, dtype=torch.bfloat16, device="cuda")
    mm = m.repeat_interleave(x.numel() // 15 + 1)[: n * 4]
    rows[:, 0] = mm
    rows[:, 1:] = x.repeat((n * 4 * 15) // x.numel() + 1)[: n * 4 * 15].view(n * 4, 15)
    rows = rows.view(n, 64)
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    pages = -(-n // 64)
    cache = torch.empty(pages, F.ls_kv4_page_bytes(lib.cfg, 64), dtype=torch.uint8, device="cuda")
    kv = F.make_paged_kv4([cache], cache.stride(0), None, 1, 64, pages)
    a, b = torch.empty_like(rows), torch.empty_like(rows)
    F.ls_kv4_append(lib.st, kv, 0, rows, -rows, 64, slots, n)
    F.ls_kv4_read_rows(lib.st, kv, 0, slots, n, a, b, 64)
    ref = O.kv4_decode(*O.kv4_encode(_f64(rows)))
    assert np.array_equal(_f64(a), ref) and np.array_equal(_f64(b), -ref)


def test_slots_outside_the_pool_are_skipped_and_flagged():
    lib = Lib()
    cache = torch.zeros(2, F.ls_kv4_page_bytes(lib.cfg, 16), dtype=torch.uint8, device="cuda")
    kv = F.make_paged_kv4([cache], cache.stride(0), None, 1, 16, 2)
    k = torch.ones(4, 256, dtype=torch.bfloat16, device="cuda")
    for bad in (32, -2, 1 << 40, -(1 << 62)):
        slots = torch.tensor([bad, -1, 3, 31], dtype=torch.int64, device="cuda")
        F.ls_kv4_append(lib.st, kv, 0, k, k, 256, slots, 4)
        assert lib.error()[1] == F.LS_DEVERR_PAGE
        lib.clear()
        out = torch.full((2, 4, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        F.ls_kv4_read_rows(lib.st, kv, 0, slots, 4, out[0], out[1], 256)
        # e4m3(1 / 6) = 11 / 64: ones are held as 6 * 11 / 64
        assert (out[:, :2] == 5).all() and (out[:, 2:] == 1.03125).all()
        assert lib.error()[1] == F.LS_DEVERR_PAGE
        lib.clear()
    F.ls_kv4_append(lib.st, kv, 0, k, k, 256, None, 0)  # no rows: nothing
    assert lib.error() == (F.LS_OK, 0)


# ---- attention -----------------------------------------------------------------------------------

def _tolerance(lib, q, k, v, ref, mass, t, scale, f32_out):
    D = lib.cfg.head_dim
    group = q.shape[1] // k.shape[1]
    kmax = np.abs(k).max(initial=0.0)
    dot = np.zeros(q.shape[:2])
    for h in range(q.shape[1]):
        if k.shape[0]:
            dot[:, h] = (np.abs(q[:, h]) @ np.abs(k[:, h // group]).T).max(-1)
    ex = (D + 8) * 2.0 ** -24 * scale * dot + D * 2.0 ** -25 * scale * np.abs(q).max(-1) * kmax
    e_out = 2.0 ** -24 if f32_out else 2.0 ** -8
    return e_out * np.abs(ref) + (2.0 ** -10 + 2 * ex[..., None] + 2 * (t + 256) * 2.0 ** -24) * mass + \
        t * 2.0 ** -33 * np.abs(v).max(initial=0.0)


def _attend(lib, cache, lengths, n, rows=None, seed=0, scale=None, q_extra=0, q_scale=1.0):
    c = lib.cfg
    b, hq, D = c.batch, c.n_q_heads, c.head_dim
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(b, n, hq * D + q_extra, generator=g, device="cuda") * q_scale).to(lib.tdtype)
    f32 = lib.tdtype == torch.float32 or (c.flags & F.LS_FLAG_OUT_F32)
    out = torch.full((b, n, hq, D), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    ws = torch.full((F.ls_verify_workspace_bytes(c, n),), 0xff, dtype=torch.uint8, device="cuda")
    d_rows = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    scale = scale or D ** -0.5
    args = (lib.st, cache.kv, 0, q, q.stride(1), n, d_rows, torch.tensor(lengths, dtype=torch.int64, device="cuda"), scale)
    F.ls_verify_attend_kv4(*args, out, ws, ws.numel())
    again = torch.full_like(out, 7.0)
    ws.fill_(0x5a)
    F.ls_verify_attend_kv4(*args, again, ws, ws.numel())
    assert torch.equal(out.nan_to_num(123.0), again.nan_to_num(123.0))
    return q, out


def _check(lib, cache, lengths, q, out, rows, n, scale=None):
    c = lib.cfg
    hq, D = c.n_q_heads, c.head_dim
    scale = scale or D ** -0.5
    f32 = out.dtype == torch.float32
    for b, t in enumerate(lengths):
        nb = n if rows is None else rows[b]
        k, v = cache.rows(b, t)
        qb = _f64(q[b])[:nb, :hq * D].reshape(nb, hq, D)
        ref, mass, _ = O.attend_rows(qb, k, v, t - nb, scale)
        got = _f64(out[b])
        assert (got[nb:] == 7.0).all()  # rows that are none stay as they were
        if nb == 0:
            continue
        exc = np.abs(got[:nb] - ref) - _tolerance(lib, qb, k, v, ref, mass, t, scale, f32)
        assert np.isfinite(got).all() and exc.max() <= 0, (b, float(exc.max()))


SHAPES = {  # kv_heads, q_heads, dim, block
    "qwen3": (8, 32, 128, 16), "mid": (2, 8, 128, 16), "narrow": (4, 16, 64, 16), "mha": (3, 3, 128, 16),
    "pair": (2, 4, 128, 32), "mqa": (1, 24, 64, 2), "wide": (2, 40, 128, 3), "most": (1, 64, 64, 1),
    "seven": (1, 7, 128, 9), "odd": (1, 55, 64, 1)}


@pytest.mark.parametrize("shape,dtype,flags,ps,n,lengths", [
    ("mid", "bf16", 0, 16, 1, [0, 1, 2, 15, 16, 17, 127, 128, 129, 1000]),
    ("mid", "bf16", 0, 32, 2, [1, 2, 300]),
    ("mid", "bf16", 0, 16, 5, [3, 5, 128, 517]),
    ("mid", "bf16", 2, 256, 6, [1, 640, 255]),
    ("mid", "bf16", 0, 128, 9, [9, 131, 2000]),
    ("mid", "bf16", 2, 16, 17, [0, 5, 17, 128, 145, 1500]),
    ("pair", "bf16", 0, 16, 33, [33, 7, 160, 1025]),
    ("mid", "bf16", 1, 64, 17, [40, 700]),
    ("qwen3", "bf16", 0, 16, 17, [1200, 333]),
    ("qwen3", "bf16", 0, 16, 1, [4001]),
    ("narrow", "bf16", 0, 64, 9, [3, 700, 1100]),
    ("narrow", "bf16", 2, 16, 1, [64, 129, 0, 2049]),
    ("narrow", "bf16", 0, 256, 17, [300, 1]),
    ("narrow", "f32", 0, 16, 5, [1, 30, 700]),
    ("mid", "f32", 0, 32, 17, [0, 17, 300]),
    ("mha", "bf16", 0, 16, 1, [5, 900]),
    ("mha", "bf16", 0, 16, 17, [17, 400]),
    ("mqa", "bf16", 0, 16, 1, [100, 1000]),
    ("mqa", "bf16", 0, 32, 3, [33, 500]),
    ("most", "bf16", 2, 16, 2, [1, 260]),
    ("most", "bf16", 0, 16, 1, [700]),
    ("wide", "bf16", 0, 16, 4, [9, 600]),
    ("mid", "bf16", 0, 16, 3, [130] * 70),
    ("mid", "bf16", 0, 16, 7, [7, 300, 1, 1025]),
    ("mid", "bf16", 0, 16, 8, [2000, 8]),
    ("seven", "bf16", 0, 32, 4, [4, 260, 901]),
    ("seven", "bf16", 2, 16, 10, [17, 3, 800]),
    ("odd", "bf16", 0, 16, 2, [2, 1, 900]),
    ("odd", "bf16", 2, 64, 1, [300]),
    ("seven", "bf16", 0, 16, 3, [129, 700]),
    ("mid", "bf16", 0, 16, 17, [20 + i % 150 for i in range(200)]),
])
def test_attention(shape, dtype, flags, ps, n, lengths):
    kvh, qh, D, block = SHAPES[shape]
    lib = Lib(batch=len(lengths), kv_heads=kvh, q_heads=qh, dim=D, block=block, dtype=dtype, flags=flags)
    cache = Cache4(lib, lengths, ps, seed=n, stride_extra=16 * (n % 3))
    q, out = _attend(lib, cache, lengths, n, q_extra=8 * n)
    _check(lib, cache, lengths, q, out, None, n)
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("shape,n", [("qwen3", 17), ("qwen3", 1), ("qwen3", 7), ("narrow", 17), ("narrow", 1)])
def test_long_lists_of_shared_pages(shape, n):
    """Twenty steps of 128 keys and more per CTA; pages that several blocks and sequences name."""
    kvh, qh, D, block = SHAPES[shape]
    lib = Lib(batch=3, kv_heads=kvh, q_heads=qh, dim=D, block=block)
    cache = Cache4(lib, [64 * 16, 0, 0], 16, seed=21)
    lengths = [24000, 9001, 18333] if D == 128 else [48000, 18001, 36333]
    cache.mb = -(-max(lengths) // 16)
    cache.table = np.random.default_rng(n).integers(0, cache.pages, (3, cache.mb), dtype=np.int32)
    cache.upload()
    q, out = _attend(lib, cache, lengths, n)
    assert lib.error() == (F.LS_OK, 0)
    # the formula in 64 bits, all rows of a KV head at once; each page decoded once
    held = [np.zeros((cache.pages, 16, kvh, D)) for _ in range(2)]
    for p in range(cache.pages):
        for h in range(kvh):
            kc, vc, ks, vs = cache.sections(p, h)
            held[0][p, :, h], held[1][p, :, h] = O.kv4_decode(kc, ks), O.kv4_decode(vc, vs)
    grp, scale = qh // kvh, D ** -0.5
    for b, t in enumerate(lengths):
        k, v = (torch.from_numpy(x[cache.table[b]].reshape(-1, kvh, D)[:t]).cuda() for x in held)
        seen = torch.arange(t, device="cuda") <= torch.arange(t - n, t, device="cuda")[:, None]
        for h in range(kvh):
            qs = q[b].double().view(n, qh, D)[:, h * grp:(h + 1) * grp]
            x = (scale * (qs @ k[:, h].T)).masked_fill(~seen[:, None], -torch.inf)
            w = torch.softmax(x, -1)
            ref, mass = w @ v[:, h], w @ v[:, h].abs()
            dot = (qs.abs() @ k[:, h].abs().T).amax(-1, keepdim=True)
            ex = (D + 8) * 2.0 ** -24 * scale * dot + D * 2.0 ** -25 * scale * qs.abs().amax(-1, keepdim=True) * k[:, h].abs().max()
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2 * ex + 2 * (t + 256) * 2.0 ** -24) * mass + t * 2.0 ** -33 * v[:, h].abs().max()
            exc = (out[b, :, h * grp:(h + 1) * grp].double() - ref).abs() - tol
            assert exc.max() <= 0, (b, h, float(exc.max()))


@pytest.mark.parametrize("shape,n,dtype", [("mid", 17, "bf16"), ("mid", 5, "bf16"), ("narrow", 17, "bf16"), ("narrow", 5, "f32")])
def test_ragged_rows(shape, n, dtype):
    """Sequences with fewer query rows than the call's, none, or more rows than tokens."""
    kvh, qh, D, block = SHAPES[shape]
    lengths, rows = [200, 64, 3, 0, 129, 50], [n, 0, 4, 2, 1, n - 1]
    lib = Lib(batch=6, kv_heads=kvh, q_heads=qh, dim=D, block=block, dtype=dtype)
    cache = Cache4(lib, lengths, 16, seed=9)
    q, out = _attend(lib, cache, lengths, n, rows=rows)
    _check(lib, cache, lengths, q, out, rows, n)
    assert (_f64(out[2])[0] == 0).all() and (_f64(out[3])[:2] == 0).all()  # rows before position 0
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("n", [1, 5, 17])
@pytest.mark.parametrize("flags", [0, 1])
def test_nothing_behind_a_row_reaches_it(n, flags):
    """NaN scales behind the length, and in the keys and values of rows a query row does not
    see, leave it alone; rows that do see one are NaN (a value's in its own 16 elements)."""
    lib = Lib(batch=2, kv_heads=2, q_heads=8, block=16, flags=flags)
    lengths = [150, 40]
    cache = Cache4(lib, lengths, 16, seed=4)
    ref_q, ref = _attend(lib, cache, lengths, n)
    for b, t in enumerate(lengths):
        for pos in range(t, cache.mb * 16):
            page = cache.table[b, pos // 16]
            if page >= 0:
                for h in range(2):
                    for sec in cache.sections(page, h)[2:]:
                        sec[pos % 16] = 0x7f
    cache.upload()
    q, out = _attend(lib, cache, lengths, n)
    assert torch.equal(out, ref)
    if n == 1:
        return
    # the last position's value group 3 of head 0, and the last position's key of head 1
    kc, vc, ks, vs = cache.sections(cache.table[0, 149 // 16], 0)
    vs[149 % 16, 3] = 0xff
    kc, vc, ks, vs = cache.sections(cache.table[0, 149 // 16], 1)
    ks[149 % 16, 0] = 0x7f
    cache.upload()
    q, out = _attend(lib, cache, lengths, n)
    assert torch.equal(out[1], ref[1]) and torch.equal(out[0, :n - 1], ref[0, :n - 1])
    last = out[0, n - 1]
    assert last[:4, 48:64].isnan().all() and last[4:].isnan().all()
    assert torch.equal(last[:4, :48], ref[0, n - 1, :4, :48]) and torch.equal(last[:4, 64:], ref[0, n - 1, :4, 64:])


@pytest.mark.parametrize("n", [1, 17])
def test_large_and_small_queries(n):
    """Queries far outside fp16's range, and logits that differ by hundreds."""
    for q_scale, scale in ((3e4, 1e-6), (1e-20, 1e18), (20.0, 0.5), (1e30, 1e-32)):
        lib = Lib(batch=1, kv_heads=1, q_heads=4, block=16, flags=F.LS_FLAG_OUT_F32)
        cache = Cache4(lib, [300], 16, seed=6, scale_std=1.5)
        q, out = _attend(lib, cache, [300], n, scale=scale, q_scale=q_scale)
        _check(lib, cache, [300], q, out, None, n, scale=scale)


@pytest.mark.parametrize("n", [1, 17])
def test_extreme_scales(n):
    """Scales from the smallest to the largest, zeros among them: the held values stay exact."""
    lib = Lib(batch=1, kv_heads=1, q_heads=4, block=16, flags=F.LS_FLAG_OUT_F32)
    cache = Cache4(lib, [200], 16, seed=8)
    rng = np.random.default_rng(3)
    for p in range(cache.pages):
        kc, vc, ks, vs = cache.sections(p, 0)
        ks[:] = rng.integers(0, 0x28, ks.shape)
        vs[:] = rng.integers(0, 0x7f, vs.shape)
    cache.upload()
    q, out = _attend(lib, cache, [200], n, q_scale=4.0)
    _check(lib, cache, [200], q, out, None, n)


def test_bad_lengths_rows_and_pages_are_flagged():
    for n, flags in ((1, 0), (17, 0), (5, F.LS_FLAG_FORCE_SIMT)):
        lib = Lib(batch=3, kv_heads=2, q_heads=8, block=16, flags=flags)
        good = [50, 40, 30]
        cache = Cache4(lib, good, 16, seed=2)
        q, ref = _attend(lib, cache, good, n)
        for bad in (-1, cache.mb * 16 + 1, 1 << 40):
            q, out = _attend(lib, cache, [50, bad, 30], n)
            assert lib.error()[1] == F.LS_DEVERR_PREFIX_LEN
            lib.clear()
            assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2]) and (out[1] == 0).all()
        q, out = _attend(lib, cache, good, n, rows=[n, n + 1, -1])
        assert lib.error()[1] == F.LS_DEVERR_ROWS
        lib.clear()
        assert torch.equal(out[:2], ref[:2]) and (out[2] == 7).all()
        old = cache.table[1, 1]
        for bad in (cache.pages, -1, 1 << 30):
            cache.table[1, 1] = bad
            cache.upload()
            q, out = _attend(lib, cache, good, n)
            assert lib.error()[1] == F.LS_DEVERR_PAGE
            lib.clear()
            cache.table[1, 1] = 0
            cache.upload()
            q, want = _attend(lib, cache, good, n)
            assert torch.equal(out, want)
        cache.table[1, 1] = old
        assert lib.error() == (F.LS_OK, 0)


def test_long_cache_past_32_bits():
    """A pool whose last pages lie more than 2^32 bytes behind its base."""
    lib = Lib(batch=2, kv_heads=2, q_heads=8, block=16)
    ps, n_pages = 16, 40
    cache = Cache4(lib, [200, 100], ps, seed=12)
    per = F.ls_kv4_page_bytes(lib.cfg, ps)
    stride = (1 << 32) // 30 // 16 * 16  # 40 pages of 143 MB: 5.7 GB
    big = torch.empty(n_pages * stride, dtype=torch.uint8, device="cuda")
    order = np.random.default_rng(0).permutation(np.arange(n_pages))[:cache.pages]
    for p in range(cache.pages):
        at = int(order[p]) * stride
        big[at:at + per] = torch.from_numpy(cache.bytes[p, :per]).cuda()
    table = np.where(cache.table >= 0, order[np.clip(cache.table, 0, cache.pages - 1)], -1).astype(np.int32)
    d_table = torch.from_numpy(table).cuda()
    for n in (1, 17):
        q, want = _attend(lib, cache, [200, 100], n)
        far = type("far", (), {"kv": F.make_paged_kv4([big], stride, d_table, cache.mb, ps, n_pages)})
        q, out = _attend(lib, far, [200, 100], n)
        assert torch.equal(out, want)
    assert lib.error() == (F.LS_OK, 0)


def test_two_streams_and_captured_calls():
    """Two calls at once with a workspace each, and a captured call replayed on changed inputs."""
    lib = Lib(batch=4, kv_heads=2, q_heads=8, block=16)
    c = lib.cfg
    lengths = [2000, 900, 0, 4100]
    cache = Cache4(lib, lengths, 16, seed=7)
    for n in (1, 17):
        sets = []
        for s in range(2):
            q, want = _attend(lib, cache, lengths, n, seed=s)
            sets.append((q, want, torch.full_like(want, 7.0), torch.empty(F.ls_verify_workspace_bytes(c, n), dtype=torch.uint8, device="cuda"),
                         torch.cuda.Stream()))
        t = torch.tensor(lengths, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        for _ in range(10):
            for q, want, out, ws, stream in sets:
                F.ls_verify_attend_kv4(lib.st, cache.kv, 0, q, q.stride(1), n, None, t, c.head_dim ** -0.5, out, ws, ws.numel(), stream)
        torch.cuda.synchronize()
        for q, want, out, ws, stream in sets:
            assert torch.equal(out, want)
        q, want, out, ws, stream = sets[0]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            F.ls_verify_attend_kv4(lib.st, cache.kv, 0, q, q.stride(1), n, None, t, c.head_dim ** -0.5, out, ws, ws.numel(), stream)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        t2 = [10, 0, 0, 4000]
        t.copy_(torch.tensor(t2))
        q.copy_(sets[1][0])
        g.replay()
        torch.cuda.synchronize()
        q2, want2 = _attend(lib, cache, t2, n, seed=1)
        assert torch.equal(out, want2)
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("n", [1, 17])
def test_a_call_after_it_sees_the_whole_output(n):
    """Short sequences: no tile is cut, so the joining kernel has no work, and the next call of the
    library (which may be scheduled early) reads the output all the same."""
    b = 64
    lib = Lib(batch=b, kv_heads=2, q_heads=2, block=16)
    lengths = [17 + i for i in range(b)]
    cache = Cache4(lib, lengths, 16, seed=14)
    q, want = _attend(lib, cache, lengths, n)
    t = torch.tensor(lengths, dtype=torch.int64, device="cuda")
    ws = torch.empty(F.ls_verify_workspace_bytes(lib.cfg, n), dtype=torch.uint8, device="cuda")
    rows = b * n
    slots = torch.arange(rows, dtype=torch.int64, device="cuda")
    dst = torch.zeros(2, -(-rows // 16), F.ls_kv4_page_bytes(lib.cfg, 16), dtype=torch.uint8, device="cuda")
    held = [F.make_paged_kv4([x], x.stride(0), None, 1, 16, x.shape[0]) for x in dst]
    F.ls_kv4_append(lib.st, held[0], 0, want, want, 256, slots, rows)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    for _ in range(50):
        out.zero_()
        dst[1].zero_()
        F.ls_verify_attend_kv4(lib.st, cache.kv, 0, q, q.stride(1), n, None, t, 128 ** -0.5, out, ws, ws.numel())
        F.ls_kv4_append(lib.st, held[1], 0, out, out, 256, slots, rows)
        assert torch.equal(dst[0], dst[1])
    assert lib.error() == (F.LS_OK, 0)


def test_refusals():
    lib = Lib(batch=2, layers=2)
    cache = Cache4(lib, [20, 30], 16)
    q = torch.zeros(2, 17, 8 * 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    t = torch.tensor([20, 30], dtype=torch.int64, device="cuda")
    ws = torch.empty(F.ls_verify_workspace_bytes(lib.cfg, 17), dtype=torch.uint8, device="cuda")
    ok = dict(kv=cache.kv, layer=0, q=q, stride=1024, n=17, t=t, scale=0.1, out=out, ws=ws, wsb=ws.numel())

    def call(**kw):
        a = {**ok, **kw}
        F.ls_verify_attend_kv4(lib.st, a["kv"], a["layer"], a["q"], a["stride"], a["n"], None, a["t"], a["scale"], a["out"], a["ws"], a["wsb"])

    def kv(base=cache.dev, stride=cache.stride, table=cache.d_table, mb=cache.mb, ps=16, pages=cache.pages):
        return F.make_paged_kv4([base, base], stride, table, mb, ps, pages)

    call()
    inv, shape, uns = F.LS_ERR_INVALID_ARG, F.LS_ERR_SHAPE, F.LS_ERR_UNSUPPORTED
    for status, kw in [
            (inv, dict(layer=2)), (inv, dict(layer=-1)), (inv, dict(q=None)), (inv, dict(out=None)), (inv, dict(ws=None)),
            (inv, dict(t=None)), (inv, dict(n=0)), (shape, dict(n=18)), (shape, dict(stride=1016)), (shape, dict(stride=1028)),
            (inv, dict(scale=0.0)), (inv, dict(scale=-1.0)), (inv, dict(scale=float("inf"))), (inv, dict(scale=float("nan"))),
            (shape, dict(wsb=ws.numel() - 1)), (inv, dict(ws=ws.data_ptr() + 16)), (inv, dict(q=q.data_ptr() + 8)),
            (inv, dict(out=out.data_ptr() + 8)), (inv, dict(t=t.data_ptr() + 4)), (inv, dict(kv=kv(base=None))),
            (inv, dict(kv=kv(base=cache.dev.data_ptr() + 8))), (shape, dict(kv=kv(stride=cache.stride - 16))),
            (shape, dict(kv=kv(stride=cache.stride + 8))), (inv, dict(kv=kv(table=None))), (inv, dict(kv=kv(mb=0))),
            (uns, dict(kv=kv(ps=8))), (uns, dict(kv=kv(ps=48))), (uns, dict(kv=kv(ps=512))), (inv, dict(kv=kv(pages=0))),
            (uns, dict(kv=kv(pages=1 << 31)))]:
        with pytest.raises(F.LsError) as e:
            call(**kw)
        assert e.value.status == status, kw
    k = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(4, dtype=torch.int64, device="cuda")
    for fn, order in ((F.ls_kv4_append, lambda k, v, st, s, n: (k, v, st, s, n)), (F.ls_kv4_read_rows, lambda k, v, st, s, n: (s, n, k, v, st))):
        for status, a in [(inv, (None, k, 256, s, 4)), (inv, (k, None, 256, s, 4)), (inv, (k, k, 256, None, 4)), (inv, (k, k, 256, s, -1)),
                          (shape, (k, k, 248, s, 4)), (shape, (k, k, 260, s, 4)), (inv, (k.data_ptr() + 2, k, 256, s, 4)),
                          (inv, (k, k, 256, s.data_ptr() + 4, 4))]:
            refused(status, fn, lib.st, cache.kv, 0, *order(*a))
        refused(inv, fn, lib.st, cache.kv, 2, *order(k, k, 256, s, 4))
        refused(uns, fn, lib.st, kv(ps=8), 0, *order(k, k, 256, s, 4))
    lib32 = Lib(kv_heads=2, q_heads=2, dim=32, dtype="f32")
    refused(uns, F.ls_kv4_append, lib32.st, cache.kv, 0, k, k, 256, s, 4)
    assert lib.error() == (F.LS_OK, 0)
