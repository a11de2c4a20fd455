"""The serving-side operators at the edges of what their header allows: references that move with
every step, idle and padded sequences, page ids that name no page, head counts whose rows are no
whole warps, calls on two streams at once."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fixed_cost_drafter_b200 as F
    import oracle as O
    from tests.serving_side import Cache4, Lib, refused
    from tests.test_gpu_kv4 import SHAPES, _attend, _check


@pytest.mark.parametrize("shape,n,flags", [("mid", 17, 0), ("mid", 17, 2), ("narrow", 17, 0), ("mid", 8, 0), ("mid", 6, 0), ("mid", 1, 0)])
def test_references_that_move_with_every_step(shape, n, flags):
    """Logits that grow by ten and more from each 64 keys to the next: every step's first weights are
    far too large (at the start of each list of keys they are infinite) and replaced by others. The
    bound is that of the attention's tests; its terms count logits of a few hundred."""
    kvh, qh, D, block = SHAPES[shape]
    lengths = [65 + 37 * (i % 23) for i in range(60)]
    lib = Lib(batch=len(lengths), kv_heads=kvh, q_heads=qh, dim=D, block=block, flags=flags)
    cache = Cache4(lib, lengths, 16, seed=5)
    for b, t in enumerate(lengths):
        for pi in range(-(-t // 16)):
            for h in range(kvh):
                kc, _, ks, _ = cache.sections(cache.table[b, pi], h)
                kc[:] = 0x22                 # ones
                ks[:] = 0x38 + pi * 16 // 64  # times 1, 1.125, 1.25 ..
    cache.upload()
    scale = 100.0 / D  # queries below have elements of one sign, 0.8 on average
    rng = np.random.default_rng(n)
    q = torch.from_numpy(rng.uniform(0.6, 1.0, (len(lengths), n, qh * D))).to(torch.bfloat16).cuda()
    f32 = bool(flags & F.LS_FLAG_OUT_F32)
    ws = torch.full((F.ls_verify_workspace_bytes(lib.cfg, n),), 0xff, dtype=torch.uint8, device="cuda")
    t = torch.tensor(lengths, dtype=torch.int64, device="cuda")
    outs = []
    for _ in range(5):
        out = torch.full((len(lengths), n, qh, D), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        F.ls_verify_attend_kv4(lib.st, cache.kv, 0, q, qh * D, n, None, t, scale, out, ws, ws.numel())
        outs.append(out)
    _check(lib, cache, lengths, q, outs[0], None, n, scale=scale)
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("heads", range(1, 9))
def test_rows_of_every_head_count(heads, dtype, dim):
    """Rows of 3, 5, 6 and 7 heads are no whole number of warps: the CTAs' last warps are filled with
    threads that have no row. Bytes equal the oracle's, and nothing else is written."""
    n, ps = 83, 16
    lib = Lib(kv_heads=heads, q_heads=heads, dim=dim, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(heads)
    k, v = (torch.randn(n, heads * dim, generator=g, device="cuda").to(lib.tdtype) for _ in range(2))
    pages = -(-n // ps) + 1
    slots = np.random.default_rng(heads).permutation(pages * ps)[:n]
    d_slots = torch.from_numpy(slots).cuda()
    per = F.ls_kv4_page_bytes(lib.cfg, ps)
    cache = torch.full((pages, per), 0xA5, dtype=torch.uint8, device="cuda")
    kv = F.make_paged_kv4([cache], per, None, 1, ps, pages)
    F.ls_kv4_append(lib.st, kv, 0, k, v, heads * dim, d_slots, n)
    want = np.full((pages, per), 0xA5, np.uint8)
    back = []
    for which, x in enumerate((k, v)):
        c, s = O.kv4_encode(x.double().cpu().numpy().reshape(n, heads, dim))
        back.append(O.kv4_decode(c, s).reshape(n, heads * dim))
        for i in range(n):
            for h in range(heads):
                sec = O.kv4_sections(want[slots[i] // ps], h, ps, dim)
                sec[which][slots[i] % ps], sec[2 + which][slots[i] % ps] = c[i, h], s[i, h]
    assert np.array_equal(cache.cpu().numpy(), want)
    out = torch.full((2, n + 1, heads * dim), 7.0, dtype=lib.tdtype, device="cuda")
    F.ls_kv4_read_rows(lib.st, kv, 0, d_slots, n, out[0], out[1], heads * dim)
    got = out.double().cpu().numpy()
    assert np.array_equal(got[0, :n], back[0]) and np.array_equal(got[1, :n], back[1]) and (got[:, n] == 7).all()
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("adapters", [True, False])
def test_projections_behind_per_layer_calls_that_do_not_wait(adapters):
    """Drafting passes back to back: the projections of one write the queries and boundary rows that
    the attention calls of the pass before, launched with LS_ATTEND_INPUTS_READY, read.
    Every pass's outputs equal those of the same pass with a synchronisation after each call."""
    b, layers, kvh, qh, D, hidden, block = 16, 4, 8, 32, 128, 512, 16
    lib = Lib(batch=b, layers=layers, kv_heads=kvh, q_heads=qh, dim=D, hidden=hidden, block=block)
    assert F.ls_attend_uses_tensor_cores(lib.st)
    g = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)
    t = torch.full((b,), 300, dtype=torch.int64, device="cuda")
    k = n(b, layers, 300, kvh * D)
    ws = torch.empty(F.ls_prefill_workspace_bytes(lib.cfg, 0, 300), dtype=torch.uint8, device="cuda")
    F.ls_prefill_summary(lib.st, k, n(b, layers, 300, kvh * D), 300 * kvh * D, kvh * D, t, 0, 300, n(b, layers, hidden), ws, ws.numel())
    w_kv, w_q = n(layers, 2 * kvh * D, hidden, std=hidden ** -0.5), n(layers, qh * D, hidden, std=hidden ** -0.5)
    bank = [n(3, layers, 16, hidden, std=hidden ** -0.5), n(3, layers, qh * D, 16), n(3, layers, 16, hidden, std=hidden ** -0.5),
            n(3, layers, 2 * kvh * D, 16), torch.ones(3, device="cuda"), torch.tensor([i % 4 - 1 for i in range(b)], dtype=torch.int32, device="cuda")]
    lora = F.make_lora(3, 16, *bank)
    lws = torch.empty(F.ls_lora_workspace_bytes(lib.cfg, 16), dtype=torch.uint8, device="cuda")
    xs = [n(b, layers, block, hidden) for _ in range(6)]
    bkv = torch.empty(b, layers, 2 * kvh * D, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(b, layers, block, qh * D, dtype=torch.bfloat16, device="cuda")
    hint = F.LS_VIEW_ALL | F.LS_ATTEND_INPUTS_READY

    def run(sync):
        outs = torch.full((len(xs), layers, b, layers, block, qh, D), 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        for i, x in enumerate(xs):
            if adapters:
                F.ls_draft_prologue_lora(lib.st, w_kv, w_q, x, lora, bkv, q, lws, lws.numel())
            else:
                F.ls_draft_prologue(lib.st, w_kv, w_q, x, bkv, q)
            if sync:
                torch.cuda.synchronize()
            for c in range(layers):  # all but the first wait for nothing
                F.ls_draft_attend_views(lib.st, 0, layers, q, bkv, bkv[:, :, kvh * D:], 2 * kvh * D, D ** -0.5,
                                        F.LS_VIEW_ALL if c == 0 else hint, outs[i, c])
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(5):
        assert torch.equal(run(False), want)
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("b,ps,pages_each", [(3, 16, 7), (64, 8, 90), (2, 16, 3000)])
def test_trim_leaves_out_ids_that_name_no_page(b, ps, pages_each):
    """Ids outside the pool among a table's returned entries are flagged and dropped: a later extend
    hands out real pages only, and takes and returns them as ever while the error word still tells."""
    rng = np.random.default_rng(b)
    num = b * pages_each + 9
    lib = Lib(batch=b)
    ids = rng.permutation(num).astype(np.int32)
    free, table = ids[:9], ids[9:].reshape(b, pages_each).copy()
    for bad in (num, -1, 1 << 30, -(1 << 31)):
        table[rng.integers(0, b), rng.integers(0, pages_each)] = bad
    table[0, 0] = table[0, -1] = num + 5
    keep = rng.integers(0, 3, b)
    keep[0] = 0
    d_table, d_held, d_count = (torch.from_numpy(x).cuda() for x in (table, np.full(b, pages_each, np.int32), np.array([9], np.int32)))
    d_free = torch.from_numpy(np.concatenate([free, np.full(num - 9, -9, np.int32)])).cuda()
    pool = F.make_page_pool(d_table, d_held, d_free, d_count, pages_each, ps, num)
    length = torch.from_numpy(keep * ps).cuda()
    gone = np.concatenate([table[i, keep[i]:] for i in range(b)])
    back = gone[(gone >= 0) & (gone < num)]
    want_free = list(free) + list(back[::-1])
    want_table = np.where(np.arange(pages_each) < keep[:, None], table, -1)

    def check():
        assert d_count.tolist() == [len(want_free)] and d_held.tolist() == keep.tolist()
        assert d_free[:len(want_free)].tolist() == want_free and np.array_equal(d_table.cpu().numpy(), want_table)

    F.ls_pages_trim(lib.st, pool, length)
    assert lib.error()[1] == F.LS_DEVERR_PAGE
    check()
    slots = torch.full((b, 2 * ps), -7, dtype=torch.int64, device="cuda")
    for clear in (False, True):
        if clear:
            lib.clear()
        F.ls_pages_extend(lib.st, pool, length, None, 2 * ps, None, slots, slots.numel())
        taken = want_free[::-1][:2 * b]
        assert (slots.view(b * 2, ps)[:, 0] // ps).tolist() == taken
        F.ls_pages_trim(lib.st, pool, length)
        check()
    assert lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("shape,n,flags", [("mid", 1, 0), ("mid", 5, 0), ("mid", 17, 0), ("narrow", 17, 0), ("mid", 17, 1)])
def test_sequences_without_rows_are_not_read(shape, n, flags):
    """The idle slots of a padded batch: their lengths are in range, their tables name no pages.
    Nothing of them is read, so nothing is flagged; the others' outputs are what they are alone."""
    kvh, qh, D, block = SHAPES[shape]
    lengths, rows = [300, 5000, 64, 40, 2000], [n, 0, n, 0, 0]
    lib = Lib(batch=5, kv_heads=kvh, q_heads=qh, dim=D, block=block, flags=flags)
    cache = Cache4(lib, lengths, 16, seed=9)
    cache.table[[1, 3, 4]] = -1
    cache.upload()
    q, out = _attend(lib, cache, lengths, n, rows=rows)
    assert lib.error() == (F.LS_OK, 0)
    _check(lib, cache, [300, 0, 64, 0, 0], q, out, rows, n)
    assert (out[[1, 3, 4]] == 7).all()
    _, bad = _attend(lib, cache, [300, -1, 64, 40, 2000], n, rows=rows)  # a length out of range still is
    assert lib.error()[1] == F.LS_DEVERR_PREFIX_LEN and torch.equal(bad, out)
    lib.clear()
    _, none = _attend(lib, cache, lengths, n, rows=[0] * 5)
    assert (none == 7).all() and lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("n", [1, 17])
def test_layers_of_the_target_beyond_the_tapped_ones(n):
    """The 4-bit cache is the target's: its layers are more than those the drafter taps. Layers the
    descriptor does not have are refused."""
    lib = Lib(batch=2, layers=2)
    lengths, layer = [200, 37], 40
    cache = Cache4(lib, lengths, 16, seed=3)
    q, want = _attend(lib, cache, lengths, n)
    per = F.ls_kv4_page_bytes(lib.cfg, 16)
    copy = torch.zeros_like(cache.dev)
    kv = F.make_paged_kv4([None] * layer + [copy], cache.stride, cache.d_table, cache.mb, 16, cache.pages)
    # rows written and read there are those of layer 0 of a like cache
    k, v = (torch.randn(50, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(50, device="cuda") + 7
    ref, got = torch.zeros_like(copy), torch.empty(4, 50, 256, dtype=torch.bfloat16, device="cuda")
    kv0 = F.make_paged_kv4([ref], cache.stride, None, 1, 16, cache.pages)
    for i, (d, l) in enumerate(((kv0, 0), (kv, layer))):
        F.ls_kv4_append(lib.st, d, l, k, v, 256, slots, 50)
        F.ls_kv4_read_rows(lib.st, d, l, slots, 50, got[2 * i], got[2 * i + 1], 256)
    assert torch.equal(copy, ref) and torch.equal(got[2:], got[:2]) and ref.any()
    out = torch.full_like(want, 7.0)
    ws = torch.empty(F.ls_verify_workspace_bytes(lib.cfg, n), dtype=torch.uint8, device="cuda")
    copy[:, :per] = cache.dev[:, :per]
    t = torch.tensor(lengths, dtype=torch.int64, device="cuda")
    args = (q, q.stride(1), n, None, t, 128 ** -0.5, out, ws, ws.numel())
    F.ls_verify_attend_kv4(lib.st, kv, layer, *args)
    assert torch.equal(out, want) and lib.error() == (F.LS_OK, 0)
    for bad in (0, layer - 1, layer + 1, 64, 1 << 30, -1):
        refused(F.LS_ERR_INVALID_ARG, F.ls_verify_attend_kv4, lib.st, kv, bad, *args)
        refused(F.LS_ERR_INVALID_ARG, F.ls_kv4_append, lib.st, kv, bad, k, v, 256, slots, 16)
        refused(F.LS_ERR_INVALID_ARG, F.ls_kv4_read_rows, lib.st, kv, bad, slots, 16, k, v, 256)


def test_adapters_of_two_states_on_two_streams():
    """Calls that overlap on the GPU, with a state and a workspace each; the next round's ids and
    inputs written on each call's own stream right before it."""
    from tests.test_gpu_lora import Case
    ids = [[0, 1, 2, -1, 2, 0], [2, -1, 0, 0, 1, 1]]
    cases = [Case(6, 16, 2, 1024, 64, 3, ids[s], seed=20 + s) for s in range(2)]
    sets = []
    for c in cases:
        xs = [c.x.clone(), -c.x, c.x.flip(0)]
        whiches = [c.which.clone(), c.which.flip(0), c.which.roll(1)]
        want = []
        for x, w in zip(xs, whiches):
            c.x.copy_(x)
            c.which.copy_(w)
            torch.cuda.synchronize()
            want.append(c.run())
            torch.cuda.synchronize()
        c.check(*want[-1])
        sets.append((c, xs, whiches, want, torch.cuda.Stream(), [c.outputs() for _ in range(12)]))
    torch.cuda.synchronize()
    for i in range(12):
        for c, xs, whiches, want, stream, outs in sets:
            with torch.cuda.stream(stream):
                c.x.copy_(xs[i % 3])
                c.which.copy_(whiches[i % 3])
                F.ls_draft_prologue_lora(c.lib.st, c.w_kv, c.w_q, c.x, c.desc, *outs[i], c.ws, c.ws.numel())
    torch.cuda.synchronize()
    for c, xs, whiches, want, stream, outs in sets:
        for i, got in enumerate(outs):
            assert torch.equal(got[0], want[i % 3][0]) and torch.equal(got[1], want[i % 3][1]), i
        assert c.lib.error() == (F.LS_OK, 0)


def test_ids_and_weights_written_before_every_call():
    """Ids and weights that the kernels right before each call write, every call's outputs compared
    with those of the same values settled long before."""
    from tests.test_gpu_lora import Case
    c = Case(16, 16, 1, 1024, 16, 4, [0] * 16, seed=7)
    whiches = [torch.tensor([(i * s) % 5 - 1 for i in range(16)], dtype=torch.int32, device="cuda") for s in (3, 2)]
    banks = [[t.clone() for t in (c.a_q, c.b_q, c.a_kv, c.b_kv, c.scale)], [-c.a_q, c.b_q * 2, -c.a_kv, c.b_kv * 0.5, c.scale + 1]]

    def put(s):
        c.which.copy_(whiches[s])
        for t, v in zip((c.a_q, c.b_q, c.a_kv, c.b_kv, c.scale), banks[s]):
            t.copy_(v)

    want = []
    for s in range(2):
        put(s)
        torch.cuda.synchronize()
        want.append(c.run())
        torch.cuda.synchronize()
        c.check(*want[s])
    assert not torch.equal(want[0][1], want[1][1])
    got = []
    for i in range(40):
        put(i % 2)
        got.append(c.run())
    for i, (bkv, q) in enumerate(got):
        assert torch.equal(bkv, want[i % 2][0]) and torch.equal(q, want[i % 2][1]), i
    assert c.lib.error() == (F.LS_OK, 0)


@pytest.mark.parametrize("n", [1, 6, 17])
def test_repeated_calls_from_fresh_states_give_the_same_bits(n):
    """Work that is split over CTAs and joined: other states, other workspaces with other contents and
    other calls beside them change no bit of the outputs."""
    lengths = [3000, 1, 517, 0, 9000]
    outs = []
    for r in range(4):
        lib = Lib(batch=5, kv_heads=8, q_heads=32)
        cache = Cache4(lib, lengths, 16, seed=6)
        q, out = _attend(lib, cache, lengths, n, seed=2)
        noise = torch.randn(1 << 24, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                noise.mul_(1.0001)
        outs.append(out)
        outs.append(_attend(lib, cache, lengths, n, seed=2)[1])
        torch.cuda.synchronize()
        assert lib.error() == (F.LS_OK, 0)
    for out in outs[1:]:
        assert torch.equal(out, outs[0])
