"""Page tables and slot maps (ls_pages_extend, ls_pages_trim) against the loops of the oracle:
whole numbers, so every comparison is for equality."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fixed_cost_drafter_b200 as F
    import oracle as O
    from tests.serving_side import Lib, refused

FLAGS = {"pool": 0x20, "rows": 0x40, "page": 0x10}
KEEP = -77  # sentinel in slots that a call leaves alone


class Pool:
    def __init__(self, b, max_blocks, ps, num, held, seed=0, count=None):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(num).astype(np.int32)
        self.ps, self.num, self.mb = ps, num, max_blocks
        self.held = np.array(held, np.int32)
        self.table = np.full((b, max_blocks), -1, np.int32)
        at = 0
        for i in range(b):
            self.table[i, :held[i]] = ids[at:at + held[i]]
            at += held[i]
        self.free = np.concatenate([ids[at:], np.full(at, -1, np.int32)])
        self.count = num - at if count is None else count
        self.up()

    def up(self):
        self.d = [torch.from_numpy(x.copy()).cuda() for x in (self.table, self.held, self.free, np.array([self.count], np.int32))]
        self.desc = F.make_page_pool(*self.d, self.mb, self.ps, self.num)

    def check(self):
        for name, got, want in zip(("table", "held", "free", "count"), self.d,
                                   (self.table, self.held, self.free, np.array([self.count]))):
            got = got.cpu().numpy()
            if name == "free":  # behind the count nothing is promised
                got, want = got[:max(self.count, 0)], want[:max(self.count, 0)]
            assert np.array_equal(got, want), name


def _flag_word(flags):
    return sum(FLAGS[f] for f in flags)


def _extend(lib, pool, length, rows, max_rows, packed, capacity=None):
    b = len(length)
    total = b * max_rows if capacity is None else capacity
    slots = torch.full((max(total, 1),), KEEP, dtype=torch.int64, device="cuda")
    begin = torch.full((b + 1,), KEEP, dtype=torch.int64, device="cuda") if packed else None
    d_rows = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    F.ls_pages_extend(lib.st, pool.desc, torch.tensor(length, dtype=torch.int64, device="cuda"), d_rows, max_rows, begin,
                      slots, total)
    use = [max_rows] * b if rows is None else rows
    pool.count, want, flags = O.pages_extend(pool.table, pool.held, pool.free, pool.count, length, use, max_rows, pool.ps, pool.num)
    got = slots.cpu().numpy()
    if packed:
        flat = [x for s in want for x in s]
        assert list(begin.cpu().numpy()) == list(np.concatenate([[0], np.cumsum([len(s) for s in want])]))
        n = min(len(flat), total)
        if len(flat) > total:
            flags = flags | {"pool"}
        assert list(got[:n]) == flat[:n] and (got[n:] == KEEP).all()
    else:
        for i, s in enumerate(want):
            assert list(got[i * max_rows:(i + 1) * max_rows]) == s + [-1] * (max_rows - len(s))
    pool.check()
    status, word = lib.error()
    assert word == _flag_word(flags), (word, flags)
    lib.clear()
    return flags


def _trim(lib, pool, length):
    F.ls_pages_trim(lib.st, pool.desc, torch.tensor(length, dtype=torch.int64, device="cuda"))
    pool.count, flags = O.pages_trim(pool.table, pool.held, pool.free, pool.count, length, pool.ps, pool.num)
    pool.check()
    assert lib.error()[1] == _flag_word(flags)
    lib.clear()


@pytest.mark.parametrize("b,ps,max_rows,packed", [
    (1, 16, 17, False), (1, 1, 5, True), (5, 24, 33, True), (16, 16, 17, False), (3, 7, 1, False),
    (300, 32, 9, True), (64, 16, 5000, True), (2, 128, 20000, False), (37, 8, 0, True)])
def test_rounds(b, ps, max_rows, packed):
    """Several rounds of extends and trims with ragged lengths, rows and kept rows."""
    rng = np.random.default_rng(b * 1000 + ps)
    lib = Lib(batch=b)
    length = rng.integers(0, 4 * ps + 1, b)
    length[0] = 0
    mb = -(-(4 * ps + 3 * max_rows + 1) // ps) + 1
    pool = Pool(b, mb, ps, b * mb + 5, -(-length // ps), seed=b)
    for _ in range(3):
        rows = rng.integers(0, max_rows + 1, b)
        _extend(lib, pool, list(length), None if not packed else list(rows), max_rows, packed)
        length = length + (rng.integers(0, rows + 1) if packed else rng.integers(0, max_rows + 1, b))
        length = np.minimum(length, (mb * ps) - max_rows)
        _trim(lib, pool, list(length))
    _trim(lib, pool, [0] * b)
    assert pool.count == pool.num


def test_extend_then_trim_restores_the_list():
    lib = Lib(batch=4)
    pool = Pool(4, 40, 16, 100, [1, 0, 3, 2], seed=3)
    free = pool.d[2].clone()
    n = pool.count
    _extend(lib, pool, [10, 0, 48, 17], None, 100, False)
    _trim(lib, pool, [10, 0, 48, 17])
    assert pool.count == n and torch.equal(pool.d[2][:n], free[:n])


def test_too_few_pages_and_sequences_behind():
    lib = Lib(batch=5)
    pool = Pool(5, 8, 16, 12, [1, 1, 1, 1, 1], seed=1)  # 7 free
    # needs 2, 4, 3 (refused), 0 (served: rows fit the held page), 1 (refused)
    assert _extend(lib, pool, [16, 16, 16, 3, 16], [32, 64, 48, 13, 1], 64, True) == {"pool"}
    assert list(pool.held) == [3, 5, 1, 1, 1]
    assert _extend(lib, pool, [0] * 5, [1] * 5, 1, True) == set()


def test_arguments_out_of_range_are_flagged():
    lib = Lib(batch=6)
    pool = Pool(6, 4, 16, 40, [1, 1, 1, 1, 1, 1])
    assert _extend(lib, pool, [5, -1, 5, 60, 5, 16], [1, 1, -1, 5, 18, 17], 17, True) == {"rows"}
    pool.held[2] = 9  # more than the table holds
    pool.up()
    assert _extend(lib, pool, [5] * 6, [1] * 6, 17, True) == {"rows"}
    _trim(lib, pool, [-1, 5, 5, 5, 5, 0])
    pool.held[2] = 1
    pool.count = pool.num + 1
    pool.up()
    _extend(lib, pool, [5] * 6, [1] * 6, 17, True)
    _trim(lib, pool, [0] * 6)  # would hold more than there are: nothing changes
    pool.count = -3
    pool.up()
    _extend(lib, pool, [5] * 6, [1] * 6, 17, True)
    _trim(lib, pool, [0] * 6)
    pool.count = 3
    pool.table[4, 0] = 40  # a page that does not exist
    pool.up()
    assert _extend(lib, pool, [5] * 6, [1] * 6, 17, True) == {"page"}


def test_slots_past_the_capacity_are_not_written():
    lib = Lib(batch=3)
    pool = Pool(3, 8, 16, 24, [0, 0, 0])
    assert _extend(lib, pool, [0, 0, 0], [10, 20, 30], 30, True, capacity=25) == {"pool"}
    assert _extend(lib, pool, [10, 20, 30], [1, 1, 1], 30, True, capacity=0) == {"pool"}


def test_positions_past_32_bits():
    """Rows far along a sequence whose pages are huge: positions and slots need 64 bits."""
    lib = Lib(batch=2)
    ps = 1 << 30
    pool = Pool(2, 6, ps, 12, [5, 4], seed=5)
    _extend(lib, pool, [5 * ps - 3, 4 * ps + 11 - ps], None, 7, False)
    ps = (1 << 30) - 1
    pool = Pool(2, 6, ps, 12, [5, 4], seed=6)
    _extend(lib, pool, [5 * ps - 3, 4 * ps - 20], None, 30, False)
    _trim(lib, pool, [4 * ps + 1, 4 * ps])


def test_lengths_of_the_state_itself():
    """d_len NULL: the lengths that the state's commits left."""
    lib = Lib(batch=3)
    lens = torch.tensor([0, 100, 37], dtype=torch.int64, device="cuda")
    k = torch.randn(3, 1, 100, 256, device="cuda").to(torch.bfloat16)
    ws = torch.empty(F.ls_prefill_workspace_bytes(lib.cfg, 0, 100), dtype=torch.uint8, device="cuda")
    F.ls_prefill_summary(lib.st, k, k, 100 * 256, 256, lens, 0, 100, None, ws, ws.numel())
    pool = Pool(3, 12, 16, 30, [0, 7, 3])
    slots = torch.empty(3, 17, dtype=torch.int64, device="cuda")
    F.ls_pages_extend(lib.st, pool.desc, None, None, 17, None, slots, 51)
    pool.count, want, _ = O.pages_extend(pool.table, pool.held, pool.free, pool.count, [0, 100, 37], [17] * 3, 17, 16, 30)
    assert slots.cpu().tolist() == want
    F.ls_pages_trim(lib.st, pool.desc, None)
    pool.count, _ = O.pages_trim(pool.table, pool.held, pool.free, pool.count, [0, 100, 37], 16, 30)
    pool.check()
    assert lib.error() == (F.LS_OK, 0)


def test_captured_and_on_another_stream():
    lib = Lib(batch=3)
    pool = Pool(3, 64, 16, 150, [1, 2, 0])
    n = torch.tensor([9, 20, 0], dtype=torch.int64, device="cuda")
    m = torch.tensor([11, 21, 2], dtype=torch.int64, device="cuda")
    slots = torch.empty(3, 17, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            F.ls_pages_extend(lib.st, pool.desc, n, None, 17, None, slots, 51)
            F.ls_pages_trim(lib.st, pool.desc, m)
    length, after = [9, 20, 0], [11, 21, 2]
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        pool.count, want, _ = O.pages_extend(pool.table, pool.held, pool.free, pool.count, length, [17] * 3, 17, 16, 150)
        assert slots.cpu().tolist() == want
        pool.count, _ = O.pages_trim(pool.table, pool.held, pool.free, pool.count, after, 16, 150)
        pool.check()
        length, after = [x + 20 for x in length], [x + 23 for x in after]
        n += 20
        m += 23
        torch.cuda.synchronize()
    assert lib.error() == (F.LS_OK, 0)


def test_refusals():
    lib = Lib(batch=2)
    pool = Pool(2, 4, 16, 8, [0, 0])
    s = torch.empty(2, 4, dtype=torch.int64, device="cuda")
    bad = F.LS_ERR_INVALID_ARG
    p = pool.d
    for desc in (F.make_page_pool(None, p[1], p[2], p[3], 4, 16, 8), F.make_page_pool(p[0], None, p[2], p[3], 4, 16, 8),
                 F.make_page_pool(p[0], p[1], None, p[3], 4, 16, 8), F.make_page_pool(p[0], p[1], p[2], None, 4, 16, 8),
                 F.make_page_pool(*p, 0, 16, 8), F.make_page_pool(*p, 4, 0, 8), F.make_page_pool(*p, 4, 16, 0),
                 F.make_page_pool(p[0].data_ptr() + 2, p[1], p[2], p[3], 4, 16, 8)):
        refused(bad, F.ls_pages_extend, lib.st, desc, None, None, 4, None, s, 8)
        refused(bad, F.ls_pages_trim, lib.st, desc, None)
    refused(F.LS_ERR_UNSUPPORTED, F.ls_pages_trim, lib.st, F.make_page_pool(*p, 4, 16, 1 << 31), None)
    refused(F.LS_ERR_UNSUPPORTED, F.ls_pages_trim, lib.st, F.make_page_pool(*p, (1 << 30) + 1, 16, 8), None)
    refused(F.LS_ERR_UNSUPPORTED, F.ls_pages_extend, lib.st, pool.desc, None, None, (1 << 30) + 1, s, s, 1 << 40)
    refused(F.LS_ERR_SHAPE, F.ls_pages_extend, lib.st, pool.desc, None, None, 4, None, s, 7)
    refused(bad, F.ls_pages_extend, lib.st, pool.desc, None, None, -1, None, s, 8)
    refused(bad, F.ls_pages_extend, lib.st, pool.desc, None, None, 4, None, None, 8)
    refused(bad, F.ls_pages_extend, lib.st, pool.desc, None, None, 4, None, s.data_ptr() + 4, 8)
    refused(bad, F.ls_pages_extend, lib.st, pool.desc, s.data_ptr() + 4, None, 4, None, s, 8)
    refused(bad, F.ls_pages_trim, lib.st, pool.desc, s.data_ptr() + 4)
    torch.cuda.synchronize()
    pool.check()
    assert lib.error() == (F.LS_OK, 0)
