"""The projections with low-rank adapters (ls_draft_prologue_lora) against the 64-bit oracle.
Bound per output element: fp32 sums of `hidden` products (hidden 2^-24 sum|w x|) and of the
adapter's two products, whose inner result is held in two bf16 parts (16 bits, 2^-16) and whose
inner sums have `hidden` and outer ones 2 `rank` terms, plus the bf16 rounding of the result:
    2^-8 |y| + (hidden + rank + 4) 2^-24 sum|w x| + (2^-16 + (hidden + 4 rank + 8) 2^-24) sum s |B| |A| |x|"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fixed_cost_drafter_b200 as F
    import oracle as O
    from tests.serving_side import Lib, refused


def _f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, batch, block, layers, hidden, rank, adapters, which, kv_heads=2, q_heads=8, dim=128, seed=0):
        self.lib = lib = Lib(batch=batch, layers=layers, kv_heads=kv_heads, q_heads=q_heads, dim=dim, hidden=hidden, block=block)
        self.nq, self.nkv, self.L, self.H, self.B, self.r, self.na, self.b = q_heads * dim, 2 * kv_heads * dim, layers, hidden, block, rank, adapters, batch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s, std=1.0):
            return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.w_kv, self.w_q = normal(layers, self.nkv, hidden, std=hidden ** -0.5), normal(layers, self.nq, hidden, std=hidden ** -0.5)
        self.a_q, self.a_kv = (normal(adapters, layers, rank, hidden, std=hidden ** -0.5) for _ in range(2))
        self.b_q, self.b_kv = normal(adapters, layers, self.nq, rank), normal(adapters, layers, self.nkv, rank)
        self.scale = torch.rand(adapters, generator=g, device="cuda") * 2 - 0.5
        self.which = torch.tensor(which, dtype=torch.int32, device="cuda")
        self.x, self.bnd = normal(batch, layers, block, hidden), normal(batch, layers, hidden)
        F.ls_prefill_summary(lib.st, None, None, 0, 0, torch.zeros(batch, dtype=torch.int64, device="cuda"), 0, 0, self.bnd, None, 0)
        self.desc = F.make_lora(adapters, rank, self.a_q, self.b_q, self.a_kv, self.b_kv, self.scale, self.which)
        self.ws = torch.full((F.ls_lora_workspace_bytes(lib.cfg, rank),), 0xff, dtype=torch.uint8, device="cuda")

    def outputs(self):
        return (torch.full((self.b, self.L, self.nkv), 7.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.b, self.L, self.B, self.nq), 7.0, dtype=torch.bfloat16, device="cuda"))

    def run(self, stream=None):
        bkv, q = self.outputs()
        F.ls_draft_prologue_lora(self.lib.st, self.w_kv, self.w_q, self.x, self.desc, bkv, q, self.ws, self.ws.numel(), stream)
        return bkv, q

    def base(self):
        bkv, q = self.outputs()
        F.ls_draft_prologue(self.lib.st, self.w_kv, self.w_q, self.x, bkv, q)
        return bkv, q

    def check(self, bkv, q):
        for got, w, x, a, bb in ((_f64(q), self.w_q, self.x, self.a_q, self.b_q),
                                 (_f64(bkv)[:, :, None], self.w_kv, self.bnd[:, :, None], self.a_kv, self.b_kv)):
            y, mag, low = O.project_lora(_f64(w), _f64(x), self.which.tolist(), _f64(a), _f64(bb), _f64(self.scale))
            tol = 2.0 ** -8 * np.abs(y) + (self.H + self.r + 4) * 2.0 ** -24 * mag + \
                (2.0 ** -16 + (self.H + 4 * self.r + 8) * 2.0 ** -24) * low
            exc = np.abs(got - y) - tol
            assert np.isfinite(got).all() and exc.max() <= 0, float(exc.max())


@pytest.mark.parametrize("batch,block,layers,hidden,rank,adapters,which", [
    (1, 1, 1, 64, 8, 1, [0]),
    (1, 16, 2, 512, 16, 3, [2]),
    (3, 16, 2, 512, 8, 2, [1, -1, 0]),
    (5, 8, 1, 1024, 24, 4, [3, 3, -1, 0, 3]),
    (16, 16, 1, 512, 16, 16, list(range(15, -1, -1))),
    (20, 16, 1, 512, 64, 5, [i % 6 - 1 for i in range(20)]),
    (7, 4, 3, 256, 40, 7, [0, 0, 0, 1, 1, 6, 5]),
    (9, 32, 1, 320, 128, 2, [0, 1, 0, 1, -1, 1, 0, 0, 1]),
    (40, 5, 1, 256, 32, 9, [(7 * i) % 10 - 1 for i in range(40)]),
    (70, 3, 1, 128, 16, 70, list(range(70))),
    (4, 16, 1, 512, 16, 2, [-1, -1, -1, -1]),
    (300, 1, 1, 128, 8, 13, [(5 * i) % 14 - 1 for i in range(300)]),
])
def test_projections(batch, block, layers, hidden, rank, adapters, which):
    c = Case(batch, block, layers, hidden, rank, adapters, which, q_heads=8 if block <= 16 else 4, seed=batch)
    bkv, q = c.run()
    c.check(bkv, q)
    c.ws.fill_(0x5a)
    again = c.run()
    assert torch.equal(bkv, again[0]) and torch.equal(q, again[1])
    base = c.base()
    for s, ad in enumerate(which):  # without an adapter: what ls_draft_prologue gives
        if ad < 0:
            assert torch.equal(bkv[s], base[0][s]) and torch.equal(q[s], base[1][s])
    assert c.lib.error() == (F.LS_OK, 0)


def test_large_projection():
    """Qwen3-8B widths, one layer: several whole waves and split boundary tiles."""
    c = Case(18, 16, 1, 4096, 16, 6, [i % 7 - 1 for i in range(18)], kv_heads=8, q_heads=32, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("rank,block", [(8, 16), (16, 5), (64, 16), (24, 32)])
def test_arguments_on_16_byte_boundaries(rank, block):
    """The documented alignment is 16 bytes: the same bits as from more aligned arguments."""
    c = Case(5, block, 2, 320, rank, 3, [2, 0, -1, 2, 1], q_heads=4, seed=11)
    want = c.run()
    c.check(*want)

    def moved(t):
        m = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape).copy_(t)
        assert m.data_ptr() % 32 == 16
        return m

    for names in (("x",), ("a_q",), ("a_kv",), ("x", "a_q", "b_q", "a_kv", "b_kv", "w_q", "w_kv")):
        kept = {n: getattr(c, n) for n in names}
        for n, t in kept.items():
            setattr(c, n, moved(t))
        c.desc = F.make_lora(c.na, c.r, c.a_q, c.b_q, c.a_kv, c.b_kv, c.scale, c.which)
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for n, t in kept.items():
            setattr(c, n, t)
    assert c.lib.error() == (F.LS_OK, 0)


def test_adapters_do_not_reach_other_sequences():
    """An adapter with infinities and NaN changes its own sequences only."""
    which = [0, 1, -1, 2, 1, 0, 2]
    c = Case(7, 5, 2, 512, 16, 3, which, seed=5)
    bkv, q = c.run()
    for t in (c.a_q, c.b_q, c.a_kv, c.b_kv):
        t[1, :, ::3] = float("nan")
        t[1, :, 1::3] = float("inf")
    b2, q2 = c.run()
    for s, ad in enumerate(which):
        if ad == 1:
            assert q2[s].isnan().any() and b2[s].isnan().any()
        else:
            assert torch.equal(bkv[s], b2[s]) and torch.equal(q[s], q2[s])
    assert c.lib.error() == (F.LS_OK, 0)


def test_ids_out_of_range_are_flagged():
    c = Case(4, 16, 1, 512, 16, 2, [0, 2, -2, 1], seed=6)
    bkv, q = c.run()
    assert c.lib.error()[1] == F.LS_DEVERR_ADAPTER
    c.lib.clear()
    base = c.base()
    for s in (1, 2):
        assert torch.equal(bkv[s], base[0][s]) and torch.equal(q[s], base[1][s])
    c.which.copy_(torch.tensor([0, -1, -1, 1]))
    again = c.run()
    assert torch.equal(bkv, again[0]) and torch.equal(q, again[1])
    assert c.lib.error() == (F.LS_OK, 0)


def test_ids_and_weights_written_just_before():
    """The adapters' ids, weights and the inputs written by the kernels right before the call."""
    c = Case(16, 16, 1, 1024, 16, 4, [0] * 16, seed=7)
    want = [(i * 3) % 5 - 1 for i in range(16)]
    new = torch.tensor(want, dtype=torch.int32, device="cuda")
    flip = -c.a_q
    c.check(*c.run())
    for _ in range(20):
        c.which.zero_()
        c.a_q.neg_()
        c.run()
        c.a_q.copy_(flip)
        c.which.copy_(new)
        bkv, q = c.run()
    c.check(bkv, q)


def test_two_streams_and_captured():
    c = Case(6, 16, 1, 512, 16, 3, [0, 1, 2, -1, 2, 0], seed=8)
    want = c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        got = c.run(side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    c.which.copy_(torch.tensor([2, -1, 0, 0, 1, 1]))
    c.x.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    c.check(*got)


def test_refusals():
    c = Case(2, 16, 1, 512, 16, 2, [0, 1])
    bkv, q = c.outputs()
    lib, na, r = c.lib, 2, 16
    inv, shape, uns = F.LS_ERR_INVALID_ARG, F.LS_ERR_SHAPE, F.LS_ERR_UNSUPPORTED
    good = [na, r, c.a_q, c.b_q, c.a_kv, c.b_kv, c.scale, c.which]

    def call(status, desc, ws=c.ws, wsb=c.ws.numel(), x=c.x, bkv=bkv):
        refused(status, F.ls_draft_prologue_lora, lib.st, c.w_kv, c.w_q, x, desc, bkv, q, ws, wsb)

    for at in range(2, 8):
        call(inv, F.make_lora(*[None if i == at else v for i, v in enumerate(good)]))
        call(inv, F.make_lora(*[v.data_ptr() + 8 if i == at else v for i, v in enumerate(good)]))
    call(inv, F.make_lora(0, *good[1:]))
    for bad in (0, 4, 12, 136):
        call(uns, F.make_lora(na, bad, *good[2:]))
    call(shape, c.desc, wsb=c.ws.numel() - 1)
    call(inv, c.desc, ws=None)
    call(inv, c.desc, ws=c.ws.data_ptr() + 16)
    call(inv, c.desc, x=None)
    call(inv, c.desc, bkv=bkv.data_ptr() + 2)
    f32 = Lib(dtype="f32", dim=64, q_heads=4)
    refused(uns, F.ls_draft_prologue_lora, f32.st, c.w_kv, c.w_q, c.x, c.desc, bkv, q, c.ws, c.ws.numel())
    assert lib.error() == (F.LS_OK, 0)
