"""A serving round of ragged requests as an engine would make it from the library's calls: pages
taken for the prompts and for each round's rows, rows written into the 4-bit cache by the slots
that came with them, the verification attention over the cache, the rows read back as the
commit's input, pages behind the accepted rows returned, the projections with every request's
adapter, the drafter's attention. The steps are compared with the oracle and with the same round
on dense rows; the whole round captured into one graph gives the bits of the eager calls."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fixed_cost_drafter_b200 as F
    import oracle as O
    from tests.serving_side import Lib

PS, L, H, HQ, D, HID, B = 16, 2, 2, 8, 128, 512, 16
SCALE = D ** -0.5


class Engine:
    def __init__(self, prompts, rounds, seed=0):
        b = self.b = len(prompts)
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lib = Lib(batch=b, layers=L, kv_heads=H, q_heads=HQ, dim=D, hidden=HID, block=B)
        self.mb = -(-(max(prompts) + rounds * (B + 1) + B + 1) // PS)
        self.num = b * self.mb
        self.table = torch.full((b, self.mb), -1, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(b, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.num, generator=g, device="cuda").int()
        self.count = torch.tensor([self.num], dtype=torch.int32, device="cuda")
        self.pool = F.make_page_pool(self.table, self.held, self.free, self.count, self.mb, PS, self.num)
        per = F.ls_kv4_page_bytes(self.lib.cfg, PS)
        self.cache = [torch.zeros(self.num, per, dtype=torch.uint8, device="cuda") for _ in range(L)]
        self.kv = F.make_paged_kv4(self.cache, per, self.table, self.mb, PS, self.num)
        self.ws = torch.empty(F.ls_verify_workspace_bytes(self.lib.cfg, B + 1), dtype=torch.uint8, device="cuda")
        n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)
        self.w_kv, self.w_q = n(L, 2 * H * D, HID, std=HID ** -0.5), n(L, HQ * D, HID, std=HID ** -0.5)
        bank = [n(3, L, 16, HID, std=HID ** -0.5), n(3, L, HQ * D, 16), n(3, L, 16, HID, std=HID ** -0.5), n(3, L, 2 * H * D, 16)]
        self.which = torch.tensor([(2 * i) % 4 - 1 for i in range(b)], dtype=torch.int32, device="cuda")
        self.bank = bank + [torch.rand(3, generator=g, device="cuda"), self.which]
        self.lora = F.make_lora(3, 16, *self.bank)
        self.lora_ws = torch.empty(F.ls_lora_workspace_bytes(self.lib.cfg, 16), dtype=torch.uint8, device="cuda")
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
        # one round's buffers
        self.rows = n(b, L, B + 1, (HQ + 2 * H) * D)  # the target's packed q, k, v of the verify rows
        self.hidden, self.x = n(b, L, B + 1, HID), n(b, L, B, HID)
        self.slots, self.new_len = z(b, B + 1, t=torch.int64), z(b, t=torch.int64)
        self.att = z(b, L, B + 1, HQ * D)
        self.vk, self.vv = z(b, L, B + 1, H, D), z(b, L, B + 1, H, D)
        self.draft = torch.randint(0, 50, (b, B), generator=g, device="cuda", dtype=torch.int32)
        self.target = torch.cat([self.draft, self.draft[:, :1]], 1).contiguous()
        self.acc, self.next = z(b, t=torch.int32), z(b, t=torch.int32)
        self.bkv, self.q, self.out = z(b, L, 2 * H * D), z(b, L, B, HQ * D), z(b, L, B, HQ, D)
        self._admit(prompts)

    def _admit(self, prompts):
        b, most = self.b, max(prompts)
        zero = torch.zeros(b, dtype=torch.int64, device="cuda")
        rows = torch.tensor(prompts, dtype=torch.int32, device="cuda")
        begin = torch.zeros(b + 1, dtype=torch.int64, device="cuda")
        total = sum(prompts)
        slots = torch.full((total,), -5, dtype=torch.int64, device="cuda")
        F.ls_pages_extend(self.lib.st, self.pool, zero, rows, most, begin, slots, total)
        packed = torch.randn(L, total, 2 * H, D, generator=self.g, device="cuda").to(torch.bfloat16)
        k = torch.zeros(b, L, most, H, D, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        for l in range(L):
            F.ls_kv4_append(self.lib.st, self.kv, l, packed[l], packed[l, :, H:], 2 * H * D, slots, total)
            for i, p in enumerate(prompts):  # what the cache holds of them becomes the state's prefix
                if p:
                    at = slots[int(begin[i]):]
                    F.ls_kv4_read_rows(self.lib.st, self.kv, l, at, p, k[i, l], v[i, l], H * D)
        self.prefix = torch.tensor(prompts, dtype=torch.int64, device="cuda")
        ws = torch.empty(F.ls_prefill_workspace_bytes(self.lib.cfg, 0, most), dtype=torch.uint8, device="cuda")
        last = torch.randn(b, L, HID, generator=self.g, device="cuda").to(torch.bfloat16)
        F.ls_prefill_summary(self.lib.st, k, v, most * H * D, H * D, self.prefix, 0, most, last, ws, ws.numel())
        self.length = self.prefix.clone()  # the engine's own copy, on the device

    def round(self, stream=None):
        st = self.lib.st
        F.ls_pages_extend(st, self.pool, None, None, B + 1, None, self.slots, self.slots.numel(), stream)
        qkv = (HQ + 2 * H) * D
        for l in range(L):
            for i in range(self.b):
                base = self.rows[i, l]
                F.ls_kv4_append(st, self.kv, l, base[:, HQ * D:], base[:, (HQ + H) * D:], qkv, self.slots[i], B + 1, stream)
        torch.add(self.length, B + 1, out=self.new_len)
        for l in range(L):  # one layer's queries of all sequences, packed
            q = self.rows[:, l].contiguous()
            out = torch.zeros(self.b, B + 1, HQ * D, dtype=torch.bfloat16, device="cuda")
            F.ls_verify_attend_kv4(st, self.kv, l, q, qkv, B + 1, None, self.new_len, SCALE, out, self.ws, self.ws.numel(), stream)
            self.att[:, l] = out
            for i in range(self.b):
                F.ls_kv4_read_rows(st, self.kv, l, self.slots[i], B + 1, self.vk[i, l], self.vv[i, l], H * D, stream)
        F.ls_commit_round(st, self.draft, self.target, self.vk, self.vv, self.hidden, self.acc, self.next, stream)
        self.length.add_(self.acc).add_(1)
        F.ls_pages_trim(st, self.pool, None, stream)
        F.ls_draft_prologue_lora(st, self.w_kv, self.w_q, self.x, self.lora, self.bkv, self.q, self.lora_ws, self.lora_ws.numel(), stream)
        F.ls_draft_attend(st, 0, L, self.q, self.bkv, self.bkv[:, :, H * D:], 2 * H * D, SCALE, self.out, stream)

    def reject(self, seed):
        """The target disagrees at a random place of every block."""
        g = torch.Generator().manual_seed(seed)
        cut = torch.randint(0, B + 1, (self.b,), generator=g)
        t = torch.cat([self.draft, self.draft[:, :1]], 1)
        for i, c in enumerate(cut.tolist()):
            if c < B:
                t[i, c] += 1
        self.target.copy_(t)
        return cut.tolist()

    def snapshot(self):
        return [t.clone() for t in (self.table, self.held, self.count, self.free[:int(self.count)], self.slots, self.att, self.vk, self.vv,
                                    self.acc, self.bkv, self.q, self.out, self.lib.arena, *self.cache)]


def _f64(t):
    return t.double().cpu().numpy()


def test_rounds_against_the_oracle():
    prompts = [40, 300, 1, 129]
    e = Engine(prompts, 4)
    lens = list(prompts)
    for r in range(4):
        cut = e.reject(r)
        e.round()
        torch.cuda.synchronize()
        table, slots = e.table.cpu().numpy(), e.slots.cpu().numpy()
        for i in range(e.b):
            # slots follow the table, pages are whole and nobody else's, those behind are returned
            assert len(set(slots[i])) == B + 1 and (slots[i] >= 0).all()
            keep = -(-(lens[i] + cut[i] + 1) // PS)
            assert int(e.held[i]) == keep and (table[i, keep:] == -1).all() and (table[i, :keep] >= 0).all()
            for l in range(L):
                # rows the cache holds, before the new ones and with them
                cache = e.cache[l].cpu().numpy()
                # (pages of rejected rows are returned, their contents stay until they are taken again)
                at = [table[i, t // PS] * PS + t % PS for t in range(lens[i])] + list(slots[i])
                k = np.stack([np.stack([O.kv4_row(cache, s, h, PS, D)[0] for h in range(H)]) for s in at])
                v = np.stack([np.stack([O.kv4_row(cache, s, h, PS, D)[1] for h in range(H)]) for s in at])
                assert np.array_equal(_f64(e.vk[i, l]), k[lens[i]:]) and np.array_equal(_f64(e.vv[i, l]), v[lens[i]:])
                rows = _f64(e.rows[i, l])
                want = O.kv4_decode(*O.kv4_encode(rows[:, HQ * D:(HQ + H) * D].reshape(B + 1, H, D)))
                assert np.array_equal(k[lens[i]:], want)
                ref, mass, _ = O.attend_rows(rows[:, :HQ * D].reshape(B + 1, HQ, D), k, v, lens[i], SCALE)
                got = _f64(e.att[i, l]).reshape(B + 1, HQ, D)
                # bf16 output, fp16 weights; logits of at most a few tens: 2 x 136 x 2^-24 x |logit| terms
                assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * mass + 1e-6).all()
        assert e.acc.tolist() == cut
        lens = [n + c + 1 for n, c in zip(lens, cut)]
        assert e.length.tolist() == lens
        ctr = e.lib.arena[: e.b * L * 3 * 8].view(torch.int64).view(e.b, L, 3)
        assert ctr[:, :, 0].tolist() == [[n] * L for n in lens]
        held = [p for i in range(e.b) for p in e.table[i, :int(e.held[i])].tolist()]
        free = e.free[:int(e.count)].tolist()
        assert sorted(held + free) == list(range(e.num))
    assert e.lib.error() == (F.LS_OK, 0)


def test_the_state_is_that_of_dense_rows():
    """The state after a round on rows read back from the cache equals one committed with the same
    rows handed over densely."""
    e, d = Engine([50, 17], 2, seed=3), Engine([50, 17], 2, seed=3)
    for r in range(2):
        e.reject(10 + r)
        d.reject(10 + r)
        e.round()
        F.ls_commit_round(d.lib.st, d.draft, d.target, e.vk, e.vv, d.hidden, d.acc, d.next)
    y = F.ls_get_layout(e.lib.cfg)
    assert torch.equal(e.lib.arena[:y.off_error], d.lib.arena[:y.off_error])
    assert torch.equal(e.lib.arena[y.off_kv:y.off_sample], d.lib.arena[y.off_kv:y.off_sample])


def test_a_captured_round_replays_like_the_eager_one():
    a, c = Engine([33, 260, 5], 4, seed=7), Engine([33, 260, 5], 4, seed=7)
    a.reject(0)
    c.reject(0)
    a.round()
    c.round()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        c.round(side)
    for r in range(1, 4):
        for e in (a, c):
            e.reject(r)
            e.rows.mul_(-0.5 * r)
            e.x.add_(0.25)
        a.round()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.snapshot(), c.snapshot()):
            assert torch.equal(x, y)
    assert a.lib.error() == (F.LS_OK, 0) and c.lib.error() == (F.LS_OK, 0)
