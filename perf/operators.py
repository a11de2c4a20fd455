"""The serving-side operators around a drafting round, as measured cases: page tables and slot
maps from request lengths, a paged KV cache held in 4 bits (rows written and read back, attention
of verify rows and of single tokens over it), and the drafter's projections with every request's
own low-rank adapter. Each has a plain torch form in 32 bits, the library's call, and a 64-bit
definition to compare both with."""

import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# Shapes of the repository's workloads: Qwen3-8B/4B heads, and the small fp32 configuration.
HEADS = {
    "qwen3": dict(kv_heads=8, q_heads=32, dim=128, dtype="bf16"),
    "mid": dict(kv_heads=2, q_heads=8, dim=128, dtype="bf16"),
    "narrow": dict(kv_heads=4, q_heads=16, dim=64, dtype="bf16"),
    "tiny": dict(kv_heads=2, q_heads=4, dim=64, dtype="f32"),
}


def listed():
    return [
        # one request alone, a drafting round of 16 + 1 rows: latency of the two calls
        dict(name="pages_round_b1", op="pages", batch=1, rows=17, lo=700, hi=5000, page=16, packed=False),
        # 16 requests at a 64K prefix, ragged, one round: pages taken for the verify rows, then trimmed
        dict(name="pages_round_b16", op="pages", batch=16, rows=17, lo=61000, hi=66000, page=16, packed=False),
        # admission of 64 requests with whole prompts up to 128K: packed slot map, pages returned at the end
        dict(name="pages_admit_b64", op="pages", batch=64, rows=131072, lo=0, hi=0, page=16, packed=True),
        # the verify rows of a round (16 requests x 17 rows) written into the cache and read back
        dict(name="rows_round", op="rows", heads="qwen3", n=272, page=16, stride_heads=48),
        # a prefill chunk of 16 x 4096 rows
        dict(name="rows_chunk", op="rows", heads="qwen3", n=65536, page=32, stride_heads=8),
        # one short request, a single token: latency
        dict(name="attend_token_b1", op="attend", heads="qwen3", batch=1, rows=1, lo=4001, hi=4001, page=16),
        # decoding 16 ragged requests at 48K-64K
        dict(name="attend_token_b16", op="attend", heads="qwen3", batch=16, rows=1, lo=49152, hi=65536, page=16),
        # the verification pass of 16 requests at 32K-64K: 17 rows each
        dict(name="attend_verify_b16", op="attend", heads="qwen3", batch=16, rows=17, lo=32768, hi=65536, page=16),
        # few rows of a small model, odd lengths
        dict(name="attend_verify_narrow", op="attend", heads="narrow", batch=5, rows=9, lo=3, hi=3333, page=64),
        # fp32 queries of the small configuration
        dict(name="attend_f32", op="attend", heads="tiny", batch=3, rows=5, lo=1, hi=700, page=16),
        # the drafting round of 16 requests, each with an adapter of its own, rank 16
        dict(name="lora_b16_r16", op="lora", batch=16, block=16, layers=4, hidden=4096, heads="qwen3", rank=16,
             adapters=16, share=0.0),
        # 64 requests over 24 adapters of rank 64, a quarter of them without one
        dict(name="lora_b64_r64", op="lora", batch=64, block=16, layers=4, hidden=4096, heads="qwen3", rank=64,
             adapters=24, share=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    # blocks of up to 16 drafts: a state holds up to 64 query rows (block x heads per KV head) of a KV head
    op = rng.choice(["pages", "rows", "attend", "attend", "lora"])
    if op == "pages":
        if rng.random() < 0.5:
            lo = _log(rng, 1, 60000)
            return dict(op="pages", batch=_log(rng, 1, 64), rows=rng.randint(1, 33), lo=lo, hi=lo + _log(rng, 1, 8000),
                        page=rng.choice([8, 16, 24, 32, 64]), packed=rng.random() < 0.3)
        return dict(op="pages", batch=_log(rng, 1, 64), rows=_log(rng, 50, 60000), lo=0, hi=rng.choice([0, 777]),
                    page=rng.choice([16, 32, 48, 128]), packed=True)
    if op == "rows":
        heads = rng.choice(sorted(HEADS))
        return dict(op="rows", heads=heads, n=_log(rng, 1, 40000), page=rng.choice([16, 32, 64, 128]),
                    stride_heads=HEADS[heads]["kv_heads"] * rng.choice([1, 2, 6]))
    if op == "attend":
        heads = rng.choice(["qwen3", "qwen3", "mid", "narrow", "tiny"])
        batch = _log(rng, 1, 32)
        hi = _log(rng, 1, max(2, min(90000, 400000 // batch) if heads != "tiny" else 2000))
        return dict(op="attend", heads=heads, batch=batch, rows=rng.choice([1, 1, 2, 5, 9, 17, 17]),
                    lo=rng.randint(0, hi), hi=hi, page=rng.choice([16, 16, 32, 64, 128]))
    batch = _log(rng, 1, 48)
    return dict(op="lora", batch=batch, block=rng.choice([1, 4, 8, 16, 16]), layers=rng.randint(1, 4),
                hidden=rng.choice([512, 1024, 2560, 4096]), heads=rng.choice(["mid", "qwen3"]),
                rank=rng.choice([8, 16, 24, 32, 64]), adapters=rng.randint(1, 24), share=rng.choice([0.0, 0.3]))


class State:
    """What a program keeps between calls: tensors, and the library's handle where it is used."""

    def __init__(self, **kw):
        self.__dict__.update(kw)

    def __del__(self):
        if getattr(self, "handle", None) is not None:
            self.lib.ls_destroy_state(self.handle)


def _library_state(s, batch, layers, heads, hidden, block):
    import fixed_cost_drafter_b200 as F
    h = HEADS[heads]
    cfg = F.make_config(batch=batch, n_layers=layers, n_kv_heads=h["kv_heads"], n_q_heads=h["q_heads"], head_dim=h["dim"],
                        hidden=hidden, block=block, window=64, scales=[64, 512], slots_per_scale=4,
                        dtype=F.LS_BF16 if h["dtype"] == "bf16" else F.LS_F32)
    s.lib, s.cfg = F, cfg
    s.arena = torch.empty(F.ls_state_bytes(cfg), dtype=torch.uint8, device=DEV)
    s.handle = F.ls_init_state(cfg, s.arena, s.arena.numel())


def _lengths(g, case):
    """Ragged lengths in [lo, hi], on the host and the device."""
    n = torch.randint(case["lo"], case["hi"] + 1, (case["batch"],), generator=g)
    return n, n.to(DEV)


def _host(seed):
    return torch.Generator().manual_seed(seed)


def _dev(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    return {"pages": _prepare_pages, "rows": _prepare_rows, "attend": _prepare_attend, "lora": _prepare_lora}[case["op"]](case, seed)


def run(s):
    if own:
        return {"pages": _own_pages, "rows": _own_rows, "attend": _own_attend, "lora": _own_lora}[s.op](s)
    return {"pages": _plain_pages, "rows": _plain_rows, "attend": _plain_attend, "lora": _plain_lora}[s.op](s)


def exact(case, seed):
    if case["op"] == "pages":  # whole numbers only
        return None
    return {"rows": _exact_rows, "attend": _exact_attend, "lora": _exact_lora}[case["op"]](prepare(case, seed))


def work(case):
    if case["op"] == "pages":
        # expected sizes: rows uniform in [1, rows] when packed, else all of them; every slot written,
        # every page id moved twice each way (taken, returned) where the round does not keep it
        b, ps = case["batch"], case["page"]
        rows = b * (case["rows"] + 1) / 2 if case["packed"] else b * case["rows"]
        pages = rows / ps + b / 2
        return {"bytes": 8 * rows + b * 44 + 16 * pages, "flops": 0}
    h = HEADS[case["heads"]]
    e = 2 if h["dtype"] == "bf16" else 4
    if case["op"] == "rows":
        elems = 2 * case["n"] * h["kv_heads"] * h["dim"]
        return {"bytes": elems * (2 * e + 2 * 9 / 16) + 8 * case["n"], "flops": 4 * elems}
    if case["op"] == "attend":
        tokens = case["batch"] * (case["lo"] + case["hi"]) / 2
        io = case["batch"] * case["rows"] * h["q_heads"] * h["dim"] * 2 * e
        return {"bytes": tokens * h["kv_heads"] * h["dim"] * 2 * 9 / 16 + io,
                "flops": 4 * tokens * case["rows"] * h["q_heads"] * h["dim"]}
    L, H, b, B, r = case["layers"], case["hidden"], case["batch"], case["block"], case["rank"]
    nq, nkv = h["q_heads"] * h["dim"], 2 * h["kv_heads"] * h["dim"]
    used = case["adapters"] * (1 - (1 - (1 - case["share"]) / case["adapters"]) ** b)
    with_one = b * (1 - case["share"])
    return {"bytes": 2 * L * (H * (nq + nkv) + used * r * (2 * H + nq + nkv) + b * B * (H + nq) + b * (H + nkv)),
            "flops": 2 * L * (b * B * H * nq + b * H * nkv + with_one * r * (B * (H + nq) + H + nkv))}


# ---- pages: block tables and slot maps ---------------------------------------------------

def _prepare_pages(case, seed):
    g = _host(seed)
    b, ps = case["batch"], case["page"]
    length, d_length = _lengths(g, case)
    if case["packed"]:
        rows = torch.randint(1, case["rows"] + 1, (b,), generator=g, dtype=torch.int32)
    else:
        rows = torch.full((b,), case["rows"], dtype=torch.int32)
    # what stays after the round: a few accepted rows of it, or nothing once an admitted batch is done
    kept = torch.minimum(torch.randint(1, 6, (b,), generator=g), rows) if case["hi"] else -length
    held = -(-length // ps)
    max_blocks = -(-(case["hi"] + case["rows"]) // ps) + 2
    num_pages = b * max_blocks + 17
    ids = torch.randperm(num_pages, generator=_dev(seed), device=DEV).int()
    first = (torch.cumsum(held, 0) - held).to(DEV)
    n_held = int(held.sum())
    j = torch.arange(max_blocks, device=DEV)
    d_held = held.to(DEV)
    at = (first[:, None] + j).clamp(max=num_pages - 1)
    table = torch.where(j < d_held[:, None], ids[at], torch.full_like(ids[at], -1)).contiguous()
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    free[: num_pages - n_held] = ids[n_held:]
    total = int(rows.sum())
    s = State(op="pages", case=case, length=d_length, rows=rows.to(DEV), after=(length + kept).to(DEV), max_rows=case["rows"],
              table=table, held=d_held.int(), free=free, page=ps, num_pages=num_pages, total=total,
              count=torch.tensor([num_pages - n_held], dtype=torch.int32, device=DEV),
              row_begin=torch.zeros(b + 1, dtype=torch.int64, device=DEV) if case["packed"] else None,
              slots=torch.full((b * case["rows"],) if case["packed"] else (b, case["rows"]), -1, dtype=torch.int64, device=DEV))
    if own:
        _library_state(s, b, 1, "mid", 512, 16)
        s.pool = s.lib.make_page_pool(s.table, s.held, s.free, s.count, max_blocks, ps, num_pages)
    return s


def _pages_out(s):
    return {"slots": s.slots, "table": s.table, "held": s.held, "free": s.free, "count": s.count,
            "row_begin": s.row_begin if s.row_begin is not None else s.held}


def _own_pages(s):
    s.lib.ls_pages_extend(s.handle, s.pool, s.length, s.rows, s.max_rows, s.row_begin, s.slots, s.slots.numel())
    s.lib.ls_pages_trim(s.handle, s.pool, s.after)
    return _pages_out(s)


def _plain_pages(s):
    ps, b = s.page, s.length.numel()
    j = torch.arange(s.table.shape[1], device=DEV)
    # extend: the pages that the new rows need come off the end of the free list, in order of the requests
    target = (s.length + s.rows + ps - 1) // ps
    need = (target - s.held).clamp(min=0)
    before = torch.cumsum(need, 0) - need
    served = before + need <= s.count
    new = served[:, None] & (j >= s.held[:, None]) & (j < target[:, None])
    src = (s.count - 1 - (before[:, None] + j - s.held[:, None])).clamp(0, s.num_pages - 1)
    s.table.copy_(torch.where(new, s.free[src], s.table))
    s.held.copy_(torch.where(served, torch.maximum(s.held, target), s.held))
    s.count.sub_((need * served).sum().int())
    if s.row_begin is not None:
        s.row_begin[1:] = torch.cumsum(s.rows, 0)
        r = torch.arange(s.total, device=DEV)
        seq = torch.searchsorted(s.row_begin[1:], r, right=True)
        pos = s.length[seq] + r - s.row_begin[seq]
        slot = s.table[seq, pos // ps].long() * ps + pos % ps
        s.slots[: s.total].copy_(torch.where(served[seq], slot, -1))
    else:
        i = torch.arange(s.slots.shape[1], device=DEV)
        pos = s.length[:, None] + i
        slot = s.table.gather(1, (pos // ps).clamp(max=s.table.shape[1] - 1)).long() * ps + pos % ps
        s.slots.copy_(torch.where((i < s.rows[:, None]) & served[:, None], slot, -1))
    # trim: pages past the lengths that stay go back to the end of the free list
    keep = (s.after + ps - 1) // ps
    back = (s.held - keep).clamp(min=0)
    before = torch.cumsum(back, 0) - back
    total = back.sum()
    gone = (j >= keep[:, None]) & (j < s.held[:, None])
    dst = torch.where(gone, s.count + total - 1 - (before[:, None] + j - keep[:, None]), s.num_pages)
    free = torch.cat([s.free, s.free[:1]])
    free.scatter_(0, dst.reshape(-1), s.table.reshape(-1))
    s.free.copy_(free[:-1])
    s.table.masked_fill_(gone, -1)
    s.held.copy_(torch.minimum(s.held, keep.int()))
    s.count.add_(total.int())
    return _pages_out(s)


# ---- the 4-bit cache ------------------------------------------------------------------------
# A page of a layer holds, per KV head, [K codes][V codes][K scales][V scales]: codes are e2m1 pairs
# (element 2i in the low half of byte i), scales e4m3, one per 16 elements of a row.

def _page_views(cache, page, dim):
    """(K codes, V codes, K scales, V scales) of cache uint8 [pages][heads][page * dim * 9 / 8]."""
    c, sc = page * dim // 2, page * dim // 16
    p, h = cache.shape[:2]
    return (cache[:, :, :c].view(p, h, page, dim // 2), cache[:, :, c:2 * c].view(p, h, page, dim // 2),
            cache[:, :, 2 * c:2 * c + sc].view(p, h, page, dim // 16), cache[:, :, 2 * c + sc:].view(p, h, page, dim // 16))


def _prepare_rows(case, seed):
    h, g = HEADS[case["heads"]], _dev(seed)
    n, ps, D, kv = case["n"], case["page"], h["dim"], h["kv_heads"]
    dtype = torch.bfloat16 if h["dtype"] == "bf16" else torch.float32
    # keys have a few channels much larger than the rest, values are even; rows lie in the projections' packed output
    wide = 1 + 7 * (torch.rand(D, generator=g, device=DEV) < 0.04)
    rows = torch.randn(n, case["stride_heads"], D, generator=g, device=DEV)
    k = (rows * wide).to(dtype)[:, :kv]
    v = torch.randn(n, case["stride_heads"], D, generator=g, device=DEV).to(dtype)[:, :kv]
    pages = -(-n // ps) + 3
    # each row's slot: consecutive places in pages of no order
    perm = torch.randperm(pages, generator=g, device=DEV)
    i = torch.arange(n, device=DEV) + int(torch.randint(0, ps, (1,), generator=_host(seed)))
    slots = perm[i // ps] * ps + i % ps
    s = State(op="rows", case=case, k=k, v=v, slots=slots, page=ps, dim=D, n=n,
              cache=torch.zeros(pages, kv, ps * D * 9 // 8, dtype=torch.uint8, device=DEV),
              k_out=torch.empty(n, kv, D, dtype=dtype, device=DEV), v_out=torch.empty(n, kv, D, dtype=dtype, device=DEV))
    if own:
        _library_state(s, 1, 1, case["heads"], 512, 16)
        s.kv4 = s.lib.make_paged_kv4([s.cache], s.cache.stride(0), None, 1, ps, pages)
    return s


def _own_rows(s):
    s.lib.ls_kv4_append(s.handle, s.kv4, 0, s.k, s.v, s.k.stride(0), s.slots, s.n)
    s.lib.ls_kv4_read_rows(s.handle, s.kv4, 0, s.slots, s.n, s.k_out, s.v_out, s.k_out.stride(0))
    return {"k": s.k_out, "v": s.v_out}


def _encode(x):
    """Codes (uint8, two per byte) and scales (uint8, e4m3) of rows [n][heads][dim]."""
    n, h, d = x.shape
    x = x.float().view(n, h, d // 16, 16)
    top = x.abs().amax(-1)
    scale = torch.where(top.isfinite(), (top / 6).clamp(max=448), math.nan).to(torch.float8_e4m3fn)
    sf = scale.float()[..., None]
    y = (x / torch.where(sf > 0, sf, 1.0)) * (sf > 0)
    m = y.abs()
    # halves go to the even code
    code = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)) | ((y < 0).byte() << 3)
    code = code.view(n, h, d)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _decode(codes, scales):
    """fp32 values [..., dim] of codes [..., dim / 2] and scales [..., dim / 16] (both bytes)."""
    lut = torch.tensor(E2M1, device=DEV)
    lut = torch.cat([lut, -lut])
    byte = torch.arange(256, device=DEV)
    pair = torch.stack([lut[byte & 15], lut[byte >> 4]], -1)
    x = pair[codes.int()].view(*scales.shape, 16)
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_rows(s):
    kc, vc, ks, vs = _page_views(s.cache, s.page, s.dim)
    page, off = s.slots // s.page, s.slots % s.page
    kc[page, :, off], ks[page, :, off] = _encode(s.k)
    vc[page, :, off], vs[page, :, off] = _encode(s.v)
    s.k_out.copy_(_decode(kc[page, :, off], ks[page, :, off]))
    s.v_out.copy_(_decode(vc[page, :, off], vs[page, :, off]))
    return {"k": s.k_out, "v": s.v_out}


def _exact_rows(s):
    def nearest(x, digits, low, top):
        """x >= 0 on the grid of floats with `digits` fraction bits, least exponent `low`, largest value `top`; halves to even."""
        e = torch.floor(torch.log2(x.clamp(min=2.0 ** (low - 8)))).clamp(min=low)
        e = torch.where(x >= torch.exp2(e + 1), e + 1, torch.where(x < torch.exp2(e), (e - 1).clamp(min=low), e))
        step = torch.exp2(e - digits)
        return (torch.round(x / step) * step).clamp(max=top)

    def held(x):
        n, h, d = x.shape
        g = x.double().view(n, h, d // 16, 16)
        sc = nearest(g.abs().amax(-1, keepdim=True) / 6, 3, -6, 448.0)
        y = nearest(g.abs() / torch.where(sc > 0, sc, 1.0), 1, 0, 6.0)
        return (torch.sign(g) * y * sc).view(n, h, d)

    return {"k": held(s.k), "v": held(s.v)}


# ---- attention over the 4-bit cache --------------------------------------------------------

def _prepare_attend(case, seed):
    h, g = HEADS[case["heads"]], _dev(seed)
    b, n, ps, D, kv, hq = case["batch"], case["rows"], case["page"], h["dim"], h["kv_heads"], h["q_heads"]
    dtype = torch.bfloat16 if h["dtype"] == "bf16" else torch.float32
    length, d_length = _lengths(_host(seed), case)
    rows = torch.full((b,), n, dtype=torch.int32)
    if n > 2:  # a request near its end drafts fewer rows
        rows[-1] = max(1, n // 2)
    blocks = -(-length // ps)
    max_blocks = int(blocks.max()) + 1
    used = int(blocks.sum())
    pages = used + 5
    perm = torch.randperm(pages, generator=g, device=DEV).int()
    j = torch.arange(max_blocks, device=DEV)
    first = (torch.cumsum(blocks, 0) - blocks).to(DEV)
    table = torch.where(j < blocks.to(DEV)[:, None], perm[(first[:, None] + j).clamp(max=pages - 1)], -1).int().contiguous()
    # codes as a group of 16 normal numbers scaled to its largest gives them; scales around 2 / 6
    weight = torch.tensor([16, 26, 24, 20, 27, 20, 13, 8], device=DEV, dtype=torch.float32)
    nib = torch.repeat_interleave(torch.arange(8, device=DEV, dtype=torch.uint8), (weight * 128 / weight.sum()).round().long())
    nib = torch.cat([nib, nib | 8])
    pick = nib[torch.linspace(0, nib.numel() - 1, 256, device=DEV).round().long()]
    cache = torch.empty(pages, kv, ps * D * 9 // 8, dtype=torch.uint8, device=DEV)
    c = ps * D
    step = max(1, (1 << 28) // (kv * c))
    for at in range(0, pages, step):
        part = cache[at:at + step]
        lo, hi = (torch.randint(0, 256, (part.shape[0], kv, c), generator=g, device=DEV, dtype=torch.uint8).int() for _ in range(2))
        part[:, :, :c] = pick[lo] | (pick[hi] << 4)
        scale = 0.33 * torch.exp(0.3 * torch.randn(part.shape[0], kv, c // 8, generator=g, device=DEV))
        part[:, :, c:] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(b, n, hq + 2 * kv, D, generator=g, device=DEV).to(dtype)  # the packed projections' output
    s = State(op="attend", case=case, q=q, n=n, rows=rows.to(DEV), length=d_length, table=table, cache=cache, page=ps,
              dim=D, kv=kv, hq=hq, scale=1 / math.sqrt(D), most=int(length.max()), out=torch.zeros(b, n, hq, D, dtype=dtype, device=DEV))
    if own:
        _library_state(s, b, 1, case["heads"], 512, max(1, min(32, n - 1)))
        s.kv4 = s.lib.make_paged_kv4([cache], cache.stride(0), table, max_blocks, ps, pages)
        s.ws = torch.empty(s.lib.ls_verify_workspace_bytes(s.cfg, n), dtype=torch.uint8, device=DEV)
    return s


def _own_attend(s):
    s.lib.ls_verify_attend_kv4(s.handle, s.kv4, 0, s.q, s.q.stride(1), s.n, s.rows, s.length, s.scale, s.out, s.ws, s.ws.numel())
    return s.out


def _plain_attend(s):
    b, kv, D, n, ps = s.length.numel(), s.kv, s.dim, s.n, s.page
    blocks = max(1, -(-s.most // ps))
    at = s.table[:, :blocks].clamp(min=0).long()
    kc, vc, ks, vs = _page_views(s.cache, ps, D)
    k = _decode(kc[at], ks[at]).transpose(1, 2).reshape(b, kv, blocks * ps, D)
    q = s.q[:, :, :s.hq].float().view(b, n, kv, s.hq // kv, D).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, D)
    t = torch.arange(blocks * ps, device=DEV)
    last = s.length[:, None] - s.rows[:, None] + torch.arange(n, device=DEV)  # [b][n]: the row's own position
    seen = t <= last[..., None]
    x = (q @ k.transpose(-1, -2)).mul_(s.scale).view(b, kv, s.hq // kv, n, -1)
    del k
    x.masked_fill_(~seen[:, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _decode(vc[at], vs[at]).transpose(1, 2).reshape(b, kv, blocks * ps, D)
    o = (p.view(b, kv, -1, blocks * ps) @ v).view(b, kv, -1, n, D) / total.clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, s.hq, D)
    real = torch.arange(n, device=DEV) < s.rows[:, None]
    s.out.copy_(torch.where(real[..., None, None], o, s.out.float()))
    return s.out


def _exact_attend(s):
    def value(codes, scales):
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
        sign = 1 - 2 * torch.floor(c / 8)
        c = c % 8
        e, m = torch.floor(c / 2), c % 2
        mag = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
        b = scales.double()
        e, m = torch.floor(b / 8), b % 8
        sc = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6)
        return sign * mag * sc.repeat_interleave(16, -1)

    out = torch.zeros(s.out.shape, dtype=torch.float64, device=DEV)
    c, sc = s.page * s.dim // 2, s.page * s.dim // 16
    for b, (length, rows) in enumerate(zip(s.length.tolist(), s.rows.tolist())):
        if not length:
            continue
        pages = s.cache[s.table[b, : -(-length // s.page)].long()].transpose(0, 1)  # [heads][pages][bytes]
        for h in range(s.kv):
            p = pages[h]
            k = value(p[:, :c].reshape(-1, s.dim // 2), p[:, 2 * c:2 * c + sc].reshape(-1, s.dim // 16))[:length]
            v = value(p[:, c:2 * c].reshape(-1, s.dim // 2), p[:, 2 * c + sc:].reshape(-1, s.dim // 16))[:length]
            group = s.hq // s.kv
            q = s.q[b, :rows, h * group:(h + 1) * group].double()
            x = torch.einsum("ngd,td->ngt", q, k) * s.scale
            pos = torch.arange(length - rows, length, device=DEV)
            seen = torch.arange(length, device=DEV) <= pos[:, None]
            x = x.masked_fill(~seen[:, None], -math.inf)
            w = torch.nan_to_num(torch.softmax(x, -1))  # a row before the first token sees nothing
            out[b, :rows, h * group:(h + 1) * group] = torch.einsum("ngt,td->ngd", w, v)
    return out


# ---- projections with low-rank adapters -----------------------------------------------------

def _prepare_lora(case, seed):
    h, g = HEADS[case["heads"]], _dev(seed)
    L, H, b, B, r, na = case["layers"], case["hidden"], case["batch"], case["block"], case["rank"], case["adapters"]
    nq, nkv = h["q_heads"] * h["dim"], 2 * h["kv_heads"] * h["dim"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(torch.bfloat16)

    which = torch.randint(0, na, (b,), generator=_host(seed), dtype=torch.int32)
    which[torch.rand(b, generator=_host(seed + 1)) < case["share"]] = -1
    s = State(op="lora", case=case, L=L, b=b, B=B, nq=nq, nkv=nkv, which=which.to(DEV),
              w_kv=normal(L, nkv, H, std=H ** -0.5), w_q=normal(L, nq, H, std=H ** -0.5),
              a_q=normal(na, L, r, H, std=H ** -0.5), b_q=normal(na, L, nq, r, std=r ** -0.5),
              a_kv=normal(na, L, r, H, std=H ** -0.5), b_kv=normal(na, L, nkv, r, std=r ** -0.5),
              scale=0.25 + 0.5 * torch.rand(na, generator=g, device=DEV), x=normal(b, L, B, H), boundary=normal(b, L, H),
              bkv=torch.empty(b, L, nkv, dtype=torch.bfloat16, device=DEV), q=torch.empty(b, L, B, nq, dtype=torch.bfloat16, device=DEV))
    if own:
        _library_state(s, b, L, case["heads"], H, B)
        # the boundary vectors of a state that holds no rows yet
        s.lib.ls_prefill_summary(s.handle, None, None, 0, 0, torch.zeros(b, dtype=torch.int64, device=DEV), 0, 0, s.boundary, None, 0)
        s.lora = s.lib.make_lora(na, r, s.a_q, s.b_q, s.a_kv, s.b_kv, s.scale, s.which)
        s.ws = torch.empty(s.lib.ls_lora_workspace_bytes(s.cfg, r), dtype=torch.uint8, device=DEV)
    return s


def _own_lora(s):
    s.lib.ls_draft_prologue_lora(s.handle, s.w_kv, s.w_q, s.x, s.lora, s.bkv, s.q, s.ws, s.ws.numel())
    return {"bkv": s.bkv, "q": s.q}


def _plain_lora(s):
    at = s.which.clamp(min=0).long()
    scale = torch.where(s.which >= 0, s.scale[at], 0.0)[:, None, None, None]

    def project(x, w, a, bb):  # x [b][L][rows][H]
        y = torch.einsum("blih,lnh->blin", x.float(), w.float())
        low = torch.matmul(x.float(), a[at].float().transpose(-1, -2))
        return y + scale * torch.matmul(low, bb[at].float().transpose(-1, -2))

    s.q.copy_(project(s.x, s.w_q, s.a_q, s.b_q))
    s.bkv.copy_(project(s.boundary[:, :, None], s.w_kv, s.a_kv, s.b_kv)[:, :, 0])
    return {"bkv": s.bkv, "q": s.q}


def _exact_lora(s):
    out = {}
    for name, x, w, a, bb in (("q", s.x, s.w_q, s.a_q, s.b_q), ("bkv", s.boundary[:, :, None], s.w_kv, s.a_kv, s.b_kv)):
        y = torch.stack([x[:, l].double() @ w[l].double().T for l in range(s.L)], 1)
        for b, ad in enumerate(s.which.tolist()):
            if ad >= 0:
                low = torch.einsum("lih,lrh->lir", x[b].double(), a[ad].double())
                y[b] += s.scale[ad].double() * torch.einsum("lir,lnr->lin", low, bb[ad].double())
        out[name] = y if name == "q" else y[:, :, 0]
    return out
