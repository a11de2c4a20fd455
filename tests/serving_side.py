"""Shared pieces of the serving-side GPU tests: a small state, page pools and 4-bit caches."""

import numpy as np
import torch

import fixed_cost_drafter_b200 as F
import oracle as O


class Lib:
    """A small drafting state and its arena."""

    def __init__(self, batch=1, layers=1, kv_heads=2, q_heads=8, dim=128, hidden=512, block=16, dtype="bf16", flags=0):
        self.cfg = F.make_config(batch=batch, n_layers=layers, n_kv_heads=kv_heads, n_q_heads=q_heads, head_dim=dim,
                                 hidden=hidden, block=block, window=64, scales=[64, 512], slots_per_scale=4,
                                 dtype=F.LS_BF16 if dtype == "bf16" else F.LS_F32, flags=flags)
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.arena = torch.empty(F.ls_state_bytes(self.cfg), dtype=torch.uint8, device="cuda")
        self.st = F.ls_init_state(self.cfg, self.arena, self.arena.numel())

    def error(self):
        return F.ls_get_error(self.st)

    def clear(self):
        F.ls_clear_error(self.st)

    def __del__(self):
        if getattr(self, "st", None):
            F.ls_destroy_state(self.st)


def refused(status, call, *args):
    try:
        call(*args)
    except F.LsError as e:
        assert e.status == status, (call.__name__, e.status)
        return
    raise AssertionError(f"{call.__name__} was not refused")


class Cache4:
    """A paged 4-bit cache of one layer whose sequences' pages lie in no order, filled from
    random bytes (codes) and scales; oracle rows are decoded from the same bytes."""

    def __init__(self, lib, lengths, page_size, seed=0, stride_extra=0, scale_std=0.5, spare=3):
        rng = np.random.default_rng(seed)
        c = lib.cfg
        self.lib, self.ps, self.D, self.H = lib, page_size, c.head_dim, c.n_kv_heads
        per = F.ls_kv4_page_bytes(c, page_size)
        self.stride = per + stride_extra
        blocks = [-(-int(n) // page_size) for n in lengths]
        self.mb = max(max(blocks), 1)
        self.pages = sum(blocks) + spare
        perm = rng.permutation(self.pages)
        self.table = np.full((len(lengths), self.mb), -1, np.int32)
        at = 0
        for b, n in enumerate(blocks):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.bytes = rng.integers(0, 256, (self.pages, self.stride), dtype=np.uint8)
        sc = np.clip(np.exp(scale_std * rng.standard_normal((self.pages, self.H, page_size * self.D // 8))) * 0.33, 0, 400)
        codes = O.kv4_encode(np.repeat(sc[..., None] * 6, 16, -1).reshape(-1, 16))[1].reshape(sc.shape)  # nearest e4m3
        for p in range(self.pages):
            for h in range(self.H):
                n = per // self.H
                self.bytes[p, h * n + page_size * self.D:(h + 1) * n] = codes[p, h]
        self.upload()

    def upload(self):
        self.dev = torch.from_numpy(self.bytes).cuda()
        self.d_table = torch.from_numpy(self.table).cuda()
        self.kv = F.make_paged_kv4([self.dev] * self.lib.cfg.n_layers, self.stride, self.d_table, self.mb, self.ps, self.pages)

    def sections(self, page, head):
        return O.kv4_sections(self.bytes[page], head, self.ps, self.D)

    def rows(self, b, n):
        """Float64 keys and values [n][H][D] of sequence b's first n positions."""
        k, v = np.zeros((n, self.H, self.D)), np.zeros((n, self.H, self.D))
        for h in range(self.H):
            for pi in range(-(-n // self.ps)):
                kc, vc, ks, vs = self.sections(self.table[b, pi], h)
                lo, hi = pi * self.ps, min(n, (pi + 1) * self.ps)
                k[lo:hi, h] = O.kv4_decode(kc, ks)[:hi - lo]
                v[lo:hi, h] = O.kv4_decode(vc, vs)[:hi - lo]
        return k, v
