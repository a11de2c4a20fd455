"""The serving-side operators without a GPU: sizes and refusals the host decides alone, the
structs the binding mirrors, and pins of their oracle."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import fixed_cost_drafter_b200 as F
import oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _cfg(**kw):
    base = dict(batch=3, n_layers=2, n_kv_heads=2, n_q_heads=8, head_dim=128, hidden=512, block=16, window=64,
                scales=[64, 512], slots_per_scale=4, dtype=F.LS_BF16)
    base.update(kw)
    return F.make_config(**base)


def test_sizes_and_their_refusals():
    assert F.ls_kv4_page_bytes(_cfg(), 16) == 2 * 16 * 144
    assert F.ls_kv4_page_bytes(_cfg(head_dim=64), 256) == 2 * 256 * 72
    for ps in (0, 8, 24, 512, -16):
        assert F.ls_kv4_page_bytes(_cfg(), ps) == 0
    assert F.ls_kv4_page_bytes(_cfg(head_dim=32), 16) == 0 and F.ls_kv4_page_bytes(_cfg(batch=0), 16) == 0
    assert F.ls_verify_workspace_bytes(_cfg(), 17) > 0
    for n in (0, 18, -1):
        assert F.ls_verify_workspace_bytes(_cfg(), n) == 0
    assert F.ls_verify_workspace_bytes(_cfg(head_dim=32), 1) == 0
    assert F.ls_lora_workspace_bytes(_cfg(), 16) > 0
    for r in (0, 4, 12, 136, -8):
        assert F.ls_lora_workspace_bytes(_cfg(), r) == 0


def test_calls_without_a_state_are_refused():
    pool = F.make_page_pool(16, 16, 16, 16, 1, 16, 1)
    kv = F.make_paged_kv4([16], 4608, 16, 1, 16, 1)
    lora = F.make_lora(1, 8, 16, 16, 16, 16, 16, 16)
    calls = [
        lambda: F.ls_pages_extend(None, pool, None, None, 1, None, 16, 3, 0),
        lambda: F.ls_pages_trim(None, pool, None, 0),
        lambda: F.ls_kv4_append(None, kv, 0, 16, 16, 256, 16, 1, 0),
        lambda: F.ls_kv4_read_rows(None, kv, 0, 16, 1, 16, 16, 256, 0),
        lambda: F.ls_verify_attend_kv4(None, kv, 0, 16, 1024, 1, None, 16, 0.1, 16, 256, 1 << 30, 0),
        lambda: F.ls_draft_prologue_lora(None, 16, 16, 16, lora, 16, 16, 256, 1 << 30, 0),
    ]
    for call in calls:
        with pytest.raises(F.LsError) as e:
            call()
        assert e.value.status == F.LS_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        F.make_paged_kv4([16] * 65, 4608, 16, 1, 16, 1)


def test_struct_mirrors(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"ls_page_pool": F.ls_page_pool, "ls_paged_kv4": F.ls_paged_kv4, "ls_lora": F.ls_lora}
    body = "".join('printf("%%zu ", sizeof(%s));' % n + "".join(
        'printf("%%zu ", offsetof(%s, %s));' % (n, f[0]) for f in s._fields_) for n, s in structs.items())
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "longspark.h"\nint main(void) {' + body + "return 0;}")
    inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run([cc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-I",
                    inc, str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for s in structs.values():
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


def test_oracle_pages_undo_each_other():
    rng = np.random.default_rng(1)
    b, mb, ps, num = 5, 9, 16, 60
    ids = rng.permutation(num)
    held = np.array([2, 0, 3, 1, 4])
    table = np.full((b, mb), -1)
    at = 0
    for i in range(b):
        table[i, :held[i]] = ids[at:at + held[i]]
        at += held[i]
    free = np.concatenate([ids[at:], np.full(at, -1)])
    length = np.array([30, 0, 48, 5, 60])
    before = (table.copy(), held.copy(), free[:num - at].copy())
    count, slots, flags = O.pages_extend(table, held, free, num - at, length, [17, 40, 1, 0, 5], 40, ps, num)
    assert not flags and [len(s) for s in slots] == [17, 40, 1, 0, 5]
    assert count == num - at - (1 + 3 + 1 + 0 + 1)
    assert slots[0][0] == table[0, 1] * ps + 14 and slots[0][2] == table[0, 2] * ps
    assert len({x for s in slots for x in s}) == 63
    count, flags = O.pages_trim(table, held, free, count, length, ps, num)
    assert not flags and count == num - at
    for x, y in zip(before, (table, held, free[:num - at])):
        assert np.array_equal(x, y)


def test_oracle_pages_refuse_in_order():
    table, held, free = np.full((3, 4), -1), np.zeros(3, int), np.arange(4)
    count, slots, flags = O.pages_extend(table, held, free, 4, np.zeros(3, int), [32, 64, 16], 64, 16, 4)
    assert flags == {"pool"} and count == 2 and list(held) == [2, 0, 0]
    assert slots[0] == [3 * 16 + i for i in range(16)] + [2 * 16 + i for i in range(16)]
    assert set(slots[1]) == {-1} and set(slots[2]) == {-1}


def test_oracle_format():
    x = np.zeros(32)
    x[:16] = [0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5]  # ties at scale 1
    c, s = O.kv4_encode(x)
    assert s[0] == 0x38 and s[1] == 0
    assert list(O.kv4_decode(c, s)[:16]) == [0, 0, 1, 1, 2, 2, 4, 4, 6, 0, -1, -1, -2, -2, -4, -4]
    y = np.random.default_rng(2).standard_normal((50, 64)) * 10.0 ** np.random.default_rng(3).integers(-4, 4, (50, 1))
    once = O.kv4_decode(*O.kv4_encode(y))
    assert np.abs(once - y).max() <= np.abs(y).max()
    top = np.abs(y.reshape(50, 4, 16)).max(-1).repeat(16, -1).reshape(50, 64)
    # half the widest code step (1 of 6) of a scale that is itself at most half a step off, or a
    # scale below the smallest normal one (2^-6): half its step 2^-9 times the largest code
    assert (np.abs(once - y) <= top / 6 * (1 + 2.0 ** -4) + 6 * 2.0 ** -10 + top * 2.0 ** -4).all()
    y[0, 3], y[1, 20] = np.inf, np.nan
    d = O.kv4_decode(*O.kv4_encode(y))
    assert np.isnan(d[0, :16]).all() and np.isfinite(d[0, 16:]).all() and np.isnan(d[1, 16:32]).all()
