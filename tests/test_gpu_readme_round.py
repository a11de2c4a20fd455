"""The serving round that the README shows, run as it stands there: a target of three layers, of which
the drafter taps two, several requests. The rows that the commit retains are those that the target
wrote, request by request and layer by layer."""

import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fixed_cost_drafter_b200 as F
    import oracle as O
    from tests.serving_side import Lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
H, HQ, D, HID, B, PS = 2, 8, 128, 512, 16, 16


def _shown():
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    return re.search(r"A serving round over a 4-bit paged cache.*?```python\n(.*?)```", text, re.S).group(1)


def test_the_round_that_the_readme_shows():
    b, tapped, target_layers, n = 3, [0, 2], 3, B + 1
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

    def zeros(*s, t=torch.bfloat16):
        return torch.zeros(*s, dtype=t, device="cuda")

    lib, twin = (Lib(batch=b, layers=len(tapped), kv_heads=H, q_heads=HQ, dim=D, hidden=HID, block=B) for _ in range(2))
    max_blocks = 4
    num_pages = b * max_blocks
    rows = normal(target_layers, b, n, (HQ + 2 * H) * D)
    draft = torch.randint(0, 50, (b, B), generator=g, device="cuda", dtype=torch.int32)
    target = torch.cat([draft, draft[:, :1]], 1).contiguous()
    target[0, 3] += 1
    target[1, 0] += 1
    ws = torch.empty(F.ls_verify_workspace_bytes(lib.cfg, n), dtype=torch.uint8, device="cuda")
    names = dict(
        F=F, st=lib.st, cfg=lib.cfg, batch=b, kv_heads=H, head_dim=D, page_size=PS, max_blocks=max_blocks, num_pages=num_pages,
        block_table=torch.full((b, max_blocks), -1, dtype=torch.int32, device="cuda"), held=zeros(b, t=torch.int32),
        free_pages=torch.randperm(num_pages, generator=g, device="cuda").int(),
        free_count=torch.tensor([num_pages], dtype=torch.int32, device="cuda"),
        layer_pages=[zeros(num_pages, F.ls_kv4_page_bytes(lib.cfg, PS), t=torch.uint8) for _ in range(target_layers)],
        tapped_layers=tapped, slots=zeros(b, n, t=torch.int64), row_stride=(HQ + 2 * H) * D, q_stride=(HQ + 2 * H) * D,
        target_projections=lambda l: (rows[l], rows[l, :, :, HQ * D:], rows[l, :, :, (HQ + H) * D:]),
        kv_len=torch.full((b,), n, dtype=torch.int64, device="cuda"), softmax_scale=D ** -0.5, out=zeros(b, n, HQ, D), ws=ws,
        verify_k=zeros(b, len(tapped), n, H, D), verify_v=zeros(b, len(tapped), n, H, D), verify_hidden=normal(b, len(tapped), n, HID),
        draft_ids=draft, target_ids=target, accept_len=zeros(b, t=torch.int32), next_token=zeros(b, t=torch.int32),
        n_adapters=2, rank=8, a_q=normal(2, 2, 8, HID, std=HID ** -0.5), b_q=normal(2, 2, HQ * D, 8), a_kv=normal(2, 2, 8, HID, std=HID ** -0.5),
        b_kv=normal(2, 2, 2 * H * D, 8), scale=torch.ones(2, device="cuda"), adapter_of=torch.tensor([0, -1, 1], dtype=torch.int32, device="cuda"),
        w_kv=normal(2, 2 * H * D, HID, std=HID ** -0.5), w_q=normal(2, HQ * D, HID, std=HID ** -0.5), x=normal(b, 2, B, HID),
        bkv=zeros(b, 2, 2 * H * D), q=zeros(b, 2, B, HQ * D),
        lora_ws=torch.empty(F.ls_lora_workspace_bytes(lib.cfg, 8), dtype=torch.uint8, device="cuda"))
    exec(_shown(), names)
    assert lib.error() == (F.LS_OK, 0)
    assert names["accept_len"].tolist() == [3, 0, B]
    dense = []
    for first, name in ((HQ * D, "verify_k"), ((HQ + H) * D, "verify_v")):
        held = rows[tapped][..., first:first + H * D].transpose(0, 1).reshape(b, len(tapped), n, H, D)
        want = O.kv4_decode(*O.kv4_encode(held.double().cpu().numpy()))
        assert np.array_equal(names[name].double().cpu().numpy(), want), name
        dense.append(torch.from_numpy(want).to(torch.bfloat16).cuda())
    # (the last layer's outputs are left in `out`)
    k, v = (O.kv4_decode(*O.kv4_encode(rows[2, :, :, f:f + H * D].reshape(b, n, H, D).double().cpu().numpy()))
            for f in (HQ * D, (HQ + H) * D))
    for i in range(b):
        ref, mass, _ = O.attend_rows(rows[2, i, :, :HQ * D].reshape(n, HQ, D).double().cpu().numpy(), k[i], v[i], 0, D ** -0.5)
        # bf16 output, fp16 weights, logits of at most a few tens: 2 x 136 x 2^-24 x |logit| terms
        assert (np.abs(names["out"][i].double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * mass + 1e-6).all()
    acc, tok = zeros(b, t=torch.int32), zeros(b, t=torch.int32)
    F.ls_commit_round(twin.st, draft, target, dense[0], dense[1], names["verify_hidden"], acc, tok)
    y = F.ls_get_layout(lib.cfg)
    assert torch.equal(lib.arena[:y.off_error], twin.arena[:y.off_error]) and torch.equal(lib.arena[y.off_kv:y.off_sample],
                                                                                         twin.arena[y.off_kv:y.off_sample])
    assert names["held"].tolist() == [-(-(a + 1) // PS) for a in (3, 0, B)]
    assert names["q"].abs().sum() > 0 and names["bkv"].abs().sum() > 0
