"""README's serving step, run as it is printed, over a prompt chunk and decode
steps with idle requests: decode lists from dsa_index_decode_paged, prompt lists
from dsa_index_prefill_paged, both into attention over the 4-bit cache."""

from pathlib import Path

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu

H_INDEX, H_ATT, PAGE, BLOCKS = 64, 24, 64, 6


def example() -> str:
    text = (Path(__file__).resolve().parent.parent / "README.md").read_text()
    blocks = [b.split("```")[0] for b in text.split("```python\n")[1:]]
    (code,) = [b for b in blocks if "dsa_block_tables" in b]
    return code


def check_row(idx, keys, q, w, topk, entries, q_att, out, lse, scale, label):
    """A row's list against the reference's index scores, and its attention."""
    m = min(topk, len(keys))
    got = idx.cpu().numpy()
    assert (got[:m] >= 0).all() and (got[m:] == -1).all() and len(set(got[:m].tolist())) == m and got[:m].max() < len(keys), label
    qd, wd, kd = q.double().cpu().numpy(), w.double().cpu().numpy(), np.stack(keys)
    want = wd @ np.maximum(qd @ kd.T, 0)
    tol = 2.0 ** -7 * (wd @ (np.abs(qd) @ np.abs(kd).T)).max()        # keys rounded once to bf16, 2^-8; as much for the sums
    assert want[got[:m]].min() >= np.sort(want)[::-1][m - 1] - 2 * tol, label
    r = ref.attend(q_att[None].double().cpu().numpy(), np.stack(entries), np.zeros((1, 1), np.int32), len(entries), [0],
                   got[None], scale)
    ref.check_attend(out[None].double().cpu().numpy(), lse[None].double().cpu().numpy(), r, label)


@pytest.mark.parametrize("topk", [40, 2048])
def test_example_runs_as_printed(topk):
    dev, B, T = "cuda", 5, 300
    n_pages = B * BLOCKS + 2
    g = torch.Generator(device=dev)
    g.manual_seed(topk)
    randn = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    ns = dict(dsa=dsa, torch=torch, n_pages=n_pages, page=PAGE, T=T, topk=topk, scale=192 ** -0.5,
              table=torch.full((B, BLOCKS), -1, dtype=torch.int32, device=dev),
              free_pages=torch.randperm(n_pages, generator=g, device=dev).int(), free_begin=i32([0]), cached=i32([0] * B),
              inv_freq=(10000.0 ** (-torch.arange(0, 64, 2, device=dev) / 64)).float(),
              k_pages=torch.zeros((n_pages, PAGE, 128), dtype=torch.bfloat16, device=dev),
              kv_pages=torch.zeros((n_pages, PAGE, 416), dtype=torch.uint8, device=dev),
              w_k=1 + 0.1 * torch.randn(128, generator=g, device=dev), b_k=0.1 * torch.randn(128, generator=g, device=dev))
    keys, ents = [[] for _ in range(B)], [[] for _ in range(B)]
    # a prompt with an empty request, decode with idle ones (the first, one in the middle), a chunk among decodes
    for step, new in enumerate(([130, 0, 3, 65, 64], [0, 1, 1, 0, 1], [1, 100, 0, 1, 1])):
        ns.update(new=i32(new), q=randn(T, H_INDEX, 128), k=randn(T, 128), latent=randn(T, 512), rope=randn(T, 64),
                  w=torch.rand((T, H_INDEX), generator=g, device=dev), q_heads=randn(T, H_ATT, 576))
        exec(example(), ns)
        torch.cuda.synchronize()
        pos, seq, n = ns["pos"].cpu().numpy(), ns["seq"].cpu().numpy(), sum(new)
        assert (seq[n:] == -1).all() and (seq[:n] >= 0).all()
        kr = ref.norm_rotate(ns["k"][:n].double().cpu().numpy()[:, None], pos[:n], ns["inv_freq"].cpu().numpy(), "layer",
                             ns["w_k"].cpu().numpy(), ns["b_k"].cpu().numpy(), 1e-6, False)[:, 0]
        er = ref.kv4_encode(ns["latent"][:n].double().cpu().numpy(), ns["rope"][:n].view(torch.int16).cpu().numpy().view(np.uint16))
        for t in range(n):
            assert pos[t] == len(keys[seq[t]])
            keys[seq[t]].append(kr[t])
            ents[seq[t]].append(er[t])
        common = lambda t, b, upto: dict(keys=keys[b][:upto], q=ns["q_idx"][t], w=ns["w"][t], topk=topk, entries=ents[b][:upto],
                                         q_att=ns["q_heads"][t], scale=ns["scale"])
        for b in range(B):
            if not new[b]:
                assert (ns["idx"][b] == -1).all() and (ns["out"][b] == 0).all() and torch.isinf(ns["lse"][b]).all()
                continue
            t = int(ns["start"][b + 1]) - 1
            check_row(ns["idx"][b], out=ns["out"][b], lse=ns["lse"][b], label=f"decode {step} {b}", **common(t, b, pos[t] + 1))
        for t in sorted({0, n // 2, n - 1, *range(0, n, 37)}):
            check_row(ns["lists"][t], out=ns["out_rows"][t], lse=ns["lse_rows"][t], label=f"chunk {step} {t}",
                      **common(t, seq[t], pos[t] + 1))
        # one row, both ways
        for b in range(B):
            if new[b]:
                t = int(ns["start"][b + 1]) - 1
                assert torch.equal(ns["idx"][b], ns["lists"][t])
        ns.update(cached=ns["seq_len"], free_begin=ns["free_end"])
