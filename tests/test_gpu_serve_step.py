"""The serving operators run together, as a prefill chunk and then decode
steps of a small batch: request layout, index preparation into the paged index
cache, latents into the 4-bit cache, the paged index decode, attention over
its Top-k lists."""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu

H_INDEX, H_ATT, PAGE, BLOCKS, TOPK = 32, 40, 64, 8, 96


def test_prefill_then_decode_steps():
    rng = np.random.default_rng(1)
    lens0 = np.array([200, 3, 64, 0, 129], np.int32)
    B, T_cap = len(lens0), 512
    n_pages = B * BLOCKS + 3
    dev = "cuda"
    pool_k = torch.zeros((n_pages, PAGE, 128), dtype=torch.bfloat16, device=dev)
    pool_kv = torch.zeros((n_pages, PAGE, 416), dtype=torch.uint8, device=dev)
    table = torch.full((B, BLOCKS), -1, dtype=torch.int32, device=dev)
    free = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda()
    begin = torch.zeros(1, dtype=torch.int32, device=dev)
    cached = torch.zeros(B, dtype=torch.int32, device=dev)
    inv_freq = torch.from_numpy((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    wk = torch.ones(128, device=dev)
    hist = [[] for _ in range(B)]        # what each request's caches should hold: (index key fp64, entry bytes)

    g = torch.Generator(device=dev)
    g.manual_seed(2)
    randn = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()
    for step in range(3):
        new = torch.from_numpy(lens0 if step == 0 else np.array([1, 1, 1, 1, 0], np.int32)).cuda()
        slot, pos, owner, start, seq, end = dsa.dsa_block_tables(cached, new, table, free, begin, n_pages, PAGE, T_cap,
                                                                 status=status)
        q, k, lat, rope = randn(T_cap, H_INDEX, 128), randn(T_cap, 128), randn(T_cap, 512), randn(T_cap, 64)
        w = torch.rand((T_cap, H_INDEX), generator=g, device=dev)
        qi, _ = dsa.dsa_index_prepare(q, k, pos, inv_freq, pool_k, slot_map=slot, k_norm="rms", k_weight=wk, status=status)
        dsa.dsa_kv4_write(lat, rope, pool_kv, slot, status=status)
        # the reference's picture of the caches
        p, o = pos.cpu().numpy(), owner.cpu().numpy()
        live = np.flatnonzero(o >= 0)
        keys = ref.norm_rotate(k[:len(live)].double().cpu().numpy()[:, None], p[:len(live)],
                               inv_freq.cpu().numpy(), "rms", None, None, 1e-6, False)[:, 0]
        ents = ref.kv4_encode(lat[:len(live)].double().cpu().numpy(),
                              rope[:len(live)].view(torch.int16).cpu().numpy().view(np.uint16))
        for r in live:
            assert p[r] == len(hist[o[r]])
            hist[o[r]].append((keys[r], ents[r]))
        # one query per request with new tokens: its last row
        last = (start[1:] - 1).long()
        seq_dec = torch.where(new > 0, seq, torch.zeros_like(seq))
        idx, score = dsa.dsa_index_decode_paged(qi[last.clamp(min=0)].contiguous(), w[last.clamp(min=0)].contiguous(),
                                                pool_k, table.clamp(min=0), seq_dec, TOPK)
        qa = randn(B, H_ATT, 576)
        out, lse = dsa.dsa_attend_kv4(qa, pool_kv, table, idx, 192 ** -0.5, status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        assert [len(h) for h in hist] == seq.cpu().tolist()
        for b in range(B):
            m = min(TOPK, len(hist[b])) if int(new[b]) else 0
            got = idx[b].cpu().numpy()
            assert (got[:m] >= 0).all() and (got[m:] == -1).all() and len(set(got[:m])) == m
            if m == 0:
                assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
                continue
            # the selected scores, from the reference's keys: queries as the index call got them (bf16), keys
            # rounded once to bf16 (2^-8 each, on sums of 128 products over 32 weighted heads)
            qd = qi[last[b]].double().cpu().numpy()
            kd = np.stack([h[0] for h in hist[b]])
            dots = qd @ kd.T
            wb = w[last[b]].double().cpu().numpy()
            want = wb @ np.maximum(dots, 0)
            tol = 2.0 ** -7 * (wb @ (np.abs(qd) @ np.abs(kd).T)).max()
            assert (np.abs(score[b, :m].double().cpu().numpy() - want[got[:m]]) <= tol).all()
            assert want[got[:m]].min() >= np.sort(want)[::-1][m - 1] - 2 * tol
            entries = np.stack([h[1] for h in hist[b]])
            r = ref.attend(qa[b:b + 1].double().cpu().numpy(), entries, np.zeros((1, 1), np.int32), len(entries),
                           [0], idx[b:b + 1].cpu().numpy(), 192 ** -0.5)
            ref.check_attend(out[b:b + 1].double().cpu().numpy(), lse[b:b + 1].double().cpu().numpy(), r, f"step {step} seq {b}")
        cached, begin = seq, end
    assert int(begin) == sum(-(-len(h) // PAGE) for h in hist)
