"""Attention over selected keys where blocks take several rows, lists split
into parts, pages have odd sizes and calls overlap (formulas and tolerances:
test_gpu_attend.py, serve_ref.py)."""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref
from tests.test_gpu_attend import SCALE, check, gpu, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("where", ["first", "last"])
def test_low_scores_with_empty_parts(H, where):
    # one row's list splits over many blocks; all scores are near -600 and all
    # but one part are empty, so a part without keys must not set the reference
    x = make(1, H, 2048, ctx=2100, seed=H)
    lat = np.full((x["entries"].shape[0], 512), 2.0)
    x["entries"] = ref.kv4_encode(lat, ref.bf16_bits(np.random.default_rng(H).standard_normal((lat.shape[0], 64))))
    q = ref.bf16_f64(x["q"])
    q[..., :512] = -8.0
    x["q"] = ref.bf16_bits(q)
    if where == "first":
        x["idx"][:, 40:] = -1
    else:
        x["idx"][:, :-40] = -1
    out, lse = check(x)
    assert (lse < -400).all() and (out.abs() > 1).all()


@pytest.mark.parametrize("page", [1, 7, 63, 1000])
@pytest.mark.parametrize("H", [16, 128])
def test_page_sizes(page, H):
    check(make(4, H, 150, B=2, ctx=333, page=page, seed=page + H, fill="holes"))


@pytest.mark.parametrize("T,H", [(160, 65), (225, 128), (90, 200), (300, 64)])
def test_more_rows_than_blocks(T, H):
    # each block works through several rows: short, long and empty lists, and
    # padding rows between them
    x = make(T, H, 300, B=5, ctx=700, seed=T, fill="ragged")
    x["row_seq"][::7] = -1
    x["idx"][11::13] = -1
    g = gpu(x)
    out = torch.full((T, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 5.0, device="cuda")
    dsa.dsa_attend_kv4(scale=SCALE, out=out, lse=lse, **g)
    want = ref.attend(ref.bf16_f64(x["q"]), x["entries"], x["table"], 64, x["row_seq"], x["idx"], SCALE)
    keep = x["row_seq"] >= 0
    ref.check_attend(out.double().cpu().numpy()[keep], lse.double().cpu().numpy()[keep], [w[keep] for w in want])
    assert (out[~torch.from_numpy(keep)] == 5).all() and (lse[~torch.from_numpy(keep)] == 5).all()


@pytest.mark.parametrize("H", [32, 128])
def test_only_padding(H):
    x = make(4, H, 40, seed=1)
    x["row_seq"][:] = -1
    out = torch.full((4, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_attend_kv4(scale=SCALE, out=out, **gpu(x))
    assert (out == 5).all()


@pytest.mark.parametrize("T,H", [(3, 128), (200, 128), (3, 24), (200, 24)])
def test_output_on_16_byte_boundaries(T, H):
    x = make(T, H, 90, B=2, seed=T + H)
    out = torch.full((T * H * 512 + 16,), 5.0, dtype=torch.bfloat16, device="cuda")
    view = out[8:-8].view(T, H, 512)
    assert view.data_ptr() % 32 == 16
    dsa.dsa_attend_kv4(scale=SCALE, out=view, **gpu(x))
    want = dsa.dsa_attend_kv4(scale=SCALE, **gpu(x))
    assert torch.equal(view, want[0]) and (out[:8] == 5).all() and (out[-8:] == 5).all()


def test_both_kinds_of_blocks_at_once():
    # few and many heads on two streams, in flight together
    xs = [make(150, 128, 300, B=2, ctx=600, seed=21), make(300, 16, 300, B=2, ctx=600, seed=22)]
    gs, alone = [gpu(x) for x in xs], []
    for x, g in zip(xs, gs):
        alone.append(dsa.dsa_attend_kv4(scale=SCALE, **g))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(dsa.dsa_attend_kv4(scale=SCALE, **gs[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for o, l in got[k]:
            assert torch.equal(o, alone[k][0]) and torch.equal(l, alone[k][1])


def test_a_list_of_one_key_many_times():
    x = make(2, 128, 700, seed=23)
    x["idx"][:] = 17
    check(x)


@pytest.mark.parametrize("T,H", [(200, 16), (160, 64), (100, 128)])
def test_replays_with_more_rows_than_blocks(T, H):
    # one workspace, replayed on changed inputs; the first row is padding in one of them
    xs = [make(T, H, 200, B=2, ctx=400, seed=s, fill=f) for s, f in ((24, "ragged"), (25, "holes"))]
    xs[1]["row_seq"][0] = -1
    g = gpu(xs[0])
    ws = torch.randint(0, 256, (dsa.dsa_attend_kv4_workspace_bytes(T, H, 200),), dtype=torch.uint8, device="cuda")
    out, lse = dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, **g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_attend_kv4(scale=SCALE, out=out, lse=lse, workspace=ws, **g)
    for x in (xs[1], xs[0], xs[1]):
        for k, v in gpu(x).items():
            g[k].copy_(v)
        out.fill_(5), lse.fill_(5)
        graph.replay()
        want = (torch.full_like(out, 5), torch.full_like(lse, 5))
        dsa.dsa_attend_kv4(scale=SCALE, out=want[0], lse=want[1], **gpu(x))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_one_sequence_table_and_long_lists():
    # far more entries than a tile ring holds, most of them listing nothing
    x = make(3, 24, 20000, ctx=3000, seed=26)
    x["idx"][np.random.default_rng(26).random(x["idx"].shape) < 0.97] = -1
    check(x)
    y = make(2, 128, 20000, ctx=3000, seed=27)
    y["idx"][:, 100:-100] = -1
    check(y)


@pytest.mark.parametrize("T,H", [(300, 128), (5, 128), (300, 64), (300, 16)])
def test_many_calls_give_the_same_bits(T, H):
    # hand-overs between warps and blocks, a few thousand of each: a stale tile would show in some call
    x = make(T, H, 900, B=3, ctx=2000, seed=T + H, fill="holes")
    g = gpu(x)
    want = dsa.dsa_attend_kv4(scale=SCALE, **g)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    for _ in range(40):
        dsa.dsa_attend_kv4(scale=SCALE, out=out, lse=lse, **g)
        off += (out != want[0]).sum() + (lse != want[1]).sum()
    assert int(off) == 0


@pytest.mark.parametrize("T,H", [(4, 16), (4, 128), (200, 16), (200, 128)])
def test_workspace_has_the_calls_status_word(T, H):
    # with and without a status word of the caller's, from a workspace of garbage; a later good call clears it
    x = make(T, H, 130, B=4, ctx=500, seed=8 + T)
    ws = torch.full((max(256, dsa.dsa_attend_kv4_workspace_bytes(T, H, 130)),), 0xA5, dtype=torch.uint8, device="cuda")
    assert dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, **gpu(x)) and dsa.dsa_index_device_status(ws) == 0
    y = dict(x, idx=x["idx"].copy())
    y["idx"][T - 1, 7] = 2 ** 31 - 1                    # past the table
    z = dict(x, row_seq=x["row_seq"].copy())
    z["row_seq"][T // 2] = 4                            # no such sequence
    w = dict(x, table=x["table"].copy())
    w["table"][:, 1] = -7                               # no such page
    for bad in (y, z, w):
        dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, **gpu(bad))
        assert dsa.dsa_index_device_status(ws) == 2
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, status=st, **gpu(bad))
        assert dsa.dsa_index_device_status(ws) == 2 and int(st) == 2
        dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, status=st, **gpu(x))
        assert dsa.dsa_index_device_status(ws) == 0 and int(st) == 2       # the caller's word collects


@pytest.mark.parametrize("T,H,n,drop", [(148, 16, 1 << 20, 25.25), (148, 64, 1 << 18, 22.0), (74, 128, 1 << 20, 25.25), (74, 128, 1 << 19, 25.5)])
def test_many_small_weights_add_up(T, H, n, drop):
    # one key at the reference and n - 1 of a weight of 2^-drop each.  Weights are fp16 times 2^7: each is off by at
    # most 2^-32 (half a subnormal step) or 2^-11 of itself, so the output by at most n 2^-32 |latent| + 2^-11 of the
    # small keys' part.  The product's fp32 accumulator takes 16 keys a step and may truncate: n / 16 steps of 2^-23
    # of the output.  The sum takes a thread's two keys (64 of a tile of 128) a step and rounds: n / 64 steps of 2^-24.
    # exp2 and the quotient: 2^-11 as in serve_ref.check_attend.  The store rounds once, 2^-8.
    lat = np.concatenate([np.full((1, 512), 1.0), np.full((63, 512), 64.0)])
    rope = np.zeros((64, 64))
    rope[1:, 0] = -drop
    x = dict(entries=ref.kv4_encode(lat, ref.bf16_bits(rope)), page=64)
    v0, v1 = ref.kv4_decode(x["entries"])[0][:2, 0]       # what the cache holds of 1 and 64
    q = torch.zeros((T, H, 576), dtype=torch.bfloat16, device="cuda")
    q[..., 512] = 1.0
    idx = torch.ones((T, n), dtype=torch.int32, device="cuda")
    idx[:, 5] = 0
    pool = torch.from_numpy(x["entries"]).cuda().view(1, 64, 416)
    zero = torch.zeros(T, dtype=torch.int32, device="cuda")
    out, lse = dsa.dsa_attend_kv4(q, pool, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), idx, float(np.log(2.0)), row_seq=zero)
    w = (n - 1) * 2.0 ** -drop
    want, want_lse = (v0 + v1 * w) / (1.0 + w), np.log1p(w)
    steps = n / 16 * 2.0 ** -23 + n / 64 * 2.0 ** -24
    tol = 2.0 ** -8 * want + (1 + 2.0 ** -8) * (n * 2.0 ** -32 * v1 + 2.0 ** -11 * v1 * w + (2.0 ** -11 + steps) * want)
    assert v1 * w / (1 + w) > 3 * tol                # the small weights would be missed
    assert float((out.double() - want).abs().max()) <= tol
    assert float((lse.double() - want_lse).abs().max()) <= n / 64 * 2.0 ** -24 + 2.0 ** -14


@pytest.mark.parametrize("T,H", [(148, 16), (148, 64), (74, 128)])
def test_equal_weights_on_the_longest_list(T, H):
    # every key the same, 2^20 of them in one part: the accumulator may truncate at each of the n / 16 steps, 2^-23 of
    # the output at most; the store rounds once, 2^-8
    n = 1 << 20
    e = ref.kv4_encode(np.full((64, 512), 1.0), ref.bf16_bits(np.zeros((64, 64))))
    v = ref.kv4_decode(e)[0][0, 0]
    zero = torch.zeros(T, dtype=torch.int32, device="cuda")
    out, lse = dsa.dsa_attend_kv4(torch.zeros((T, H, 576), dtype=torch.bfloat16, device="cuda"),
                                  torch.from_numpy(e).cuda().view(1, 64, 416), zero.view(T, 1),
                                  torch.zeros((T, n), dtype=torch.int32, device="cuda"), 1.0, row_seq=zero)
    assert float((out.double() - v).abs().max()) <= v * (2.0 ** -8 + n / 16 * 2.0 ** -23)
    assert float((lse.double() - np.log(n)).abs().max()) <= n / 64 * 2.0 ** -24 + 2.0 ** -18


@pytest.mark.parametrize("T,H", [(2, 16), (200, 64), (3, 128)])
def test_the_largest_scales(T, H):
    # scores stay moderate: rows of zeros, and rows so small that a scale near fp32's largest brings them back
    x = make(T, H, 150, ctx=400, seed=T)
    q = ref.bf16_f64(x["q"]) * 2.0 ** -125
    q[:, ::3] = 0
    x["q"] = ref.bf16_bits(q)
    check(x, scale=3.0e38)
    check(x, scale=-3.0e38)
