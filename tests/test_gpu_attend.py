"""Attention over selected keys of the 4-bit latent cache against fp64."""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def make(T, H, n, B=1, ctx=500, page=64, seed=0, fill="full", q_gain=1.0):
    rng = np.random.default_rng(seed)
    blocks = -(-ctx // page)
    n_pages = B * blocks + 2
    N = n_pages * page
    lat = ref.bf16_f64(ref.bf16_bits(rng.standard_normal((N, 512)) * (0.5 + rng.random(512))))
    x = dict(q=ref.bf16_bits(rng.standard_normal((T, H, 576)) * q_gain), page=page,
             entries=ref.kv4_encode(lat, ref.bf16_bits(rng.standard_normal((N, 64)))),
             table=rng.permutation(n_pages)[:B * blocks].reshape(B, blocks).astype(np.int32),
             row_seq=rng.integers(0, B, T).astype(np.int32))
    idx = np.stack([rng.choice(ctx, n, replace=n > ctx) for _ in range(T)]).astype(np.int32)
    if fill == "ragged":                       # list t holds t * 37 mod (n + 1) keys: row 0 none
        idx[np.arange(n)[None] >= (np.arange(T)[:, None] * 37) % (n + 1)] = -1
    elif fill == "holes":
        idx[rng.random((T, n)) < 0.6] = -1
    elif fill == "late":                       # nothing but the last entry
        idx[:, :-1] = -1
    x["idx"] = idx
    return x


def gpu(x):
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return dict(q=g(x["q"].view(np.int16)).view(torch.bfloat16), kv_pages=g(x["entries"]).view(-1, x["page"], 416),
                block_table=g(x["table"]), idx=g(x["idx"]), row_seq=g(x["row_seq"]))


def check(x, scale=SCALE, label=""):
    r = dsa.dsa_attend_kv4(scale=scale, **gpu(x))
    torch.cuda.synchronize()
    want = ref.attend(ref.bf16_f64(x["q"]), x["entries"], x["table"], x["page"], x["row_seq"], x["idx"], scale)
    ref.check_attend(r[0].double().cpu().numpy(), r[1].double().cpu().numpy(), want, label)
    return r


@pytest.mark.parametrize("H", [1, 7, 8, 16, 17, 32, 33, 64, 65, 96, 128, 200, 256])
def test_heads(H):
    check(make(3, H, 200, seed=H))


@pytest.mark.parametrize("n", [1, 2, 15, 63, 64, 65, 127, 128, 129, 192, 193, 500, 1000, 2048])
def test_list_lengths(n):
    check(make(2, 64, n, ctx=1500 if n < 1500 else 2500, seed=n))
    check(make(1, 5, n, ctx=1500, seed=n + 1))


@pytest.mark.parametrize("fill", ["ragged", "holes", "late"])
@pytest.mark.parametrize("H,n", [(16, 130), (128, 64), (64, 333)])
def test_masks(fill, H, n):
    check(make(12, H, n, B=3, ctx=400, page=48, seed=n + H, fill=fill))


def test_empty_lists():
    x = make(5, 64, 100, seed=1)
    x["idx"][[0, 3, 4]] = -1
    out, lse = check(x)
    assert (out[[0, 3, 4]] == 0).all() and torch.isinf(lse[[0, 3, 4]]).all()
    x["idx"][:] = -(2 ** 31)
    out, lse = check(x)
    assert (out == 0).all()


@pytest.mark.parametrize("rows", [1, 5, 149, 400])
def test_many_rows(rows):
    check(make(rows, 24, 80, B=4, ctx=700, page=192, seed=rows, fill="ragged"))


def test_repeated_entries_count_as_often_as_listed():
    x = make(2, 16, 90, seed=2)
    x["idx"][:, 10:60] = x["idx"][:, :1]
    check(x)


@pytest.mark.parametrize("gain", [8.0, 200.0])
def test_peaked_scores(gain):
    # one key takes nearly all the weight, and the maximum keeps rising along
    # the list (the running maximum moves in every tile)
    x = make(3, 32, 512, ctx=600, seed=3, q_gain=gain)
    q, lat = ref.bf16_f64(x["q"]), ref.kv4_decode(x["entries"])[0]
    for t in range(3):
        slots = x["table"][x["row_seq"][t]][x["idx"][t] // 64].astype(np.int64) * 64 + x["idx"][t] % 64
        order = np.argsort(lat[slots] @ q[t, 0, :512])
        x["idx"][t] = x["idx"][t][order if t < 2 else order[::-1]]
    check(x)


def test_scales():
    x = make(2, 16, 100, seed=4)
    for scale in (0.0, -0.07, 1e-30, 3.0):
        check(x, scale)


def test_query_magnitudes():
    # rows whose size differs by many powers of two, zero rows, subnormal and huge ones
    x = make(2, 16, 100, seed=5)
    q = ref.bf16_f64(x["q"])
    q *= 2.0 ** np.linspace(-120, 2, 16)[None, :, None]
    q[0, 3] = 0
    q[1, 5, :512] = 0                            # rotary part alone
    q[1, 6, 512:] = 0
    q[0, 7, :512] *= 2.0 ** -100
    x["q"] = ref.bf16_bits(q)
    check(x)
    x["q"] = ref.bf16_bits(ref.bf16_f64(x["q"]) * 2.0 ** 110)
    check(x, scale=2.0 ** -110)


def test_padding_rows_are_left_alone():
    x = make(9, 64, 70, B=2, seed=6)
    x["row_seq"][[2, 7, 8]] = -1
    g = gpu(x)
    out = torch.full((9, 64, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 64), 5.0, device="cuda")
    dsa.dsa_attend_kv4(scale=SCALE, out=out, lse=lse, **g)
    want = ref.attend(ref.bf16_f64(x["q"]), x["entries"], x["table"], 64, x["row_seq"], x["idx"], SCALE)
    keep = x["row_seq"] >= 0
    ref.check_attend(out.double().cpu().numpy()[keep], lse.double().cpu().numpy()[keep], [w[keep] for w in want])
    assert (out[[2, 7, 8]] == 5).all() and (lse[[2, 7, 8]] == 5).all()


def test_sequence_default_is_the_row():
    x = make(6, 16, 64, B=8, seed=7)
    x["row_seq"] = np.arange(6, dtype=np.int32)
    a = check(x)
    g = gpu(x)
    g.pop("row_seq")
    b = dsa.dsa_attend_kv4(scale=SCALE, **g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_pages_positions_and_sequences_are_flagged():
    x = make(4, 16, 128, B=4, ctx=500, seed=8)
    x["row_seq"] = np.arange(4, dtype=np.int32)
    x["table"][0, 2] = -7
    x["table"][1, 1] = x["entries"].shape[0] // 64
    x["idx"][2, 5] = x["table"].shape[1] * 64
    x["idx"][2, 6] = 2 ** 31 - 1
    for row in range(3):
        y = dict(x, row_seq=np.where(np.arange(4) == row, x["row_seq"], 3).astype(np.int32))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        dsa.dsa_attend_kv4(scale=SCALE, status=st, **gpu(y))
        assert int(st) == 2, row
        check(y)
    y = dict(x, row_seq=np.array([4, 3, 3, 3], np.int32))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((4, 16, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_attend_kv4(scale=SCALE, status=st, out=out, **gpu(y))
    assert int(st) == 2 and (out[0] == 5).all() and not (out[1:] == 5).all()


def test_unselected_garbage_does_not_leak():
    # NaN codes, scales and rotary values in entries that no list names
    x = make(4, 32, 100, ctx=400, seed=9, fill="holes")
    want = check(x)
    used = set()
    for t in range(4):
        p = x["idx"][t][x["idx"][t] >= 0]
        used |= set((x["table"][x["row_seq"][t]][p // 64].astype(np.int64) * 64 + p % 64).tolist())
    rest = np.setdiff1d(np.arange(x["entries"].shape[0]), sorted(used))
    y = dict(x, entries=x["entries"].copy())
    y["entries"][rest] = 0xFF
    got = dsa.dsa_attend_kv4(scale=SCALE, **gpu(y))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_do_not_depend_on_the_batch_around_them():
    x = make(40, 64, 256, B=3, ctx=600, seed=10)
    full = check(x)
    y = dict(x)
    for k in ("q", "idx", "row_seq"):
        y[k] = x[k].copy()
    y["q"][1:] = 0x4000
    y["idx"][1:] = -1
    part = dsa.dsa_attend_kv4(scale=SCALE, **gpu(y))
    assert torch.equal(full[0][0], part[0][0]) and torch.equal(full[1][0], part[1][0])
    again = dsa.dsa_attend_kv4(scale=SCALE, **gpu(x))
    assert torch.equal(full[0], again[0]) and torch.equal(full[1], again[1])


def test_offsets_past_32_bits():
    n = (1 << 32) // 416 + 2000
    pages = n // 100
    pool = torch.zeros((pages, 100, 416), dtype=torch.uint8, device="cuda")
    x = make(2, 16, 90, ctx=200, page=100, seed=11)
    e = torch.from_numpy(x["entries"]).cuda().view(-1, 100, 416)
    pool[pages - e.shape[0]:] = e
    x["table"] += pages - e.shape[0]
    g = dict(gpu(x), kv_pages=pool)
    r = dsa.dsa_attend_kv4(scale=SCALE, **g)
    x["table"] -= pages - e.shape[0]
    want = ref.attend(ref.bf16_f64(x["q"]), x["entries"], x["table"], 100, x["row_seq"], x["idx"], SCALE)
    ref.check_attend(r[0].double().cpu().numpy(), r[1].double().cpu().numpy(), want)


def test_streams_and_workspaces():
    # calls in flight on two streams, each with its workspace; a workspace of
    # garbage; the same results as alone
    xs = [make(30, 128, 300, B=2, ctx=600, seed=s) for s in (12, 13)]
    gs = [gpu(x) for x in xs]
    alone = [check(x) for x in xs]
    need = dsa.dsa_attend_kv4_workspace_bytes(30, 128, 300)
    ws = [torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda") for _ in xs]
    outs = [(torch.empty_like(a[0]), torch.empty_like(a[1])) for a in alone]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, w, o, s in zip(gs, ws, outs, streams):
            with torch.cuda.stream(s):
                dsa.dsa_attend_kv4(scale=SCALE, workspace=w, out=o[0], lse=o[1], **g)
    torch.cuda.synchronize()
    for o, a in zip(outs, alone):
        assert torch.equal(o[0], a[0]) and torch.equal(o[1], a[1])


@pytest.mark.parametrize("T,H", [(1, 128), (40, 16)])
def test_replays_in_a_graph(T, H):
    xs = [make(T, H, 700, B=2, ctx=1000, seed=s, fill=f) for s, f in ((14, "full"), (15, "ragged"))]
    xs[1]["table"] = xs[1]["table"]
    g = gpu(xs[0])
    out, lse = dsa.dsa_attend_kv4(scale=SCALE, **g)
    ws = torch.empty(max(256, dsa.dsa_attend_kv4_workspace_bytes(T, H, 700)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_attend_kv4(scale=SCALE, out=out, lse=lse, workspace=ws, **g)
    for x in (xs[1], xs[0]):
        for k, v in gpu(x).items():
            g[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.attend(ref.bf16_f64(x["q"]), x["entries"], x["table"], 64, x["row_seq"], x["idx"], SCALE)
        ref.check_attend(out.double().cpu().numpy(), lse.double().cpu().numpy(), want)
