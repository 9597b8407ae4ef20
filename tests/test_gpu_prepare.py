"""Index preparation (norms, rotation, slots) against the formulas in fp64.

Tolerance: statistics are fp32 sums of 128 terms (8 in order, then a tree: 12
roundings), the root and its factor 4, weight and bias 2, the rotation 3 with
cos and sin within 2^-22: fewer than 40 roundings of 2^-24 on values of at
most twice the row's largest magnitude before rotation, under 2^-17 of it.
The layer norm subtracts the mean first: its roundings scale with the raw
row's largest magnitude over its deviation, which the bound carries.  The
store rounds once: bf16 2^-8, E4M3 2^-4 (2^-10 below its normal range), of
the value.
"""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


def make(T, H, rot, q_norm, k_norm, seed, far=1_000_000, pad=0):
    rng = np.random.default_rng(seed)
    x = dict(q=ref.bf16_bits(rng.standard_normal((T, H, 128)) * 1.5), k=ref.bf16_bits(rng.standard_normal((T, 128)) * 2 + 0.3),
             pos=(rng.integers(0, far, T)).astype(np.int32), rot=rot,
             inv_freq=(10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32),
             slot=rng.permutation(T + 11)[:T].astype(np.int32), n=T + 11, q_norm=q_norm, k_norm=k_norm)
    for s, n in (("q", q_norm), ("k", k_norm)):
        x[s + "_weight"] = (1 + 0.2 * rng.standard_normal(128)).astype(np.float32) if n != "none" else None
        x[s + "_bias"] = (0.2 * rng.standard_normal(128)).astype(np.float32) if n == "layer" else None
    if pad:
        x["pos"][-pad:] = -1
        x["slot"][-pad:] = -1
    return x


def gpu(a):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a)).cuda()
    return t.view(torch.bfloat16) if a.dtype == np.uint16 else t


def call(x, interleaved, fp8, slots=True, status=None, q_out=None):
    kw = {k: (gpu(x[k]) if not isinstance(x[k], str) else x[k]) for k in
          ("q_norm", "q_weight", "q_bias", "k_norm", "k_weight", "k_bias")}
    T, H, n = *x["q"].shape[:2], x["n"]
    a = (gpu(x["q"]), gpu(x["k"]), gpu(x["pos"]), gpu(x["inv_freq"]))
    kw.update(slot_map=gpu(x["slot"]) if slots else None, interleaved=interleaved, eps=1e-6, status=status)
    if not fp8:
        k_out = torch.full((n, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        q_out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda") if q_out is None else a[0]
        r = dsa.dsa_index_prepare(*a, k_out, q_out=q_out, **kw)
        torch.cuda.synchronize()
        return r[0].double().cpu().numpy(), r[1].double().cpu().numpy()
    k_out, ks = torch.full((n, 128), 0x38, dtype=torch.uint8, device="cuda"), torch.full((n,), 7.0, device="cuda")
    q_out, qs = torch.full((T, H, 128), 0x38, dtype=torch.uint8, device="cuda"), torch.full((T, H), 7.0, device="cuda")
    dsa.dsa_index_prepare_fp8(*a, k_out, ks, q_out=q_out, q_scale_out=qs, **kw)
    torch.cuda.synchronize()
    return tuple(v.cpu().numpy() for v in (q_out, qs, k_out, ks))


def bound(raw, y, norm):
    """2^-17 of the largest magnitude before rotation, grown by the layer norm's cancellation."""
    top = np.abs(y).max(-1, keepdims=True) * 2
    if norm == "layer":
        dev = raw.std(-1, keepdims=True) + 1e-3
        top = top * (1 + np.abs(raw).max(-1, keepdims=True) / dev)
    return 2.0 ** -17 * top


def check_bf16(got, raw, y, norm, label):
    err, tol = np.abs(got - y), 2.0 ** -8 * np.abs(y) + bound(raw, y, norm)
    assert (err <= tol).all(), f"{label}: {(err - tol).max()}"


def check_fp8(code, scale, raw, y, norm, label):
    amax = np.abs(y).max(-1)
    want = np.where(amax > 0, np.maximum(amax / 448, 2.0 ** -126), 1.0)
    slack = bound(raw, y, norm)
    assert (np.abs(scale - want) <= slack[..., 0] / 448 + 2.0 ** -23 * want).all(), label
    got = ref.E4M3[code] * scale[..., None].astype(np.float64)
    tol = 2.0 ** -4 * np.abs(y) * (1 + 2.0 ** -10) + 2.0 ** -10 * want[..., None] + 2 * slack
    assert np.isfinite(got).all() and (np.abs(got - y) <= tol).all(), label


NORMS = [("none", "layer"), ("rms", "rms"), ("layer", "none")]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,rot,norms", [
    (1, 1, 64, 0), (1, 64, 64, 0), (2, 32, 32, 1), (3, 7, 16, 2), (5, 17, 96, 1), (64, 64, 64, 0), (147, 33, 128, 2),
    (148, 65, 64, 1), (201, 3, 0, 1), (150, 256, 48, 2),
])
def test_prepare(T, H, rot, norms, interleaved, fp8):
    qn, kn = NORMS[norms]
    x = make(T, H, rot, qn, kn, seed=T * 1000 + H, pad=T // 4)
    live = x["pos"] >= 0
    raw_q, raw_k = ref.bf16_f64(x["q"]), ref.bf16_f64(x["k"])
    yq = ref.norm_rotate(raw_q, x["pos"], x["inv_freq"], qn, x["q_weight"], x["q_bias"], 1e-6, interleaved)[live]
    yk = ref.norm_rotate(raw_k[:, None], x["pos"], x["inv_freq"], kn, x["k_weight"], x["k_bias"], 1e-6, interleaved)[live, 0]
    at = x["slot"][live]
    rest = np.setdiff1d(np.arange(x["n"]), at)
    if fp8:
        qc, qs, kc, ks = call(x, interleaved, True)
        check_fp8(qc[live], qs[live], raw_q[live], yq, qn, "q")
        check_fp8(kc[at], ks[at], raw_k[live], yk, kn, "k")
        assert (qc[~live] == 0x38).all() and (qs[~live] == 7).all() and (kc[rest] == 0x38).all() and (ks[rest] == 7).all()
    else:
        q, k = call(x, interleaved, False)
        check_bf16(q[live], raw_q[live], yq, qn, "q")
        check_bf16(k[at], raw_k[live], yk, kn, "k")
        assert (q[~live] == 7).all() and (k[rest] == 7).all()      # padding and other slots as they were


def test_prepare_in_place_and_without_slots():
    x = make(70, 64, 64, "rms", "layer", seed=3)
    a, b = call(x, False, False), call(x, False, False, q_out="in place")
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    c = call(x, False, False, slots=False)
    assert np.array_equal(c[1][:70], a[1][x["slot"]]) and (c[1][70:] == 7).all()


def test_prepare_far_positions():
    # a fraction of a turn at positions up to 2^31 - 1: fp64 angles, not fp32
    x = make(40, 32, 64, "none", "none", seed=4)
    x["pos"] = np.linspace(2 ** 31 - 4000, 2 ** 31 - 1, 40).astype(np.int32)
    y = ref.norm_rotate(ref.bf16_f64(x["q"]), x["pos"], x["inv_freq"], "none", None, None, 0, True)
    check_bf16(call(x, True, False)[0], ref.bf16_f64(x["q"]), y, "none", "far")


def test_prepare_zero_and_tiny_rows():
    x = make(6, 32, 64, "none", "none", seed=5)
    x["q"][1], x["k"][2] = 0, 0
    x["q"][3] = 0x0001                              # the smallest subnormal
    x["q"][4] = 0x7F00                              # close to the largest
    qc, qs, kc, ks = call(x, False, True)
    # zeros stay zeros in value; 0 cos - 0 sin is -0 where sin is negative
    assert (ref.E4M3[qc[1]] == 0).all() and (ref.E4M3[kc[x["slot"][2]]] == 0).all()
    assert (qs[1] == 1).all() and ks[x["slot"][2]] == 1
    assert np.isfinite(ref.E4M3[qc]).all() and (qs[3] == np.float32(2.0 ** -126)).all()
    y = ref.norm_rotate(ref.bf16_f64(x["q"]), x["pos"], x["inv_freq"], "none", None, None, 0, False)
    check_fp8(qc[4:5], qs[4:5], y[4:5], y[4:5], "none", "large")


def test_prepare_flags_bad_slots():
    x = make(9, 32, 64, "none", "rms", seed=6)
    x["slot"][2], x["slot"][5] = x["n"], -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = call(x, False, False, status=st)
    assert int(st) == 2
    ok = np.setdiff1d(np.arange(9), [2, 5])
    assert (np.delete(k, x["slot"][ok], 0) == 7).all() and not (q == 7).all(-1).any()


def test_prepare_replays_in_a_graph():
    xs = [make(33, 64, 64, "rms", "layer", seed=s, pad=5 * (s == 8)) for s in (7, 8)]
    ins = [gpu(xs[0][k]) for k in ("q", "k", "pos", "inv_freq", "slot", "q_weight", "k_weight", "k_bias")]
    k_out = torch.zeros((xs[0]["n"], 128), dtype=torch.bfloat16, device="cuda")
    q_out = torch.zeros_like(ins[0])
    go = lambda: dsa.dsa_index_prepare(*ins[:4], k_out, slot_map=ins[4], q_norm="rms", q_weight=ins[5], k_norm="layer",
                                       k_weight=ins[6], k_bias=ins[7], q_out=q_out)
    go()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for x in xs[::-1]:
        for dst, k in zip(ins, ("q", "k", "pos", "inv_freq", "slot", "q_weight", "k_weight", "k_bias")):
            dst.copy_(gpu(x[k]))
        q_out.fill_(7)
        graph.replay()
        want = call(x, False, False)
        assert np.array_equal(q_out.double().cpu().numpy(), want[0])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,rot,norms", [(1203, 5, 64, 1), (1190, 33, 32, 0), (1185, 64, 128, 2), (1184, 1, 16, 1)])
def test_prepare_many_tokens(T, H, rot, norms, interleaved, fp8):
    # enough tokens that a block takes a group of them; the last group is short
    # and padding rows end inside a group
    test_prepare(T, H, rot, norms, interleaved, fp8)


def test_prepare_many_tokens_in_place():
    x = make(1300, 20, 64, "rms", "rms", seed=31, pad=7)
    a = call(x, False, False)
    b = call(x, False, False, q_out="in place")
    assert np.array_equal(a[0][:-7], b[0][:-7]) and np.array_equal(a[1], b[1])
    assert np.array_equal(b[0][-7:], ref.bf16_f64(x["q"])[-7:])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H", [(40, 5), (320, 33), (1300, 4)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
def test_prepare_norms_over_their_range(norm, eps, T, H, fp8):
    # magnitudes over the whole range of a norm; then single rows beyond it, which are flagged and change no other
    rng = np.random.default_rng(T)
    x = make(T, H, 64, norm, norm, seed=T)
    size = 2.0 ** rng.integers(-46, 56, (T, H + 1))
    x["q"] = ref.bf16_bits(ref.bf16_f64(x["q"]) * size[:, :H, None])
    x["k"] = ref.bf16_bits(ref.bf16_f64(x["k"]) * size[:, H:])

    def run(x):
        a = [gpu(x[k]) for k in ("q", "k", "pos", "inv_freq")]
        kw = dict(slot_map=gpu(x["slot"]), eps=eps, q_norm=norm, k_norm=norm, status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                  **{k: gpu(x[k]) for k in ("q_weight", "q_bias", "k_weight", "k_bias")})
        if fp8:
            k_out, ks = torch.zeros((x["n"], 128), dtype=torch.uint8, device="cuda"), torch.zeros(x["n"], device="cuda")
            r = [t.cpu().numpy() for t in dsa.dsa_index_prepare_fp8(*a, k_out, ks, **kw)]
            return (r[0], r[2][x["slot"]], r[1], r[3][x["slot"]]), int(kw["status"])
        k_out = torch.zeros((x["n"], 128), dtype=torch.bfloat16, device="cuda")
        q, k = dsa.dsa_index_prepare(*a, k_out, **kw)
        return (q.double().cpu().numpy(), k.double().cpu().numpy()[x["slot"]]), int(kw["status"])

    good, st = run(x)
    assert st == 0
    raw_q, raw_k = ref.bf16_f64(x["q"]), ref.bf16_f64(x["k"])
    yq = ref.norm_rotate(raw_q, x["pos"], x["inv_freq"], norm, x["q_weight"], x["q_bias"], eps, False)
    yk = ref.norm_rotate(raw_k[:, None], x["pos"], x["inv_freq"], norm, x["k_weight"], x["k_bias"], eps, False)[:, 0]
    # bound() sees the rows at a size where its own floor of the deviation does not count
    unit = lambda r: r / np.abs(r).max(-1, keepdims=True)
    for i, (raw, y, name) in enumerate(((unit(raw_q), yq, "q"), (unit(raw_k), yk, "k"))):
        if fp8:
            check_fp8(good[i], good[2 + i], raw, y, norm, name)
        else:
            check_bf16(good[i], raw, y, norm, name)
    for e in (62, 100, 120) + ((-54, -90, -125) if eps == 0 else ()):
        for name, at in (("q", (T // 2, H - 1)), ("k", (T - 1,))):
            y = dict(x, **{name: x[name].copy()})
            row = rng.standard_normal(128)
            y[name][at] = ref.bf16_bits(row / np.sqrt((row * row).mean()) * 2.0 ** e)
            got, st = run(y)
            assert st == 8, (e, name)
            for i, (g, w) in enumerate(zip(got, good)):
                if "qk"[i % 2] == name:
                    g[at] = w[at]
                assert np.array_equal(g, w)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,rot,norms", [(297, 33, 64, 0), (301, 64, 32, 1), (741, 5, 128, 2), (999, 40, 64, 1)])
def test_prepare_tokens_in_small_groups(T, H, rot, norms, fp8):
    test_prepare(T, H, rot, norms, False, fp8)
