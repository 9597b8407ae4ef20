"""Non-finite inputs of the serving calls: status bit 3 (value 8), nothing else
disturbed, and no bit for finite inputs of any size."""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref
from tests import test_gpu_attend as att
from tests import test_gpu_prepare as prep
from tests.test_gpu_kv4 import bf, rows

pytestmark = pytest.mark.gpu

BAD = [0x7FC0, 0xFFC1, 0x7F80, 0xFF80]        # NaNs and infinities in bf16


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", BAD)
def test_cache_rows(bad):
    lat, rope = rows(33, 4)                                  # rotary bits: any
    pool = torch.zeros((40, 1, 416), dtype=torch.uint8, device="cuda")
    slot = torch.arange(33, dtype=torch.int32, device="cuda")
    st = word()
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot, status=st)
    assert int(st) == 0
    want = pool.clone()
    lat[17, 37] = bad
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot, status=st)
    assert int(st) == 8
    same = torch.arange(40, device="cuda") != 17
    assert torch.equal(pool[same], want[same])
    slot[17], st = -1, word()                                # padding
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot, status=st)
    assert int(st) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,norm", [(5, 33, "none"), (5, 7, "layer"), (1300, 3, "rms"), (310, 40, "rms")])
def test_prepared_rows(T, H, norm, fp8):
    x = prep.make(T, H, 64, norm, norm, seed=T, pad=2)
    st = word()
    good = prep.call(x, False, fp8, status=st)
    assert int(st) == 0
    for what, at in (("q", (T - 4, H - 1, 5)), ("k", (1, 99))):
        for bad in BAD:
            y, st = dict(x, **{what: x[what].copy()}), word()
            y[what][at] = bad
            got = prep.call(y, False, fp8, status=st)
            assert int(st) == 8, (what, hex(bad))
            row = (T - 4, H - 1) if what == "q" else x["slot"][1]
            for g, w, which in zip(got, good, "qqkk" if fp8 else "qk"):
                if which == what:
                    g[row] = w[row]
                assert np.array_equal(g, w)
    y, st = dict(x, q=x["q"].copy(), k=x["k"].copy()), word()
    y["q"][-1], y["k"][-1] = BAD[0], BAD[2]                  # padding is not looked at
    prep.call(y, False, fp8, status=st)
    assert int(st) == 0


@pytest.mark.parametrize("T,H", [(1, 16), (200, 16), (150, 64), (1, 128), (100, 128), (3, 70)])
@pytest.mark.parametrize("bad", BAD)
def test_attention(T, H, bad):
    x = att.make(T, H, 200, ctx=600, seed=T + H)
    ws = torch.empty(max(256, dsa.dsa_attend_kv4_workspace_bytes(T, H, 200)), dtype=torch.uint8, device="cuda")
    want = dsa.dsa_attend_kv4(scale=att.SCALE, workspace=ws, **att.gpu(x))
    assert dsa.dsa_index_device_status(ws) == 0
    y = dict(x, q=x["q"].copy())
    y["q"][0, H - 1, 100] = bad
    got = dsa.dsa_attend_kv4(scale=att.SCALE, workspace=ws, **att.gpu(y))
    assert dsa.dsa_index_device_status(ws) == 8
    assert torch.equal(got[0][1:], want[0][1:]) and torch.equal(got[0][0, :H - 1], want[0][0, :H - 1])
    assert torch.equal(got[1][1:], want[1][1:])
    y, st = dict(x, q=x["q"].copy()), word()
    y["q"][0, :, 512:] = ref.bf16_bits(np.full((H, 64), -1.0))
    y["entries"] = x["entries"].copy()
    y["entries"][:, 288 + 2 * 9: 288 + 2 * 9 + 2] = np.array([bad], np.uint16).view(np.uint8)   # every key: all -inf too
    dsa.dsa_attend_kv4(scale=att.SCALE, workspace=ws, status=st, **att.gpu(y))
    assert dsa.dsa_index_device_status(ws) == 8 and int(st) == 8


def test_a_nan_block_in_the_cache_shows():
    x = att.make(2, 16, 100, ctx=300, seed=3)
    row, slot = 1, int(x["table"][0, x["idx"][1, 50] // 64]) * 64 + int(x["idx"][1, 50]) % 64
    x["idx"][0][x["idx"][0] == x["idx"][1, 50]] = -1
    want = dsa.dsa_attend_kv4(scale=att.SCALE, **att.gpu(x))
    x["entries"][slot, 256 + 3] = 0x7F
    st = word()
    got = dsa.dsa_attend_kv4(scale=att.SCALE, status=st, **att.gpu(x))
    assert int(st) == 8 and torch.equal(got[0][0], want[0][0]) and torch.isnan(got[0][row]).any()


def test_empty_lists_and_large_finite_inputs_set_nothing():
    for T, H in ((3, 16), (200, 16), (3, 128), (90, 128)):
        x = att.make(T, H, 64, ctx=200, seed=H)
        x["idx"][::2] = -1
        x["q"] = ref.bf16_bits(ref.bf16_f64(x["q"]) * 1e6)
        st = word()
        dsa.dsa_attend_kv4(scale=att.SCALE, status=st, **att.gpu(x))
        assert int(st) == 0
