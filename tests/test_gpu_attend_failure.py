"""Attention's bounded waits, run out on purpose by the host-armed injection (the
list warps stop behind their first tiles; nothing faults or hangs): every role
of the kernels gives up, the launch returns, the status words carry the timeout
bit, and the next call is exact."""

import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests.test_gpu_attend import SCALE, check, gpu, make

pytestmark = pytest.mark.gpu

LIMIT_NS = 50_000_000  # 50 ms


# one row and split lists, rows for every block and more, lists of one tile (the wait is between rows) and of several
@pytest.mark.parametrize("n", [40, 1000])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 40), (200, 16), (200, 32), (200, 64), (1, 128), (9, 100), (160, 128)])
def test_waits_give_up_and_the_next_call_is_exact(T, H, n):
    x = make(T, H, n, B=2, ctx=1500, seed=T + H)
    g = gpu(x)
    ws = torch.full((max(256, dsa.dsa_attend_kv4_workspace_bytes(T, H, n)),), 0x5A, dtype=torch.uint8, device="cuda")
    want = dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, **g)
    assert dsa.dsa_index_device_status(ws) == 0
    dsa.dsa_test_inject_wait_timeout(LIMIT_NS)
    dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, **g)
    torch.cuda.synchronize()
    assert dsa.dsa_index_device_status(ws) == 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dsa.dsa_test_inject_wait_timeout(LIMIT_NS)
    dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, status=st, **g)
    assert int(st) == 1
    got = dsa.dsa_attend_kv4(scale=SCALE, workspace=ws, **g)
    assert dsa.dsa_index_device_status(ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if T < 10:
        check(x)


def test_row_numbers_past_their_field():
    # some 400 rows a block: the row number that travels with a tile has 8 bits
    T, n = 60_000, 3
    x = make(1, 1, n, ctx=300, seed=1)
    g = gpu(x)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    q = torch.randn((T, 1, 576), generator=gen, device="cuda").bfloat16()
    idx = torch.randint(0, 300, (T, n), generator=gen, device="cuda", dtype=torch.int32)
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    seq[::11] = -1
    out = torch.full((T, 1, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_attend_kv4(q, g["kv_pages"], g["block_table"], idx, SCALE, row_seq=seq, out=out)
    want = torch.full_like(out, 5.0)
    for a in range(0, T, 148):                     # one row a block
        b = min(a + 148, T)
        dsa.dsa_attend_kv4(q[a:b], g["kv_pages"], g["block_table"], idx[a:b], SCALE, row_seq=seq[a:b], out=want[a:b])
    assert torch.equal(out, want) and (out[::11] == 5).all() and not (out[1::11] == 5).all(-1).any()
