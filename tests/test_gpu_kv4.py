"""The 4-bit latent cache: stored bytes equal the 64-bit reference's, rows read
back are exact."""

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


def bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def rows(T, seed):
    rng = np.random.default_rng(seed)
    lat = rng.standard_normal((T, 512)) * np.exp(rng.standard_normal((T, 1)))
    # exact ties, zeros of both signs, blocks below and above the scale's range
    lat[rng.random((T, 512)) < 0.05] = 0.0
    lat[:, 16:32] = np.round(lat[:, 16:32] * 4) / 4
    lat[:, 16] = 6.0
    lat[:, 32:48] *= 1e-4
    lat[:, 48:64] *= 1e5
    lat[:, 64:80] = -0.0
    return ref.bf16_bits(lat), rng.integers(0, 1 << 16, (T, 64)).astype(np.uint16)


@pytest.mark.parametrize("T,page,pad", [(1, 64, 0), (7, 1, 2), (64, 64, 0), (65, 192, 7), (1201, 64, 13)])
def test_write_and_read(T, page, pad):
    lat, rope = rows(T, T)
    n_pages = -(-T // page) + 2
    rng = np.random.default_rng(T + 1)
    slot = rng.permutation(n_pages * page)[:T].astype(np.int32)
    slot[T - pad:] = -1
    pool = torch.full((n_pages, page, 416), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.from_numpy(slot).cuda()
    assert dsa.dsa_kv4_write(bf(lat), bf(rope), pool, s, status=st) is pool
    back = [torch.full((T, w), 3.0, dtype=torch.bfloat16, device="cuda") for w in (512, 64)]
    dsa.dsa_kv4_read(pool, s, *back, status=st)
    torch.cuda.synchronize()
    want = np.full((n_pages * page, 416), 0xA5, np.uint8)
    live = slot >= 0
    want[slot[live]] = ref.kv4_encode(ref.bf16_f64(lat[live]), rope[live])
    assert np.array_equal(pool.cpu().numpy().reshape(-1, 416), want) and int(st) == 0
    dec, _ = ref.kv4_decode(want[slot[live]])
    assert np.array_equal(back[0].double().cpu().numpy()[live], dec)
    assert np.array_equal(back[1].view(torch.int16).cpu().numpy().view(np.uint16)[live], rope[live])
    assert (back[0].cpu()[~live] == 3).all() and (back[1].cpu()[~live] == 3).all()


def test_every_code_and_scale_reads_exactly():
    # 127 scales x all codes, laid down as bytes
    e = np.zeros((127, 416), np.uint8)
    e[:, :256] = np.arange(256)
    e[:, 256:288] = np.arange(127)[:, None]
    pool = torch.from_numpy(e).cuda().view(127, 1, 416)
    lat, _ = dsa.dsa_kv4_read(pool, torch.arange(127, dtype=torch.int32, device="cuda"))
    assert np.array_equal(lat.double().cpu().numpy(), ref.kv4_decode(e)[0])


def test_bad_slots_are_skipped_and_flagged():
    lat, rope = rows(5, 3)
    pool = torch.zeros((1, 8, 416), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    slot = torch.tensor([0, 8, 2, 2 ** 31 - 1, -1], dtype=torch.int32, device="cuda")
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot, status=st)
    assert int(st) == 2 and not pool[0, [1, 3, 4, 5, 6, 7]].any() and pool[0, 0].any() and pool[0, 2].any()
    st.zero_()
    out = [torch.full((5, w), 3.0, dtype=torch.bfloat16, device="cuda") for w in (512, 64)]
    dsa.dsa_kv4_read(pool, slot, *out, status=st)
    assert int(st) == 2 and (out[0][[1, 3, 4]] == 3).all()
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot)          # without a status word
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    n = (1 << 32) // 416 + 1000                               # a pool of more than 4 GiB
    pool = torch.empty((n, 1, 416), dtype=torch.uint8, device="cuda")
    slot = torch.tensor([n - 1, 3, n - 500], dtype=torch.int32, device="cuda")
    pool[[3, n - 500, n - 1]] = 0
    lat, rope = rows(3, 9)
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot)
    got = pool[slot.long()].cpu().numpy().reshape(3, 416)
    assert np.array_equal(got, ref.kv4_encode(ref.bf16_f64(lat), rope))
    back, _ = dsa.dsa_kv4_read(pool, slot)
    assert np.array_equal(back.double().cpu().numpy(), ref.kv4_decode(got)[0])


@pytest.mark.parametrize("T", [1, 9, 2000])
def test_nan_stays_and_infinity_saturates(T):
    # a NaN (of either sign, at any place of its block) makes the block NaN and no other; an infinity is the largest value
    lat, rope = rows(T, 21)
    rng = np.random.default_rng(T)
    at = rng.integers(0, 512, T)
    lat[np.arange(T), at] = np.where(np.arange(T) % 2, 0x7FC0, 0xFF81)
    inf = (at + 16 * (1 + rng.integers(0, 30, T))) % 512
    lat[np.arange(T), inf] = np.where(np.arange(T) % 3, 0x7F80, 0xFF80)
    pool = torch.zeros((T, 1, 416), dtype=torch.uint8, device="cuda")
    slot = torch.arange(T, dtype=torch.int32, device="cuda")
    dsa.dsa_kv4_write(bf(lat), bf(rope), pool, slot)
    x = ref.bf16_f64(lat).reshape(T, 32, 16)
    nan_block = np.isnan(x).any(-1)
    fill = np.where(np.isinf(x), np.sign(x) * 1e6, np.where(nan_block[..., None], 0.0, x)).reshape(T, 512)
    want = ref.kv4_encode(fill, rope)
    want[:, 256:288][nan_block] = 0x7F
    got = pool.cpu().numpy().reshape(T, 416)
    codes = want[:, :256].reshape(T, 32, 8)
    codes[nan_block] = 0
    assert np.array_equal(got, want)
    back, _ = dsa.dsa_kv4_read(pool, slot)
    assert np.array_equal(back.double().cpu().numpy(), ref.kv4_decode(want)[0], equal_nan=True)
    assert (torch.isnan(back).reshape(T, 32, 16).all(-1).cpu().numpy() == nan_block).all()
