"""Host side of the serving operators: argument refusals (no GPU is touched)
and the 64-bit references' own pins."""

import ctypes
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import sparse_attention_token_03_b200 as dsa
from tests import serve_ref as ref

P = ctypes.c_void_p
d = P(4096)


def tables(L, B=4, table=d, blocks=8, n_free=9, begin=P(512), n_pages=64, page=64, T=16, out=d, seq=P(1024), end=P(2048),
           status=None, cached=P(256)):
    return L.dsa_block_tables(cached, P(8192), B, table, blocks, d, n_free, begin, n_pages, page, T, out, out, out, d, seq,
                              end, status, None)


def test_block_tables_refusals():
    L = dsa.lib()
    assert tables(L, B=0) == -1 and tables(L, B=65537) == -1
    assert tables(L, blocks=0) == -1 and tables(L, page=0) == -1 and tables(L, n_pages=0) == -1
    assert tables(L, n_pages=1 << 25) == -1          # n_pages * page_size reaches 2^31
    assert tables(L, n_pages=1 << 62) == -1          # and must not wrap
    assert tables(L, blocks=1 << 25) == -1
    assert tables(L, T=-1) == -1 and tables(L, T=1 << 30) == -1 and tables(L, n_free=-1) == -1
    assert tables(L, table=None) == -1 and tables(L, out=None) == -1 and tables(L, begin=None) == -1
    assert tables(L, status=P(6)) == -1 and tables(L, table=P(18)) == -1
    assert tables(L, end=P(512)) == -1 and tables(L, seq=P(256)) == -1     # aliases
    assert b"alias" in L.dsa_last_error_string()


def prepare(L, T=4, H=64, width=128, rot=64, qn=0, qw=None, qb=None, kn=2, kw=None, kb=None, eps=1e-6, slots=d, n=64,
            q=d, k=d, q_out=d, k_out=d, freq=d, fp8=False, scale=d):
    a = (q, k, d, freq, rot, T, H, width, qn, qw, qb, kn, kw, kb, eps, 0, slots, n, q_out)
    if fp8:
        return L.dsa_index_prepare_fp8(*a, scale, k_out, scale, None, None)
    return L.dsa_index_prepare(*a, k_out, None, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_prepare_refusals(fp8):
    L = dsa.lib()
    go = lambda **kw: prepare(L, fp8=fp8, **kw)
    assert go(width=64) == -2 and go(H=0) == -2 and go(H=257) == -2
    assert go(rot=8) == -2 and go(rot=144) == -2 and go(rot=-16) == -2
    assert go(qn=3) == -2 and go(kn=-1) == -2
    assert go(qw=d) == -1 and go(qb=d) == -1 and go(kn=0, kb=d) == -1     # weight or bias without a norm
    assert go(eps=-1.0) == -1 and go(eps=float("nan")) == -1
    assert go(T=-1) == -1 and go(T=1 << 30) == -1 and go(n=-1) == -1 and go(n=1 << 31) == -1
    assert go(slots=None, n=3) == -1                                       # row t to slot t needs n_slots >= T
    assert go(q=None) == -1 and go(k=None) == -1 and go(freq=None) == -1 and go(k_out=None) == -1
    assert go(q=P(8)) == -1 and go(k_out=P(8)) == -1 and go(kw=P(8)) == -1
    assert go(T=0, q=None, k=None, q_out=None, k_out=None) == 0
    if fp8:
        assert go(scale=None) == -1


def test_kv4_refusals():
    L = dsa.lib()
    for f in (lambda lat=d, rope=d, kv=d, n=8, slots=d, T=4, st=None: L.dsa_kv4_write(lat, rope, kv, n, slots, T, st, None),
              lambda lat=d, rope=d, kv=d, n=8, slots=d, T=4, st=None: L.dsa_kv4_read(kv, n, slots, T, lat, rope, st, None)):
        assert f(T=-1) == -1 and f(T=1 << 31) == -1 and f(n=-1) == -1 and f(n=1 << 31) == -1
        assert f(lat=None) == -1 and f(rope=None) == -1 and f(kv=None) == -1 and f(slots=None) == -1
        assert f(lat=P(8)) == -1 and f(kv=P(16)) == -1 and f(st=P(2)) == -1
        assert f(T=0, lat=None, rope=None, kv=None, slots=None) == 0


def attend(L, q=d, kv=d, n_pages=8, page=64, table=d, B=2, blocks=4, seq=d, idx=d, T=2, H=16, n=128, scale=0.1, out=d,
           lse=d, ws=d, need=None, st=None):
    need = L.dsa_attend_kv4_workspace_bytes(T, H, n) if need is None else need
    return L.dsa_attend_kv4(q, kv, n_pages, page, table, B, blocks, seq, idx, T, H, n, scale, out, lse, ws, need, st, None)


def test_attend_refusals():
    L = dsa.lib()
    assert attend(L, H=0) == -2 and attend(L, H=257) == -2
    assert attend(L, n=0) == -1 and attend(L, n=(1 << 30) + 1, need=1 << 40) == -1 and attend(L, T=-1) == -1 and attend(L, T=1 << 31, need=1 << 40) == -1
    assert attend(L, page=0) == -1 and attend(L, n_pages=1 << 31) == -1 and attend(L, blocks=1 << 28) == -1
    assert attend(L, scale=float("inf")) == -1 and attend(L, scale=float("nan")) == -1
    assert attend(L, B=0) == -1 and attend(L, seq=None, T=3) == -1
    for name in ("q", "kv", "table", "idx", "out", "ws"):
        assert attend(L, **{name: None}) == -1, name
    assert attend(L, q=P(8)) == -1 and attend(L, kv=P(16)) == -1 and attend(L, out=P(8)) == -1
    assert attend(L, ws=P(128)) == -1 and attend(L, st=P(2)) == -1 and attend(L, lse=P(2)) == -1
    need = L.dsa_attend_kv4_workspace_bytes(2, 16, 128)
    assert need >= 256 and attend(L, need=need - 1) == -3
    assert L.dsa_attend_kv4_workspace_bytes(2, 0, 128) == 0 and L.dsa_attend_kv4_workspace_bytes(2, 16, 0) == 0
    assert attend(L, T=0, q=None, idx=None, out=None, ws=None) == 0


def test_attend_refuses_lists_longer_than_its_sums_hold():
    L = dsa.lib()
    for n in ((1 << 20) + 1, 1 << 22, 1 << 30):
        assert attend(L, n=n, need=1 << 40) == -1 and b"2^20" in L.dsa_last_error_string()
        assert L.dsa_attend_kv4_workspace_bytes(2, 16, n) == 0
    assert L.dsa_attend_kv4_workspace_bytes(2, 16, 1 << 20) > 256


def test_binding_refuses_wrong_tensors():
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32)
    with pytest.raises(ValueError):   # not on a CUDA device
        dsa.dsa_index_prepare(q, q[:, 0].contiguous(), i, f, torch.zeros((2, 128), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        dsa.dsa_index_prepare(q.float(), q[:, 0].contiguous(), i, f, torch.zeros((2, 128), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        dsa.dsa_kv4_read(torch.zeros((2, 64, 416)), i)
    with pytest.raises(ValueError):
        dsa.dsa_kv4_read(torch.zeros((2, 64, 416), dtype=torch.uint8), i)
    with pytest.raises(TypeError):
        dsa.dsa_attend_kv4(q, torch.zeros((2, 64, 416), dtype=torch.int8), i, i, 1.0)
    with pytest.raises(TypeError):
        dsa.dsa_block_tables(i.long(), i, i.view(2, 1), i, i[:1], 4, 64, 8)


def test_library_does_not_need_the_native_host_side():
    # no object, no compiler: the index calls load as they are, the serving calls warn once and check in Python
    code = """
import os, warnings
from pathlib import Path
os.environ["CXX"] = "/bin/false"
import torch
import sparse_attention_token_03_b200 as dsa
from sparse_attention_token_03_b200 import build
build.BINDING = Path("/nonexistent/none.so")
with warnings.catch_warnings():
    warnings.simplefilter("error")
    assert dsa.dsa_index_prefill_workspace_bytes(4, 4, 64, 128, 8) > 0
    assert dsa.lib(build_if_missing=False) is dsa.lib()
slots = torch.zeros(2, dtype=torch.int32)
for i in range(2):
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        try:
            dsa.dsa_kv4_read(torch.zeros((2, 64, 416), dtype=torch.uint8), slots)
            raise SystemExit("accepted a CPU tensor")
        except ValueError as e:
            assert "CUDA" in str(e)
    assert [w.category for w in seen] == ([RuntimeWarning] if i == 0 else []), seen
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=Path(__file__).resolve().parent.parent, timeout=300)


def test_native_host_side_is_built_for_one_torch_and_python(tmp_path, monkeypatch):
    from sparse_attention_token_03_b200 import build
    tag = sys.implementation.cache_tag
    assert build.BINDING == build.binding_path(torch.__version__, tag)
    # an object of another torch or Python is another file: it is neither loaded nor taken for this one's
    other = [build.binding_path(torch.__version__, "cpython-399"), build.binding_path("9.9.9", tag)]
    assert len({build.BINDING, *other}) == 3
    monkeypatch.setattr(build, "PKG", tmp_path)
    for p in other:
        (tmp_path / p.name).write_bytes(b"")
    monkeypatch.setattr(build, "BINDING", build.binding_path(torch.__version__, tag))
    assert build.binding_stale()


def test_reference_formats():
    # E4M3 against torch's own conversion; E2M1 rounding at its midpoints (ties to the even code)
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(ref.E4M3, t, equal_nan=True)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    assert list(ref.nearest_even(mids, ref.E2M1)) == [0, 2, 2, 4, 4, 6, 6, 7]
    # what the cache holds is exact: encoding a decoded row changes nothing
    rng = np.random.default_rng(5)
    x = ref.bf16_f64(ref.bf16_bits(rng.standard_normal((9, 512)) * np.exp(rng.standard_normal((9, 1)) * 2)))
    e = ref.kv4_encode(x, rng.integers(0, 1 << 15, (9, 64)))
    lat, _ = ref.kv4_decode(e)
    # half a step of E2M1 (1 at the largest code's scale) and the scale's own rounding by 2^-4
    assert (np.abs(lat - x) <= np.repeat(np.abs(x.reshape(9, 32, 16)).max(-1), 16, 1) * (1 / 6 + 2.0 ** -4)).all()
    assert np.array_equal(lat, ref.bf16_f64(ref.bf16_bits(lat)))
