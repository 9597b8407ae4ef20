"""The serving calls' native host side: what it leaves to the Python checks
gives the same results, and its errors are the library's."""

import pytest
import torch

import sparse_attention_token_03_b200 as dsa

pytestmark = pytest.mark.gpu


class Sub(torch.Tensor):
    pass


def tokens(T=9, H=32):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    i = torch.arange(T, device="cuda", dtype=torch.int32)
    return dict(q=r(T, H, 128).bfloat16(), k=r(T, 128).bfloat16(), position=i * 100, inv_freq=torch.rand(32, device="cuda"),
                w=1 + 0.1 * r(128), latent=r(T, 512).bfloat16(), rope=r(T, 64).bfloat16(), slot=i.flip(0).contiguous())


def test_subclasses_and_parameters_give_the_same():
    x = tokens()
    call = lambda q, w: dsa.dsa_index_prepare(q, x["k"], x["position"], x["inv_freq"],
                                              torch.zeros((9, 128), dtype=torch.bfloat16, device="cuda"),
                                              q_norm="rms", q_weight=w)
    a = call(x["q"], x["w"])
    b = call(x["q"].as_subclass(Sub), torch.nn.Parameter(x["w"]))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_fp8_tensors_and_bytes_give_the_same():
    x, got = tokens(), []
    for t in (torch.uint8, torch.float8_e4m3fn):
        k = torch.zeros((9, 128), dtype=torch.uint8, device="cuda").view(t)
        q = torch.zeros((9, 32, 128), dtype=torch.uint8, device="cuda").view(t)
        r = dsa.dsa_index_prepare_fp8(x["q"], x["k"], x["position"], x["inv_freq"], k,
                                      torch.ones(9, device="cuda"), q_out=q)
        assert r[0] is q and r[2] is k
        got.append([u.view(torch.uint8) if u.element_size() == 1 else u for u in r])
    assert all(torch.equal(u, v) for u, v in zip(*got))


def test_outputs_are_given_back():
    x = tokens()
    kv = torch.zeros((2, 16, 416), dtype=torch.uint8, device="cuda")
    assert dsa.dsa_kv4_write(x["latent"], x["rope"], kv, x["slot"]) is kv
    lat, rope = torch.empty_like(x["latent"]), torch.empty_like(x["rope"])
    r = dsa.dsa_kv4_read(kv, x["slot"], latent_out=lat, rope_out=rope)
    assert r[0] is lat and r[1] is rope
    assert all(torch.equal(u, v) for u, v in zip(dsa.dsa_kv4_read(kv, x["slot"]), r))
    q = torch.randn((9, 16, 576), device="cuda").bfloat16()
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    seq = torch.zeros(9, dtype=torch.int32, device="cuda")
    idx = torch.arange(9, dtype=torch.int32, device="cuda").repeat(9, 1)
    a = dsa.dsa_attend_kv4(q, kv, table, idx, 0.1, row_seq=seq)
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    b = dsa.dsa_attend_kv4(q, kv, table, idx, 0.1, row_seq=seq, out=out, lse=lse)
    assert b[0] is out and b[1] is lse and torch.equal(a[0], out) and torch.equal(a[1], lse)


def test_layout_outputs_given_or_not():
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = lambda: torch.tensor([[3, -1, -1], [5, 6, -1]], dtype=torch.int32, device="cuda")
    args = lambda t: (i(60, 100), i(10, 1), t, i(7, 8, 9), i(0), 10, 64, 13)
    t1, t2 = table(), table()
    a = dsa.dsa_block_tables(*args(t1))
    outs = [torch.full_like(u, 99) for u in a]
    b = dsa.dsa_block_tables(*args(t2), *outs)
    assert all(u is v for u, v in zip(b, outs))
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and torch.equal(t1, t2)
    a[0].fill_(-5)                               # parts of one allocation, but tensors of their own
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2]) and a[0].shape == (13,)


def test_the_librarys_errors():
    x = tokens()
    kv = torch.zeros((2, 16, 416), dtype=torch.uint8, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(dsa.DSAError):
        dsa.dsa_block_tables(i, i, i.view(2, 1), i, i[:1], 4, 0, 8)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_attend_kv4(torch.zeros((1, 300, 576), dtype=torch.bfloat16, device="cuda"), kv, i.view(1, 2),
                           i.view(1, 2), 1.0)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_index_prepare(x["q"], x["k"], x["position"], x["inv_freq"][:3].contiguous(),
                              torch.zeros((9, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        dsa.dsa_kv4_write(x["latent"][:, ::2].contiguous(), x["rope"], kv, x["slot"])
    with pytest.raises(ValueError):
        dsa.dsa_kv4_write(x["latent"].t().contiguous().t(), x["rope"], kv, x["slot"])
    with pytest.raises(TypeError):
        dsa.dsa_kv4_read(kv, x["slot"].long())


def test_python_checks_alone_give_the_same(monkeypatch):
    # every serving call with the native host side and, as where it cannot be built, without it
    x = tokens(70)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    seq, q_att = torch.zeros(70, dtype=torch.int32, device="cuda"), torch.randn((70, 40, 576), device="cuda").bfloat16()

    def step():
        table = i(3, -1, -1).view(1, 3)
        out = list(dsa.dsa_block_tables(i(20), i(70), table, i(0, 1, 2), i(0), 4, 64, 75)) + [table]
        slot = out[0][:70].contiguous()
        pool = torch.zeros((4, 64, 128), dtype=torch.bfloat16, device="cuda")
        out += dsa.dsa_index_prepare(x["q"], x["k"], x["position"], x["inv_freq"], pool, slot_map=slot, k_norm="rms", k_weight=x["w"])
        k8, ks = torch.zeros((4, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((4, 64), device="cuda")
        out += dsa.dsa_index_prepare_fp8(x["q"], x["k"], x["position"], x["inv_freq"], k8, ks, slot_map=slot, interleaved=True)
        kv = dsa.dsa_kv4_write(x["latent"], x["rope"], torch.zeros((4, 64, 416), dtype=torch.uint8, device="cuda"), slot)
        out += [kv, *dsa.dsa_kv4_read(kv, slot)]
        idx = torch.arange(20, 90, dtype=torch.int32, device="cuda").repeat(70, 1)
        return out + list(dsa.dsa_attend_kv4(q_att, kv, table, idx, 0.1, row_seq=seq))

    a = step()
    assert dsa._serve is not dsa._NoBinding
    monkeypatch.setattr(dsa, "_serve", dsa._NoBinding)
    b = step()
    assert len(a) == len(b) and all(torch.equal(u, v) for u, v in zip(a, b))
