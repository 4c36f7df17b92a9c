"""What the table extension and the norm-and-rotation call refuse, on the host:
no library call is made for them."""
import pytest
import torch

import mla_decode_context_gb300 as dcp

I32, I64, BF, F32 = torch.int32, torch.int64, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def launch(*a):
        raise AssertionError("reached the library")
    monkeypatch.setattr(dcp, "_launch", launch)


def extend_args(**kw):
    a = dict(block_table=torch.zeros((2, 4), dtype=I32), seq_lens=torch.zeros(2, dtype=I32),
             query_start_loc=torch.zeros(3, dtype=I32), free_blocks=torch.zeros(9, dtype=I32),
             free_count=torch.zeros(1, dtype=I32), free_left=torch.zeros(1, dtype=I32),
             positions=torch.zeros(5, dtype=I32), slot_mapping=torch.zeros(5, dtype=I64), block_size=16)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,kind", [
    (dict(), ValueError),  # (host tensors)
    (dict(block_table=torch.zeros((2, 4), dtype=I64)), TypeError),
    (dict(block_table=torch.zeros((3, 4), dtype=I32)), ValueError),
    (dict(block_table=torch.zeros((4, 2), dtype=I32).t()), ValueError),
    (dict(block_table=torch.zeros((3, 2, 4), dtype=I32), D=2), ValueError),
    (dict(query_start_loc=torch.zeros(2, dtype=I32)), ValueError),
    (dict(seq_lens=torch.zeros(2, dtype=I64)), TypeError),
    (dict(free_blocks=torch.zeros((3, 3), dtype=I32)), ValueError),
    (dict(free_count=torch.zeros(2, dtype=I32)), ValueError),
    (dict(free_left=torch.zeros(1, dtype=I64)), TypeError),
    (dict(positions=torch.zeros(5, dtype=I64)), TypeError),
    (dict(slot_mapping=torch.zeros(4, dtype=I64)), ValueError),
    (dict(slot_mapping=torch.zeros(5, dtype=I32)), TypeError),
    (dict(dev_error=torch.zeros(0, dtype=I32)), ValueError),
    (dict(block_size=1 << 32), ValueError),
    (dict(interleave=1 << 31), ValueError),
    (dict(block_table=None), TypeError),
])
def test_extend_refuses(bad, kind):
    with pytest.raises(kind):
        dcp.dcp_cache_extend(**extend_args(**bad))


def rope_args(**kw):
    a = dict(ql_nope=torch.zeros((5, 3, 512), dtype=BF), q_pe=torch.zeros((5, 3, 64), dtype=BF),
             q_out=torch.zeros((5, 3, 576), dtype=BF), kv_c=torch.zeros((5, 512), dtype=BF),
             k_pe=torch.zeros((5, 64), dtype=BF), norm_weight=torch.zeros(512, dtype=BF),
             positions=torch.zeros(5, dtype=I32), cos_sin=torch.zeros((8, 64)), slot_mapping=torch.zeros(5, dtype=I64),
             kv_cache=torch.zeros((2, 16, 576), dtype=BF))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,kind", [
    (dict(), ValueError),  # (host tensors)
    (dict(ql_nope=None), ValueError),  # q_out's width is the decode query's
    (dict(q_pe=None), TypeError),
    (dict(q_out=None), TypeError),
    (dict(q_out=torch.zeros((5, 3, 64), dtype=BF)), ValueError),
    (dict(ql_nope=torch.zeros((5, 2, 512), dtype=BF)), ValueError),
    (dict(q_pe=torch.zeros((5, 3, 64))), TypeError),
    (dict(kv_c=torch.zeros((512, 5), dtype=BF).t()), ValueError),
    (dict(k_pe=torch.zeros((4, 64), dtype=BF)), ValueError),
    (dict(norm_weight=torch.zeros(512)), TypeError),
    (dict(norm_weight=torch.zeros(64, dtype=BF)), ValueError),
    (dict(positions=torch.zeros(5, dtype=I64)), TypeError),
    (dict(positions=torch.zeros(4, dtype=I32)), ValueError),
    (dict(cos_sin=torch.zeros((8, 32))), ValueError),
    (dict(cos_sin=torch.zeros((8, 64), dtype=BF)), TypeError),
    (dict(cos_sin=torch.zeros((0, 64))), ValueError),
    (dict(slot_mapping=torch.zeros(5, dtype=I32)), TypeError),
    (dict(kv_cache=torch.zeros((2, 16, 576), dtype=torch.uint8)), TypeError),
    (dict(kv_scale=torch.zeros((2, 16))), ValueError),
    (dict(dev_error=torch.zeros(0, dtype=I32)), ValueError),
])
def test_norm_rope_refuses(bad, kind):
    with pytest.raises(kind):
        dcp.dcp_norm_rope_cache(**rope_args(**bad))


# the C entries, with addresses that are never followed
def c_extend(L, **kw):
    a = dict(table=0x1000, W=4, stride=4, per=0, shard_stride=0, seq=0x2000, qsl=0x3000, B=2, T=5, bs=16, D=4, I=1,
             d0=0, Dn=4, free=0x4000, F=9, count=0x5000, left=0x5000, pos=0x6000, slots=0x7000)
    a.update(kw)
    return L.dcp_cache_extend(*a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(D=0), dict(D=33), dict(I=0), dict(bs=0), dict(d0=-1), dict(Dn=0), dict(d0=1), dict(F=-1),
    dict(table=None), dict(seq=None), dict(qsl=None), dict(free=None), dict(count=None), dict(left=None),
    dict(pos=None), dict(slots=None), dict(W=0), dict(W=(1 << 20) + 1, stride=1 << 21), dict(stride=3),
    dict(per=1, shard_stride=7)])
def test_extend_c_refuses(bad):
    assert c_extend(dcp.lib(), **bad) == 1


def c_rope(L, **kw):
    a = dict(ql=0x1000, ql_t=512, ql_h=5 * 512, qp=0x2000, qp_t=192, qp_h=64, qo=0x3000, qo_t=3 * 576, qo_h=576, c=0x4000,
             c_t=576, k=0x5000, k_t=576, w=0x6000, eps=1e-6, pos=0x7000, cs=0x8000, top=100, il=1, slots=0x9000, T=5,
             H=3, cache=0xa000, kind=0, scale=None, n=32)
    a.update(kw)
    return L.dcp_norm_rope_cache(*a.values(), None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), 0), (dict(T=-1), 1), (dict(H=-1), 1), (dict(n=0), 1), (dict(top=0), 1), (dict(kind=2), 2),
    (dict(c=None), 1), (dict(k=None), 1), (dict(pos=None), 1), (dict(cs=None), 1), (dict(slots=None), 1),
    (dict(cache=None), 1), (dict(kind=1), 1), (dict(H=0), 1), (dict(qp=None), 1), (dict(qo=None), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(c_t=-576), 1), (dict(c_t=570), 3), (dict(k_t=4), 3),
    (dict(w=0x6008), 3), (dict(cs=0x8004), 3), (dict(cache=0xa008), 3), (dict(ql_h=4), 3), (dict(qo_h=512), 1),
    (dict(qo_t=576), 1), (dict(ql=None, qo_h=64, qo_t=128), 1), (dict(qo=0x3008), 3), (dict(qp_t=-64), 1)])
def test_norm_rope_c_refuses(bad, status):
    assert c_rope(dcp.lib(), **bad) == status
