"""What chunk attention and the weight's layout refuse, on the host: no library
call is made for them, or none that launches."""
import pytest
import torch

import mla_decode_context_gb300 as dcp

I32, BF = torch.int32, torch.bfloat16


def args(**kw):
    a = dict(q=torch.zeros((5, 3, 192), dtype=BF), kv_cache=torch.zeros((2, 16, 576), dtype=BF),
             block_table=torch.zeros((2, 4), dtype=I32), seq_lens=torch.zeros(2, dtype=I32),
             query_start_loc=torch.zeros(3, dtype=I32), packed_kv_b=torch.zeros((3, 8, 256, 64), dtype=BF),
             out=torch.zeros((5, 3, 128), dtype=BF), lse=torch.zeros((5, 3)), workspace=None, scale=1.0, total_len=9)
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,kind", [
    (dict(), ValueError),  # (host tensors)
    (dict(q=torch.zeros((5, 3, 576), dtype=BF)), ValueError),
    (dict(q=torch.zeros((5, 3, 192))), TypeError),
    (dict(q=torch.zeros((5, 192, 3), dtype=BF).transpose(1, 2)), ValueError),
    (dict(kv_cache=torch.zeros((2, 16, 576), dtype=torch.uint8)), TypeError),
    (dict(kv_cache=torch.zeros((32, 576), dtype=BF)), ValueError),
    (dict(kv_scale=torch.zeros((2, 16))), ValueError),
    (dict(block_table=torch.zeros((3, 2, 4), dtype=I32), D=2), ValueError),
    (dict(block_table=torch.zeros((1, 4), dtype=I32)), ValueError),
    (dict(block_table=torch.zeros((2, 4), dtype=torch.int64)), TypeError),
    (dict(query_start_loc=torch.zeros(2, dtype=I32)), ValueError),
    (dict(packed_kv_b=torch.zeros((2, 8, 256, 64), dtype=BF)), ValueError),
    (dict(packed_kv_b=torch.zeros((3 * 256, 512), dtype=BF)), ValueError),
    (dict(out=torch.zeros((5, 3, 512), dtype=BF)), ValueError),
    (dict(out=torch.zeros((5, 3, 128), dtype=torch.float16)), TypeError),
    (dict(lse=torch.zeros((3, 5))), ValueError),
    (dict(dev_error=torch.zeros(0, dtype=I32)), ValueError),
    (dict(D=1 << 32), ValueError),
])
def test_refuses(bad, kind, monkeypatch):
    def launch(*a):
        raise AssertionError("reached the library")
    monkeypatch.setattr(dcp, "_launch", launch)
    with pytest.raises(kind):
        dcp.dcp_mla_chunk_attention(**args(**bad))


@pytest.mark.parametrize("w,packed,kind", [
    ((512, 512), (2, 8, 256, 64), ValueError),  # (host tensors)
    ((500, 512), (2, 8, 256, 64), ValueError), ((512, 576), (2, 8, 256, 64), ValueError),
    ((512, 512), (1, 8, 256, 64), ValueError), ((0, 512), (0, 8, 256, 64), ValueError)])
def test_layout_refuses(w, packed, kind):
    with pytest.raises(kind):
        dcp.dcp_pack_kv_b(torch.zeros(w, dtype=BF), torch.zeros(packed, dtype=BF))
    with pytest.raises(ValueError):
        dcp.pack_kv_b(torch.zeros((512, 512), dtype=BF), 3)


# the C entries, with addresses that are never followed
def call(L, **kw):
    a = dict(q=0x1000, qt=3 * 192, qh=192, kv=0x2000, kind=0, sc=None, nb=4, bs=16, table=0x3000, W=4, stride=4, per=0,
             shard_stride=0, D=2, I=1, seq=0x4000, qsl=0x5000, B=2, T=5, H=3, total=100, scale=0.07, w=0x6000,
             out=0x7000, dt=0, lse=0x8000, ws=0x10000, n=1 << 40)
    a.update(kw)
    return L.dcp_mla_chunk_attention(*a.values(), None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 0), (dict(T=0), 0), (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(H=1025), 1),
    (dict(total=-1), 1), (dict(total=1 << 40), 1), (dict(total=1 << 36, H=1024), 1), (dict(D=0), 1), (dict(D=33), 1),
    (dict(I=0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(kind=3), 2), (dict(dt=5), 2),
    (dict(q=None), 1), (dict(kv=None), 1), (dict(table=None), 1), (dict(seq=None), 1), (dict(qsl=None), 1),
    (dict(w=None), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(kind=1), 1), (dict(nb=0), 1), (dict(bs=0), 1),
    (dict(W=0), 1), (dict(stride=3), 1), (dict(qt=-192), 1), (dict(per=1, shard_stride=7), 1), (dict(q=0x1008), 3),
    (dict(qh=196), 3), (dict(out=0x7008), 3), (dict(ws=0x10008), 3), (dict(w=0x6004), 3), (dict(ws=None), 5),
    (dict(n=1000), 5)])
def test_c_refuses(bad, status):
    assert call(dcp.lib(), **bad) == status


def test_workspace_sizes():
    size = dcp.dcp_chunk_attention_workspace_size
    assert size(0, 5, 16, 0) == 0 and size(3, 0, 16, 100) == 0
    assert 0 < size(1, 9, 16, 9) < 1 << 21  # (a tile a head, its keys' remainders, no pieces)
    assert size(1, 512, 16, 4000) < size(1, 512, 128, 4000) <= size(2, 512, 128, 8000)
    assert size(1, 2048, 128, 1 << 20) < 5 << 30  # (passes over the heads)
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, 0, 1), (1, 1, 1, -1), (1, 1, 1, 1 << 60)):
        with pytest.raises(dcp.DCPError):
            size(*bad)
    with pytest.raises(ValueError):
        size(1 << 32, 1, 1, 1)
    L = dcp.lib()
    one = size(2, 5, 1, 100)
    assert call(L, n=one - 1) == 5
