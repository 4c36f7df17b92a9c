"""What the table extension refuses of a count of held blocks, on the host."""
import pytest
import torch

from tests.test_step_refusals_cpu import extend_args
import mla_decode_context_gb300 as dcp

I32 = torch.int32


@pytest.mark.parametrize("bad,kind", [
    (dict(held=torch.zeros(2, dtype=I32)), ValueError),  # (host tensors)
    (dict(held=torch.zeros(3, dtype=I32)), ValueError),
    (dict(held=torch.zeros((1, 2), dtype=I32)), ValueError),
    (dict(held=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(held=[0, 0]), TypeError),
    (dict(held=torch.zeros(2, dtype=I32), block_table=torch.zeros((3, 2, 4), dtype=I32), D=3), ValueError),
    (dict(held=torch.zeros((2, 3), dtype=I32), block_table=torch.zeros((3, 2, 4), dtype=I32), D=3), ValueError)])
def test_refuses(bad, kind, monkeypatch):
    def launch(*a):
        raise AssertionError("reached the library")
    monkeypatch.setattr(dcp, "_launch", launch)
    with pytest.raises(kind):
        dcp.dcp_cache_extend(**extend_args(**bad))


def call(L, **kw):
    a = dict(table=0x1000, W=4, stride=4, per=0, shard_stride=0, seq=0x2000, qsl=0x3000, B=2, T=5, bs=16, D=4, I=1,
             d0=0, Dn=4, free=0x4000, F=9, count=0x5000, left=0x5000, held=0x8000, pos=0x6000, slots=0x7000)
    a.update(kw)
    return L.dcp_cache_extend_v2(*a.values(), None, None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(bs=0), dict(table=None), dict(count=None), dict(pos=None), dict(W=0),
                                 dict(per=1, shard_stride=7)])
def test_c_refuses(bad):
    assert call(dcp.lib(), **bad) == 1
