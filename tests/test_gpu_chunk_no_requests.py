"""A step without requests: rows of no request are zeros and -inf."""
import pytest
import torch

import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu


def tensors(T, H, local):
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    return dict(q=torch.full((T, H, 192), float("nan"), dtype=torch.bfloat16, device="cuda"),
                kv_cache=torch.zeros((2, 16, 576), dtype=torch.bfloat16, device="cuda"),
                block_table=e.view(3, 0, 4) if local else e.view(0, 4), seq_lens=e,
                query_start_loc=torch.zeros(1, dtype=torch.int32, device="cuda"),
                packed_kv_b=torch.zeros((H, 8, 256, 64), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,local", [(1, 1, False), (5, 3, False), (1001, 7, True)])
def test_rows_are_padding(T, H, local, dtype):
    t = tensors(T, H, local)
    kw = dict(scale=0.1, total_len=0, D=3 if local else 1)
    # twice the rows: the others stay as they were
    big, big_lse = torch.full((2 * T, H, 128), 7.0, dtype=dtype, device="cuda"), torch.full((2 * T, H), 7.0, device="cuda")
    dcp.dcp_mla_chunk_attention(**t, out=big[:T], lse=big_lse[:T], workspace=None, **kw)
    assert (big[:T] == 0).all() and (big_lse[:T] == -torch.inf).all()
    assert (big[T:] == 7).all() and (big_lse[T:] == 7).all()
    # the allocating form, on memory that held something else
    torch.full((T, H, 128), 7.0, dtype=dtype, device="cuda")
    out, lse = dcp.chunk_attention(**t, out_dtype=dtype, **kw)
    assert (out == 0).all() and (lse == -torch.inf).all()


def test_on_a_side_stream_and_captured():
    t = tensors(5, 3, False)
    out, lse = torch.full((5, 3, 128), 7.0, device="cuda"), torch.full((5, 3), 7.0, device="cuda")

    def call(**kw):
        dcp.dcp_mla_chunk_attention(**t, out=out, lse=lse, workspace=None, scale=0.1, total_len=0, **kw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.fill_(7), lse.fill_(7)
    graph.replay()
    assert (out == 0).all() and (lse == -torch.inf).all()
    out.fill_(7), lse.fill_(7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert (out == 0).all() and (lse == -torch.inf).all()
    out.fill_(7), lse.fill_(7)
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side.cuda_stream)
    side.synchronize()
    assert (out == 0).all() and (lse == -torch.inf).all()


def test_no_rows():
    t = tensors(0, 3, False)
    out, lse = dcp.chunk_attention(**t, scale=0.1, total_len=0)
    assert out.shape == (0, 3, 128) and lse.shape == (0, 3)
