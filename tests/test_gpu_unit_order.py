"""The launch order of the decodes' units lives in a workspace that holds no
partials, int32 words at any 4-byte aligned address."""
import pytest
import torch

import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G
from tests.test_gpu_select import S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [0, 4, 8, 12])
@pytest.mark.parametrize("windowed", [False, True], ids=["plain", "windowed"])
def test_order_of_units_at_a_4_byte_aligned_address(windowed, offset):
    B, H = 200, 16
    inp = wl.make_decode_inputs(S("order", seed=140, B=B, seq_lens=tuple(1 + (37 * b) % 90 for b in range(B)), H=H, D=1))
    t = G.to_device(inp)
    O, O2 = (torch.empty((1, B, H, 512), device="cuda") for _ in range(2))
    lse, lse2 = (torch.empty((1, B, H), device="cuda") for _ in range(2))
    buf = torch.full((4096,), -1, dtype=torch.int32, device="cuda")
    kw = dict(D=1, interleave=1, scale=inp["scale"], max_seq_len=inp["max_seq_len"], max_q_len=1)
    call = dcp.dcp_mla_decode_partial_v2
    if windowed:
        call, kw = dcp.dcp_mla_decode_partial_window, dict(kw, window=40, num_sinks=2)
    args = t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["query_start_loc"]
    call(*args, O, lse, workspace=buf[offset // 4:], **kw)
    call(*args, O2, lse2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    units = B + 1 if windowed else B  # (windowed: one more for the rows of no request)
    order = buf.cpu()[offset // 4:]
    assert sorted(order[:units].tolist()) == list(range(units)) and (order[units:] == -1).all()
