"""GPU checks of the windowed and tree decodes over shard layouts: ranges of a
tree decode's shards by themselves, and interleave periods past 31 bits, which
the CUDA-core kernel takes.

Tolerances: 2^-8 max|v| + 1e-3 (softmax weights in bf16, the rest fp32), LSE
1e-3."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G
from tests.test_gpu_select import S, kernel, random_trees, run  # noqa: F401
from tests.test_gpu_select_calls import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    (S("global", seed=220, B=2, seq_lens=(700, 90), q_len=(9, 3), H=16, D=5, interleave=3), 0, 0),
    (S("window", seed=221, B=2, seq_lens=(2500, 40), q_len=7, H=128, D=3), 900, 4),
    (S("local", seed=222, B=2, seq_lens=(500, 133), q_len=20, H=16, D=4, interleave=5, layout="local"), 60, 2),
    (S("fp8", seed=223, B=1, seq_lens=(900,), q_len=12, H=64, D=4, kv_dtype="fp8_e4m3"), 0, 0),
], ids=lambda c: c[0].name)
def test_ranges_of_a_trees_shards(case, kernel):  # noqa: F811
    spec, W, n = case
    inp = wl.make_decode_inputs(spec)
    t = G.to_device(inp)
    B, T, H, D = inp["B"], inp["T"], inp["H"], inp["D"]
    vis = random_trees(np.random.default_rng(spec.seed), inp)
    mask = dcp.pack_tree_mask(torch.from_numpy(vis)).cuda()
    ref_O, ref_lse = oracle.decode_partial_select(inp, W, n, vis)
    size = dcp.dcp_decode_select_workspace_size(B, T, H, D, inp["max_seq_len"], inp["max_q_len"], W, n)
    for d0 in range(D):
        for count in sorted({1, D - d0}):
            table = t["block_table"]
            if table.dim() == 3:
                table = table[d0:d0 + count]
            O = torch.empty((count, T, H, 512), device="cuda")
            lse = torch.empty((count, T, H), device="cuda")
            dcp.dcp_mla_decode_partial_tree(
                t["q"], t["kv_cache"], table, t["seq_lens"], t["query_start_loc"], mask, O, lse, D=D,
                interleave=inp["interleave"], scale=inp["scale"], window=W, num_sinks=n,
                max_seq_len=inp["max_seq_len"], max_q_len=inp["max_q_len"], kv_scale=t.get("kv_scale"),
                shard_begin=d0, shard_count=count, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
            torch.cuda.synchronize()
            check(inp, O, lse, (ref_O[d0:d0 + count], ref_lse[d0:d0 + count]), "shards %d+%d" % (d0, count))


@pytest.mark.parametrize("D,interleave", [(1, 0x7fffffff), (2, 1 << 30), (3, 0x7fffffff)])
def test_interleave_periods_past_31_bits(D, interleave):
    """Every token is shard 0's; the other shards are empty."""
    inp = wl.make_decode_inputs(S("period", seed=224, B=2, seq_lens=(300, 40), q_len=5, H=16, D=1))
    inp = dict(inp, D=D, interleave=interleave)
    t = G.to_device(inp)
    vis = random_trees(np.random.default_rng(224), inp)
    for W, tree in ((0, None), (50, None), (50, vis)):
        O, lse, err = run(inp, t, W, 3, tree)
        assert err == 0
        check(inp, O, lse, oracle.decode_partial_select(inp, W, 3, tree), "period")
