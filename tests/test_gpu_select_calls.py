"""GPU checks of the ways in which the windowed and tree decodes may be called:
outputs aligned to 16 bytes only, shards computed one at a time in workspaces
of exactly the stated size, more units than fit at once (ordered, and without
room for the order), rows of no request, scales that are no powers of two, a
stream argument, strided inputs, captured steps replayed on new lengths, and a
wait that runs out.

Tolerances: LSE 1e-3 as for the other decodes.  Outputs: the tensor cores take
the softmax weights p_t in bf16, each off by half a step at most (2^-8 of
itself), while their sum stays fp32, so an output is off by at most
2^-8 sum_t p_t |v_t| <= 2^-8 max|v|, reached where one token outweighs the rest
(p close to 1 and |v| its largest: 0.012 at |v| = 3.46); 1e-3 besides for the
fp32 sums (at most 4,000 terms of 2^-24) and for weights that are scaled down
and rounded again, which are below 2^-8 of the largest.  A bf16 output adds half
a step of its own, 2^-8 of the value.  A code times a scale that is no power of
two is rounded to bf16 on the tensor cores, so there the oracle gets the rounded
rows."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G
from tests.test_gpu_select import S, kernel, random_trees, run  # noqa: F401

pytestmark = pytest.mark.gpu


def check(inp, O, lse, ref, what):
    O_ref, lse_ref = ref
    got, gl = O.float().cpu().numpy(), lse.cpu().numpy()
    empty = lse_ref == -np.inf
    assert np.array_equal(gl == -np.inf, empty) and (got[empty] == 0).all(), what
    live = ~empty
    v = oracle.kv_rows_f64(inp)[:, :512]
    tol = 2.0 ** -8 * np.abs(v[np.isfinite(v)]).max(initial=0) + 1e-3
    tol = tol + (2.0 ** -8 * np.abs(O_ref[live]) if O.dtype == torch.bfloat16 else 0.0)
    assert np.abs(gl[live] - lse_ref[live]).max(initial=0) <= G.ATT_LSE_ABS, what
    assert (np.abs(got[live] - O_ref[live]) <= tol).all(), what


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,q_len,W", [(128, 1, 60), (16, 3, 2), (33, 2, 5000)])
def test_output_aligned_to_16_bytes_only(kernel, dt, H, q_len, W):
    inp = wl.make_decode_inputs(S("al", seed=80, B=2, seq_lens=(300, 0), q_len=q_len, H=H, D=2, extra_rows=1))
    t = G.to_device(inp)
    T = inp["T"]
    n = 2 * T * H * 512
    off = 16 // dt.itemsize
    buf = torch.full((n + 2 * off,), 7.0, dtype=dt, device="cuda")
    O = buf[off:off + n].view(2, T, H, 512)
    assert O.data_ptr() % 32 == 16
    lse = torch.empty((2, T, H), dtype=torch.float32, device="cuda")
    kw = dict(D=2, interleave=1, scale=inp["scale"], window=W, num_sinks=3, max_seq_len=300, max_q_len=q_len)
    ws = torch.empty(dcp.dcp_decode_select_workspace_size(2, T, H, 2, 300, q_len, W, 3), dtype=torch.uint8, device="cuda")
    dcp.dcp_mla_decode_partial_window(t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["query_start_loc"], O,
                                      lse, workspace=ws, **kw)
    torch.cuda.synchronize()
    check(inp, O, lse, oracle.decode_partial_select(inp, W, 3), "aligned")
    assert (buf[:off] == 7).all() and (buf[off + n:] == 7).all()


@pytest.mark.parametrize("case", [
    (S("one_long", seed=81, B=1, seq_lens=(9000,), q_len=2, H=128, block_size=64, D=5), 0, 0),
    (S("window", seed=82, B=2, seq_lens=(4000, 700), q_len=3, H=16, D=8, interleave=16), 1500, 4),
    (S("local", seed=83, B=1, seq_lens=(3000,), q_len=1, H=128, D=3, interleave=3, layout="local"), 0, 0),
    (S("many", seed=84, B=30, seq_lens=tuple(100 + 70 * b for b in range(30)), q_len=1, H=128, D=3), 0, 0),
], ids=lambda c: c[0].name)
def test_shards_alone_in_the_stated_workspace(case):
    """Each range of shards by itself, in a workspace of exactly the stated
    size with a guard behind it, gives the oracle's partials of those shards."""
    spec, W, n = case
    inp = wl.make_decode_inputs(spec)
    t = G.to_device(inp)
    B, T, H, D = inp["B"], inp["T"], inp["H"], inp["D"]
    ref_O, ref_lse = oracle.decode_partial_select(inp, W, n)
    size = dcp.dcp_decode_select_workspace_size(B, T, H, D, inp["max_seq_len"], inp["max_q_len"], W, n)
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    for d0 in range(D):
        for count in sorted({1, (D - d0 + 1) // 2, D - d0}):
            table = t["block_table"]
            if table.dim() == 3:
                table = table[d0:d0 + count]
            O = torch.empty((count, T, H, 512), dtype=torch.float32, device="cuda")
            lse = torch.empty((count, T, H), dtype=torch.float32, device="cuda")
            dcp.dcp_mla_decode_partial_window(
                t["q"], t["kv_cache"], table, t["seq_lens"], t["query_start_loc"], O, lse, D=D,
                interleave=inp["interleave"], scale=inp["scale"], window=W, num_sinks=n,
                max_seq_len=inp["max_seq_len"], max_q_len=inp["max_q_len"], shard_begin=d0, shard_count=count,
                workspace=ws[:size])
            torch.cuda.synchronize()
            check(inp, O, lse, (ref_O[d0:d0 + count], ref_lse[d0:d0 + count]), "shards %d+%d" % (d0, count))
            assert (ws[size:] == 255).all()


def test_more_units_than_fit_with_and_without_room_for_their_order():
    """1,600 units of very different lengths: sorted (the workspace holds the
    order) and in index order, bit for bit the same."""
    rng = np.random.default_rng(85)
    seq = tuple(int(x) for x in rng.integers(0, 400, 200))
    inp = wl.make_decode_inputs(S("units", seed=85, B=200, seq_lens=seq, q_len=2, H=64, D=8))
    t = G.to_device(inp)
    size = dcp.dcp_decode_select_workspace_size(200, inp["T"], 64, 8, inp["max_seq_len"], 2, 0, 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    O, lse, err = run(inp, t, 0, 0, workspace=ws)
    assert err == 0
    check(inp, O, lse, oracle.decode_partial_select(inp, 0, 0), "ordered")
    O2, lse2, err = run(inp, t, 0, 0, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert err == 0 and torch.equal(O, O2) and torch.equal(lse, lse2)
    # a workspace at an odd address holds no order
    odd = torch.empty(size + 16, dtype=torch.uint8, device="cuda")[1:]
    O2, lse2, err = run(inp, t, 0, 0, workspace=odd)
    assert err == 0 and torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,extra", [(1, 1), (1, 300), (40, 77)])
def test_rows_of_no_request(kernel, B, extra):
    inp = wl.make_decode_inputs(S("pad", seed=86, B=B, seq_lens=tuple(30 + 11 * b for b in range(B)), q_len=3, H=16,
                                  D=2, extra_rows=extra))
    t = G.to_device(inp)
    O, lse, err = run(inp, t, 40, 2)
    assert err == 0
    check(inp, O, lse, oracle.decode_partial_select(inp, 40, 2), "padding")


def test_scales_that_are_no_powers_of_two(kernel):
    inp = wl.make_decode_inputs(S("scale", seed=87, B=2, seq_lens=(500, 90), q_len=4, H=128, D=2,
                                  kv_dtype="fp8_e4m3"))
    inp["kv_scale"] = (inp["kv_scale"] * np.random.default_rng(87).uniform(0.6, 1.4, inp["kv_scale"].shape)).astype(np.float32)
    t = G.to_device(inp)
    vis = random_trees(np.random.default_rng(87), inp)
    ref = inp
    if kernel == "tc":
        rows = wl.f32_to_bf16_bits(oracle.kv_rows_f64(inp).astype(np.float32))
        ref = dict(inp, kv_cache=rows.reshape(inp["kv_cache"].shape), kv_scale=None, kv_dtype="bf16")
    for tree in (None, vis):
        O, lse, err = run(inp, t, 200, 3, tree)
        assert err == 0
        check(inp, O, lse, oracle.decode_partial_select(ref, 200, 3, tree), "scales")


def test_stream_argument_and_strided_inputs():
    """A stream argument (an object or its address) runs there, allocations
    included; q, the table and the mask may be slices of wider tensors."""
    inp = wl.make_decode_inputs(S("str", seed=88, B=2, seq_lens=(2500, 300), q_len=4, H=16, D=2, block_size=64))
    t = G.to_device(inp)
    T = inp["T"]
    vis = random_trees(np.random.default_rng(88), inp)
    ref = oracle.decode_partial_select(inp, 900, 3, vis)
    q = torch.full((T, 16 + 3, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:, :16] = t["q"]
    table = torch.full((2, t["block_table"].shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    table[:, :-5] = t["block_table"]
    mask = torch.full((T, 4), -1, dtype=torch.int64, device="cuda")
    mask[:, :1] = dcp.pack_tree_mask(torch.from_numpy(vis)).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream, None):
        O, lse = dcp.decode_partial_tree(q[:, :16], t["kv_cache"], table[:, :-5], t["seq_lens"], t["query_start_loc"],
                                         mask[:, :2], D=2, interleave=1, scale=inp["scale"], window=900, num_sinks=3,
                                         max_seq_len=2500, max_q_len=4, stream=stream)
        torch.cuda.synchronize()
        check(inp, O, lse, ref, "stream")
    cu = torch.tensor([0, 100, 250], dtype=torch.int32, device="cuda")
    want = dcp.latent_cache_read(t["kv_cache"], t["block_table"], cu, 250)
    s.wait_stream(torch.cuda.current_stream())
    got = dcp.latent_cache_read(t["kv_cache"], t["block_table"], cu, 250, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(want, got)


def test_captured_step_replays_on_other_lengths():
    """A captured decode and combine replayed with other lengths, rows and
    masks in the same buffers: as fresh calls, bit for bit."""
    inp = wl.make_decode_inputs(S("cap", seed=89, B=3, seq_lens=(900, 450, 600), q_len=5, H=16, D=2, block_size=64))
    t = G.to_device(inp)
    rng = np.random.default_rng(89)
    masks = [dcp.pack_tree_mask(torch.from_numpy(random_trees(rng, inp, k))).cuda() for k in ("tree", "odd", "tree")]
    mask = masks[0].clone()

    def step():
        O, lse = dcp.decode_partial_tree(t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["query_start_loc"],
                                         mask, D=2, interleave=1, scale=inp["scale"], window=300, num_sinks=2,
                                         max_seq_len=900, max_q_len=5)
        return (O, lse) + dcp.lse_combine(O, lse, t["seq_lens"], t["query_start_loc"])
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for k, (seq, qsl) in enumerate([((900, 450, 600), (0, 5, 10, 15)), ((3, 0, 900), (0, 1, 1, 6)),
                                    ((64, 65, 31), (0, 5, 8, 9))]):
        t["seq_lens"].copy_(torch.tensor(seq, dtype=torch.int32))
        t["query_start_loc"].copy_(torch.tensor(qsl, dtype=torch.int32))
        mask.copy_(masks[k])
        for r in res:
            r.fill_(float("nan"))
        g.replay()
        fresh = step()
        torch.cuda.synchronize()
        # (request 2 at 900 tokens sees 40 that were never written, NaN in its
        # last block, and blocks that its table lacks: NaN in both)
        for a, b in zip(res, fresh):
            assert torch.allclose(a, b, rtol=0, atol=0, equal_nan=True)
        seen = 1 if k == 1 else 15
        assert not torch.isnan(res[0][:, :seen]).any()


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """The tensor-core kernel's waits are bounded: with a barrier that nobody
    signals the call returns, reports the timeout and leaves the context
    usable."""
    inp = wl.make_decode_inputs(S("stall", seed=90, B=1, seq_lens=(300,), q_len=2, H=128, D=1))
    t = G.to_device(inp)
    for fp8 in (False, True):
        if fp8:
            inp = wl.make_decode_inputs(S("stall8", seed=90, B=1, seq_lens=(300,), q_len=2, H=128, D=1,
                                          kv_dtype="fp8_e4m3"))
            t = G.to_device(inp)
        monkeypatch.setenv("DCP_TEST_STALL_WAIT", "1")
        _, _, err = run(inp, t, 100, 2)
        assert err & dcp.DEVERR_TIMEOUT
        monkeypatch.delenv("DCP_TEST_STALL_WAIT")
        O, lse, err = run(inp, t, 100, 2)
        assert err == 0
        check(inp, O, lse, oracle.decode_partial_select(inp, 100, 2), "after")


def test_many_pairs_in_few_splits_are_the_plain_decode():
    """320 rows of 32 heads (10,240 pairs, merged a warp each) over 9,000
    tokens in two to four splits, on a chain: the partials of the decode without
    selection, within twice the attention tolerances."""
    inp = wl.make_decode_inputs(S("merge", seed=91, B=2, seq_lens=(9000, 8000), q_len=160, H=32, D=1, block_size=64))
    t = G.to_device(inp)
    size = dcp.dcp_decode_select_workspace_size(2, 320, 32, 1, 9000, 160, 0, 0)
    assert 2 <= size // (320 * 32 * 2052) <= 4
    want, want_lse = G.run_decode(inp, t)[:2]
    for dt in (torch.float32, torch.bfloat16):
        O, lse, err = run(inp, t, 0, 0, out_dtype=dt)
        assert err == 0
        step = 0.0 if dt == torch.float32 else 2.0 ** -8
        assert ((O.float() - want).abs() <= 2 * G.ATT_OUT_ABS + step * want.abs()).all()
        assert (lse - want_lse).abs().max().item() <= 2 * G.ATT_LSE_ABS


def test_captured_call_of_ordered_units_replays():
    """The kernel that orders the units and the decode that sets up alongside
    it, captured once and replayed on other lengths: as a fresh call, bit for
    bit, also when replays follow one another without a pause."""
    inp = wl.make_decode_inputs(S("ordered", seed=92, B=60, seq_lens=(200,) * 60, q_len=1, H=128, D=8))
    t = G.to_device(inp)
    rng = np.random.default_rng(92)
    size = dcp.dcp_decode_select_workspace_size(60, 60, 128, 8, 200, 1, 90, 3)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def call():
        return dcp.decode_partial_window(t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["query_start_loc"],
                                         D=8, interleave=1, scale=inp["scale"], window=90, num_sinks=3,
                                         max_seq_len=200, max_q_len=1, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        O, lse = call()
    for _ in range(4):
        seq = rng.integers(0, 201, 60).astype(np.int32)
        t["seq_lens"].copy_(torch.from_numpy(seq))
        O.fill_(float("nan"))
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        O2, lse2 = call()
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
    check(inp, O, lse, oracle.decode_partial_select(dict(inp, seq_lens=seq), 90, 3), "ordered")
