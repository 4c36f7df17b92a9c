"""GPU checks of the windowed and tree decodes on latents that are not finite,
on both kernels: a row that sees a NaN has a NaN output and a NaN LSE, also
where that token is all it sees of a shard, a split or a tile, and the combine
and the split merge pass both on; rows that do not see it are as without it.

Finite rows: 2^-8 max|v| + 1e-3 (each softmax weight is off by half a bf16
step at most, the rest is fp32), LSE 1e-3."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G
from tests.test_gpu_select import S, kernel, run  # noqa: F401

pytestmark = pytest.mark.gpu


def _poison(inp, b, p):
    """A copy of the inputs with request b's latent at position p all NaN."""
    kv = inp["kv_cache"].copy()
    bs = inp["block_size"]
    kv[inp["block_table"][b, p // bs], p % bs] = wl.FP8_NAN if inp["kv_dtype"] == "fp8_e4m3" else wl.BF16_NAN
    return dict(inp, kv_cache=kv)


def _check(inp, O, lse, ref, what):
    """NaN, empty and finite (row, head) pairs exactly where the oracle has them."""
    O_ref, lse_ref = ref
    got, gl = O.float().cpu().numpy(), lse.cpu().numpy()
    assert np.array_equal(np.isnan(gl), np.isnan(lse_ref)), what + ": NaN LSEs"
    assert np.array_equal(gl == -np.inf, lse_ref == -np.inf), what + ": empty pairs"
    nan, empty = np.isnan(lse_ref), lse_ref == -np.inf
    assert nan.any() and np.isnan(got[nan]).all() and (got[empty] == 0).all(), what
    live = ~nan & ~empty
    v = oracle.kv_rows_f64(inp)[:, :512]
    tol = 2.0 ** -8 * np.abs(v[np.isfinite(v)]).max(initial=0) + 1e-3
    assert np.abs(gl[live] - lse_ref[live]).max(initial=0) <= G.ATT_LSE_ABS, what
    assert np.abs(got[live] - O_ref[live]).max(initial=0) <= tol, what


def _check_combined(O, lse, t, lse_ref):
    out, out_lse = G.run_combine(O, lse, t, torch.float32)
    nan = np.isnan(lse_ref).any(0)
    assert np.array_equal(np.isnan(out_lse.cpu().numpy()), nan)
    assert np.isnan(out.cpu().numpy()[nan]).all() and np.isfinite(out.cpu().numpy()[~nan]).all()


def _chain_mask(n):
    return np.tril(np.ones((n, n), bool))


# (spec, window, sinks, tree mask, position of the NaN)
ALONE = [
    (S("one_token", seed=100, B=1, seq_lens=(1,), H=128, D=1), 0, 0, None, 0),
    (S("one_token_h16", seed=101, B=1, seq_lens=(1,), H=16, D=1), 5, 2, None, 0),
    (S("one_tree_row", seed=102, B=1, seq_lens=(1,), H=128, D=1), 0, 0, _chain_mask(1), 0),
    (S("window_1", seed=103, B=1, seq_lens=(100,), H=128, D=1), 1, 0, None, 99),
    (S("window_1_rows", seed=104, B=1, seq_lens=(100,), q_len=3, H=16, D=2), 1, 0, None, 98),
    (S("one_token_of_a_shard", seed=105, B=1, seq_lens=(9,), H=128, D=8), 0, 0, None, 1),
    (S("own_token_of_a_shard", seed=106, B=1, seq_lens=(300,), q_len=2, H=16, D=8), 3, 0, None, 299),
    # rows 20 and on of the tree have left the prefix: of the first tile they
    # see the sink alone, of the others their own branch
    (S("sink_before_finite_tiles", seed=107, B=1, seq_lens=(300,), q_len=61, H=16, D=1), 20, 1, _chain_mask(61), 0),
    (S("sink_and_window_h128", seed=108, B=1, seq_lens=(500,), H=128, D=1), 60, 1, None, 0),
    # the last tile holds the one token
    (S("tail_tile", seed=109, B=1, seq_lens=(65,), H=128, D=1), 0, 0, None, 64),
]


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("case", ALONE, ids=lambda c: c[0].name)
def test_a_nan_is_kept(case, kv_dtype, kernel):  # noqa: F811
    spec, W, n, tree, p = case
    inp = _poison(wl.make_decode_inputs(S(**{**spec.__dict__, "kv_dtype": kv_dtype})), 0, p)
    t = G.to_device(inp)
    with np.errstate(invalid="ignore"):
        ref = oracle.decode_partial_select(inp, W, n, tree)
    O, lse, err = run(inp, t, W, n, tree)
    assert err == 0
    _check(inp, O, lse, ref, spec.name)
    _check_combined(O, lse, t, ref[1])


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3"])
def test_a_nan_that_fills_the_first_tiles_is_kept(kernel, kv_dtype):  # noqa: F811
    """33 NaN sinks: a whole tile and a token of the next, then finite ones."""
    inp = wl.make_decode_inputs(S("tiles", seed=110, B=1, seq_lens=(400,), H=128, D=1, kv_dtype=kv_dtype))
    for p in range(33):
        inp = _poison(inp, 0, p)
    O, lse, err = run(inp, G.to_device(inp), 50, 33)
    assert err == 0 and torch.isnan(O).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("tree", [False, True], ids=["window", "tree"])
def test_a_nan_alone_in_the_last_split_is_kept(kernel, tree):  # noqa: F811
    """A bound of 600 tokens is cut into splits of whole tiles; a context of
    32 k + 1 tokens, k = 4 among them, leaves the row's own token alone in its
    last tile and, for some k, in its last split."""
    inp = wl.make_decode_inputs(S("split", seed=111, B=1, seq_lens=(600,), H=128, D=1))
    assert dcp.dcp_decode_select_workspace_size(1, 1, 128, 1, 600, 1) > 2 * 128 * 2052  # two splits at least
    mask = np.ones((1, 1), bool) if tree else None
    for k in range(1, 19):
        cut = dict(_poison(inp, 0, 32 * k), seq_lens=np.array([32 * k + 1], np.int32))
        for dt in (torch.float32, torch.bfloat16):
            O, lse, err = run(cut, G.to_device(cut), 0, 0, mask, out_dtype=dt)
            assert err == 0 and torch.isnan(lse).all() and torch.isnan(O).all(), k
