"""GPU checks of the windowed and tree decodes where the largest score comes
late: the running maxima of the tensor-core kernel's two softmax groups move at
different tiles, and tiles of a smaller maximum are brought to the scale of a
larger one.

Tolerance: each softmax weight is rounded to bf16 once (half a step, 2^-8 of
itself; bringing it to another scale moves its exponent only), their sum stays
fp32, so an output is off by at most 2^-8 sum_t p_t |v_t| <= 2^-8 max|v|, and
1e-3 for the fp32 sums.  LSE 1e-3."""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from tests import gpu_util as G
from tests.test_gpu_select import S, kernel, run  # noqa: F401

pytestmark = pytest.mark.gpu


def _scored(spec, bits_of, values=None):
    """Inputs whose token at position p scores bits_of(p)[0] + bits_of(p)[1]
    (both rounded to bf16) in powers of two, in every row and head, on top of
    what the seeded draws of dims 0-511 score times `values` (None: ones for
    values and no score of their own)."""
    def rows(b, pos):
        x = np.ones((len(pos), 576), np.float32)
        if values is not None:
            x[:, :512] = np.random.default_rng([spec.seed, b]).standard_normal((len(pos), 512), dtype=np.float32)
        hi, lo = bits_of(pos)
        x[:, 512:] = 0
        x[:, 512], x[:, 513] = hi, lo
        return wl.f32_to_bf16_bits(x)
    inp = wl.make_decode_inputs(spec, rows)
    q = np.zeros((inp["T"], spec.H, 576), np.float32)
    if values is not None:
        q[:, :, :512] = values * np.random.default_rng(spec.seed + 1000).standard_normal((inp["T"], spec.H, 512),
                                                                                         dtype=np.float32)
    q[:, :, 512:514] = 1.0
    inp["q"], inp["scale"] = wl.f32_to_bf16_bits(q), math.log(2.0)
    return inp


def _check(inp, window, sinks, tree=None):
    vmax = np.abs(oracle.kv_rows_f64(inp)[:, :512])
    vmax = vmax[np.isfinite(vmax)].max()
    O_ref, lse_ref = oracle.decode_partial_select(inp, window, sinks, tree)
    O, lse, err = run(inp, G.to_device(inp), window, sinks, tree)
    live = lse_ref != -np.inf
    assert err == 0 and np.array_equal(lse.cpu().numpy() != -np.inf, live)
    assert np.abs(lse.cpu().numpy()[live] - lse_ref[live]).max() <= G.ATT_LSE_ABS
    off = np.abs(O.cpu().numpy()[live] - O_ref[live]).max()
    assert off <= 2.0 ** -8 * vmax + 1e-3, off


@pytest.mark.parametrize("jump", [1.00555, 2.00555, 3.0035, 0.7])
def test_weights_are_rounded_once(kernel, jump):  # noqa: F811
    """Four tiles.  The second's maximum is 8.5 bits above the first's, the
    third's `jump` above that, and the fourth, most of the row's weight, is at
    the second's plus 0.0056763: 1.0039424 in its scale, just above half a step
    over 1, and (jump 1.00555) in the third's just above half a step again."""
    def bits(pos):
        tile, i = pos // 32, pos % 32
        hi = np.where(tile == 0, 0.0, np.where(tile == 3, 8.5, np.where(i == 7, 8.5 + math.floor(jump), -200.0)))
        lo = np.where(tile == 3, 0.0056763, np.where((tile == 2) & (i == 7), jump - math.floor(jump), 0.0))
        hi[(tile == 1) & (i == 7)] = 8.5
        return hi, lo
    _check(_scored(S("once", seed=120, B=1, seq_lens=(128,), H=128, D=1), bits), 0, 0)


def _zeros(pos):
    return np.zeros(len(pos))


SHAPES = {
    "ramp": lambda pos: (20.0 * pos / 2000, _zeros(pos)),
    "fall": lambda pos: (20.0 - 20.0 * pos / 2000, _zeros(pos)),
    "needle_tile_4": lambda pos: (np.where(pos == 4 * 64 + 9, 12.0, 0.0), _zeros(pos)),
    "needle_tile_5": lambda pos: (np.where(pos == 5 * 64 + 9, 14.0, 0.0), _zeros(pos)),
    "wide": lambda pos: (5.0 * np.random.default_rng(7).standard_normal(4096)[pos], _zeros(pos)),
    "steps": lambda pos: (8.3 * (pos // 200), _zeros(pos)),
    "far": lambda pos: (np.where(pos % 500 == 77, 300.0 * (pos // 500 + 1), 0.0), _zeros(pos)),
}


@pytest.mark.parametrize("H,q_len,D,window,sinks", [(128, 1, 2, 0, 0), (16, 5, 2, 1300, 4), (64, 2, 1, 700, 60)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_scores_that_grow_through_the_context(kernel, shape, H, q_len, D, window, sinks):  # noqa: F811
    spec = S(shape, seed=130, B=2, seq_lens=(2000, 777), q_len=q_len, H=H, D=D, block_size=64)
    inp = _scored(spec, SHAPES[shape], values=0.05)
    _check(inp, window, sinks)
    if q_len > 1:
        tree = np.tile(np.tril(np.ones((q_len, q_len), bool)), (2, 1))
        _check(inp, window, sinks, tree)
