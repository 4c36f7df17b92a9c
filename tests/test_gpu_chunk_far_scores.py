"""Scores far below a row's largest, and rows that see nothing but such scores."""
import math

import pytest
import torch

from tests import chunk_reference as ref
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu
Q0 = 2.0 ** 12  # the queries' first rope element


def run(st):
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=st["total"], out_dtype=torch.float32)
    torch.cuda.synchronize()
    return out, lse


def inputs(L, n, far, key):
    """Tokens `far` get scores of 1 to 4 times Q0 x key x scale (and what their other
    dims add), the others' first rope element is 0."""
    st = ref.make(seq=[L], q=[n], H=2, bs=64, seed=31)
    st["q"][:, :, 128] = (Q0 * (1 + torch.arange(n, device="cuda") % 16 / 16)).to(torch.bfloat16)[:, None]
    rows = torch.from_numpy(ref.rows_of(st, 0)).cuda()
    st["cache"].view(-1, 576)[:, 512] = 0
    # 1 to 2 times the key and Q0: products with the scale that no fp32 number is
    at = rows[far]
    st["cache"].view(-1, 576)[at, 512] = (key * (1 + torch.arange(len(at), device="cuda") * 37 % 127 / 128 + 1 / 128)).to(torch.bfloat16)
    return st, rows


# 1,300 tokens: one piece, 4,000: pieces that are joined; keys of -4e7, -3e8 and -5e9 in score, and -inf
@pytest.mark.parametrize("L,n", [(1300, 3), (1300, 200), (4000, 1), (4000, 150)])
@pytest.mark.parametrize("key", [-2.0 ** 17, -2.0 ** 20, -2.0 ** 24, -math.inf])
@pytest.mark.parametrize("part", ["first", "second", "middle"])
def test_far_tokens_weigh_nothing(L, n, key, part):
    far = {"first": slice(0, L // 2), "second": slice(L // 2, L - n), "middle": slice(700, 1000)}[part]
    st, rows = inputs(L, n, far, key)
    out, lse = run(st)
    # the reference without these tokens: a table without them would be another order, so
    # their weights are set to 0 by the same keys, and the tolerances are those of ordinary ones
    want, want_lse, _, _ = ref.reference(st)
    st["cache"].view(-1, 576)[rows[far], 512] = 0
    st["q"][:, :, 128] = 0
    _, _, tol, tol_lse = ref.reference(st)
    # A row's elements are f16 after its largest came to 1: half a step of 2^-24 below
    # 2^-14, times 2^12, is 2^-13 an element, times 192 keys of about 1 (mean 0.8) and the scale: 1.4e-3.
    ds = 2.0 ** -13 * 192 * 0.8 * st["scale"]
    assert ((lse.double() - want_lse).abs() <= tol_lse + ds).all()
    # (values' magnitudes average below 1, and weights add up to 1)
    assert ((out.double() - want).abs() <= tol + 2 * ds).all()


@pytest.mark.parametrize("L,n", [(1, 1), (200, 200), (1300, 3), (4000, 1), (4000, 150)])
@pytest.mark.parametrize("key", [-2.0 ** 18, -2.0 ** 24, -math.inf])
def test_rows_with_nothing_but_far_tokens_are_nan(L, n, key):
    st, _ = inputs(L, n, slice(0, L), key)
    out, lse = run(st)
    assert out.isnan().all() and lse.isnan().all()


def test_rows_that_see_a_near_token_and_rows_before_it():
    """One ordinary token among far ones: rows from it on are finite (its value), rows
    before it NaN; a request without rows to see keeps zeros and -inf."""
    st, rows = inputs(400, 120, slice(0, 400), -2.0 ** 20)
    at = 330
    st["cache"].view(-1, 576)[rows[at], 512] = 0
    out, lse = run(st)
    sees = torch.arange(280, 400) >= at
    assert out[~sees].isnan().all() and lse[~sees].isnan().all()
    kv = st["cache"].view(-1, 576)[rows[at]].double()
    for h in range(2):
        v = st["w"][256 * h + 128:256 * h + 256].double() @ kv[:512]
        # f16 value and weight (2^-11 each), and 1e-5 of 512 products' sum of magnitudes (0.8 x 0.035 each)
        assert ((out[sees][:, h].double() - v).abs() <= 2.0 ** -10 * 1.01 * v.abs() + 1e-5 * 15).all()


@pytest.mark.parametrize("power", [0, 60, 120, 125])
def test_a_scale_of_zero_weighs_all_alike(power):
    """Queries up to bf16's largest, every score 0."""
    st = ref.make(seq=[300, 20], q=[150, 20], H=2, seed=32)
    st["q"] = (st["q"].double() * 2.0 ** power).to(torch.bfloat16)
    st["scale"] = 0.0
    out, lse = run(st)
    ref.check(out, lse, ref.reference(st))


@pytest.mark.parametrize("L", [1300, 4000])  # in one piece, in pieces
@pytest.mark.parametrize("past", [-40.0, -4.0, 0.0])
def test_rows_at_the_border_are_nan_in_pieces_too(L, past):
    """All scores (the same for every token) within a few units of the border, 2^25 in
    base 2, on its far side."""
    st = ref.make(seq=[L], q=[2], H=1, bs=64, seed=33)
    st["q"].zero_()
    st["cache"].view(-1, 576)[:, 512] = -1
    st["q"][:, :, 128] = 2.0 ** 12
    st["scale"] = (2.0 ** 25 - past) / 2.0 ** 12 / math.log2(math.e)
    # the factor of a score: fp32 product of the scale and log2 e, off by 2 x 2^-24 of it: 4 at 2^25
    out, lse = run(st)
    if past < -4:
        assert out.isnan().all() and lse.isnan().all()
    else:  # either side
        assert torch.equal(out.isnan(), out.isnan()[:1, :1, :1].expand_as(out)) and torch.equal(out.isnan()[..., 0], lse.isnan())
