"""Keys past f16's largest number: every row that sees one is NaN, whatever the
signs of its products, and no other row changes."""
import pytest
import torch

from tests import chunk_reference as ref
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu
DIM, HEAD, BACK = 7, 0, 20  # the key dim and head that overflow, the token: BACK before the last


def run(st):
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=st["total"], kv_scale=st["kv_scale"])
    torch.cuda.synchronize()
    return out, lse


def inputs(L, value, q_value, fp8=False):
    """One key element of `value` x 1024 at one token and head, times queries of
    q_value; the token's other keys and values stay ordinary."""
    st = ref.make(seq=[L], q=[40], H=2, bs=64, seed=21, fp8=fp8)
    row = int(ref.rows_of(st, 0)[L - 1 - BACK])
    st["w"][256 * HEAD + DIM] = 0
    st["w"][256 * HEAD + DIM, 0] = 1024
    st["q"][:, :, DIM] = q_value
    st["cache"].view(-1, 576)[:, 0] = 0
    if fp8:  # code 0x7e: 448
        st["cache"].view(-1, 576)[row, 0] = 0x7e
        st["kv_scale"].view(-1)[row] = value / 448
    else:
        st["cache"].view(-1, 576)[row, 0] = value
    return st, row


# 300 tokens in one piece with key remainders, 1,025 without, 9,000 in pieces that are joined
@pytest.mark.parametrize("L", [300, 1025, 9000])
@pytest.mark.parametrize("value", [70.0, -70.0, float("inf")])
@pytest.mark.parametrize("q_value", [-1e-4, 1e-4, -2.0])
def test_rows_that_see_it_are_nan(L, value, q_value):
    st, row = inputs(L, value, q_value)
    out, lse = run(st)
    sees = torch.zeros(40, dtype=torch.bool)
    sees[40 - 1 - BACK:] = True
    heads = slice(None) if value == float("inf") else HEAD  # (an infinite latent is infinite, or NaN, in every key)
    assert out[sees][:, heads].isnan().all() and lse[sees][:, heads].isnan().all()
    st["cache"].view(-1, 576)[row, 0] = 0  # an ordinary token in its place
    clean, clean_lse = run(st)
    assert clean.isfinite().all() and clean_lse.isfinite().all()
    assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], clean_lse[~sees])


def test_rows_that_see_it_are_nan_fp8():
    st, _ = inputs(1025, 70.0, -1e-4, fp8=True)
    out, _ = run(st)
    assert out[40 - 1 - BACK:, HEAD].isnan().all() and out[:40 - 1 - BACK].isfinite().all()
    assert out[:, 1 - HEAD].isfinite().all()


@pytest.mark.parametrize("L", [300, 1025])
def test_the_largest_key_is_ordinary(L):
    """65,280 = 1,024 x 63.75, below f16's largest: finite, and its share of the scores
    counts (-1e-4 in bf16 times it times the scale: about -0.47)."""
    st, _ = inputs(L, 63.75, -1e-4)
    out, lse = run(st)
    assert out.isfinite().all()
    # 65,280 is exact in f16 and a single product; the reference's bound would take it for
    # every token's, so the bound is that without it, and 1e-5 of what it adds
    _, want, _, _ = ref.reference(st)
    st["cache"].view(-1, 576)[:, 0] = 0
    _, _, _, tol = ref.reference(st)
    assert ((lse.double() - want).abs() <= tol + 1e-5).all()
