"""Chunk attention against the tight reference: units in pieces, several passes over
the heads with units in pieces, decoding rows among chunks."""
import pytest
import torch

from tests import chunk_reference as ref
from tests.chunk_tight import tight_check, tight_reference
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu


def run(st, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=st["total"], kv_scale=st["kv_scale"], D=st["D"],
                                   interleave=st["I"], out_dtype=torch.float32, dev_error=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out, lse


CASES = {
    "one_row_in_pieces": dict(seq=[20000], q=[1], H=2),
    "rows_in_pieces": dict(seq=[9000, 10], q=[130, 10], H=2),
    "two_tiles_of_rows": dict(seq=[6000], q=[256], H=1),
    "odd_rows_and_tokens": dict(seq=[5003], q=[391], H=1),
    "whole_prompt": dict(seq=[3000], q=[3000], H=2),
    "not_cut": dict(seq=[1400], q=[9], H=3),
    "key_remainders": dict(seq=[1024, 700, 130], q=[40, 300, 130], H=2),
    "either_side_of_the_border": dict(seq=[1024, 1025], q=[40, 40], H=2),
    "decodes_among_chunks": dict(seq=[2500, 7000, 130, 4100, 9], q=[1, 300, 130, 1, 1], H=2),
    "fp8": dict(seq=[4000, 300], q=[70, 300], H=2, fp8=True),
    "shard_tables": dict(seq=[4000, 1500], q=[70, 3], H=2, D=8, I=3, local=True),
    "blocks_of_one": dict(seq=[2000], q=[5], H=1, bs=1),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_against_the_tight_reference(name):
    st = ref.make(**{"bs": 64, "seed": 52, **CASES[name]})
    tight_check(*run(st), tight_reference(st))


@pytest.mark.parametrize("heads", [1, 2, 3])
def test_passes_of_unequal_heads_with_units_in_pieces(heads):
    """A workspace for 1, 2 or 3 of 5 heads: passes of 1, of 2, 2 and 1, of 3 and 2.
    Each pass cuts its units for its own number of heads."""
    st = ref.make(seq=[9000, 3000, 400], q=[130, 40, 30], H=5, bs=64, seed=53)
    n = dcp.dcp_chunk_attention_workspace_size(3, st["T"], heads, st["total"])
    assert n < dcp.dcp_chunk_attention_workspace_size(3, st["T"], 5, st["total"])
    want = tight_reference(st)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    got = run(st, workspace=ws)
    tight_check(*got, want)
    again = run(st, workspace=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    tight_check(*run(st), want)


@pytest.mark.parametrize("L", [1000, 1200, 4000])
def test_a_row_that_sees_little_but_one_token(L):
    """Keys of requests of more than 1,024 tokens are off by half a step of f16, 2^-11 of
    an element: a row that attends to one token has all of that in its log-sum-exp,
    and no more; shorter requests' keys are off by 2^-22."""
    st = ref.make(seq=[L], q=[6], H=2, bs=64, seed=54)
    st["scale"] = 1.0
    kv = ref.latents(st, ref.rows_of(st, 0))
    for h in range(2):  # queries along one token's keys
        k = kv[:, :512] @ st["w"][256 * h:256 * h + 128].double().T
        for r in range(6):
            t = (37 + 157 * r) % (L - 6)
            st["q"][r, h, :128] = k[t].to(torch.bfloat16)
            st["q"][r, h, 128:] = kv[t, 512:].to(torch.bfloat16)
    out, lse = run(st)
    for h in range(2):
        k = torch.cat([kv[:, :512] @ st["w"][256 * h:256 * h + 128].double().T, kv[:, 512:]], 1)
        q = st["q"][:, h].double()
        s = (q @ k.T).masked_fill(torch.arange(L, device="cuda")[None, :] > L - 6 + torch.arange(6, device="cuda")[:, None], -torch.inf)
        z = torch.logsumexp(s, 1)
        top = s.argmax(1)
        assert (torch.exp(s.amax(1) - z) > 0.99).all()
        size = (q[:, :128] * k[top, :128]).abs().sum(1)
        # fp32 sums of 192 products: 12 steps (20 with remainders), 2^-23 of up to the whole sum each
        bound = size * (2.0 ** -11 if L > 1024 else 2.0 ** -22) + 20 * 2.0 ** -23 * (q * k[top]).abs().sum(1) + 2.0 ** -20 * z.abs()
        assert ((lse[:, h].double() - z).abs() <= bound).all()
