"""Chunk attention against the fp64 reference (chunk_reference.py, which also
derives the tolerances)."""
import numpy as np
import pytest
import torch

from tests import chunk_reference as ref
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu


def run(st, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw.setdefault("total_len", st["total"])
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], kv_scale=st["kv_scale"], D=st["D"], interleave=st["I"],
                                   dev_error=err, **kw)
    torch.cuda.synchronize()
    return out, lse, int(err)


CASES = {
    "one_token": dict(seq=[1], q=[1], H=1),
    "short_prompt": dict(seq=[9], q=[9], H=3),
    "tile_of_rows_and_tokens": dict(seq=[128], q=[128], H=2),
    "one_past_a_tile": dict(seq=[129], q=[129], H=1),
    "unit_of_rows": dict(seq=[256], q=[256], H=1),
    "one_past_a_unit": dict(seq=[257], q=[257], H=2),
    "decode_rows": dict(seq=[300, 1, 129, 128], q=[1, 1, 1, 1], H=5),
    "chunk_on_context": dict(seq=[777], q=[200], H=3),
    "long_context_few_rows": dict(seq=[3001], q=[7], H=2),
    "ragged": dict(seq=[40, 513, 130, 700], q=[40, 3, 129, 261], H=2, pad=5),
    "rows_before_the_context": dict(seq=[3, 130, 1], q=[9, 300, 2], H=2),
    "no_tokens_no_rows": dict(seq=[0, 50, 0, 20], q=[3, 10, 0, 0], H=2, pad=300),
    "blocks_of_one": dict(seq=[150, 3], q=[20, 3], H=1, bs=1),
    "odd_blocks": dict(seq=[150, 391], q=[20, 300], H=2, bs=7),
    "fp8": dict(seq=[300, 77], q=[50, 77], H=3, fp8=True),
    "fp8_any_scale": dict(seq=[300, 77], q=[50, 77], H=2, fp8=True, pow2=False, bs=64),
    "shard_tables": dict(seq=[300, 77, 5], q=[50, 70, 5], H=2, D=3, I=4, local=True),
    "shard_tables_fp8": dict(seq=[513, 64], q=[13, 60], H=1, D=8, I=64, local=True, fp8=True, bs=64),
    "one_table_many_shards": dict(seq=[300], q=[50], H=2, D=8, I=2),
    "many_requests": dict(seq=[(37 * i) % 190 for i in range(70)], q=[(5 * i) % 9 for i in range(70)], H=1),
    "sharp_scores": dict(seq=[400], q=[150], H=2, q_scale=30.0),
    "many_heads": dict(seq=[140], q=[30], H=67),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_against_the_reference(name):
    st = ref.make(**CASES[name])
    want = ref.reference(st)
    out, lse, err = run(st)
    assert err == 0
    ref.check(out, lse, want)
    out32, lse32, _ = run(st, out_dtype=torch.float32)
    ref.check(out32, lse32, want)
    assert torch.equal(lse32.nan_to_num(), lse.nan_to_num()) and torch.equal(out32.to(torch.bfloat16), out)


@pytest.mark.parametrize("scale", [0.0, -0.0722, 3.0, -2.0])
def test_scales(scale):
    st = ref.make(seq=[300, 20], q=[150, 20], H=2, seed=1)
    st["scale"] = scale
    out, lse, _ = run(st)
    ref.check(out, lse, ref.reference(st))


def test_strided_queries_and_longer_bounds():
    st = ref.make(seq=[300, 20], q=[150, 20], H=3, seed=2)
    wide = torch.zeros((3, 171, 200), dtype=torch.bfloat16, device="cuda")
    q = wide.transpose(0, 1)[:170, :, :192]
    q.copy_(st["q"])
    st["q"] = q
    out, lse, err = run(st, total_len=5000)
    ref.check(out, lse, ref.reference(st))
    assert err == 0


def test_passes_over_the_heads_are_the_same():
    st = ref.make(seq=[300, 20, 500], q=[150, 20, 5], H=7, seed=3)
    out, lse, _ = run(st)
    ref.check(out, lse, ref.reference(st))
    n = dcp.dcp_chunk_attention_workspace_size(3, st["T"], 7, st["total"])
    one = dcp.dcp_chunk_attention_workspace_size(3, st["T"], 1, st["total"])
    for size in (one, one + (n - one) // 3, n - 16, n, n + 1000):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        o, l, _ = run(st, workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
    with pytest.raises(dcp.DCPError):
        run(st, workspace=torch.empty(one - 16, dtype=torch.uint8, device="cuda"))


def test_a_context_that_does_not_fit_is_not_seen():
    st = ref.make(seq=[300, 2000, 100], q=[30, 40, 20], H=2, seed=4)
    out, lse, err = run(st, total_len=600)
    assert err == dcp.DEVERR_SEQ_TOO_LONG
    ref.check(out, lse, ref.reference(st, skip_requests=(1, 2)))


def test_bad_blocks_are_skipped():
    st = ref.make(seq=[300, 150], q=[60, 30], H=2, seed=5)
    st["table"][0, 3], st["table"][0, 18], st["table"][1, 0] = -1, st["cache"].shape[0], 1 << 30
    out, lse, err = run(st)
    assert err == dcp.DEVERR_BAD_BLOCK
    ref.check(out, lse, ref.reference(st))
    st["table"][1] = -5  # a request without any block
    out, lse, err = run(st)
    ref.check(out, lse, ref.reference(st))
    st = ref.make(seq=[300], q=[60], H=2, seed=5)
    full = st["table"]
    st["table"] = full[:, :10].contiguous()  # columns missing
    out, lse, err = run(st)
    assert err == dcp.DEVERR_BAD_BLOCK
    st["table"] = torch.cat([full[:, :10], torch.full_like(full[:, 10:], -1)], 1)
    ref.check(out, lse, ref.reference(st))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dim", [5, 560])
def test_nonfinite_latents_reach_only_the_rows_that_see_them(value, dim):
    st = ref.make(seq=[300, 150], q=[200, 150], H=2, seed=6)
    clean_out, clean_lse, _ = run(st)
    rows = ref.rows_of(st, 0)
    st["cache"].view(-1, 576)[int(rows[210]), dim] = value  # the token of row 110 of request 0
    out, lse, _ = run(st)
    keep = torch.ones(350, dtype=torch.bool)
    keep[110:200] = False
    assert torch.equal(out[keep], clean_out[keep]) and torch.equal(lse[keep], clean_lse[keep])
    hit = ~keep
    if dim < 512:
        assert out[hit].isnan().all() and lse[hit].isnan().all()
    else:  # an infinite score: weight 0 where it is negative, NaN else
        s = st["q"][hit][..., 128 + dim - 512].double().cuda() * st["scale"] * value
        lost = ~(s == -torch.inf)
        assert out[hit][lost].isnan().all() and out[hit][~lost].isfinite().all() and lse[hit][~lost].isfinite().all()


def test_nonfinite_queries_stay_in_their_rows():
    st = ref.make(seq=[300], q=[200], H=2, seed=7)
    out, lse, _ = run(st)
    st["q"][50, 1, 3] = float("nan")
    o, l, _ = run(st)
    assert o[50, 1].isnan().all() and l[50, 1].isnan()
    o[50, 1], l[50, 1] = out[50, 1], lse[50, 1]
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_unused_cache_rows_may_hold_anything():
    st = ref.make(seq=[300, 77], q=[50, 77], H=2, seed=8)
    want = ref.reference(st)
    used = np.concatenate([ref.rows_of(st, b) for b in range(2)])
    other = torch.ones(st["cache"].shape[0] * st["bs"], dtype=torch.bool)
    other[torch.from_numpy(used)] = False
    st["cache"].view(-1, 576)[other.cuda()] = float("nan")
    out, lse, _ = run(st)
    ref.check(out, lse, want)


def test_the_same_as_the_decode_with_absorbed_queries():
    """Both forms of one attention: bf16 roundings of keys, values and weights on
    this side, of absorbed queries and outputs on that one."""
    st = ref.make(seq=[700, 90], q=[3, 2], H=16, bs=64, seed=9, q_scale=1.0)
    out, lse, _ = run(st)
    w = st["w"].view(16, 256, 512)
    ql = torch.einsum("thk,hkc->thc", st["q"][..., :128].float(), w[:, :128].float())
    q = torch.cat([ql.to(torch.bfloat16), st["q"][..., 128:]], 2)
    O, l = dcp.decode_partial(q, st["cache"], st["table"], st["seq"], st["qsl"], D=1, interleave=1, scale=st["scale"],
                              max_seq_len=700, max_q_len=3)
    o = torch.einsum("thc,hvc->thv", O[0], w[:, 128:].float())
    _, _, tol, tol_l = ref.reference(st)
    assert ((out.float() - o).abs() <= 2 * tol + 2.0 ** -7 * o.abs()).all()
    assert ((lse - l[0]).abs() <= 2 * tol_l + 0.01).all()


def test_captured_streams_and_two_calls_at_once():
    st = [ref.make(seq=[300, 77], q=[50, 77], H=2, seed=s) for s in (10, 11)]
    eager = [run(s) for s in st]
    packed = [dcp.pack_kv_b(s["w"]) for s in st]

    def call(i, **kw):
        s = st[i]
        return dcp.chunk_attention(s["q"], s["cache"], s["table"], s["seq"], s["qsl"], packed[i], scale=s["scale"],
                                   total_len=s["total"], **kw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(0), call(1)]
    for _ in range(2):
        graph.replay()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        pair = [call(i, stream=side[i]) for i in range(2)]
    torch.cuda.synchronize()
    for (o, l, _), a, b in zip(eager, got, pair):
        assert torch.equal(o, a[0]) and torch.equal(l, a[1]) and torch.equal(o, b[0]) and torch.equal(l, b[1])


def test_more_units_than_fit_at_once_and_repeatable():
    st = ref.make(seq=[900, 2000, 30], q=[800, 600, 30], H=60, bs=64, seed=12)
    out, lse, _ = run(st)
    again = run(st)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    few = dict(st, H=2, q=st["q"][:, 57:59].contiguous(), w=st["w"][57 * 256:59 * 256].contiguous())
    ref.check(out[:, 57:59].contiguous(), lse[:, 57:59].contiguous(), ref.reference(few))
