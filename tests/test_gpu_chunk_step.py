"""A prefill chunk's step as it is used: tables extended, latents normed, turned
and written, queries turned in place, attention over the cache; then a decode
step on the same cache.  And its parts at the ends of their ranges."""
import math

import numpy as np
import pytest
import torch

from tests import chunk_reference as ref
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu
H, BS, EPS = 5, 16, 1e-6


def rotated(x, pos, cs):
    """fp64 [T, .., 64], pairs (2i, 2i + 1) as complex numbers."""
    a = cs[pos].double()
    turn = torch.complex(a[:, :32], a[:, 32:]).view(len(pos), *([1] * (x.dim() - 2)), 32)
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], 32, 2)) * turn
    return torch.view_as_real(z).flatten(-2)


def step_inputs(g, T):
    def rand(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    return dict(kv=rand(T, 576), q=rand(T, H, 192))


@pytest.mark.parametrize("fp8,D,I,local", [(False, 1, 1, False), (True, 1, 1, False), (True, 3, 4, True), (False, 2, 1, False)])
def test_two_chunks_and_a_decode_step(fp8, D, I, local):
    """Requests prefill in two chunks; every row of both is compared with exact
    attention over the latents that the cache holds."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, blocks = 3, 200
    cache = torch.zeros((blocks, BS, 576), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    scale = torch.ones((blocks, BS), device="cuda") if fp8 else None
    table = torch.full((D, B, 20) if local else (B, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor([blocks], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ang = torch.arange(1000, device="cuda", dtype=torch.float64)[:, None] * 1000.0 ** (-torch.arange(32, device="cuda") / 32.0)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    weight = (1 + 0.1 * torch.empty(512, device="cuda").normal_(generator=g)).to(torch.bfloat16)
    w = (torch.empty((H * 256, 512), device="cuda").normal_(generator=g) / 512 ** 0.5).to(torch.bfloat16)
    packed = dcp.pack_kv_b(w)
    sm = 1 / math.sqrt(192)
    seq = [0, 0, 0]
    for q_lens in ([150, 0, 33], [37, 290, 1]):
        seq = [a + b for a, b in zip(seq, q_lens)]
        T = sum(q_lens) + 3  # three padded rows
        x = step_inputs(g, T)
        seq_d = torch.tensor(seq, dtype=torch.int32, device="cuda")
        qsl = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda")
        pos, slots = dcp.cache_extend(table, seq_d, qsl, free, count, T, BS, D=D, interleave=I, dev_error=err)
        raw = x["q"].clone()
        dcp.norm_rope_cache(x["kv"][:, :512], x["kv"][:, 512:], slots, cache, pos, cs, norm_weight=weight, eps=EPS,
                            q_pe=x["q"][..., 128:], q_out=x["q"][..., 128:], kv_scale=scale, dev_error=err)
        out, lse = dcp.chunk_attention(x["q"], cache, table, seq_d, qsl, packed, scale=sm, total_len=sum(seq),
                                       kv_scale=scale, D=D, interleave=I, dev_error=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        st = dict(seq_h=seq, q_h=q_lens, H=H, bs=BS, D=D, I=I, local=local, scale=sm, kv_scale=scale, table=table,
                  seq=seq_d, qsl=qsl, T=T, cache=cache, q=x["q"], w=w)
        ref.check(out, lse, ref.reference(st))
        # the queries and rows that attention saw are the exact ones, rounded
        n = sum(q_lens)
        p = pos[:n].long()
        want = rotated(raw[:n, :, 128:], p, cs)
        assert ((x["q"][:n, :, 128:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6 * want.abs().max()).all()
        assert torch.equal(x["q"][..., :128], raw[..., :128]) and torch.equal(x["q"][n:], raw[n:])
        c = x["kv"][:n, :512].double()
        c = c / (c.pow(2).mean(1, keepdim=True) + EPS).sqrt() * weight.double()
        row = torch.cat([c, rotated(x["kv"][:n, 512:], p, cs)], 1)
        flat = cache.view(-1, 576)[slots[:n]]
        if fp8:
            s = scale.view(-1)[slots[:n]].double()[:, None]
            assert ((flat.view(torch.float8_e4m3fn).double() * s - row).abs() <= 2.0 ** -4 * row.abs() + 2.0 ** -10 * s + 1e-5).all()
        else:
            assert ((flat.double() - row).abs() <= 2.0 ** -8 * row.abs() + 1e-5).all()
    if D > 1 and not local:
        return
    # a decode step of each request on the same cache, and the chunk's form of it
    seq = [s + 1 for s in seq]
    x = step_inputs(g, B)
    seq_d = torch.tensor(seq, dtype=torch.int32, device="cuda")
    qsl = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    pos, slots = dcp.cache_extend(table, seq_d, qsl, free, count, B, BS, D=D, interleave=I)
    up = w.view(H, 256, 512).float()
    ql = torch.einsum("thk,hkc->thc", x["q"][..., :128].float(), up[:, :128]).to(torch.bfloat16)
    q = dcp.norm_rope_cache(x["kv"][:, :512], x["kv"][:, 512:], slots, cache, pos, cs, norm_weight=weight, eps=EPS,
                            ql_nope=ql, q_pe=x["q"][..., 128:], kv_scale=scale)
    O, l = dcp.decode_partial(q, cache, table, seq_d, qsl, D=D, interleave=I, scale=sm, max_seq_len=max(seq),
                              max_q_len=1, kv_scale=scale)
    o, l = dcp.lse_combine(O, l, seq_d, qsl, out_dtype=torch.float32)
    o = torch.einsum("thc,hvc->thv", o, up[:, 128:])
    full = torch.cat([x["q"][..., :128], q[..., 512:]], 2).contiguous()
    out, lse = dcp.chunk_attention(full, cache, table, seq_d, qsl, packed, scale=sm, total_len=sum(seq), kv_scale=scale,
                                   D=D, interleave=I)
    # (the decode's queries, weights and, from FP8, latents are bf16: a few 2^-8 of sums of ~1)
    assert (out.float() - o).abs().max() <= 0.03 and (lse - l).abs().max() <= 0.01


def test_cache_rows_past_32_bits():
    """A cache of more than 2^32 bytes, its last blocks in use: written, read and
    attended to."""
    blocks, bs = 60000, 64
    cache = torch.zeros((blocks, bs, 576), dtype=torch.bfloat16, device="cuda")
    assert cache.numel() * 2 > 1 << 32
    st = ref.make(seq=[300, 70], q=[60, 70], H=2, bs=bs, seed=1)
    n = st["cache"].shape[0]
    cache[blocks - n:] = st["cache"]
    st["table"] = torch.where(st["table"] >= 0, st["table"] + blocks - n, st["table"])
    st["cache"] = cache
    rows = torch.from_numpy(np.concatenate([ref.rows_of(st, b) for b in range(2)])).cuda()
    new = torch.randn((len(rows), 576), device="cuda").to(torch.bfloat16)
    dcp.norm_rope_cache(new[:, :512], new[:, 512:], rows, cache, torch.full((len(rows),), -1, dtype=torch.int32, device="cuda"),
                        torch.zeros((1, 64), device="cuda"))
    assert torch.equal(cache.view(-1, 576)[rows], new)
    out, lse = dcp.chunk_attention(st["q"], cache, st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=st["total"])
    ref.check(out, lse, ref.reference(st))


def test_more_requests_than_the_plan_keeps():
    """1,500 requests: the plan reads its scans back from global memory."""
    seq = [(29 * i) % 170 for i in range(1500)]
    q = [(3 * i) % 4 for i in range(1500)]
    st = ref.make(seq=seq, q=q, H=1, bs=64, seed=2)
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=st["total"])
    ref.check(out, lse, ref.reference(st))


@pytest.mark.parametrize("lead,T_cut", [(5, 0), (300, 0), (0, 30), (7, 50)])
def test_rows_before_the_first_request_and_rows_cut_off(lead, T_cut):
    """query_start_loc that starts past row 0 (rows of no request before it), or that
    ends past the last row of the query (only the rows that exist are computed)."""
    st = ref.make(seq=[300, 77], q=[60, 77], H=2, bs=64, seed=7)
    want = ref.reference(st)
    T = lead + 137 - T_cut
    q = torch.zeros((T, 2, 192), dtype=torch.bfloat16, device="cuda")
    q[lead:] = st["q"][:137 - T_cut]
    out, lse = dcp.chunk_attention(q, st["cache"], st["table"], st["seq"], st["qsl"] + lead, dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=st["total"])
    assert (out[:lead] == 0).all() and (lse[:lead] == -torch.inf).all()
    ref.check(out[lead:], lse[lead:], [x[:137 - T_cut] for x in want])


def test_nothing_to_see():
    st = ref.make(seq=[0, 0], q=[3, 300], H=2, seed=3, pad=7)
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], dcp.pack_kv_b(st["w"]),
                                   scale=st["scale"], total_len=0)
    assert (out == 0).all() and (lse == -torch.inf).all()


@pytest.mark.parametrize("seq,q", [([20000], [1]), ([9000, 10], [130, 10]), ([3000], [3000]), ([1024, 1025], [40, 40])])
def test_long_contexts_in_pieces(seq, q):
    """Few rows over long contexts are cut along the tokens and joined; the border of
    the key remainders."""
    st = ref.make(seq=seq, q=q, H=2, bs=64, seed=4, pad=1)
    packed = dcp.pack_kv_b(st["w"])

    def run(**kw):
        return dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], packed, scale=st["scale"],
                                   total_len=st["total"], **kw)
    out, lse = run()
    ref.check(out, lse, ref.reference(st))
    out32, lse32 = run(out_dtype=torch.float32)
    ref.check(out32, lse32, ref.reference(st))
    for _ in range(3):
        o, l = run()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_nonfinite_latent_in_a_long_context():
    """Rows that see it are NaN through the pieces' join, the others unchanged."""
    st = ref.make(seq=[9000], q=[40], H=2, bs=64, seed=5)
    packed = dcp.pack_kv_b(st["w"])

    def run():
        return dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], packed, scale=st["scale"],
                                   total_len=9000)
    out, lse = run()
    st["cache"].view(-1, 576)[int(ref.rows_of(st, 0)[8980]), 3] = float("inf")
    o, l = run()
    assert torch.equal(o[:20], out[:20]) and torch.equal(l[:20], lse[:20])
    assert o[20:].isnan().all() and l[20:].isnan().all()


def test_extreme_queries_and_keys():
    """Query rows of any magnitude (each scaled by its own power of 2); rows with
    scores past 2e7 and rows that see keys past f16's largest are NaN, no others."""
    st = ref.make(seq=[300], q=[64], H=1, bs=64, seed=6)
    power = torch.randint(-120, 100, (64, 1, 1), device="cuda").double()
    st["q"] = (st["q"].double() * 2.0 ** power).to(torch.bfloat16)
    st["scale"] = 1.0
    ok = (power.view(-1) < -3).nonzero().view(-1)  # (where scores do not single out one token)
    packed = dcp.pack_kv_b(st["w"])
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], packed, scale=1.0, total_len=300)
    o, l, tol, tol_l = ref.reference(st)
    assert ((out.double() - o).abs() <= tol + 2.0 ** -8 * (o.abs() + tol))[ok].all()
    assert ((lse.double() - l).abs() <= tol_l)[ok].all()
    far, near = l.view(-1) > 3e7, l.view(-1) < 1.5e7
    assert out[far].isnan().all() and lse[far].isnan().all() and out[near].isfinite().all() and lse[near].isfinite().all()
    assert far.any() and (near & (l.view(-1) > 1e4)).any()
    st["cache"].view(-1, 576)[int(ref.rows_of(st, 0)[250]), :512] *= 2.0 ** 18
    st["scale"] = 2.0 ** -20
    out, lse = dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], packed, scale=2.0 ** -20,
                                   total_len=300)
    _, l, _, _ = ref.reference(st)
    sees = (torch.arange(236, 300) >= 250).cuda()
    assert out[sees].isnan().all() and out[~sees & (l.view(-1) < 1.5e7)].isfinite().all()
