"""Norm, rotation, concat and cache write in one launch, against fp64.

Tolerances: fp32 arithmetic of a few operations (the mean's sum of 512 squares
among them) is within 1e-6 of the value (of the pair's length for a rotation);
then one rounding, half a step: bf16 2^-8 of the value, E4M3 2^-4 of it and
half of its least step, 2^-10 of the scale."""
import numpy as np
import pytest
import torch

import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(T, H, query, fp8, seed=0, top=200, spare=5, bs=16):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    kv = rand(T, 576) * 3
    nb = (T + spare + bs - 1) // bs
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T]
    slots = torch.where(torch.arange(T, device="cuda") % 7 == 3, torch.full_like(slots, -1), slots)
    ang = torch.rand((top, 32), generator=g, device="cuda", dtype=torch.float64) * 6.28
    st = dict(kv_c=kv[:, :512], k_pe=kv[:, 512:], slots=slots,
              positions=torch.randint(0, top, (T,), generator=g, device="cuda").to(torch.int32),
              cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(), weight=rand(512) + 1,
              cache=torch.full((nb, bs, 576), 7, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda"),
              scale=torch.full((nb, bs), 3.0, device="cuda") if fp8 else None, ql=None, q=None)
    if query:
        st["q"] = rand(T, H, 192)[..., 128:]
    if query == "decode":
        st["ql"] = rand(H, T, 512).transpose(0, 1)
    return st


def rotated(x, pos, cs, pairs):
    """x fp64 [T, .., 64] turned as complex numbers; positions outside the table: as it is."""
    live = (pos >= 0) & (pos < len(cs))
    a = cs[np.where(live, pos, 0)].astype(np.float64)
    turn = np.where(live[:, None], a[:, :32] + 1j * a[:, 32:], 1.0)
    turn = turn.reshape(turn.shape[0], *([1] * (x.ndim - 2)), 32)
    z = (x[..., 0::2] + 1j * x[..., 1::2] if pairs else x[..., :32] + 1j * x[..., 32:]) * turn
    out = np.empty_like(x)
    if pairs:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    else:
        out[..., :32], out[..., 32:] = z.real, z.imag
    length = np.repeat(np.abs(z), 2, -1) if pairs else np.concatenate([np.abs(z)] * 2, -1)
    return out, length


def f64(t):
    return t.double().cpu().numpy()


def rows64(st, norm, pairs):
    x = f64(st["kv_c"])
    if norm:
        x = x / np.sqrt((x * x).mean(1, keepdims=True) + EPS) * f64(st["weight"])
    r, length = rotated(f64(st["k_pe"]), st["positions"].cpu().numpy(), st["cos_sin"].cpu().numpy(), pairs)
    return np.concatenate([x, r], 1), np.concatenate([np.abs(x), length], 1)


def check_cache(st, norm, pairs, before, before_scale):
    row, size = rows64(st, norm, pairs)
    slots = st["slots"].cpu().numpy()
    live = slots >= 0
    fp8 = st["scale"] is not None
    flat = st["cache"].reshape(-1, 576)
    got = f64(flat.view(torch.float8_e4m3fn) if fp8 else flat)
    other = np.ones(len(got), bool)
    other[slots[live]] = False
    assert torch.equal(flat[torch.from_numpy(other).cuda()], before.reshape(-1, 576)[torch.from_numpy(other).cuda()])
    err = 1e-6 * size[live]
    if fp8:
        s = f64(st["scale"]).reshape(-1)
        assert (s[other] == f64(before_scale).reshape(-1)[other]).all()
        s = s[slots[live]][:, None]
        top = np.abs(row[live]).max(1, keepdims=True)
        assert (np.log2(s) % 1 == 0).all()
        some = top[:, 0] > 0
        assert (top <= 256 * s * (1 + 1e-6)).all() and (top > 128 * s * (1 - 1e-6))[some].all() and (s[~some] == 1).all()
        assert (np.abs(got[slots[live]] * s - row[live]) <= err + 2.0 ** -4 * np.abs(row[live]) + 2.0 ** -10 * s).all()
    else:
        assert (np.abs(got[slots[live]] - row[live]) <= err + 2.0 ** -8 * np.abs(row[live])).all()


def check_query(got, st, pairs):
    r, length = rotated(f64(st["q"]), st["positions"].cpu().numpy(), st["cos_sin"].cpu().numpy(), pairs)
    if st["ql"] is not None:
        assert torch.equal(got[..., :512], st["ql"])
        got = got[..., 512:]
    assert (np.abs(f64(got) - r) <= 1e-6 * length + 2.0 ** -8 * np.abs(r)).all()


def call(st, norm, pairs, **kw):
    return dcp.norm_rope_cache(st["kv_c"], st["k_pe"], st["slots"], st["cache"], st["positions"], st["cos_sin"],
                               norm_weight=st["weight"] if norm else None, eps=EPS, ql_nope=st["ql"], q_pe=st["q"],
                               interleaved=pairs, kv_scale=st["scale"], **kw)


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,query", [(1, 0, None), (1, 1, "decode"), (1, 128, "decode"), (9, 6, "decode"),
                                       (37, 33, "decode"), (1, 1, "pe"), (5, 17, "pe"), (301, 20, "pe"), (77, 0, None)])
def test_rows_and_queries(T, H, query, fp8, pairs):
    for norm in (True, False):
        st = make(T, H, query, fp8, seed=T + H)
        before, scale = st["cache"].clone(), None if st["scale"] is None else st["scale"].clone()
        q = call(st, norm, pairs)
        torch.cuda.synchronize()
        check_cache(st, norm, pairs, before, scale)
        if query:
            check_query(q, st, pairs)
        else:
            assert q is None


@pytest.mark.parametrize("pairs", [True, False])
def test_rope_parts_turned_in_place(pairs):
    st = make(23, 37, "pe", False, seed=3)
    whole = torch.randn((23, 37, 192), device="cuda").to(torch.bfloat16)
    st["q"] = whole[..., 128:]
    want, keep = whole.clone(), st["q"].clone()
    assert call(st, True, pairs, q_out=st["q"]) is st["q"]
    torch.cuda.synchronize()
    assert torch.equal(whole[..., :128], want[..., :128])
    st["q"] = keep
    check_query(whole[..., 128:], st, pairs)


def test_heads_outside_tokens():
    """Output laid out [H, T, ..], and a query whose heads are a slice."""
    for query, width in (("decode", 576), ("pe", 64)):
        st = make(11, 5, query, False, seed=4)
        out = torch.full((5, 12, width + 8), 5.0, dtype=torch.bfloat16, device="cuda")
        q = out.transpose(0, 1)[:11, :, :width]
        call(st, True, True, q_out=q)
        torch.cuda.synchronize()
        check_query(q, st, True)
        assert (out[:, 11] == 5).all() and (out[..., width:] == 5).all()


def test_positions_outside_the_table():
    st = make(10, 3, "decode", False, seed=5)
    st["positions"][2], st["positions"][6] = -1, 1 << 30
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = st["cache"].clone()
    q = call(st, True, True, dev_error=err)
    torch.cuda.synchronize()
    check_cache(st, True, True, before, None)
    check_query(q, st, True)
    assert int(err) == dcp.DEVERR_BAD_POSITION
    st["positions"][6] = 0
    err.zero_()
    call(st, True, True, dev_error=err)
    assert int(err) == 0


def test_slot_past_the_cache():
    st = make(10, 0, None, True, seed=6)
    st["slots"][1] = st["cache"].shape[0] * st["cache"].shape[1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before, scale = st["cache"].clone(), st["scale"].clone()
    call(st, True, True, dev_error=err)
    torch.cuda.synchronize()
    st["slots"][1] = -1
    check_cache(st, True, True, before, scale)
    assert int(err) == dcp.DEVERR_BAD_BLOCK


@pytest.mark.parametrize("fp8", [False, True])
def test_zero_tiny_and_nonfinite_rows(fp8):
    """A row of zeros, the least magnitudes, and infinities or NaN in one row,
    which the others do not see."""
    st = make(16, 0, None, fp8, seed=7)
    kv = torch.randn((16, 576), device="cuda").to(torch.bfloat16)
    kv[0] = 0
    kv[1] *= 2.0 ** -120
    kv[4, 5], kv[5, 550], kv[6, 2] = float("nan"), float("inf"), float("-inf")
    st.update(kv_c=kv[:, :512], k_pe=kv[:, 512:], slots=torch.arange(16, device="cuda"))
    call(st, False, True)
    torch.cuda.synchronize()
    flat = st["cache"].reshape(-1, 576)
    got = flat.view(torch.float8_e4m3fn).double() * st["scale"].reshape(-1, 1).double() if fp8 else flat.double()
    assert not got[4, 5].isfinite() and not got[6, 2].isfinite() and not got[5, 550:552].isfinite().any()
    row, _ = rows64(st, False, True)
    row, got = row[:16], got[:16].cpu().numpy()
    ok = np.isfinite(row)
    ok[5, 550:552] = False
    assert np.isfinite(got[ok]).all() and (got[0] == 0).all()
    s = st["scale"].reshape(-1)[:16].double().cpu().numpy()[:, None] if fp8 else 0 * row[:, :1]
    # (below 2^-126 a bf16 step is 2^-133 whatever the value, so half a step 2^-134, which
    # is more than 2^-8 of it: the least row's turned parts come down to there)
    tol = 2.0 ** (-4 if fp8 else -8) * np.abs(row) + 2.0 ** -10 * s + 1e-6 * np.abs(row).max(1, keepdims=True) + 2.0 ** -134
    assert (np.abs(got - row) <= tol)[:4][ok[:4]].all() and (np.abs(got - row) <= tol)[7:].all()


def test_captured_streams_and_the_decode_behind_it():
    """Captured with the decode that reads its rows; the same as the eager calls
    and as the concat of parts normed and turned before."""
    T, H = 4, 16
    st = make(T, H, "decode", False, seed=8, bs=64, spare=300)
    st["slots"] = torch.arange(T, device="cuda") * 64 + 20
    st["cache"].normal_()
    table = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    seq = torch.full((T,), 21, dtype=torch.int32, device="cuda")
    qsl = torch.arange(T + 1, dtype=torch.int32, device="cuda")

    def step():
        q = call(st, True, True)
        return q, dcp.decode_partial(q, st["cache"], table, seq, qsl, D=1, interleave=1, scale=0.07, max_seq_len=21,
                                     max_q_len=1)

    q0, (O0, l0) = step()
    torch.cuda.synchronize()
    row, size = rows64(st, True, True)
    parts = torch.from_numpy(row).cuda().to(torch.bfloat16)
    cache = st["cache"].clone()
    q1 = dcp.decode_concat_cache(st["ql"], torch.from_numpy(rotated(f64(st["q"]), st["positions"].cpu().numpy(),
                                 st["cos_sin"].cpu().numpy(), True)[0]).cuda().to(torch.bfloat16),
                                 parts[:, :512].contiguous(), parts[:, 512:].contiguous(), st["slots"], cache)
    assert (q1.double() - q0.double()).abs().max() <= 2.0 ** -7 * q0.abs().max()  # a step, where fp32 fell on the other side
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q2, (O2, l2) = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, q0) and torch.equal(O2, O0) and torch.equal(l2, l0)
    side = torch.cuda.Stream()
    q3 = call(st, True, True, stream=side)
    side.synchronize()
    assert torch.equal(q3, q0)
