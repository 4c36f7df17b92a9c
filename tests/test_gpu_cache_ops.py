"""GPU checks of the quantising cache write and the cache read-back against the
64-bit oracle.  Codes, scales and copies are exact; a value read back from an
fp8 cache is code x scale rounded once (half a step: 2^-24 relative in fp32,
2^-8 in bf16; exact when the scale is a power of two and the output fp32)."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _rows(rng, n, spread=8.0):
    x = rng.standard_normal((n, 576), dtype=np.float32)
    return wl.f32_to_bf16_bits(x * np.exp(rng.uniform(-spread, spread, (n, 1))).astype(np.float32))


def _t(bits):
    return G.bf16_tensor(bits)


def _host(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _special_rows():
    """Rows where a quantiser can go wrong: zeros, one value, exactly 256 s and
    just above, ties, the smallest and largest bf16, infinities and NaN."""
    b = wl.f32_to_bf16_bits(np.random.default_rng(1).standard_normal((12, 576), dtype=np.float32))
    f = lambda v: wl.f32_to_bf16_bits(np.array([v], dtype=np.float32))[0]  # noqa: E731
    b[0] = 0
    b[1] = 0
    b[1, 575] = f(-3.0)
    b[2, 0] = f(256.0)
    b[3, 0] = f(258.0)                       # the next bf16: the scale doubles
    b[4, :8] = [f(v) for v in (256, 17, 19, 21, -25, 2 ** -10, -3 * 2 ** -10, 2 ** -9)]
    b[5] = 0x0001                            # the least subnormal
    b[6] = 0x8001
    b[6, 9] = 0x007F
    b[7, 3] = 0x7F7F                         # the largest finite
    b[8, 3], b[8, 4] = 0x7F80, 0xFF80
    b[9, 511], b[9, 512] = 0x7FC0, 0xFFC1
    b[10] = 0x7FC0
    b[11] = 0x8000
    return b


@pytest.mark.parametrize("T,H", [(1, 0), (5, 1), (67, 33), (64, 128), (1031, 0)])
def test_fp8_write_matches_oracle(T, H):
    rng = np.random.default_rng(100 * T + H)
    x = _rows(rng, T)
    nb, bs = T // 8 + 3, 16
    slots = rng.choice(nb * bs, size=T, replace=False).astype(np.int64)
    slots[2::5] = -1 - slots[2::5]
    codes = rng.integers(0, 256, (nb, bs, 576), dtype=np.uint8)
    scale = rng.random((nb, bs), dtype=np.float32)
    codes_ref, scale_ref = oracle.concat_cache_fp8(x[:, :512], x[:, 512:], slots, codes, scale)
    wide = _t(np.concatenate([x, x[:, :64]], axis=1))  # both parts as slices of a wider row
    codes_d, scale_d = torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.from_numpy(slots).cuda()
    if H == 0:
        dcp.latent_cache_write(wide[:, :512], wide[:, 512:576], at, codes_d, kv_scale=scale_d, dev_error=err)
    else:
        ql, qp = rng.integers(0, 0x7F00, (H, T, 512), dtype=np.uint16), rng.integers(0, 0x7F00, (T, H, 64), dtype=np.uint16)
        q = dcp.decode_concat_cache(_t(ql).transpose(0, 1), _t(qp), wide[:, :512], wide[:, 512:576], at, codes_d,
                                    dev_error=err, kv_scale=scale_d)
        assert np.array_equal(_host(q), np.concatenate([ql.transpose(1, 0, 2), qp], axis=2))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(scale_d.cpu().numpy(), scale_ref)
    assert np.array_equal(codes_d.cpu().numpy(), codes_ref)


def test_fp8_write_of_special_rows():
    x = _special_rows()
    n = len(x)
    codes_d = torch.zeros((n, 1, 576), dtype=torch.uint8, device="cuda")
    scale_d = torch.zeros((n, 1), device="cuda")
    dcp.latent_cache_write(_t(x[:, :512]), _t(x[:, 512:]), torch.arange(n, device="cuda"), codes_d, kv_scale=scale_d)
    codes, scale = oracle.quantize_rows(x)
    assert np.array_equal(scale_d.cpu().numpy()[:, 0], scale)
    got = codes_d.cpu().numpy()[:, 0]
    nan = (codes & 0x7F) == 0x7F
    assert ((got[nan] & 0x7F) == 0x7F).all()  # either NaN code
    assert np.array_equal(got[~nan], codes[~nan])


def test_write_bf16_cache_alone_and_bad_slots():
    rng = np.random.default_rng(8)
    x = _rows(rng, 9)
    nb, bs = 2, 8
    for fp8 in (False, True):
        slots = np.array([3, -1, 15, 16, 0, -9, 1 << 40, 7, 8], dtype=np.int64)
        ok = np.where(slots < nb * bs, slots, -1)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if fp8:
            c, s = np.full((nb, bs, 576), 3, np.uint8), np.full((nb, bs), 2.0, np.float32)
            c_ref, s_ref = oracle.concat_cache_fp8(x[:, :512], x[:, 512:], ok, c, s)
            cd, sd = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
            dcp.latent_cache_write(_t(x)[:, :512], _t(x)[:, 512:], torch.from_numpy(slots).cuda(), cd, sd, err)
            assert np.array_equal(cd.cpu().numpy(), c_ref) and np.array_equal(sd.cpu().numpy(), s_ref)
        else:
            c = _rows(rng, nb * bs).reshape(nb, bs, 576)
            q = np.zeros((9, 1, 512), np.uint16)
            _, c_ref = oracle.concat_cache(q, q[:, :, :64], x[:, :512], x[:, 512:], ok, c)
            cd = _t(c)
            dcp.latent_cache_write(_t(x)[:, :512], _t(x)[:, 512:], torch.from_numpy(slots).cuda(), cd, dev_error=err)
            assert np.array_equal(_host(cd), c_ref)
        assert int(err.item()) == dcp.DEVERR_BAD_BLOCK


def test_written_fp8_cache_is_the_generators():
    """The write gives byte for byte the cache that the fp8 decode's inputs are
    made with, so the decode's own parity holds for it."""
    spec = wl.DecodeSpec("w", seed=33, B=2, seq_lens=(70, 33), H=1, block_size=16, kv_dtype="fp8_e4m3")
    f, b = wl.make_decode_inputs(spec), wl.make_decode_inputs(wl.DecodeSpec("w", seed=33, B=2, seq_lens=(70, 33), H=1,
                                                                            block_size=16))
    live = np.concatenate([f["block_table"][r, np.arange(n) // 16] * 16 + np.arange(n) % 16 for r, n in ((0, 70), (1, 33))])
    x = b["kv_cache"].reshape(-1, 576)[live]
    # the generator quantises the fp32 draws: start from its values on a grid both hold exactly
    back = (oracle.fp8_e4m3_to_f64(f["kv_cache"].reshape(-1, 576)[live]) * f["kv_scale"].reshape(-1)[live][:, None])
    x = wl.f32_to_bf16_bits(back.astype(np.float32))
    codes, scale = oracle.quantize_rows(x)
    cd, sd = torch.zeros((103, 1, 576), dtype=torch.uint8, device="cuda"), torch.zeros((103, 1), device="cuda")
    dcp.latent_cache_write(_t(x[:, :512]), _t(x[:, 512:]), torch.arange(103, device="cuda"), cd, kv_scale=sd)
    assert np.array_equal(cd.cpu().numpy()[:, 0], codes) and np.array_equal(sd.cpu().numpy()[:, 0], scale)
    got = oracle.fp8_e4m3_to_f64(cd.cpu().numpy()[:, 0]) * sd.cpu().numpy()
    assert np.array_equal(got, back)  # requantising a held value loses nothing


READS = [
    # (seed, seqs, starts, block_size, D, I, local, fp8)
    (1, (37, 1, 0, 300), (0, 0, 0, 13), 16, 1, 1, False, False),
    (2, (37, 129), (36, 0), 1, 4, 3, False, True),
    (3, (250, 40, 77), (7, 40, 70), 8, 4, 3, True, True),
    (4, (500,), (0,), 64, 8, 64, True, False),
    (5, tuple(1 + b % 3 for b in range(70)), (0,) * 70, 4, 2, 1, False, True),
    (6, (2049, 5), (1, 5), 64, 3, 1, True, False),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", READS, ids=lambda c: str(c[0]))
def test_read_back_matches_oracle(case, out_dtype):
    seed, seqs, starts, bs, D, I, local, fp8 = case
    inp = wl.make_decode_inputs(wl.DecodeSpec("r", seed=seed, B=len(seqs), seq_lens=seqs, H=1, block_size=bs, D=D,
                                              interleave=I, layout="local" if local else "global",
                                              kv_dtype="fp8_e4m3" if fp8 else "bf16"))
    if fp8 and seed % 2:  # scales that are not powers of two: one rounding
        inp["kv_scale"] = (inp["kv_scale"] * np.random.default_rng(seed).uniform(0.6, 1.0, inp["kv_scale"].shape)
                           ).astype(np.float32)
    t = G.to_device(inp)
    starts = np.asarray(starts, np.int32)
    cu = np.concatenate([[0], np.cumsum(inp["seq_lens"] - starts)]).astype(np.int32)
    N = int(cu[-1])
    st, cud = torch.from_numpy(starts).cuda(), torch.from_numpy(cu).cuda()
    rows = oracle.kv_rows_f64(inp)
    # the fp32 product, then (bf16) one more rounding
    step = 2.0 ** -24 + (2.0 ** -8 if out_dtype == torch.bfloat16 else 0.0)
    for shards in ([range(D)] if D == 1 else [range(D), range(1, 2)]):
        tab = t["block_table"][shards.start:shards.stop] if local else t["block_table"]
        ref = oracle.cache_read(rows, tab.cpu().numpy(), bs, starts, cu, D, I, shards, local)
        buf = torch.full((N + 5, 584), 7.0, dtype=out_dtype, device="cuda")  # strided rows, spare rows
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        dcp.dcp_latent_cache_read(t["kv_cache"], tab, cud, buf[:, :576], seq_starts=st, kv_scale=t.get("kv_scale"),
                                  D=D, interleave=I, shard_begin=shards.start, shard_count=len(shards), dev_error=err)
        got = buf.double().cpu().numpy()
        assert int(err.item()) == 0
        assert (got[N:] == 7).all() and (got[:, 576:] == 7).all()  # nothing else is written
        assert (np.abs(got[:N, :576] - ref) <= step * np.abs(ref)).all()
        if not fp8:
            assert np.array_equal(got[:N, :576], ref)


def test_read_back_flags_what_it_cannot_find():
    cache = torch.ones((4, 8, 576), dtype=torch.bfloat16, device="cuda")
    tab = torch.tensor([[0, 9, -1], [1, 2, 3]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 24, 34], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, -2], dtype=torch.int32, device="cuda")
    for name, c, s, n in (("block ids", cu, None, 34), ("negative", cu, starts, 34),
                          ("past the table", torch.tensor([0, 8, 40], dtype=torch.int32, device="cuda"), None, 40)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = dcp.latent_cache_read(cache, tab, c, n, seq_starts=s, dev_error=err)
        assert int(err.item()) == dcp.DEVERR_BAD_BLOCK, name
        got = out[:, 0].float().cpu().numpy()
        if name == "past the table":
            want = [1] * 8 + [1] * 24 + [0] * 8
        else:
            want = [1] * 8 + [0] * 16 + ([0] * 2 + [1] * 8 if s is not None else [1] * 10)
        assert list(got) == want, name


def test_read_back_without_requests_or_rows():
    cache = torch.ones((1, 1, 576), dtype=torch.bfloat16, device="cuda")
    none = torch.zeros((0, 1), dtype=torch.int32, device="cuda")
    out = torch.full((3, 576), 5.0, device="cuda")
    dcp.dcp_latent_cache_read(cache, none, torch.zeros(1, dtype=torch.int32, device="cuda"), out)
    dcp.dcp_latent_cache_read(cache, torch.zeros((2, 1), dtype=torch.int32, device="cuda"),
                              torch.zeros(3, dtype=torch.int32, device="cuda"), out)  # two empty ranges
    assert (out == 5).all()
    assert dcp.latent_cache_read(cache, none, torch.zeros(1, dtype=torch.int32, device="cuda"), 0).shape == (0, 576)


def test_write_and_read_captured_on_another_stream():
    rng = np.random.default_rng(3)
    x = _rows(rng, 50)
    kc, kp = _t(x[:, :512]), _t(x[:, 512:])
    codes, scale = torch.zeros((7, 8, 576), dtype=torch.uint8, device="cuda"), torch.ones((7, 8), device="cuda")
    slots = torch.arange(50, device="cuda").flip(0)
    tab, cu = torch.arange(7, dtype=torch.int32, device="cuda")[None], torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    out = torch.zeros((50, 576), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dcp.latent_cache_write(kc, kp, slots, codes, kv_scale=scale)
        dcp.dcp_latent_cache_read(codes, tab, cu, out, kv_scale=scale)
    for k in range(2):
        x = _rows(rng, 50)
        kc.copy_(_t(x[:, :512]))
        kp.copy_(_t(x[:, 512:]))
        g.replay()
        torch.cuda.synchronize()
        c, sc = oracle.quantize_rows(x)
        want = oracle.fp8_e4m3_to_f64(c) * sc[:, None]
        assert np.array_equal(out.double().cpu().numpy()[::-1], want)
