"""Quantising cache write and cache read-back, without a GPU: the oracle's
quantiser against torch's conversion and the input generator's, its read-back
against the walker, and what the two entry points refuse before any launch."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from mla_decode_context_gb300 import build_lib

pytestmark = pytest.mark.cpu


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return dcp.lib()


def test_quantiser_oracle_is_the_generators_and_torchs():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 576), dtype=np.float32) * np.exp(rng.uniform(-30, 30, (40, 1))).astype(np.float32)
    x[3] = 0
    x[4, 1:] = 0
    x[5, :7] = [448.0, 256.0, -256.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]  # 256 exactly, ties, the last subnormal
    bits = wl.f32_to_bf16_bits(x)
    codes, scale = oracle.quantize_rows(bits)
    ref_codes, ref_scale = wl.quantize_fp8_e4m3((bits.astype(np.uint32) << 16).view(np.float32))
    assert np.array_equal(scale, ref_scale)
    assert np.array_equal(codes, ref_codes)
    assert np.abs(oracle.fp8_e4m3_to_f64(codes)).max() <= 256


def test_quantiser_oracle_on_non_finite_rows():
    bits = wl.f32_to_bf16_bits(np.full((2, 576), 3.0, np.float32))
    bits[0, 5], bits[0, 6], bits[0, 7] = 0x7F80, 0xFF80, 0x7FC0  # inf, -inf, NaN
    bits[1] = 0x7FC0
    codes, scale = oracle.quantize_rows(bits)
    assert list(codes[0, 5:8]) == [0x7F] * 3 and (codes[1] == 0x7F).all()
    assert scale[0] == 2.0 ** -6 and scale[1] == 1.0  # 3 <= 256 * 2^-6 = 4
    assert (oracle.fp8_e4m3_to_f64(codes[0, :5]) * scale[0] == 3.0).all()


def test_read_back_oracle_is_the_walker_and_shards_add_up():
    spec = dict(seed=9, B=2, seq_lens=(37, 20), H=1, block_size=8, D=3, interleave=2)
    g = wl.make_decode_inputs(wl.DecodeSpec("g", **spec))
    loc = wl.make_decode_inputs(wl.DecodeSpec("l", layout="local", **spec))
    cu, starts = np.array([0, 30, 41]), np.array([7, 3])
    whole = oracle.cache_read(oracle.kv_rows_f64(g), g["block_table"], 8, starts, cu)
    for b, (lo, n) in enumerate(((7, 30), (3, 11))):
        rows = oracle.gather_latents(g["kv_cache"], g["block_table"][b], 8, np.arange(lo, lo + n))
        assert np.array_equal(whole[cu[b]:cu[b + 1]], rows)
    parts = [oracle.cache_read(oracle.kv_rows_f64(loc), loc["block_table"][d:d + 1], 8, starts, cu, 3, 2, [d], True)
             for d in range(3)]
    assert np.array_equal(sum(parts), whole)


def _write(L, **kw):
    a = dict(qn=0x1000, qn_t=512, qn_h=512, qp=0x2000, qp_t=64, qp_h=64, kc=0x3000, kc_t=512, kp=0x4000, kp_t=64,
             slot=0x5000, T=2, H=1, qo=0x6000, qo_t=576, cache=0x7000, dt=1, sc=0x8000, nslots=16, err=None)
    a.update(kw)
    return L.dcp_decode_concat_cache_v2(a["qn"], a["qn_t"], a["qn_h"], a["qp"], a["qp_t"], a["qp_h"], a["kc"],
                                        a["kc_t"], a["kp"], a["kp_t"], a["slot"], a["T"], a["H"], a["qo"], a["qo_t"],
                                        a["cache"], a["dt"], a["sc"], a["nslots"], a["err"], None)


def test_write_refusals_before_launch(L):
    assert _write(L, T=0) == 0
    assert _write(L, T=-1) == 1 and _write(L, H=-1) == 1 and _write(L, nslots=0) == 1
    assert _write(L, dt=2) == 2
    assert _write(L, sc=None) == 1                     # an fp8 cache needs scales
    assert _write(L, sc=0x8002) == 3
    assert _write(L, slot=None) == 1 and _write(L, qo=None) == 1 and _write(L, kc=None) == 1
    assert _write(L, H=0) == 1                         # cache alone, yet query pointers given
    assert _write(L, qo_t=575) == 1 and _write(L, kc_t=-8) == 1
    assert _write(L, kc_t=516) == 3 and _write(L, qn=0x1008) == 3 and _write(L, cache=0x7004) == 3


def _read(L, **kw):
    a = dict(kv=0x1000, dt=0, sc=None, nb=4, bs=16, tab=0x2000, w=4, ws=4, loc=0, ss=0, D=4, I=1, d0=0, dn=4,
             starts=None, cu=0x3000, B=2, N=5, out=0x4000, odt=0, os=576, err=None)
    a.update(kw)
    return L.dcp_latent_cache_read(a["kv"], a["dt"], a["sc"], a["nb"], a["bs"], a["tab"], a["w"], a["ws"], a["loc"],
                                   a["ss"], a["D"], a["I"], a["d0"], a["dn"], a["starts"], a["cu"], a["B"], a["N"],
                                   a["out"], a["odt"], a["os"], a["err"], None)


def test_read_refusals_before_launch(L):
    assert _read(L, B=0) == 0 and _read(L, N=0) == 0
    assert _read(L, B=-1) == 1 and _read(L, N=-1) == 1
    assert _read(L, D=0) == 1 and _read(L, D=33) == 1 and _read(L, I=0) == 1
    assert _read(L, dt=5) == 2 and _read(L, odt=5) == 2
    assert _read(L, dt=1) == 1                         # an fp8 cache needs scales
    assert _read(L, kv=None) == 1 and _read(L, cu=None) == 1 and _read(L, out=None) == 1
    assert _read(L, nb=0) == 1 and _read(L, bs=0) == 1 and _read(L, ws=3) == 1 and _read(L, os=575) == 1
    assert _read(L, d0=-1) == 1 and _read(L, d0=1) == 1 and _read(L, dn=0) == 1
    assert _read(L, loc=1, ss=7) == 1                  # shards' tables would overlap
    assert _read(L, kv=0x1008) == 3 and _read(L, out=0x4004) == 3 and _read(L, os=580) == 3
    assert _read(L, odt=1, os=578) == 3


def test_wrappers_check_types_and_shapes_before_the_device():
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    cache, codes = torch.zeros((2, 8, 576), dtype=bf), torch.zeros((2, 8, 576), dtype=torch.uint8)
    kc, kp, slots = torch.zeros((3, 512), dtype=bf), torch.zeros((3, 64), dtype=bf), torch.zeros(3, dtype=torch.int64)
    sc = torch.ones((2, 8))
    w = dcp.latent_cache_write
    with pytest.raises(TypeError, match="kv_scale"):
        w(kc, kp, slots, codes)
    with pytest.raises(ValueError, match="kv_scale"):
        w(kc, kp, slots, cache, kv_scale=sc)
    with pytest.raises(ValueError, match="num_blocks, block_size"):
        w(kc, kp, slots, codes, kv_scale=torch.ones(16))
    with pytest.raises(TypeError, match="kv_c"):
        w(kc.float(), kp, slots, codes, kv_scale=sc)
    with pytest.raises(ValueError, match="disagree"):
        w(kc, kp[:2], slots, codes, kv_scale=sc)
    with pytest.raises(ValueError, match="slot_mapping"):
        w(kc, kp, slots.int(), codes, kv_scale=sc)
    with pytest.raises(TypeError, match="q_pe"):       # a query needs all of its tensors
        dcp.dcp_decode_concat_cache_v2(torch.zeros((3, 2, 512), dtype=bf), None, kc, kp, slots, None, cache)
    with pytest.raises(ValueError, match="CUDA"):
        w(kc, kp, slots, codes, kv_scale=sc)
    tab, cu, out = torch.zeros((2, 4), dtype=i32), torch.zeros(3, dtype=i32), torch.zeros((5, 576), dtype=bf)
    r = dcp.dcp_latent_cache_read
    with pytest.raises(TypeError, match="cu_lens"):
        r(cache, tab, cu.long(), out)
    with pytest.raises(TypeError, match="out"):
        r(cache, tab, cu, out.half())
    with pytest.raises(ValueError, match="block_table"):
        r(cache, tab[:1], cu, out)
    with pytest.raises(ValueError, match="seq_starts"):
        r(cache, tab, cu, out, seq_starts=cu)
    with pytest.raises(ValueError, match="576"):
        r(cache, tab, cu, out[:, :512])
    with pytest.raises(ValueError, match="shards"):
        r(cache, tab, cu, out, D=2, shard_begin=2)
    with pytest.raises(ValueError, match="CUDA"):
        r(cache, tab, cu, out)
