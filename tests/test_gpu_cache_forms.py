"""GPU checks of forms of the cache write and read-back: the write of a bf16 cache
with the decode query, and output rows before the first request.  Byte copies:
exact."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G
from tests.test_gpu_cache_ops import _host, _rows, _t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (67, 33), (64, 128), (1000, 4)])
def test_bf16_write_with_the_query(T, H):
    rng = np.random.default_rng(200 * T + H)
    x = _rows(rng, T)
    nb, bs = T // 8 + 3, 16
    cache = _rows(rng, nb * bs).reshape(nb, bs, 576)
    slots = rng.choice(nb * bs, size=T, replace=False).astype(np.int64)
    slots[2::5] = -1 - slots[2::5]
    ql, qp = rng.integers(0, 0x7F00, (H, T, 512), dtype=np.uint16), rng.integers(0, 0x7F00, (T, H, 64), dtype=np.uint16)
    q_ref, cache_ref = oracle.concat_cache(ql.transpose(1, 0, 2), qp, x[:, :512], x[:, 512:], slots, cache)
    wide = _t(np.concatenate([x, x[:, :64]], axis=1))
    cache_d = _t(cache)
    buf = torch.full((T + 1, H + 1, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dcp.dcp_decode_concat_cache_v2(_t(ql).transpose(0, 1), _t(qp), wide[:, :512], wide[:, 512:576],
                                   torch.from_numpy(slots).cuda(), buf[:T, :H], cache_d, dev_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(_host(buf[:T, :H]), q_ref) and np.array_equal(_host(cache_d), cache_ref)
    assert (buf[T:] == 7).all() and (buf[:, H:] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("first", [1, 7, 8, 33])
def test_output_rows_before_the_first_request_are_left(fp8, first):
    inp = wl.make_decode_inputs(wl.DecodeSpec("r", seed=210, B=2, seq_lens=(37, 21), H=1, block_size=8,
                                              kv_dtype="fp8_e4m3" if fp8 else "bf16"))
    t = G.to_device(inp)
    cu = np.array([first, first + 37, first + 58], np.int32)
    out = torch.full((first + 58 + 9, 576), 7.0, device="cuda")
    dcp.dcp_latent_cache_read(t["kv_cache"], t["block_table"], torch.from_numpy(cu).cuda(), out,
                              kv_scale=t.get("kv_scale"))
    want = oracle.cache_read(oracle.kv_rows_f64(inp), inp["block_table"], 8, (0, 0), cu)
    got = out.double().cpu().numpy()
    assert (got[:first] == 7).all() and (got[first + 58:] == 7).all()
    assert np.array_equal(got[first:first + 58], want[first:])
