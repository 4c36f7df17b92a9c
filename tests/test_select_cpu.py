"""Windowed and tree decodes without a GPU: the oracle's visible positions
against brute force and special cases, the mask packing, the workspace query,
and what the entry points refuse before any launch."""
import ctypes

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


def test_visible_positions():
    v = oracle.visible_positions
    assert list(v(10, 1, 0, 3, 2)) == [0, 1, 7, 8, 9]
    assert list(v(10, 4, 0, 3, 0)) == [4, 5, 6]           # L = 7
    assert list(v(3, 1, 0, 5, 2)) == [0, 1, 2]
    assert list(v(2, 4, 0)) == [] and list(v(2, 4, 3)) == [0, 1]
    bits = np.array([1, 0, 1, 1], bool)
    assert list(v(8, 4, 3, tree_bits=bits)) == [0, 1, 2, 3, 4, 6, 7]
    assert list(v(8, 4, 3, 2, 1, tree_bits=bits)) == [0, 6, 7]
    assert list(v(8, 4, 3, 4, 0, tree_bits=bits)) == [3, 4, 6, 7]  # ranks, not positions
    assert list(v(2, 4, 3, tree_bits=bits)) == [0, 1]              # rows 0, 1 lie before the context


def test_select_oracle_reduces_to_the_decode_oracle():
    inp = wl.make_decode_inputs(wl.DecodeSpec("r", seed=3, B=2, seq_lens=(40, 9), q_len=3, H=2, block_size=8, D=3,
                                              interleave=2))
    O, lse, _ = oracle.decode_partial(inp)
    vis = np.tile(np.tril(np.ones((3, 3), bool)), (2, 1))
    for kw in (dict(), dict(window=100), dict(tree=vis), dict(tree=vis, window=64, sinks=3)):
        O2, lse2 = oracle.decode_partial_select(inp, **kw)
        assert np.array_equal(lse, lse2) and np.array_equal(np.nan_to_num(O), np.nan_to_num(O2))


def test_select_oracle_by_masked_softmax():
    """Against a dense torch softmax with the mask written out as a matrix."""
    inp = wl.make_decode_inputs(wl.DecodeSpec("m", seed=4, B=1, seq_lens=(30,), q_len=5, H=3, block_size=8, D=1))
    rng = np.random.default_rng(4)
    vis = rng.random((5, 5)) < 0.5
    kv = torch.from_numpy(oracle.gather_latents(inp["kv_cache"], inp["block_table"][0], 8, np.arange(30)))
    q = torch.from_numpy(oracle.bf16_to_f64(inp["q"]))
    see = torch.zeros((5, 30), dtype=torch.bool)
    for r in range(5):
        seq = list(range(25)) + [25 + k for k in range(5) if vis[r, k]]
        for rank, p in enumerate(seq):
            see[r, p] = rank < 2 or rank >= len(seq) - 7
    s = torch.einsum("thk,pk->thp", q, kv) * inp["scale"]
    s = s.masked_fill(~see[:, None, :], -float("inf"))
    O, lse = oracle.decode_partial_select(inp, 7, 2, vis)
    assert np.allclose(lse[0], torch.logsumexp(s, -1).numpy(), atol=1e-12)
    assert np.allclose(O[0], (torch.softmax(s, -1) @ kv[:, :512]).numpy(), atol=1e-12)


def test_pack_tree_mask():
    rng = np.random.default_rng(0)
    for n in (1, 63, 64, 65, 200):
        v = rng.random((7, n)) < 0.5
        m = dcp.pack_tree_mask(torch.from_numpy(v)).numpy().view(np.uint64)
        assert m.shape == (7, (n + 63) // 64)
        assert all(bool((int(m[r, k // 64]) >> (k % 64)) & 1) == v[r, k] for r in range(7) for k in range(n))
    assert dcp.pack_tree_mask(torch.zeros((3, 0), dtype=torch.bool)).shape == (3, 1)
    with pytest.raises(TypeError):
        dcp.pack_tree_mask(torch.zeros((3, 4)))


def _call(L, entry="window", **kw):
    a = dict(q=0x1000, qs=128 * 576, kv=0x2000, dt=0, sc=None, nb=4, bs=16, tab=0x3000, w=4, ws=4, loc=0, ss=0, d0=0,
             dn=4, seq=0x4000, qsl=0x5000, B=2, T=2, H=128, msl=37, mql=1, D=4, I=1, scale=0.07, mask=0x8000, ms=1,
             win=8, sinks=1, O=0x6000, odt=1, lse=0x7000, wk=None, wb=0, err=None)
    a.update(kw)
    args = [a[k] for k in ("q", "qs", "kv", "dt", "sc", "nb", "bs", "tab", "w", "ws", "loc", "ss", "d0", "dn", "seq",
                           "qsl", "B", "T", "H", "msl", "mql", "D", "I", "scale")]
    args += [a["mask"], a["ms"]] if entry == "tree" else []
    args += [a[k] for k in ("win", "sinks", "O", "odt", "lse", "wk", "wb", "err")]
    return getattr(L, "dcp_mla_decode_partial_" + entry)(*args, None)


@pytest.mark.parametrize("entry", ["window", "tree"])
def test_refusals_before_launch(L, entry):
    def c(**kw):
        return _call(L, entry, **kw)
    assert c(B=0) == 0 and c(T=0) == 0
    assert c(win=-1) == 1 and c(sinks=-1) == 1
    assert c(q=None) == 1 and c(D=0) == 1 and c(D=33) == 1 and c(I=0) == 1 and c(H=0) == 1 and c(H=1025) == 1
    assert c(mql=0) == 1 and c(scale=float("inf")) == 1
    assert c(d0=1) == 1 and c(dn=0) == 1
    assert c(dt=3) == 2 and c(odt=3) == 2 and c(dt=1) == 1
    assert c(q=0x1008) == 3 and c(O=0x6004) == 3 and c(kv=0x2004) == 3
    assert c(msl=65) == 4                                    # needs 5 columns of 16 > 4
    # one long request: split partials need a workspace
    big = dict(B=1, T=1, msl=120000, bs=64, w=1875, ws=1875, D=8, dn=8, win=0)
    assert c(**big) == 5 and c(**big, wk=0x9000, wb=100) == 5
    assert c(**big, wk=0x9008, wb=1 << 30) == 3


def test_tree_refusals_before_launch(L):
    assert _call(L, "tree", mask=None) == 1
    assert _call(L, "tree", mask=0x8004) == 3
    assert _call(L, "tree", mql=65, ms=1) == 1               # two words a row
    assert _call(L, "tree", mql=257, ms=9) == 1              # at most 256 rows


def test_workspace_query(L):
    f = dcp.dcp_decode_select_workspace_size
    assert f(0, 0, 128, 8, 1000, 1) == 0
    assert f(1, 1, 128, 1, 120000, 1) > f(1, 1, 128, 1, 120000, 1, 1024, 4) > 0   # a window bounds what is split
    # rows that share a unit leave more of the GPU to splits
    assert f(1, 8, 16, 1, 120000, 8) / 16 > f(1, 8, 128, 1, 120000, 8) / 128
    for bad in ((-1, 1, 128, 8, 10, 1), (1, 1, 0, 8, 10, 1), (1, 1, 128, 33, 10, 1), (1, 1, 128, 8, 10, 0),
                (1, 1, 128, 8, 10, 1, -1, 0), (1, 1, 128, 8, 10, 1, 1, -1)):
        with pytest.raises(dcp.DCPError):
            f(*bad)


def test_workspace_query_covers_every_interleave(L):
    """A workspace of the queried size is never refused (status 5), whatever
    the interleave, shard range and window; without a device a call that gets
    past its checks ends in a CUDA error."""
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not memory")
    rng = np.random.default_rng(0)
    for _ in range(3000):
        B, H, D = int(rng.integers(1, 65)), int(rng.choice([1, 5, 16, 40, 64, 128])), int(rng.choice([1, 2, 5, 8, 32]))
        q = int(rng.choice([1, 2, 4, 17, 64]))
        msl, win, sinks = int(np.exp(rng.uniform(0, 12))), int(rng.choice([0, 1, 100, 5000])), int(rng.choice([0, 4, 900]))
        n = dcp.dcp_decode_select_workspace_size(B, B * q, H, D, msl, q, win, sinks)
        st = _call(L, "tree", B=B, T=B * q, H=H, D=D, dn=D, I=int(rng.choice([1, 3, 64, 10000])), mql=q, msl=msl, win=win,
                   sinks=sinks, bs=64, w=4096, ws=4096, qs=H * 576, wk=0x9000 if n else None, wb=n, ms=4)
        assert st == 6, (B, H, D, q, msl, win, sinks)


def _args(**kw):
    a = dict(q=torch.zeros((2, 16, 576), dtype=torch.bfloat16), kv=torch.zeros((4, 16, 576), dtype=torch.bfloat16),
             tab=torch.zeros((2, 4), dtype=torch.int32), seq=torch.zeros(2, dtype=torch.int32),
             qsl=torch.zeros(3, dtype=torch.int32), O=torch.zeros((4, 2, 16, 512)), lse=torch.zeros((4, 2, 16)),
             mask=torch.zeros((2, 1), dtype=torch.int64), sc=None, mql=1)
    a.update(kw)
    return a


@pytest.mark.parametrize("tree", [False, True])
def test_wrappers_check_shapes_before_the_device(tree):
    def call(**kw):
        a = _args(**kw)
        f = dcp.dcp_mla_decode_partial_tree if tree else dcp.dcp_mla_decode_partial_window
        f(a["q"], a["kv"], a["tab"], a["seq"], a["qsl"], *([a["mask"]] if tree else []), a["O"], a["lse"], D=4,
          interleave=1, scale=0.1, window=5, num_sinks=1, max_seq_len=37, max_q_len=a["mql"], kv_scale=a["sc"])
    for bad, msg in ((dict(tab=torch.zeros((1, 4), dtype=torch.int32)), "disagree on B"),
                     (dict(kv=torch.zeros((64, 576), dtype=torch.bfloat16)), "kv_cache"),
                     (dict(O=torch.zeros((4, 2, 16, 256))), "O_part")):
        with pytest.raises(ValueError, match=msg):
            call(**bad)
    if tree:
        with pytest.raises(TypeError, match="tree_mask"):
            call(mask=torch.zeros((2, 1), dtype=torch.int32))
        with pytest.raises(ValueError, match="tree_mask"):
            call(mql=65)
        with pytest.raises(ValueError, match="tree_mask"):
            call(mask=torch.zeros((1, 1), dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        call()


def test_entry_points_take_uint64_masks():
    names = dict((n, a) for n, _, a in dcp.EXPORTS)
    assert len(names["dcp_mla_decode_partial_tree"]) == len(names["dcp_mla_decode_partial_window"]) + 2
    assert names["dcp_mla_decode_partial_tree"][24:26] == [ctypes.c_void_p, ctypes.c_int64]
