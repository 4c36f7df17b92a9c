"""Host-side checks of the windowed and tree decodes' calls: the stated
workspace covers every range of shards, the largest launches are refused by
the size query and the call alike, and the allocating forms' defaults."""
import numpy as np
import pytest
import torch

import mla_decode_context_gb300 as dcp
from tests.test_select_cpu import L, _call  # noqa: F401


def test_workspace_query_covers_every_range_of_shards(L):  # noqa: F811
    """As the check over every interleave, for fewer computed shards than D."""
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not memory")
    rng = np.random.default_rng(1)
    for _ in range(3000):
        B, H, D = int(rng.integers(1, 65)), int(rng.choice([1, 5, 16, 40, 64, 128])), int(rng.choice([2, 5, 8, 32]))
        q, dn = int(rng.choice([1, 2, 4, 17, 64])), int(rng.integers(1, D + 1))
        msl, win, sinks = int(np.exp(rng.uniform(0, 12))), int(rng.choice([0, 1, 100, 5000])), int(rng.choice([0, 4, 900]))
        n = dcp.dcp_decode_select_workspace_size(B, B * q, H, D, msl, q, win, sinks)
        st = _call(L, "tree", B=B, T=B * q, H=H, D=D, dn=dn, I=int(rng.choice([1, 3, 64, 10000])), mql=q, msl=msl,
                   win=win, sinks=sinks, bs=64, w=4096, ws=4096, qs=H * 576, wk=0x9000 if n else None, wb=n, ms=4)
        assert st == 6, (B, H, D, dn, q, msl, win, sinks)


def test_too_many_units_are_refused_by_the_query_and_the_call(L):  # noqa: F811
    with pytest.raises(dcp.DCPError) as e:
        dcp.dcp_decode_select_workspace_size(64, 64, 128, 8, 1000, 1 << 22)
    assert e.value.status == 1
    assert _call(L, "window", B=64, T=64, H=128, D=8, dn=8, mql=1 << 22, qs=128 * 576, wk=0x9000, wb=1 << 40) == 1


def test_default_row_bound_of_a_tree(monkeypatch):
    """T rows at most, what a mask row can name, and what a call takes."""
    seen = []
    monkeypatch.setattr(dcp, "_decode_select", lambda *a: seen.append(a[15]))  # max_q_len
    for T, words, want in ((1, 1, 1), (7, 1, 7), (100, 1, 64), (100, 2, 100), (400, 4, 256), (400, 9, 256)):
        q = torch.zeros((T, 1, 576), dtype=torch.bfloat16)
        cache = torch.zeros((1, 16, 576), dtype=torch.bfloat16)
        dcp.decode_partial_tree(q, cache, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                torch.zeros(2, dtype=torch.int32), torch.zeros((T, words), dtype=torch.int64), D=1,
                                interleave=1, scale=1.0)
        assert seen[-1] == want
