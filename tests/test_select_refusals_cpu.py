"""What the windowed and tree decodes refuse before any launch, beyond the checks
of each argument by itself."""
import pytest

import mla_decode_context_gb300 as dcp
from tests.test_select_cpu import L, _call  # noqa: F401


def test_mask_rows_must_hold_every_row_of_a_request(L):  # noqa: F811
    """Also with one query row: a request's bounds (device data) may name more
    rows than the call has, and the mask words read go by them."""
    for T in (1, 2):
        assert _call(L, "tree", B=1, T=T, mql=65, ms=1) == 1
        assert _call(L, "tree", B=1, T=T, mql=256, ms=3) == 1
        assert _call(L, "tree", B=1, T=T, mql=1, ms=0) == 1
        assert _call(L, "tree", B=1, T=T, mql=1, ms=-1) == 1


def _args(tree):
    import torch
    q = torch.zeros((2, 16, 576), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    args = [q, torch.zeros((4, 16, 576), dtype=torch.bfloat16), i32(2, 4), i32(2), i32(3)]
    return args + ([torch.zeros((2, 1), dtype=torch.int64)] if tree else [])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("name", ["window", "num_sinks", "max_seq_len", "max_q_len", "interleave", "D", "shard_begin"])
@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 5, -(1 << 32) + 5])
def test_numbers_past_32_bits_are_refused(tree, name, value):
    """The C entries take int32: a larger number would be cut to its low bits
    (2^32 + 5 tokens to a window of 5)."""
    import torch
    f = dcp.dcp_mla_decode_partial_tree if tree else dcp.dcp_mla_decode_partial_window
    kw = dict(D=4, interleave=1, scale=0.1, window=5, num_sinks=1, max_seq_len=37, max_q_len=1, shard_begin=0,
              shard_count=4)
    with pytest.raises(ValueError, match="32 bits"):
        f(*_args(tree), torch.zeros((4, 2, 16, 512)), torch.zeros((4, 2, 16)), **dict(kw, **{name: value}))
    if name in ("window", "num_sinks", "max_seq_len", "max_q_len", "D"):
        sizes = dict(B=1, T=2, H=16, D=4, max_seq_len=37, max_q_len=1, window=5, num_sinks=1)
        with pytest.raises(ValueError, match="32 bits"):
            dcp.dcp_decode_select_workspace_size(**dict(sizes, **{name: value}))


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 2, -(1 << 32) + 2])
def test_a_read_interleave_past_32_bits_is_refused(value):
    import torch
    cache, i32 = torch.zeros((2, 8, 576), dtype=torch.bfloat16), torch.int32
    with pytest.raises(ValueError, match="32 bits"):
        dcp.dcp_latent_cache_read(cache, torch.zeros((1, 4), dtype=i32), torch.zeros(2, dtype=i32),
                                  torch.zeros((5, 576), dtype=torch.bfloat16), D=2, interleave=value)


def test_default_context_bound_fits_32_bits(monkeypatch):
    """A table of more slots than an int32 length can reach bounds nothing."""
    import torch
    seen = []
    monkeypatch.setattr(dcp, "_decode_select", lambda *a: seen.append(a[14]))  # max_seq_len
    monkeypatch.setattr(dcp, "dcp_decode_select_workspace_size", lambda *a: 0)
    args = _args(False)
    args[2] = torch.zeros((1, 1), dtype=torch.int32).expand(2, 1 << 29)
    dcp.decode_partial_window(*args, D=4, interleave=1, scale=0.1, window=5, max_q_len=1)
    dcp.decode_partial_window(*_args(False), D=4, interleave=1, scale=0.1, window=5, max_q_len=1)
    assert seen == [0x7fffffff, 64]
