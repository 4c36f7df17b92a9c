"""The tight reference notices what the wide one lets through: a lost or doubled
tile at a piece's border, a lost token, keys rounded to bf16.  On the CPU: the
mistakes are planted in the reference."""
import pytest
import torch

from tests import chunk_reference as ref
from tests.chunk_tight import tight_check, tight_reference

TILE = 128


def case(L, n):
    return ref.make(seq=[L], q=[n], H=1, bs=64, seed=51, device="cpu")


def dense(parts, T):
    out, lse = torch.zeros((T, 1, 128), dtype=torch.float64), torch.full((T, 1), -torch.inf, dtype=torch.float64)
    for rows, h, o, z, _, _ in parts:
        out[rows, h], lse[rows, h] = o, z
    return out, lse


@pytest.mark.parametrize("L,n,pieces", [(20000, 1, 26), (9000, 3, 11), (1600, 2, 2)])
def test_lost_or_doubled_tiles_at_the_borders_are_noticed(L, n, pieces):
    st = case(L, n)
    want = tight_reference(st)
    tight_check(*dense(want, n), want)
    tiles = -(-L // TILE)
    for i in range(1, pieces):
        j = tiles * i // pieces
        for tile, weight in ((j, 0.0), (j - 1, 0.0), (j, 2.0), (j - 1, 2.0)):
            times = torch.ones(L)
            times[TILE * tile:TILE * (tile + 1)] = weight
            with pytest.raises(AssertionError):
                tight_check(*dense(tight_reference(st, times), n), want)


def test_a_lost_token_is_noticed():
    """One of the tenth that weighs most.  (Scores have a deviation of 0.0722 x 1.5 x
    sqrt(192) = 1.5, so the heaviest tenth has p > exp(1.28 x 1.5 - 1.5^2 / 2) / 9000 =
    2.5e-4, and losing one moves the output by p |v|, 2.5e-4 x 11; the tolerance is
    about 1e-3 of |out| = sqrt(sum p^2) |v| = 0.03 x 11.  The lightest ones move it by
    less than a rounding.)"""
    st = case(9000, 1)
    want = tight_reference(st)
    kv = ref.latents(st, ref.rows_of(st, 0))
    k = torch.cat([kv[:, :512] @ st["w"][:128].double().T, kv[:, 512:]], 1)
    order = (st["q"][0, 0].double() @ k.T).argsort()
    for t in order[[8100, 8500, 8900, 8999]].tolist():
        times = torch.ones(9000)
        times[t] = 0
        with pytest.raises(AssertionError):
            tight_check(*dense(tight_reference(st, times), 1), want)


def test_keys_in_bf16_are_noticed():
    st = case(9000, 4)
    want = tight_reference(st)
    half = torch.Tensor.to

    def coarse(x, dtype, *a, **kw):  # f16 -> bf16
        return half(x, torch.bfloat16 if dtype is torch.float16 else dtype, *a, **kw)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.Tensor, "to", coarse)
        rough = tight_reference(st)
    with pytest.raises(AssertionError):
        tight_check(*dense(rough, 4), want)
