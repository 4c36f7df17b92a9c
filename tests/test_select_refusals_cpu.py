"""What the windowed and tree decodes refuse before any launch, beyond the checks
of each argument by itself."""
from tests.test_select_cpu import L, _call  # noqa: F401


def test_mask_rows_must_hold_every_row_of_a_request(L):  # noqa: F811
    """Also with one query row: a request's bounds (device data) may name more
    rows than the call has, and the mask words read go by them."""
    for T in (1, 2):
        assert _call(L, "tree", B=1, T=T, mql=65, ms=1) == 1
        assert _call(L, "tree", B=1, T=T, mql=256, ms=3) == 1
        assert _call(L, "tree", B=1, T=T, mql=1, ms=0) == 1
        assert _call(L, "tree", B=1, T=T, mql=1, ms=-1) == 1
