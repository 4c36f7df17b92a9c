"""Small cases of `perf/more_operators.py`: its plain forms (on the CPU) and the
library's calls (on a GPU) against its exact results.

Tolerances.  Tables, positions and slots are whole numbers: equal.  Rows and
queries: one rounding, half a step of the value (bf16 2^-8, E4M3 2^-4 and 2^-10
of a scale for its subnormals), and 1e-5 of the largest for fp32 arithmetic.
Attention outputs are bf16 (2^-8) of fp32 sums: 1e-4 for a few hundred terms.
The library's values and softmax weights are f16 besides: 2^-11 of the largest
value each, and 1e-3 from the scores' own errors; log-sum-exps 1e-4 of
themselves, for contexts this short."""
import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")


def _module(device, own):
    spec = importlib.util.spec_from_file_location("more_operator_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEVICE, m.own = device, own
    return m


CASES = {
    "extend": lambda m: m._extend("", 5, 3, 9, 0, 50, 4, 2, 3, True),
    "extend_one": lambda m: m._extend("", 1, 1, 1, 999, 999, 64, 1, 1, False),
    "extend_shards": lambda m: m._extend("", 6, 1, 20, 0, 50, 16, 8, 1, True),
    "extend_blocks_of_one": lambda m: m._extend("", 4, 2, 2, 5, 5, 1, 2, 1, False),
    "rope_decode": lambda m: m._rope("", 5, 3, "decode", False, True, True, 100),
    "rope_decode_fp8_halves": lambda m: m._rope("", 9, 33, "decode", True, True, False, 100),
    "rope_chunk": lambda m: m._rope("", 5, 17, "pe", True, True, False, 100),
    "rope_alone_no_norm": lambda m: m._rope("", 40, 0, "none", True, False, True, 100),
    "chunk": lambda m: m._chunk("", 1, 9, 9, 0, 0, 2, False, 1, 1, False, 16, 0),
    "chunk_fp8_shards": lambda m: m._chunk("", 3, 1, 9, 0, 40, 2, True, 2, 3, True, 4, 2),
    "chunk_one_table": lambda m: m._chunk("", 2, 5, 9, 3, 40, 2, False, 2, 3, False, 4, 2),
    "chunk_long": lambda m: m._chunk("", 2, 100, 300, 200, 900, 2, False, 1, 1, False, 64, 0),
}


def _compare(m, case, got, want, own):
    assert len(got) == len(want)
    want = [torch.as_tensor(w).double().cpu() for w in want]
    types = [g.dtype for g in got]
    got = [g.double().cpu() for g in got]
    for g, w in zip(got, want):
        assert tuple(g.shape) == tuple(w.shape)
    if case["op"] == "extend":
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    elif case["op"] == "rope":
        if case["fp8"]:
            assert torch.equal(got[-1], want[-1])
            got, want, types = got[:-1], want[:-1], types[:-1]
        for g, w, t in zip(got, want, types):
            step = 2.0 ** -4 if t == torch.float8_e4m3fn else 2.0 ** -8
            tiny = 2.0 ** -10 if t == torch.float8_e4m3fn else 0.0
            assert ((g - w).abs() <= step * w.abs() + tiny + 1e-5 * w.abs().max()).all()
    else:
        live = want[1] != -torch.inf
        assert torch.equal(got[1] != -torch.inf, live) and (got[0][~live] == 0).all()
        assert ((got[1] - want[1]).abs() <= 1e-4 * (1 + want[1].abs()))[live].all()
        tol = 1e-4 + 2.0 ** -8 * want[0].abs()
        if own:
            w = m.prepare(case, 3)["w"].double()
            top = 6.0 * w.norm(dim=1).max().cpu()  # of a value: latents are normal numbers
            tol = tol + 1e-3 + 2 * 2.0 ** -11 * top
        assert ((got[0] - want[0]).abs() <= tol)[live].all()


@pytest.mark.parametrize("name", sorted(CASES))
def test_plain_form_is_the_exact_result(name):
    m = _module("cpu", False)
    case = CASES[name](m)
    _compare(m, case, m.run(m.prepare(case, 3)), m.exact(case, 3), False)


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_library_calls_are_the_exact_result(name):
    m = _module("cuda", True)
    case = CASES[name](m)
    got = m.run(m.prepare(case, 3))
    torch.cuda.synchronize()
    _compare(m, case, got, m.exact(case, 3), True)
