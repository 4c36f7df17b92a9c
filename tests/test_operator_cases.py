"""Small cases of `perf/operators.py`: its plain forms (on the CPU) and the
library's calls (on a GPU) against its exact results.

Tolerances: written caches and queries are exact.  A row read back is code x
scale rounded once (2^-8 of the value in bf16; exact in fp32 with power-of-two
scales).  Attention outputs are bf16, half a step of the value (2^-8), and the
plain form's sums fp32: 1e-4 for a few hundred terms.  The library's softmax
weights are bf16 besides: 2^-8 of the largest value, and 1e-3."""
import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


def _module(device, own):
    spec = importlib.util.spec_from_file_location("operator_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEVICE, m.own = device, own
    return m


CASES = {
    "write_q": lambda m: m._write("", 5, 3, 7),
    "write_alone": lambda m: m._write("", 37, 0, 20),
    "read_bf16_f32": lambda m: m._read("", 3, 5, 60, False, "float32", 16),
    "read_fp8_bf16": lambda m: m._read("", 2, 40, 90, True, "bfloat16", 64),
    "read_fp8_f32": lambda m: m._read("", 5, 1, 9, True, "float32", 1),
    "read_bf16_bf16": lambda m: m._read("", 1, 30, 30, False, "bfloat16", 16),
    "window": lambda m: m._attend("", "window", 2, 30, 90, 3, True, 16, 2, 1, 25, 2, False, 16),
    "window_fp8": lambda m: m._attend("", "window", 1, 77, 77, 1, False, 128, 3, 4, 50, 0, True, 16),
    "window_past_context": lambda m: m._attend("", "window", 2, 10, 33, 2, False, 8, 1, 1, 300, 5, False, 16),
    "tree": lambda m: m._attend("", "tree", 2, 40, 80, 9, True, 16, 2, 1, 0, 0, False, 16),
    "tree_window_fp8": lambda m: m._attend("", "tree", 1, 70, 70, 12, False, 33, 1, 1, 20, 3, True, 16),
    "tree_longer_than_context": lambda m: m._attend("", "tree", 2, 1, 70, 66, True, 4, 2, 64, 0, 0, False, 64),
}


def _compare(m, case, got, want, own):
    got, want = (list(x) if isinstance(x, (tuple, list)) else [x] for x in (got, want))
    assert len(got) == len(want)
    want = [torch.as_tensor(w).double().cpu() for w in want]
    types = [g.dtype for g in got]
    got = [g.double().cpu() for g in got]
    for g, w in zip(got, want):
        assert tuple(g.shape) == tuple(w.shape)
    if case["op"] == "write":
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    elif case["op"] == "read":
        assert ((got[0] - want[0]).abs() <= (2.0 ** -8 if types[0] == torch.bfloat16 else 0.0) * want[0].abs()).all()
    else:
        live = want[1] != -torch.inf
        assert torch.equal(got[1] != -torch.inf, live) and (got[0][~live] == 0).all()
        assert (got[1] - want[1])[live].abs().max() <= 1e-3
        tol = 1e-4 + 2.0 ** -8 * want[0].abs()
        if own:
            tol = tol + 1e-3 + 2.0 ** -8 * m._values64(m.prepare(case, 3))[:, :512].abs().max().cpu()
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
