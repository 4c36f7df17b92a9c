"""The barrier protocol of the windowed and tree decodes' persistent kernel, run
under random interleavings on the CPU (`tests/select_protocol_model.py`), in
both cache forms and over lists of short and long units; and each planted
mistake is caught."""
import random

import pytest

from tests import select_protocol_model as M

FORMS = [True, False]
FORM_IDS = ["bf16", "fp8"]


def _sizes(rng):
    return [rng.choice((1, 1, 1, 2, 2, 3, 4, 5, 7, 12)) for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("decoupled", FORMS, ids=FORM_IDS)
@pytest.mark.parametrize("first", range(0, 240, 40))
def test_protocol_holds_under_random_completion_order(first, decoupled):
    for seed in range(first, first + 40):
        M.run(_sizes(random.Random(seed)), seed, decoupled=decoupled)


@pytest.mark.parametrize("decoupled", FORMS, ids=FORM_IDS)
@pytest.mark.parametrize("sizes", [[1] * 20, [2] * 12, [40], [1, 30, 1, 1, 17], [53, 2]], ids=str)
def test_protocol_holds_on_uniform_and_lopsided_lists(sizes, decoupled):
    for seed in range(12):
        M.run(sizes, seed, decoupled=decoupled)


@pytest.mark.parametrize("mutation,decoupled", [(m, f) for m, form in M.MUTATIONS.items() for f in FORMS
                                                if form is None or form == f])
def test_planted_protocol_mistake_is_caught(mutation, decoupled):
    for seed in range(1500):
        rng = random.Random(seed)
        sizes = [1] * rng.randint(6, 16) if seed % 3 == 0 else _sizes(rng) + [1] * (seed % 2)
        try:
            M.run(sizes, seed, mutation, decoupled=decoupled)
        except M.ProtocolError:
            return
    pytest.fail("no interleaving exposed the planted mistake %r" % mutation)
