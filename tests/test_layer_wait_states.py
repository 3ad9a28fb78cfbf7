"""Wait states behind the matrix operations of the integer products and of
attention over a shared prefix, counted in the compiled code as for the other
sources: v_mfma_i32_16x16x64_i8 has four passes, as the 16 x 16 bf16 operation,
and its result may be used by another kind of instruction eight wait states
later; v_mfma_f32_32x32x16_bf16 has eight, and needs twelve."""
import concurrent.futures as cf

import pytest

from tests import test_wait_states as base

NEEDED = {"int8.hip": ("v_mfma_i32_16x16x64_i8", 8), "prefix.hip": ("v_mfma_f32_32x32x16_bf16", 12)}


@pytest.fixture(scope="module")
def compiled():
    with cf.ThreadPoolExecutor(len(NEEDED)) as ex:
        return dict(zip(NEEDED, ex.map(base.compile_source, NEEDED)))


@pytest.mark.parametrize("src", list(NEEDED))
def test_results_are_not_used_early(compiled, src, monkeypatch):
    op, needed = NEEDED[src]
    monkeypatch.setattr(base, "FAR", needed + 4)
    code, labels = base.parse(compiled[src])
    products = [i for i, t in enumerate(code) if t.startswith(op)]
    assert len(products) > 100
    early = [(code[i], n) for i, n in ((i, base.nearest_use(code, labels, i)) for i in products) if n < needed]
    assert not early, "%d of %d results are used too early: %s" % (len(early), len(products), early[:3])
