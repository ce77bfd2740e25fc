"""The rule that chooses a form of the attention, as the header states it, and
the split of a row tile's tokens, both from the kernels' own header."""
import numpy as np
import pytest

from tests import kv4_forms as forms
from tests.test_kv4_forms_gpu import MANY_ONE


def test_the_rule_is_the_one_that_the_header_names():
    g = np.random.default_rng(1)
    seen = set()
    for _ in range(4000):
        Hk, G, B, mq = (int(np.exp(g.uniform(0, t))) for t in (2.5, 3.5, 6, 6))
        D, P = int(g.choice([64, 128, 256])), int(g.choice([32, 64, 256]))
        width = int(np.exp(g.uniform(0, 8)))
        rows = B * mq * Hk * G
        few = mq * G <= 64 or rows <= 4096 or rows * (width * P // 32) <= 2 ** 20
        for window in (0, 500):
            p = forms.plan(Hk * G, Hk, D, P, width, B, mq, window)
            assert p.few == few and p.rows == (16 if few else 64) * p.mt and p.tiles * p.rows >= mq * G
            seen.add((p.few, p.mt, p.list, p.budget > 0))
    # every kind there is: budget or none, a list or sums, one or two tiles of 16 rows a wave
    assert seen == {(True, m, l, b) for m in (1, 2) for l, b in ((False, False), (False, True), (True, True))} | {
        (False, m, b, b) for m in (1, 2) for b in (False, True)}


@pytest.mark.parametrize("step", [1, 2])
def test_parts_hold_every_tile_once(step):
    for tiles in list(range(1, 70)) + [157, 4094, 4095, 2 ** 26 - 1]:
        for parts in list(range(1, 40)) + [512]:
            at = 0
            for i in range(parts):
                first, last = forms.part(tiles, parts, i, step)
                assert first == at and first <= last <= tiles and (last == tiles or (last - first) % step == 0)
                at = last
            assert at == tiles


@pytest.mark.parametrize("case", MANY_ONE, ids=[c[0] for c in MANY_ONE])
def test_shapes_of_the_form_for_many_rows(case):
    """The cases beside the kernels' tests reach the kernel that they are about: one tile of 16 rows a wave."""
    name, B, mq, Hk, G, width, window, dealt = case
    for D in (64, 128, 256):
        p = forms.plan(Hk * G, Hk, D, 32, width, B, mq, window)
        assert not p.few and p.mt == 1 and p.list == (p.budget > 0) == dealt
