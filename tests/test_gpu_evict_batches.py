"""Evictions of batches that one CTA per sequence takes, with heads in several
turns and pages for each of its sizes; and of few sequences, which take a CTA
per row."""
import random

import pytest

from tests import test_gpu_paged8 as paged8

pytestmark = pytest.mark.gpu

BATCHES = [  # sequences, Hkv, page, max_pages, keep, keep_first, keep_last
    (21, 8, 16, 40, 12, 1, 2),
    (24, 24, 32, 250, 100, 2, 3),
    (22, 48, 16, 300, 140, 0, 1),      # more heads than three turns take
    (70, 11, 16, 1000, 400, 3, 1),
    (160, 1, 64, 513, 60, 0, 1),
    (20, 8, 16, 40, 12, 1, 2),         # a CTA per row from here on
    (9, 33, 16, 1024, 500, 1, 1),
    (1, 5, 16, 512, 200, 0, 1),
]


@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"{c[0]}x{c[1]}x{c[3]}-keep{c[4]}")
@pytest.mark.parametrize("kind", ["spread", "ties", "wild"])
def test_evict_of_batches(case, kind):
    B, Hkv, page, P, keep, first, last = case
    rng = random.Random(B)
    lens = [rng.choice((0, 1, keep * page, keep * page + 1, P * page, rng.randrange(P * page))) for _ in range(B)]
    paged8.test_evict((Hkv, page, P, lens, keep, first, last), kind)
