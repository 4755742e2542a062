"""The linear products' rounds, restated on the host: every item of a launch goes to one CTA pair once."""
import random

import pytest

from float_plan import items, plan, two_products, work_item


def played(C, n0, n1, rest, gap):
    seen = {}
    for c in range(C):
        k = 0
        while (w := work_item(k, c, C, n0, n1, rest, gap)) is not None:
            seen[w] = seen.get(w, 0) + 1
            k += 1
    return seen


@pytest.mark.parametrize("sms", [148, 152])
def test_every_item_of_two_products_once(sms):
    rng = random.Random(1)
    shared = gaps = 0
    for _ in range(400):
        B, IC, OC = (rng.choice([64, 256, 300, 1000, 2048, 8192]) + rng.randrange(64) for _ in range(3))
        two = two_products(B, IC, OC, sms)
        if two is None:
            continue
        _, n0, n1, C, rest, gap = two
        seen = played(C, n0, n1, rest, gap)
        assert len(seen) == n0 + n1 and set(seen.values()) == {1}, (B, IC, OC)
        assert set(seen) == {(0, i) for i in range(n0)} | {(1, i) for i in range(n1)}
        shared += 1
        gaps += gap > 1
    assert shared > 100 and gaps > 30


@pytest.mark.parametrize("n0,n1", [(1, 1), (76, 1), (75, 400), (77, 3), (152, 9), (153, 1000), (3, 2), (500, 75)])
@pytest.mark.parametrize("gap", [1, 2, 7])
def test_every_item_once_at_the_edges(n0, n1, gap):
    C = min(76, n0 + n1)
    rest = n0 % C
    seen = played(C, n0, n1, rest, gap if rest else 0)
    assert len(seen) == n0 + n1 and set(seen.values()) == {1}


def test_slices_cover_k_with_none_empty():
    rng = random.Random(2)
    for _ in range(500):
        M, N, K = (rng.randrange(1, 9000) for _ in range(3))
        p = plan(M, N, K, rng.random() < 0.5, 152)
        blocks = -(-K // 64)
        assert items(M, N, p) > 0 and p[2] * p[3] >= blocks > (p[2] - 1) * p[3]
