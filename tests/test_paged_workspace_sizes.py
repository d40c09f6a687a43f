"""A paged-attention workspace made for the largest batch does for every smaller
one: a server keeps one while sequences come and go."""

import random

from test_serve_refusals import cp  # noqa: F401


def test_sizes_grow_with_the_batch(cp):  # noqa: F811
    size = cp._lib.cpattn_paged_attn_workspace_size
    rng = random.Random(1)
    for _ in range(4000):
        Hk = rng.choice([1, 2, 4, 8, 16, 200])
        H, D = Hk * rng.choice([1, 2, 3, 5, 8, 16, 17, 32, 33, 71, 128]), rng.choice([64, 128])
        B = rng.choice([1, 2, 31, 32, 33, 64, 100, 1500])
        most = rng.choice([0, 1, 2, 3, 4, 8, 16, 33, 129, 1000])
        T = rng.choice([0, B, B * most, rng.randint(0, B * most + 1)])
        whole = size(T, B, H, Hk, D, most)
        less = (rng.randint(0, T), rng.choice([rng.randint(0, B), min(B, 32)]),
                rng.choice([0, most // 2, min(most, 1), rng.randint(0, most)]))
        if rng.random() < 0.5:
            less = (rng.choice([T, less[0]]), less[1], rng.choice([most, less[2]]))
        assert size(less[0], less[1], H, Hk, D, less[2]) <= whole, (T, B, H, Hk, D, most, less)
