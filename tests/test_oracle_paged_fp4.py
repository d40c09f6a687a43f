"""Pins of the 4-bit cache's oracle (oracle/paged_fp4.py), CPU only."""

import numpy as np
import torch

from oracle import paged_fp4 as o4


def test_the_8_bit_floats_are_the_types():
    byte = torch.arange(256, dtype=torch.uint8)
    want = byte.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o4.E4M3, want, equal_nan=True)


def test_rounding_to_8_bits_is_the_types():
    rng = np.random.default_rng(0)
    x = np.abs(rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000))
    x = np.concatenate([x, (o4.E4M3[:126] + o4.E4M3[1:127]) / 2])     # halves
    x = np.clip(x, 2.0 ** -9, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o4.nearest(x, o4.E4M3[:127]), want)


def test_halves_go_to_the_even_code():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert o4.nearest(x, o4.GRID).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert o4.nearest(x + 1e-9, o4.GRID).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert o4.nearest(x - 1e-9, o4.GRID).tolist() == [0, 1, 2, 3, 4, 5, 6]


def test_by_hand():
    """Sixteen features with largest 6: scale 1; with largest 12 and unit 4: 3 / 6."""
    x = np.array([6, -6, 5, -5.1, 3.5, 3.4, -2.5, 2.6, 1.75, 1.2, -0.75, 0.7, 0.25, -0.26, 0, 1.0])
    code, scale = o4.quantise(x)
    assert scale.tolist() == [0x38]
    assert code.tolist() == [7, 15, 6, 15, 6, 5, 12, 5, 4, 2, 10, 1, 0, 9, 0, 2]
    code2, scale2 = o4.quantise(2 * x, 4.0)
    assert scale2.tolist() == [0x30] and np.array_equal(code2, code)
    assert np.array_equal(o4.values(code2, scale2, 4.0), 2 * o4.values(code, scale))
    assert o4.quantise(np.zeros(16))[1].tolist() == [1]          # the smallest, 2^-9
    assert o4.quantise(np.full(16, 1e6))[1].tolist() == [0x7E]   # 448
    assert o4.quantise(np.array([np.nan] + [1.0] * 15))[1].tolist() == [0x7F]


def test_values_quantise_to_themselves():
    """A group that holds a 6 comes back bit for bit."""
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (50, 128)).astype(np.uint8)
    code[code == 8] = 0
    code[:, ::16] = 7
    scale = rng.integers(1, 127, (50, 8)).astype(np.uint8)
    again, s = o4.quantise(o4.values(code, scale, 0.25), 0.25)
    assert np.array_equal(again, code) and np.array_equal(s, scale)


def test_every_byte_of_a_page_has_one_use():
    for D in (64, 128):
        for size in (16, 32):
            seen = np.zeros(size * 9 * D // 16, dtype=int)
            for r in range(size):
                for f in range(D):
                    at, high = o4.code_place(r, f, D)
                    seen[at] += 1 + 16 * high
                for j in range(D // 16):
                    seen[o4.scale_place(r, j, D)] += 18
            assert (seen == np.where(seen == 18, 18, 17 + 1)).all() and (seen > 0).all()


def test_write_then_unpack():
    rng = np.random.default_rng(2)
    for D in (64, 128):
        cache = rng.integers(0, 256, (3, 2, 32, 9 * D // 16)).astype(np.uint8)
        before = o4.unpack(cache, D)
        code, scale = o4.quantise(rng.normal(size=D))
        o4.write(cache, 1, 1, 19, code, scale)
        after = o4.unpack(cache, D)
        assert np.array_equal(after[1, 19, 1], o4.values(code, scale))
        after[1, 19, 1] = before[1, 19, 1]
        assert np.array_equal(after, before, equal_nan=True)


def test_what_is_lost():
    """Normally distributed features keep all but 9.5 % (RMS)."""
    x = np.random.default_rng(3).normal(size=(2000, 128))
    e = o4.values(*o4.quantise(x)) - x
    assert 0.093 < np.sqrt((e ** 2).mean() / (x ** 2).mean()) < 0.097
