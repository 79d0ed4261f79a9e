"""Pins of the oracle's 4-bit format (CPU only): values, rounding, layout."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention, e2m1, e4m3


def test_all_codes_against_the_table_of_the_format():
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    got = e2m1.lut()
    assert got[:8].tolist() == want and got[8:].tolist() == [-v for v in want]
    assert np.signbit(got[8]) and not np.signbit(got[0])


def test_nearest_even_by_brute_force():
    grid = e2m1.lut()[:8]
    for n in range(0, 8 * 64):
        a = Fraction(n, 64)
        best = min(range(8), key=lambda i: (abs(a - Fraction(grid[i])), i % 2))
        assert int(e2m1.nearest_even(float(a), grid)) == best, a
    assert int(e2m1.nearest_even(np.inf, grid)) == 7


def test_group_scale_and_codes_of_a_hand_made_group():
    x = np.zeros(128)
    x[:4] = [6.0, -3.0, 2.5, 0.25]     # group 0: s = 1; 2.5 ties to 2, 0.25 to 0
    x[16:18] = [1.0, -1.0 / 12]        # group 1: s = E4M3(1/6) = 0.171875; 1/s = 5.82 -> 6
    codes, scales = e2m1.encode(x, 1.0)
    assert scales[0] == 0x38 and e4m3.lut()[scales[1]] == 0.171875 and not scales[2:].any()
    assert codes[0] == 7 | (13 << 4) and codes[1] == 4 | (0 << 4)
    assert codes[8] == 7 | (9 << 4)    # (1/12) / 0.171875 = 0.485 -> 0.5
    back = e2m1.decode_slices(e2m1.pack(np.tile(codes, (16, 1)), np.tile(scales, (16, 1))))
    assert back.shape == (16, 128)
    assert back[3, 0] == 6 and back[3, 1] == -3 and back[3, 2] == 2 and back[3, 16] == 6 * 0.171875


def test_special_values():
    x = np.ones((4, 128))
    x[0, 3] = np.nan
    x[1, 20] = np.inf
    x[2] = 0.0
    x[3, :16] = 1e-9                   # the group's scale underflows to 0
    codes, scales = e2m1.encode(x, 1.0)
    assert scales[0, 0] == 0x7F and scales[0, 1] == scales[3, 1]
    assert scales[1, 1] == 0x7E and (codes[1, 10] & 15) == 7
    assert not codes[2].any() and not scales[2].any() and not scales[3, 0] and not codes[3, :8].any()


def test_error_of_a_round_trip_is_bounded():
    # |x| <= 6.25 s t after the scale's own rounding (E4M3: half a step is 2^-4), so the
    # error is half the widest step, 1 s, or the part cut off at 6: at most 1.0 s
    rng = np.random.default_rng(1)
    x = rng.standard_normal((64, 128)) * np.exp(rng.uniform(-2, 2, (64, 1)))
    codes, scales = e2m1.encode(x, 0.5)
    y = 0.5 * e2m1.decode_slices(e2m1.pack(codes.reshape(4, 16, 64), scales.reshape(4, 16, 8))).reshape(64, 128)
    s = 0.5 * np.repeat(e4m3.lut()[scales], 16, axis=1)
    assert np.all(np.abs(x - y) <= 1.0 * s + 1e-12)


@pytest.mark.parametrize("n_t", [1, 3])
def test_attention_equals_the_fp8_oracle_on_values_both_formats_hold(n_t):
    # codes 0, 1, 2, 3 of group scale 1 are E4M3 values: the same cache in both formats
    rng = np.random.default_rng(2)
    nb, hkv, ctx = 6, 2, [37, 5, 0]
    nib = rng.integers(0, 4, (nb, hkv, 16, 128)) + 8 * rng.integers(0, 2, (nb, hkv, 16, 128))
    packed = e2m1.pack((nib[..., 0::2] + 16 * nib[..., 1::2]).astype(np.uint8),
                       np.full((nb, hkv, 16, 8), 0x38, np.uint8))
    table = {v: i for i, v in enumerate(e4m3.lut()[:127])}
    fp8 = np.vectorize(lambda c: table[abs(e2m1.lut()[c])] + (128 if c & 8 else 0))(nib).astype(np.uint8)
    bt = np.array([[4, 1, 2], [5, -1, -1], [-1, -1, -1]], np.int32)
    q = rng.standard_normal((3, n_t, 8, 128)).astype(np.float16)
    fn = attention.paged_decode_attention_multi
    want = fn(q, fp8, fp8, bt, np.array(ctx, np.int32), 0.5, 0.25, None, kv_dtype="e4m3")
    got = e2m1.paged_decode_attention(q, packed, packed, bt, ctx, 0.5, 0.25)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)
