"""The three e5m2 terms of a softmax weight (split_e5m2x4 of csrc/kv8_decode.cuh) in numpy, over
the whole range: what decode's bounds count for them."""
import numpy as np


def upper_byte(x):
    """The e5m2 value in the upper byte of an f16."""
    return (x.view(np.uint16) & np.uint16(0xff00)).view(np.float16)


def three_terms(w):
    x = w.astype(np.float32).astype(np.float16)
    hi = upper_byte(x)
    rest = ((x - hi) * np.float16(8)).astype(np.float16)
    mid = upper_byte(rest)
    rest = ((rest - mid) * np.float16(8)).astype(np.float16)
    lo = upper_byte((rest.view(np.uint16) + np.uint16(0x80)).view(np.float16))
    return [t.astype(np.float64) for t in (hi, mid, lo)]


def test_a_weight_is_off_by_half_a_step_of_nine_bits_or_the_floor():
    rng = np.random.default_rng(0)
    every_f16 = np.arange(0x7401, dtype=np.uint16).view(np.float16).astype(np.float64)  # to 2^14
    w = np.concatenate([every_f16, (every_f16[1:] + every_f16[:-1]) / 2,
                        np.exp2(rng.uniform(-40, 14, 200000)), [0.0, 2.0 ** 14 * (1 + 2.0 ** -20)]])
    hi, mid, lo = three_terms(w)
    for t in (hi, mid, lo):  # none leaves e5m2, the largest is 57344
        assert np.all(np.isfinite(t)) and t.min() >= 0 and t.max() <= 57344
    err = np.abs(hi + mid / 8 + lo / 64 - w)
    assert np.all(err <= np.maximum(1.25 * 2.0 ** -9 * w, 1.25 * 2.0 ** -23))
