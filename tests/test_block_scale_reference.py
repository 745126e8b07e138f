"""The 64-bit reference of the block-scaled caches against PyTorch's E4M3 cast and closed forms (no GPU)."""

import numpy as np
import torch

import block_scale_reference as R


def test_codes_match_the_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(R.CODES))
    assert np.array_equal(t[~np.isnan(t)], R.CODES[~np.isnan(t)])


def test_encode_matches_the_cast_inside_the_range():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * np.exp2(rng.integers(-14, 8, 20000))).astype(np.float32)
    mids = (R.CODES[:126] + R.CODES[1:127]) / 2  # every tie
    x = np.concatenate([np.clip(x, -448, 448), mids, -mids, R.CODES[:127], [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x), want)


def test_encode_saturates_and_keeps_nan():
    assert list(R.encode(np.array([449.0, 1e9, np.inf, -np.inf]))) == [0x7E, 0x7E, 0x7E, 0xFE]
    assert R.encode(np.array([np.nan]))[0] == 0x7F


def test_needed_exponent_is_the_smallest():
    rng = np.random.default_rng(1)
    values = np.concatenate([np.exp2(rng.uniform(-70, 120, 2000)), 448.0 * np.exp2(np.arange(-60.0, 60.0)),
                             np.nextafter(448.0 * np.exp2(np.arange(-60.0, 60.0)), np.inf), [0.0, 1e-300]])
    for a in values:
        e = R.needed_exp(float(a))
        assert a <= 448.0 * 2.0 ** e
        assert e == R.MIN_EXP or a > 448.0 * 2.0 ** (e - 1)
