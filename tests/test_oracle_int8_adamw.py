"""Pins of the oracles of the 8-bit layer and of AdamW: closed forms, small cases by hand, grids by search."""

from fractions import Fraction

import numpy as np

from oracle import adamw, int8


def _bf16(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).bfloat16().double().numpy()


def test_int8_codes_are_the_exact_quotients_rounded_to_even():
    rng = np.random.default_rng(0)
    M = _bf16(rng.standard_normal((40, 60)) * np.exp(rng.uniform(-60, 60, (40, 1))))
    M[0, :3] = [2.0, 1.0, -1.0]
    M[0, 3:] = 0.0                       # 127 * 1 / 2 = 63.5, a tie
    codes, scales = int8.quantize_rows(M)
    for i in range(M.shape[0]):
        a = max(abs(Fraction(float(x))) for x in M[i])
        for j in range(M.shape[1]):
            assert codes[i, j] == round(127 * Fraction(float(M[i, j])) / a)   # Python rounds ties to even
        assert scales[i] == np.float32(float(a) / 127.0)
    assert list(codes[0, :3]) == [127, 64, -64]


def test_int8_edges():
    M = np.array([[0.0, 0.0, 0.0], [np.nan, 1.0, -np.inf], [np.inf, np.nan, np.nan], [2.0 ** -149, 0, 2.0 ** -126]])
    codes, scales = int8.quantize_rows(M)
    assert codes.tolist() == [[0, 0, 0], [0, 127, -127], [127, 0, 0], [0, 0, 1]]
    assert scales[0] == scales[2] == scales[3] == np.float32(2.0 ** -126) and scales[1] == np.float32(1 / 127)


def test_int8_product_by_hand():
    out = int8.product([[127, -128], [0, 3]], [0.5, 2.0], [[1, 1], [-128, 2]], [1.0, 0.25])
    assert out.tolist() == [[-0.5, (127 * -128 - 256) * 0.125], [6.0, 3.0]]


def test_state_codes_round_trip_and_are_sorted():
    for signed in (True, False):
        mag = adamw.magnitudes(signed)
        assert np.all(np.diff(mag) > 0)
        n = len(mag)
        codes = np.arange(n).astype(np.uint8)
        E = np.full(-(-n // 128), 140, np.uint8)
        x = adamw.decode(codes, E, signed)
        back, Eb = adamw.encode(x[-128:], signed)          # the block that holds the largest code
        assert np.array_equal(back, codes[-128:]) and Eb[0] == 140
        assert x[-1] == 1.875 * 2.0 ** 13                   # 2^(E - 127) <= largest < 2^(E - 126)


def test_state_encode_is_the_nearest_code():
    rng = np.random.default_rng(1)
    for signed, octaves in ((True, 25), (False, 45)):
        x = rng.standard_normal(1280) * 2.0 ** rng.uniform(-octaves, 0, 1280)
        if not signed:
            x = np.abs(x)
        codes, E = adamw.encode(x, signed)
        mag = adamw.magnitudes(signed)
        t = (np.abs(x).reshape(-1, 128) / (2.0 ** (E.astype(float) - (144 if signed else 160)))[:, None]).reshape(-1)
        best = np.abs(mag[None, :] - t[:, None]).argmin(1)
        if not signed:
            best = np.maximum(best, 1)                       # a positive second moment keeps code 1
        assert np.array_equal(codes & 127 if signed else codes, best)


def test_state_stochastic_rounding_is_unbiased():
    x = np.linspace(0.6, 1.9, 128)
    fields = np.arange(65536)
    lo = np.zeros(128)
    for f in fields[::64] + 32:
        lo += adamw.decode(*adamw.encode(x, True, np.full(128, f)), True)
    # the fields are 1024 equidistant points: off by a thousandth of a step (1/8 at most here)
    inner = x < 1.75                                         # the top code is clamped
    assert np.abs(lo / 1024 - x)[inner].max() < 2.0 ** -3 / 1000


def test_state_edges():
    x = np.zeros(200)
    x[3], x[130], x[131] = np.nan, np.inf, 1e-300
    for signed in (True, False):
        codes, E = adamw.encode(x, signed)
        assert codes[3] == codes[130] == 0 and E.tolist() == [16, 16]
        assert codes[131] == (0 if signed else 1)
    codes, E = adamw.encode(np.array([1e60, 1.0]), False)
    assert codes.tolist() == [255, 1] and E[0] == 254


def test_adamw_first_step_moves_by_the_learning_rate():
    g = np.array([3.0, -0.01, 7e-4])
    m, v = adamw.moments(np.zeros(3), np.zeros(3), g, 0.9, 0.99)
    p = adamw.parameter(np.ones(3), m, v, 1, 0.1, 0.9, 0.99, 0.0, 0.5)
    assert np.allclose(p, 0.95 - 0.1 * np.sign(g), rtol=0, atol=1e-14)
