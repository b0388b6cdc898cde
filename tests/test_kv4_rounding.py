"""The append's way to a code (a rounded reciprocal, a product, its mantissa cut to 11 bits)
decides like the exact quotient for every bf16 magnitude under every scale (CPU, exhaustive)."""

import numpy as np


def test_codes_of_every_value_under_every_scale():
    byte = np.arange(1, 127)
    scales = np.where(byte >> 3 == 0, (byte & 7) * 2.0 ** -9, (8 + (byte & 7)) * 2.0 ** ((byte >> 3) - 10.0))
    x = (np.arange(0x0000, 0x7F80, dtype=np.uint32) << 16).view(np.float32)
    borders = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))

    def code(y):                                         # to the nearest e2m1 value, ties to even
        return sum((y >= b) if up else (y > b) for b, up in borders)

    for s in scales:
        with np.errstate(over="ignore"):
            y = x * (np.float32(1) / np.float32(s))
        y = ((y.view(np.uint32) + np.uint32(0x1000)) & np.uint32(0xFFFFE000)).view(np.float32)
        assert np.array_equal(code(y.astype(np.float64)), code(x.astype(np.float64) / s)), s
