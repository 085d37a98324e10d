"""8-bit integer quantizer and product, restated plainly in fp64.

A line (a row of M) with amax = max |x| over its finite entries has a = max(amax, 127 * 2^-126),
scale = fp32(a / 127) and codes rint(127 x / a), ties to even; NaN -> 0, +-inf -> +-127.
"""

import numpy as np

MIN_AMAX = 127.0 * 2.0 ** -126


def quantize_rows(M):
    """(codes int8, scales fp32) of the rows of M (fp32 or bf16 values, as any float array)."""
    M = np.asarray(M, dtype=np.float64)
    mag = np.where(np.isfinite(M), np.abs(M), 0.0)
    a = np.maximum(mag.max(axis=1), MIN_AMAX)
    # 254 |x| and (2 q + 1) a are exact: fp32 values have 24 bits, the factors 8
    q = np.floor(127.0 * mag / a[:, None])
    q = np.minimum(q, 127.0)
    for _ in range(2):      # the quotient itself is rounded and may have crossed an integer
        q = np.where(127.0 * mag < q * a[:, None], q - 1, q)
        q = np.where((127.0 * mag >= (q + 1) * a[:, None]) & (q < 127), q + 1, q)
    left, right = 254.0 * mag, (2.0 * q + 1.0) * a[:, None]
    q = q + ((left > right) | ((left == right) & (q % 2 == 1)))
    q = np.where(np.isinf(M), 127.0, q)
    codes = np.where(np.isnan(M), 0.0, np.copysign(q, M))
    return codes.astype(np.int8), (a / 127.0).astype(np.float32)


def product(A, sa, B, sb):
    """fp32(fp32(fp32(sum) * sa[i]) * sb[j]) with the exact integer sum."""
    acc = np.asarray(A, dtype=np.float64) @ np.asarray(B, dtype=np.float64).T    # below 2^53: exact
    out = acc.astype(np.float32) * np.asarray(sa, dtype=np.float32)[:, None]
    return out * np.asarray(sb, dtype=np.float32)[None, :]


def product_error_bound(A, B, sa, sb):
    """Largest difference of the product of the decoded operands from that of the matrices A and B
    themselves (rows contracted): every decoded entry is off by half a step at most."""
    a, b = np.abs(np.asarray(A, dtype=np.float64)), np.abs(np.asarray(B, dtype=np.float64))
    k = a.shape[1]
    ha, hb = 0.5 * np.asarray(sa, dtype=np.float64), 0.5 * np.asarray(sb, dtype=np.float64)
    return (a.sum(1)[:, None] * hb[None, :] + ha[:, None] * b.sum(1)[None, :] + k * np.outer(ha, hb)) * (1 + 2.0 ** -20)
