"""The scale of an e4m3 block, max|x| / 448 in float32, as fp8_block_scale forms it for a maximum in
[2^-100, 2^100]: q0 = RN(a r) with r = RN(1 / 448), e = fma(-448, q0, a) (exact), q = fma(e, r, q0). On
the CPU, for every float32 significand and exponents over that range, it equals the division."""
import numpy as np


def test_three_instructions_equal_the_division():
    r = np.float32(1) / np.float32(448)
    bits = np.arange(1 << 23, dtype=np.uint32)
    for e in (-100, -61, -14, -1, 0, 7, 30, 99):
        a = (bits | np.uint32((127 + e) << 23)).view(np.float32)
        q0 = a * r
        # float64 holds a - 448 q0 and the last product and sum exactly enough for one rounding: 448 has
        # 3 significant bits, e at most 24, r 24, and q0 + e r at most 24 + 49 bits apart by their sizes'
        # ratio of 2^23, so a wrong rounding would need q0 + e r within 2^-53 of a tie
        err = (a.astype(np.float64) - 448.0 * q0.astype(np.float64)).astype(np.float32)
        q = (q0.astype(np.float64) + err.astype(np.float64) * np.float64(r)).astype(np.float32)
        assert np.array_equal(q, a / np.float32(448)), e
