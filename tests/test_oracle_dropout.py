"""The dropout oracle's generator against published known answers, and the mask's statistics."""
import numpy as np

from oracle import dropout as od


def test_known_answers():
    """Counter, key and result of Philox4x32-10 as its authors publish them."""
    f = 0xFFFFFFFF
    for c, k, want in (((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
                       ((f, f, f, f), (f, f), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
                       ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
                        (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        got = od.philox4x32([np.array([v], dtype=np.uint32) for v in c], k)
        assert tuple(int(v[0]) for v in got) == want


def test_mask_statistics():
    """The share kept is 1 - p within five standard deviations, in every column class, and rows differ."""
    T, H = 512, 403
    for p in (0.1, 0.5, 0.9):
        m = od.keep(T, H, p, 12345, 7)
        assert abs(m.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / m.size)
        for k in range(4):
            part = m[:, k::4]
            assert abs(part.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / part.size)
    assert not np.array_equal(m[0], m[1])
    assert np.all(od.keep(3, 5, 0.0, 1, 2)) and od.keep(0, 5, 0.5, 1, 2).shape == (0, 5)
    assert np.array_equal(od.keep(4, 40, 0.3, 9, 8)[2:], od.keep(2, 40, 0.3, 9, 8, row0=2))
    assert not np.array_equal(od.keep(4, 40, 0.3, 9, 8), od.keep(4, 40, 0.3, 9, 8 + 2 ** 32))
    assert not np.array_equal(od.keep(4, 40, 0.3, 9, 8), od.keep(4, 40, 0.3, 9 + 2 ** 32, 8))
