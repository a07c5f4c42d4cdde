"""Pins of the dropout oracle (oracle/drop.py)."""
import numpy as np
import pytest

from oracle import drop as orc


@pytest.mark.parametrize("ctr,key,want", [
    # the known answers published with the generator (Random123, Philox4x32-10)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(ctr, key, want):
    got = orc.philox4x32(np.array(ctr, np.uint64)[None], key)[0]
    assert [int(v) for v in got] == list(want)


def test_element_layout_by_hand():
    # element j of row r: group r ceil(cols / 8) + j / 8, bits 16 (j % 2) of word (j % 8) / 2
    rows, cols, seed, offset = 5, 19, 0x1234567890ABCDEF, (7 << 32) | 3
    k = orc.keep(rows, cols, 0.5, seed, offset)
    for r, j in [(0, 0), (0, 7), (0, 8), (1, 0), (2, 18), (4, 13)]:
        g = r * 3 + j // 8
        w = orc.philox4x32(np.array([[g, 0, 3, 7]], np.uint64), (0x90ABCDEF, 0x12345678))[0]
        bits = (int(w[(j % 8) // 2]) >> (16 * (j % 2))) & 0xFFFF
        assert bool(k[r, j]) == (bits >= 32768), (r, j)


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_share_and_mean(p):
    k = orc.keep(400, 768, p, 11, 12)
    n = k.size
    q = 1 - orc.threshold(p) / 65536
    # 6 standard deviations of a binomial share
    assert abs(k.mean() - q) <= 6 * np.sqrt(q * (1 - q) / n)
    if p < 1:
        assert float(orc.scale(p)) * q == pytest.approx(1.0, abs=1e-6)


def test_masks_of_other_offsets_seeds_and_neighbours_are_unlike():
    a = orc.keep(64, 768, 0.5, 1, 1)
    for b in (orc.keep(64, 768, 0.5, 1, 2), orc.keep(64, 768, 0.5, 2, 1), orc.keep(64, 768, 0.5, 1, 1 << 32),
              orc.keep(64, 768, 0.5, 1 << 32, 1)):
        assert abs((a == b).mean() - 0.5) <= 6 * 0.5 / np.sqrt(a.size)
    assert abs((a[1:] == a[:-1]).mean() - 0.5) <= 6 * 0.5 / np.sqrt(a[1:].size)
    assert abs((a[:, 1:] == a[:, :-1]).mean() - 0.5) <= 6 * 0.5 / np.sqrt(a[:, 1:].size)


def test_threshold_rounds_to_even_and_rows_agree():
    assert orc.threshold(0.5) == 32768 and orc.threshold(1.0) == 65536
    assert orc.threshold(2.0 ** -17) == 0 and orc.threshold(3 * 2.0 ** -17) == 2
    whole = orc.keep(50, 13, 0.3, 5, 6)
    assert np.array_equal(orc.keep_rows([3, 49, 20], 13, 0.3, 5, 6), whole[[3, 49, 20]])


def test_dropout_is_its_own_gradient():
    r = np.random.default_rng(0)
    x, dy, res = r.standard_normal((3, 6, 21))
    y = orc.dropout(x, 0.4, 1, 2, res)
    dx = orc.dropout(dy, 0.4, 1, 2)
    h = 1e-6
    for i, j in [(0, 0), (5, 20), (3, 9), (2, 2)]:
        xp = x.copy()
        xp[i, j] += h
        num = ((orc.dropout(xp, 0.4, 1, 2, res) - y) * dy).sum() / h
        assert num == pytest.approx(dx[i, j], abs=1e-6)
