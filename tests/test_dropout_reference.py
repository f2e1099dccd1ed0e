"""The dropout mask's definition (tests/block_reference.py) against the generator's published
known answers (the Random123 distribution's test vectors of Philox4x32-10)."""
import numpy as np
import pytest

from block_reference import keep_mask, philox4x32, threshold


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_known_answers(counter, key, words):
    got = philox4x32([np.array([c], dtype=np.uint64) for c in counter], key)
    assert [int(w[0]) for w in got] == list(words)


def test_a_window_is_a_part_of_the_whole():
    whole = keep_mask(1000, 0.5, 7, 8)
    for first in (1, 6, 8, 13, 500):
        assert np.array_equal(keep_mask(100, 0.5, 7, 8, first), whole[first:first + 100])
    assert threshold(0.1) == 6554 and threshold(0.0) == 0 and threshold(1.0) == 65536
