"""Split plans of the longest lengths and the sizes of their workspaces (no GPU): every length up to the last one that
32 bits hold."""

import ctypes

import pytest

OK, INVALID, WORKSPACE = 0, 1, 3
I, SZ, P, I64 = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int64
LONGEST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from mla_absorbed_decode_absorb_gb300 import build
    return ctypes.CDLL(build.build())


def asked(call, out, *args):
    assert call(*args, ctypes.byref(out)) == OK
    return out.value


@pytest.mark.parametrize("length", [LONGEST, LONGEST - 1, LONGEST - 61, LONGEST - 62, LONGEST - 63, LONGEST - 64])
def test_masked_plans_of_the_longest_lengths(lib, length):
    pages = -(-length // 64)
    for split in (0, 1, 1 << 19, 1 << 20, 1 << 25, LONGEST):
        n = asked(lib.mla_masked_num_splits, I(0), 2, 3, length, 0, 0, split)
        assert 1 <= n <= 64
        if split >= 1 << 19:
            assert n == -(-pages // split)
        size = asked(lib.mla_masked_workspace_size, SZ(0), 2, 3, length, 0, 0, split)
        assert size >= (2 * 3 * n * 128 * (512 * 4 + 4) if n > 1 else 0)
        # a window's view does not grow with the length
        for window, sinks in ((1024, 0), (1024, 300), (LONGEST, LONGEST)):
            view = min(pages, (window + 2 + 62) // 64 + 1 + -(-sinks // 64))
            n = asked(lib.mla_masked_num_splits, I(0), 2, 3, length, window, sinks, split)
            assert 1 <= n <= 64 and (split < 8 or window == LONGEST or n == -(-view // split))
