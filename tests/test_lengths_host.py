"""Split plans of the longest lengths and the sizes of their workspaces (no GPU): every length up to the last one that
32 bits hold."""

import ctypes

import pytest

OK, UNSUPPORTED, WORKSPACE = 0, 2, 3
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


A = 1 << 20  # a valid-looking address: every check comes before the device is touched


@pytest.mark.parametrize("B,n_q,max_kv_len,window,sinks,split", [
    (4, 3, 1000, 0, 0, 4), (1, 1, 4096, 0, 0, 1), (3, 64, 5000, 700, 5, 3), (129, 7, 300, 0, 0, 2)])
def test_masked_workspace_holds_the_partials_and_no_less(lib, B, n_q, max_kv_len, window, sinks, split):
    """512 float32 values and a float32 log-sum-exp of each query, split and head, either rounded up to 256 bytes; one byte
    less is refused."""
    plan = (B, n_q, max_kv_len, window, sinks, split)
    n = asked(lib.mla_masked_num_splits, I(0), *plan)
    size = asked(lib.mla_masked_workspace_size, SZ(0), *plan)
    rows = B * n_q * n * 128
    assert n > 1 and rows * (512 * 4 + 4) <= size < rows * (512 * 4 + 4) + 2 * 256
    attend = lib.mla_decode_attn_masked_partial
    attend.argtypes = [P, P, I64, P, I, P, P, P, I, I, I, I, I, I, P, SZ, P, P, P]
    pages = -(-max_kv_len // 64)

    def args(ws, b):
        return A, A, pages, A, pages, A, None, None, window, sinks, B, n_q, max_kv_len, split, ws, b, A, A, None
    assert attend(*args(A, size - 1)) == WORKSPACE and attend(*args(None, size)) == WORKSPACE
    assert attend(*args(A + 8, size)) == WORKSPACE


@pytest.mark.parametrize("length", [LONGEST, LONGEST - 1, LONGEST - 62, LONGEST - 63, LONGEST - 64])
def test_causal_plans_of_the_longest_lengths(lib, length):
    pages = -(-length // 64)
    for split in (0, 1, 1000, 1 << 20, 1 << 25, LONGEST - 1, LONGEST):
        n = asked(lib.mla_decode_num_splits, I(0), 2, 3, length, split)
        assert n == -(-pages // split) if split else 1 <= n <= 256
        size = asked(lib.mla_decode_workspace_size, SZ(0), 2, 3, length, split)
        assert size >= (2 * 3 * n * 128 * (512 * 2 + 4) if n > 1 else 0)
    assert asked(lib.mla_decode_num_splits, I(0), 8, 4, 300, LONGEST) == 1  # one split of all pages


@pytest.mark.parametrize("length", [LONGEST, LONGEST - 64, LONGEST - 127, LONGEST - 128, 1 << 24])
def test_prompts_of_the_longest_lengths_are_refused(lib, length):
    """128 heads' rows of one sequence pass 32 bits."""
    stride = 1 << 25
    decompress, attend = lib.mla_decompress_kv, lib.mla_prefill_attn
    decompress.argtypes = [P, I64, P, I, P, I, I, P, P, P, P, P]
    attend.argtypes = [P, P, P, P, I, P, P, I, P, I64, P, I, P, I, I, P, P, P]
    assert decompress(A, 8, A, stride, A, 1, length, A, A, A, A, None) == UNSUPPORTED
    assert attend(A, A, A, A, 300, A, A, length, A, 8, A, stride, A, 1, 70, A, A, None) == UNSUPPORTED
    windowed, prompt = lib.mla_decompress_kv_window, lib.mla_prefill_attn_window
    windowed.argtypes = [P, I64, P, I, P, I, I, I, I, I, P, P, P, P, P]
    prompt.argtypes = [P, P, P, P, I, P, P, I, P, I64, P, I, P, I, I, I, I, P, P, P]
    assert windowed(A, 8, A, stride, A, 1, 70, length, 64, 4, A, A, A, A, None) == UNSUPPORTED
    assert prompt(A, A, A, A, 300, A, A, length, A, 8, A, stride, A, 1, 70, 64, 4, A, A, None) == UNSUPPORTED
