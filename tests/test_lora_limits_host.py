"""The largest numbers of tokens and adapters, refused before the device is touched (the pointers are never
dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
MOST = 0x7fff0000  # SPOPS_LORA_MAX_COUNT


@pytest.fixture(scope="module")
def lib():
    from unstructured_sparse_linear_gb300 import _lib, build
    build.build()
    return _lib.load()


@pytest.mark.parametrize("tokens,n", [(2 ** 31 - 1, 1), (MOST + 1, 1), (5, 2 ** 31 - 2), (5, MOST + 1), (2 ** 31 - 31, 8)])
def test_counts_that_32_bit_steps_would_pass(lib, tokens, n):
    """The kernels step past the last token and the last adapter in 32 bits: by up to 1024."""
    assert lib.spops_lora_plan_size(tokens, n) == 0
    assert lib.spops_lora_plan_build(P(0x1000), tokens, n, P(0x2000), 1 << 62, None) == 2
    assert str(max(tokens, n)).encode() in lib.spops_last_error()
    assert lib.spops_lora_add(P(0x100000), 64, P(0x200000), P(0x300000), None, 1.0, 2, tokens, 64, 32, 4, n, None, 32,
                              P(0x500000), 32, None, P(0x600000), None) == 2
    assert lib.spops_lora_grad(P(0x100000), 32, P(0x200000), 64, P(0x300000), P(0x400000), None, 1.0, 2, tokens, 64, 32, 4,
                               n, None, None, 64, P(0x500000), 64, None, None, P(0x800000), P(0x900000), 1 << 62, None) == 2
    import unstructured_sparse_linear_gb300 as sp
    with pytest.raises(ValueError, match="tokens >= 0"):
        sp.lora_plan(None, n, tokens=tokens, device="cuda:0")


def test_sizes_up_to_the_limit(lib):
    words = 2 * MOST + 3 * (MOST + 2)
    assert lib.spops_lora_plan_size(MOST, MOST) > 4 * words
