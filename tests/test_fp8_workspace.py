"""Sizes of the FP8 operators' workspaces: a buffer for a batch serves every smaller one (CPU only)."""

import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_quantize_gb300 import _lib, build
    build.build()
    return _lib.load()


# the widths of the products' tiles change at 0.5, 12 and 52 slots per expert, the order of the slots
# at 262144 slots (and with 1024 experts): every token count around them
CASES = [(8, 128, 2048, 768, 2000), (2, 8, 272, 128, 500), (4, 4, 1040, 512, 200), (1, 1, 256, 128, 300), (1, 2048, 48, 128, 120000),
         (8, 60, 400, 256, 40000), (3, 7, 48, 144, 100000)]


@pytest.mark.parametrize("c", CASES)
def test_layer_workspace_never_falls(lib, c):
    k, E, H, I, most = c
    size = [lib.ft_moe_layer_fp8_workspace_bytes(T, k, E, H, I) for T in range(1, most + 1)]
    falls = [T + 2 for T in range(most - 1) if size[T + 1] < size[T]]
    assert size[0] > 0 and not falls, f"smaller than for one token less at {falls[:5]}"


@pytest.mark.parametrize("c", CASES)
def test_product_workspace_never_falls(lib, c):
    k, E, K, _, most = c
    size = [lib.ft_moe_fp8_workspace_bytes(T, k, E, K) for T in range(1, most + 1)]
    falls = [T + 2 for T in range(most - 1) if size[T + 1] < size[T]]
    assert size[0] > 0 and not falls, f"smaller than for one token less at {falls[:5]}"
