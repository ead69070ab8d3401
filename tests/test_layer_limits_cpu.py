"""Sizes past what the layer operators' kernels number or a launch can hold
are refused on the host (no kernel is launched)."""
import os

import pytest

UNSUP = 5


@pytest.fixture(scope="module")
def lib():
    from fine_grained_fp8_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load_library()


def test_adapter_output_tiles_are_numbered_in_32_bits(lib):
    f = lib.fp8_adapter_linear_workspace
    assert f(1 << 23, 1 << 23, 128, 8, 1) == -1              # 2^16 x 2^15 tiles of 128 x 256
    assert f((1 << 23) - 128, 1 << 23, 128, 8, 1) > 0
    assert f(64, 1 << 23, 128, 8, 1) > 0


def test_adapter_launches_hold_less_than_2_32_threads(lib):
    f = lib.fp8_adapter_linear_workspace
    # 16 tokens and a share of K (8 of them from 29 K blocks on) for 512 threads
    assert f(1 << 24, 128, 29 * 128, 8, 1) == -1
    assert f((1 << 24) - 16, 128, 29 * 128, 8, 1) > 0
    assert f(1 << 24, 128, 28 * 128, 8, 1) > 0               # 7 shares


def test_expert_launches_hold_less_than_2_32_threads(lib):
    f = lib.fp8_moe_few_tokens_workspace
    # 16 channels of an expert for 512 threads, and one workgroup for the routing
    assert f(1, 128, 1 << 17, 1024, 1024, 1) == -1
    assert f(1, 128, (1 << 17) - 128, 1024, 1024, 1) > 0
    st = lib.fp8_moe_few_tokens(1, 128, 1 << 17, 1024, 0, 1024, 1, None, 128, None, 128, None, 0, 1, 1.0, None, None, None,
                                None, None, 0, 128, None, None, None, 0, None)
    assert st == UNSUP
