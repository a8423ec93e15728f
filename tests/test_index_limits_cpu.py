"""CPU: sizes whose index arithmetic would pass 32 bits inside a kernel are refused
on the host, before anything is launched."""
import ctypes

import pytest
import torch

import varlen_flashattention_forward_gb300 as fa
from varlen_flashattention_forward_gb300 import build_ext

P = ctypes.c_void_p
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return fa.load_library()


def select(lib, capacity, budget):
    return lib.fa_paged_kv_select(P(0x1000), P(0x2000), 1, 1, capacity, budget, 4, 16, P(0x3000),
                                  P(0x4000), None)


# A cluster of 8 CTAs of 256 threads goes through a row's keys, and through its
# budget, 2048 at a time: an index may pass the end by that much.
STRIDE = 8 * 256


@pytest.mark.parametrize("past", [1, 255, 256, 257, 1024, STRIDE - 1])
def test_select_refuses_rows_whose_strides_pass_32_bits(lib, past):
    n = MOST - STRIDE + past
    assert select(lib, n, 64) == fa.FA_ERR_UNSUPPORTED
    assert select(lib, 256, n) == fa.FA_ERR_UNSUPPORTED
    assert select(lib, n, n) == fa.FA_ERR_UNSUPPORTED


def test_select_takes_the_largest_rows_that_fit(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
    assert select(lib, MOST - STRIDE, 64) in none
    assert select(lib, MOST - STRIDE, MOST - STRIDE) in none


def tree(lib, total, words=1):
    return lib.fa_draft_tree(P(0x1000), P(0x2000), P(0x3000), 1, total, words, P(0x4000), None, None)


# 1024 blocks of 64 threads go through a sequence's nodes 65536 at a time.
NODES = 1024 * 64


@pytest.mark.parametrize("past", [1, 63, 64, 1000, NODES - 1, NODES])
def test_draft_tree_refuses_nodes_whose_strides_pass_32_bits(lib, past):
    assert tree(lib, MOST - NODES + past) == fa.FA_ERR_UNSUPPORTED


def test_draft_tree_takes_as_many_nodes_as_fit(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert tree(lib, MOST - NODES) in (fa.FA_ERR_LAUNCH, fa.FA_ERR_ARCH)
