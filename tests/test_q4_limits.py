"""Limits of the decode over the 4-bit cache that its launcher keeps on the host (no GPU)."""
import ctypes

import pytest

from sparse_attention_flux_b200 import build, flux


@pytest.fixture(scope="module")
def lib():
    build.build(quiet=True)
    return flux.lib()


@pytest.mark.parametrize("d", [64, 128])
def test_no_more_ctas_than_the_merge_buffer_has_weights(lib, d):
    """The last merge of a row keeps a weight for each part and head in a part of shared memory that
    holds 320 parts; the launcher makes no more CTAs than that, and the workspace follows."""
    workspace = lib._ZN4flux25decode_q4_workspace_bytesEii     # by head_dim and SMs, as the launcher counts
    workspace.argtypes, workspace.restype = [ctypes.c_int, ctypes.c_int], ctypes.c_size_t
    a_cta = workspace(d, 148) // 296
    assert workspace(d, 148) == 296 * a_cta and workspace(d, 160) == 320 * a_cta
    assert workspace(d, 161) == workspace(d, 1000) == 320 * a_cta
