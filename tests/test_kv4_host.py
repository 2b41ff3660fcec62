"""CPU checks of the 4-bit cache's entry points: refusals come before any GPU call."""
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not __import__("os").path.exists(
    "/usr/local/cuda/bin/nvcc"), reason="nvcc not available")


@pytest.fixture(scope="module")
def abi():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_retrieval_host_gb300 import abi as a
    return a


@pytest.mark.parametrize("bad", [dict(shared_kv=True), dict(head_dim=512), dict(head_dim=64), dict(device="cpu")])
def test_a_4_bit_cache_that_is_not_offered_is_refused(bad):
    from sparse_retrieval_host_gb300.paged import PagedKV4
    with pytest.raises(ValueError):
        PagedKV4(**{**dict(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1), **bad})


def test_null_handles_of_the_new_calls(abi):
    lib = abi.load()
    n = None
    assert lib.kv4_append(n, n, n, n, n, 1, n, 0, n, 0, 1, n) == abi.SRH_ERR_INVALID
    assert lib.kv4_read(n, n, n, n, n, n, 1, n, 0, n, 0, 1, n) == abi.SRH_ERR_INVALID
    assert lib.kv8_read(n, n, n, n, n, n, 1, n, 0, n, 0, 1, n) == abi.SRH_ERR_INVALID
    assert lib.kv4_attend(n, n, n, n, n, 1, n, 0, 1, 1, 1.0, 0, n, 0, n) == abi.SRH_ERR_INVALID
    assert lib.kv8_norm_rope_axes(n, n, n, 1, 128, n, 0, 1, n, n, 0, 0, 0, 0.0, n) == abi.SRH_ERR_INVALID
