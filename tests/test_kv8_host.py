"""CPU checks of the paged 8-bit cache's entry points: refusals come before any
GPU call, so none of these needs a device."""
import ctypes
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


GOOD = dict(batch=4, n_kv_heads=2, head_dim=128, block_tokens=16, n_blocks=8, max_blocks=4, shared_kv=0, block_stride=0)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(batch=4097), dict(n_kv_heads=0), dict(n_kv_heads=257), dict(head_dim=64), dict(head_dim=192),
    dict(head_dim=1024), dict(block_tokens=8), dict(block_tokens=48), dict(block_tokens=256), dict(n_blocks=0),
    dict(max_blocks=0), dict(max_blocks=1 << 27), dict(shared_kv=2), dict(block_stride=4080), dict(block_stride=4096 + 8),
    dict(block_stride=-16), dict(block_stride=1 << 40)])
def test_bad_configs(abi, bad):
    cfg = abi.Kv8Config(**{**GOOD, **bad})
    out = ctypes.c_void_p(1)
    lib = abi.load()
    assert lib.kv8_create(ctypes.byref(cfg), ctypes.byref(out)) == abi.SRH_ERR_INVALID and not out.value
    assert lib.kv8_last_error(None)
    with pytest.raises(abi.SrhError) as ei:
        abi.kv8_create(cfg)
    assert ei.value.code == abi.SRH_ERR_INVALID


def test_null_handles(abi):
    lib = abi.load()
    assert lib.kv8_create(None, None) == abi.SRH_ERR_INVALID
    assert lib.kv8_check_error(None) == abi.SRH_ERR_INVALID
    lib.kv8_destroy(None)


def test_three_terms_hold_a_weight():
    """What the attention's weights are split into: two e5m2 terms cut off an fp16 value and one rounded are within 2^-9 of
    it, or half of e5m2's smallest step."""
    import torch
    h = torch.arange(0x7B00, dtype=torch.int16).view(torch.float16)        # up to 57,344
    rest = h.clone()
    for _ in range(2):
        rest = (rest.float() - (rest.view(torch.int16) & -256).view(torch.float16).float()).half()
    rest = rest.double() - rest.to(torch.float8_e5m2).double()
    assert (rest.abs() <= (2.0 ** -9 * h.double()).clamp(min=2.0 ** -17)).all()


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_a_cache_on_no_gpu_is_refused(device):
    from sparse_retrieval_host_gb300.paged import PagedKV8
    with pytest.raises(ValueError, match="CUDA device"):
        PagedKV8(batch=1, n_kv_heads=1, head_dim=128, block_tokens=16, n_blocks=1, max_blocks=1, device=device)
