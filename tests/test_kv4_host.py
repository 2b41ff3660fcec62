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


SCRATCH = r"""
#include <cstdio>
#include "kv8_internal.cuh"
using namespace srh::kv8;
// A call of so many heads that only the many-row kernel serves it, over a handle whose scratch lacks `part`.
int main() {
    for (int dim = 128; dim <= 256; dim += 128)
        for (int part = 0; part < 3; ++part) {
            Cache c{};
            c.cfg = kv8_config{1, 1, dim, 16, 1, 1, 0, 0};
            c.sm_count = 152;
            c.bs_log2 = 4;
            attend4_scratch(c.sm_count, &c.part_o_floats, &c.part_ml_floats, &c.meta_n, &c.arrived_n);
            if (part == 0) c.part_o_floats = 0;
            if (part == 1) c.part_ml_floats = 0;
            if (part == 2) c.meta_n = 100;
            std::printf("%d ", (int)launch_attend4(c, kv4_pool{}, nullptr, nullptr, nullptr, 1, nullptr, 40 * dim, 1, 40, 1.f, 0,
                                                   nullptr, 40 * dim, nullptr));
        }
    return 0;
}
"""


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="host code alone, where nothing can be launched")
def test_a_call_without_its_scratch_is_refused_before_any_launch(abi, tmp_path):
    """cudaErrorInvalidValue (1), not what a launch without a device gives."""
    import os
    import subprocess

    from sparse_retrieval_host_gb300 import build
    src, exe = tmp_path / "scratch.cu", tmp_path / "scratch"
    src.write_text(SCRATCH)
    subprocess.run([build._nvcc(), *build.ARCH, *build.FLAGS, "-I", build.CSRC, str(src), build.LIB, "-o", str(exe),
                    "-Xlinker", f"-rpath={os.path.dirname(build.LIB)}"], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert got.split() == ["1"] * 6
