"""Which kernel an expert product runs with (no GPU): the rules of ep_choice.h,
compiled for the host."""
import os
import subprocess

import pytest

from combine_ep_prepare_amd import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ep_choice.h"
int main(int argc, char** argv) {
  auto n = [&](int i) { return std::strtoll(argv[i], nullptr, 10); };
  epmi::Dims d{};
  d.T = n(2); d.K = (int)n(3); d.E = (int)n(4); d.cap = n(5); d.H = n(6); d.dtype = (int)n(8);
  std::printf("%d", (int)epmi::kernel_of((epmi::Product)n(1), d, n(7), 256));
}
"""
FEW, T256, T256_ONCE, T128, T128_ONCE, T64 = range(6)
FORWARD, ROW_GRAD, WEIGHT_GRAD = range(3)
BF16, FP16, FP32 = range(3)


@pytest.fixture(scope="module")
def kernel(tmp_path_factory):
    work = tmp_path_factory.mktemp("choice")
    source, program = work / "choice.hip", work / "choice"
    source.write_text(PROGRAM)
    subprocess.run([_build.hipcc(), "-std=c++17", f"--offload-arch={_build.ARCH}", "-I",
                    os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, "-o", str(program),
                    str(source)], check=True, capture_output=True)

    def choose(product, T, K, E, cap, H, N, dtype=BF16):
        args = [str(v) for v in (product, T, K, E, cap, H, N, dtype)]
        return int(subprocess.run([str(program), *args], check=True, capture_output=True).stdout)
    return choose


def test_rows_are_those_that_the_capacity_holds(kernel):
    """A rank's 32 of 256 experts, 8 routes a token: an eighth of the routes are
    its own, and the capacity is a quarter above that."""
    def share(T, product=FORWARD):
        return kernel(product, T, 8, 32, T * 5 // 4, 7168, 4096)
    assert share(64) == share(100) == share(300) == FEW            # up to 12 rows an expert
    assert share(512) == share(1024) == share(2048) == T128_ONCE   # 20, 40, 80
    assert share(4096) == share(32768) == T256                     # 160, 1280
    assert share(512, ROW_GRAD) == T128_ONCE
    assert share(1024, ROW_GRAD) == T256
    assert share(16384, WEIGHT_GRAD) == T256_ONCE                  # 640
    assert share(32768, WEIGHT_GRAD) == T256
    # a capacity for every route says nothing of the share
    assert kernel(FORWARD, 64, 8, 32, 64 * 8, 7168, 4096) == T128_ONCE


def test_rules_at_their_borders(kernel):
    def rows(r, product=FORWARD, dtype=BF16):
        return kernel(product, r * 16, 8, 128, r * 128, 2048, 1536, dtype)
    for dtype in (BF16, FP16):
        assert [rows(r, dtype=dtype) for r in (1, 12, 13, 104, 105, 256)] == \
            [FEW, FEW, T128_ONCE, T128_ONCE, T256, T256]
        assert [rows(r, ROW_GRAD, dtype) for r in (1, 32, 33, 256)] == \
            [T128_ONCE, T128_ONCE, T256, T256]
        assert [rows(r, WEIGHT_GRAD, dtype) for r in (1, 768, 769)] == \
            [T256_ONCE, T256_ONCE, T256]
    assert [rows(r, dtype=FP32) for r in (1, 12, 129, 1000)] == [T128] * 4
    # grids of one tile of 256 rows a CU, and of less
    assert [kernel(ROW_GRAD, r * 4, 8, 32, r * 32, 2048, 1536) for r in (33, 104, 105)] == \
        [T128_ONCE, T128_ONCE, T256]
    assert [kernel(FORWARD, r * 4, 8, 32, r * 32, 2048, 1536) for r in (104, 105, 128, 129)] == \
        [T128_ONCE, T128, T128, T256]
    assert kernel(FORWARD, 640, 8, 31, 5120, 2048, 1536) == T128   # 186 of 192
    # small grids: one expert of 256 rows, 4096 x 4096
    assert kernel(FORWARD, 256, 1, 1, 256, 4096, 4096) == T64
    assert kernel(FORWARD, 256, 1, 1, 256, 4096, 4096, FP32) == T64
    # no row at all
    assert kernel(FORWARD, 0, 8, 128, 0, 2048, 1536) == FEW
    assert kernel(ROW_GRAD, 0, 8, 128, 0, 2048, 1536) == T64
