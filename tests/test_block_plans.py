"""CPU: which kernels the block operators' calls take, where tests or a launch's limits hang on it."""
import subprocess

import pytest

from block_scaled_fp4_e2m1_amd import binding, build
from test_gpu_block_tiles import SHAPES


def fused(M, N, K):
    """Whether int8_quantize_gemm quantises inside the product's workgroups: it needs no workspace then."""
    return binding.load().bsfp4_int8_quantize_gemm_workspace_size(M, N, K) == 0


@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_fused_quantiser_by_rows(M):
    """Up to where the rows and their codes fit in LDS."""
    K = 9216 // M
    assert fused(M, 512, K) and not fused(M, 512, K + 16) and not fused(M + 1, 512, K)


@pytest.mark.parametrize("M,K,last", [(1, 512, 16384), (1, 1024, 16384), (1, 2048, 32768), (1, 4096, 131072),
                                      (2, 1024, 8192), (2, 4096, 16384), (3, 1024, 5456), (4, 2304, 4096)])
def test_fused_quantiser_by_columns(M, K, last):
    """Every workgroup quantises the rows again: past some width two launches take over."""
    assert fused(M, last, K) and not fused(M, last + 8, K)


def test_fused_quantiser_within_a_launch():
    """32 threads per column, fewer than 2^32 in a launch, for every width that is admitted."""
    assert not any(fused(M, 1 << p, K) for M in (1, 2, 3, 4) for p in range(27, 30) for K in range(16, 9217, 16))


#: the planner's own host code, for 256 compute units
PLANNER = r"""
#include <cstdio>
#include "rows_gemm.h"
using namespace bsfp4;
int main() {
  const char* const names[] = {"256", "256x128", "128", "deep", "64x128", "64"};
  long long m, n, kbytes;
  while (std::scanf("%lld %lld %lld", &m, &n, &kbytes) == 3) {
    const TilePlan p = plan_tile(m, n, kbytes, 256);
    std::printf("%s|%s", rows_ok(m, n, kbytes) ? "rows" : "tiles", names[p.kind]);
    if (p.splits > 1) std::printf(" split");
    if (p.cut_m) std::printf(" rows+%s", names[p.rest]);
    if (p.cut_n) std::printf(" cols+%s", names[p.rest]);
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    d = tmp_path_factory.mktemp("planner")
    (d / "plan.hip").write_text(PLANNER)
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-w",
                    f"-I{build.ROOT}/include", f"-I{build.CSRC}", str(d / "plan.hip"), "-o", str(d / "plan")], check=True)

    def plans(shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        return subprocess.run([d / "plan"], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    return plans


def test_tile_shapes_reach_their_plans(planner):
    """The tile tests' shapes are named after the kernel, split and part launch that they are to reach."""
    for label, (rows, n, kbytes) in SHAPES.items():
        # the 8-bit product, the 8-bit gated one, the bf16 gated one
        assert planner([(rows - less, n, kbytes) for less in (3, 1, 2)]) == [f"tiles|{label}"] * 3, label
        # dx: rows - 3 tokens, sums over 2 I = kbytes / 2; dW13: `rows` weight rows, sums over kbytes / 2 tokens
        got = planner([(rows - 3, n, kbytes // 4 * 4), (rows // 2 * 2, n, kbytes // 2 * 2)])
        assert [g.split("|")[1] for g in got] == [label] * 2, label


def test_tile_shapes_cover_the_kernels(planner):
    """Every tile kernel alone, split over K where it can be, and as the rest of a part launch."""
    kinds = {"256", "256x128", "128", "deep", "64x128", "64"}
    assert kinds <= set(SHAPES) and {f"{k} split" for k in kinds} <= set(SHAPES)
    assert {label.split("+")[1] for label in SHAPES if "+" in label} >= kinds - {"256"}
