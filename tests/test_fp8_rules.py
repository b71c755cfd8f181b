"""CPU: what the host rules of the E4M3 operators promise to each other, by the rules' own code."""
import subprocess

from block_scaled_fp4_e2m1_amd import build
from test_gpu_fp8_moe import GROUPS
from test_gpu_fp8_plans import HEIGHTS

FEW_ROWS = r"""
#include <cstdio>
#include "fp8_plan.h"
using namespace bsfp4;
int main() {
  long long inside = 0, apart = 0;
  for (long long m = 1; m <= 5; m++)
    for (long long k = 16; k <= 16384; k += 16)
      for (long long n = 8; n <= 1 << 21; n += n < 1 << 15 ? 8 : 1 << 9)
        if (fp8_rows_quant_ok(m, n, k)) {
          inside++;
          if (!fp8_on_rows(false, false, m, n, k) && apart++ == 0) std::printf("%lld x %lld x %lld\n", m, n, k);
        }
  std::printf("%lld %lld\n", inside, apart);
}
"""


def run(tmp_path, source, text=""):
    (tmp_path / "rule.hip").write_text(source)
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-w", f"-I{build.ROOT}/include",
                    f"-I{build.CSRC}", str(tmp_path / "rule.hip"), "-o", str(tmp_path / "rule")], check=True)
    return subprocess.run([tmp_path / "rule"], input=text, capture_output=True, text=True, check=True).stdout.splitlines()


def test_rows_quantised_inside_are_rows(tmp_path):
    """Where the quantiser runs inside the product, the product alone takes the same kernel: the same order of sums."""
    lines = run(tmp_path, FEW_ROWS)
    inside, apart = map(int, lines[-1].split())
    assert inside > 100000 and apart == 0, lines


HEIGHT = r"""
#include <cstdio>
#include "fp8_plan.h"
int main() {
  long long gated, rows, n, e, cus;
  while (std::scanf("%lld %lld %lld %lld %lld", &gated, &rows, &n, &e, &cus) == 5)
    std::printf("%d\n", (int)bsfp4::fp8_tall_tiles(gated, rows, n, e, (int)cus));
}
"""


def test_grouped_heights(tmp_path):
    """The shapes that are to run on tall tiles and on tiles of 64 rows do, with either epilogue; the border moves with the chip."""
    shapes, want = [], []
    for tall, groups in ((True, HEIGHTS), (False, GROUPS)):
        for counts, behind, N, _ in groups:
            rows = sum(counts) + behind
            shapes += [(0, rows, N, len(counts), 256), (1, rows, N // 2, len(counts), 256)]
            want += [tall] * 2
    for gated in (0, 1):
        # 48 experts of 60 rows: (2880 + 1536) / 64 = 69 row tiles of 8 columns' blocks, 552 in all
        for cus in (32, 256, 304):
            shapes.append((gated, 2880, 1024, 48, cus))
            want.append(552 > (cus if gated else 2 * cus))
    text = "\n".join(" ".join(map(str, s)) for s in shapes)
    assert [int(v) for v in run(tmp_path, HEIGHT, text)] == want
