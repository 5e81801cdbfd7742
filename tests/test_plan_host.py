"""The kernels that calls are sent to, from the header that the library takes
the choice from."""
import shutil
import subprocess

import pytest

from bit_diffusion_transformer_nvfp4_b200 import build
from plan_shapes import ATTENTION, PRODUCTS

PROGRAM = """
#include <cstdio>
#include "plan.h"
int main() {
  const int clusters[9] = {0, 148, 74, 48, 33, 26, 22, 18, 15};
  long op, a, b, c;
  while (std::scanf("%ld %ld %ld %ld", &op, &a, &b, &c) == 4) {
    if (op == 0)
      std::printf("%d %d\\n", w4a4::fp8_gemm_plan(a, b, c, 148),
                  w4a4::fp8_small_splits(w4a4::ceil_div(b, 128), w4a4::ceil_div(c, 128), 148));
    else
      std::printf("%d 0\\n", w4a4::xattn_splits(a, b, c, 148, clusters));
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs a C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cc").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{build.CSRC}", str(d / "plan.cc"), "-o", str(d / "plan")],
                   check=True)

    def ask(rows):
        text = "".join(" ".join(map(str, r)) + "\n" for r in rows)
        out = subprocess.run([str(d / "plan")], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def test_products_reach_the_kernels_they_are_listed_for(plan):
    got = plan([(0, M, N, K) for M, N, K, _, _ in PRODUCTS])
    for (M, N, K, kernel, slices), (k, s) in zip(PRODUCTS, got, strict=True):
        assert (k, s) == (kernel, slices), (M, N, K)
    # every instantiation, with every number of slices that it can have
    few = {(next(t for t in (16, 32, 64, 128) if M <= t), s) for M, _, _, k, s in PRODUCTS if k == 0}
    assert few == {(t, s) for t in (16, 32, 64, 128) for s in (1, 2, 4, 8)}
    assert {k for _, _, _, k, _ in PRODUCTS} == {0, 64, 128, 256}


def test_choice_over_the_range(plan):
    """Few rows only to 128 tokens, always to 16; slices within the K steps and a cluster."""
    sizes = [(M, N, K) for M in (1, 16, 17, 64, 100, 128, 129, 500, 9000) for N in (8, 136, 1000, 9216, 65536, 1 << 23)
             for K in (16, 128, 400, 6144, 1 << 20)]
    for (M, N, K), (k, s) in zip(sizes, plan([(0, *x) for x in sizes]), strict=True):
        assert k in (0, 64, 128, 256)
        if M > 128 or N > 65535 * 128:
            assert k != 0
        elif M <= 16:
            assert k == 0
        assert s in (1, 2, 4, 8) and s <= -(-K // 128)


def test_attention_forms(plan):
    def row(batch, sq, sk, heads, kv_heads):
        pack = 1
        while pack < 32 and heads // kv_heads % (2 * pack) == 0:
            pack *= 2
        return 1, sq * pack, batch * (heads // pack), -(-sk // 128)

    got = plan([row(b, sq, sk, h, hk) for b, _, sq, sk, h, hk, _, _ in ATTENTION])
    for case, (splits, _) in zip(ATTENTION, got, strict=True):
        assert (splits > 0) == case[-1], case
