"""The choice between the kernels of one product: the shapes that the GPU tests mean
for a kernel do get it, on the MI355X's 256 CUs."""

import os
import shutil
import subprocess

import pytest

import tile_shapes as ts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fine_grained_block_fp8q_amd", "csrc")
CUS = 256

SOURCE = """
#include <cstdio>
#include "tile_choice.hpp"
int main() {
  char kind[8];
  long M, W, K;
  while (std::scanf("%7s %ld %ld %ld", kind, &M, &W, &K) == 4)
    std::printf("%d\\n", kind[0] == 'i' ? fp8q::pick_i8(M, W, K, CUS) : fp8q::pick_gated(M, W, K, CUS));
  for (const fp8q::TileVariant& v : fp8q::kI8Variants) std::printf("i8 %d\\n", v.tile);
  for (const fp8q::TileVariant& v : fp8q::kGatedVariants) std::printf("gated %d\\n", v.tile);
}
"""


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("choice")
    (d / "pick.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", f"-DCUS={CUS}", "-I", CSRC, str(d / "pick.cpp"), "-o",
                    str(d / "pick")], check=True)

    def run(asked):
        """[(kind, M, weight rows, K)] -> (tiles, {kind: its tiles})"""
        text = "".join("%s %d %d %d\n" % a for a in asked)
        out = subprocess.run([str(d / "pick")], input=text, capture_output=True, text=True,
                             check=True).stdout.splitlines()
        have = {"i8": set(), "gated": set()}
        for line in out[len(asked):]:
            kind, tile = line.split()
            have[kind].add(int(tile))
        return [int(x) for x in out[:len(asked)]], have
    return run


def test_shapes_get_the_kernel_they_are_meant_for(pick):
    K = ts.I8_LARGEST_SUM_K
    meant = [(tile, ("i8", M, N, K)) for tile, (M, N) in ts.I8_LARGEST_SUM.items()]
    meant += [(tile, ("i8",) + s) for tile, s in ts.I8_LONG_K.items()]
    meant += [(tile, ("i8", M, 2 * F, K)) for tile, (M, F, K) in ts.I8_GATED_LONG_K.items()]
    meant += [(tile, ("gated", M, 2 * F, K)) for tile, (M, F, K) in ts.GATED_LONG_K.items()]
    got, _ = pick([a for _, a in meant])
    assert [(g, a) for g, (_, a) in zip(got, meant)] == meant


def test_every_kernel_has_its_shapes(pick):
    _, have = pick([])
    for shapes in (ts.I8_LARGEST_SUM, ts.I8_LONG_K, ts.I8_GATED_LONG_K):
        assert set(shapes) == have["i8"] | {0}
    assert set(ts.GATED_LONG_K) == have["gated"] | {0}


def test_single_tokens_take_the_kernel_for_few_rows(pick):
    asked = [(k, M, W, K) for k in ("i8", "gated") for M in (1, 16) for W in (256, 65536)
             for K in (128, 57344)]
    assert not any(pick(asked)[0])
