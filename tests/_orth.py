"""Sizes of the orthogonalised update that reach every instance of its products' kernels, and the plan of a size: the library's own cost
model, compiled for the host."""
import functools
import os
import subprocess
import tempfile

import matrix_state_nonlinear_m2rnn_amd as m2

# batch, m, n: sides a few short of whole tiles
SIZES = [(1, 129, 126), (1, 127, 510), (12, 701, 120), (48, 189, 192), (6, 310, 1277), (20, 125, 1085), (24, 640, 317), (64, 190, 509),
         (32, 255, 1214), (24, 187, 830), (48, 381, 383), (6, 4799, 573), (32, 511, 510), (5, 767, 4670), (64, 382, 380), (5, 893, 6590),
         (16, 959, 958), (2, 1341, 17983), (3, 2559, 2557), (2, 2237, 20926)]

_SOURCE = r"""
#include <cstdio>
#include "m2rnn_orth_plan.h"
int main() {
  long b, m, n;
  while (std::scanf("%ld %ld %ld", &b, &m, &n) == 3) {
    const m2rnn::OrthCuts p(b, m, n);
    std::printf("%d %d %d %d\n", p.gram.shape, p.gram.splits, p.poly.shape, p.next.shape);
  }
  std::printf("%d\n", m2rnn::kShapeCount);
}
"""


@functools.lru_cache(None)
def plans(sizes):
    """For each (batch, m, n): (shape of X X^T, its parts, shape of b A + c A A, shape of B X); and how many shapes there are."""
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "plan.cpp"), os.path.join(d, "plan")
        with open(src, "w") as f:
            f.write(_SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(os.path.dirname(m2.__file__), "csrc"), src, "-o", exe], check=True)
        out = subprocess.run([exe], input="\n".join("%d %d %d" % s for s in sizes), capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, line.split())) for line in out.splitlines()]
    return rows[:-1], rows[-1][0]
