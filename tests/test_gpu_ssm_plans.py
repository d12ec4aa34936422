"""The selective scan's kernel variants and launch plans that the small cases of test_gpu_ssm.py do not reach, on the
GPU against the fp64 oracle: every padded K with every V, several heads (or column blocks) in one workgroup of the
backward, heads split unevenly over workgroups, partial sums that take the tree of slices.

Tolerances are those of test_gpu_ssm.py, with one rounding more for each head that shares a query/key: their parts
of dq and dk are added one after the other, in registers and over the planes of split heads.
"""
import os
import re

import numpy as np
import pytest

from oracle import ssm

import matrix_state_nonlinear_m2rnn_amd as m2
from _gpu import say, torch_cuda
from test_gpu_ssm import bounds, check, make, on_gpu, oracle_in, run

pytestmark = pytest.mark.gpu


def compare(size, dtype, seed, lens=None):
    import torch
    d = make(*size, dtype, seed=seed)
    ls = None if lens is None else np.array(lens)
    ref = dict(zip(("y", "H_T"), ssm.fwd(*oracle_in(d), lens=ls)))
    ref.update(ssm.bwd(*oracle_in(d), d["dy"], d["dH_T"], lens=ls))
    tol = bounds(d, dtype, ls, True)
    B, T, N, G, K, V = size
    L = 64 if dtype == "bf16" else 32
    ops = K + V + L + 4 * -(-T // L) + 96
    for n in ("dq", "dk"):
        tol[n] = tol[n] * ((ops + N // G) / ops)
    tl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    check(run(on_gpu(d, dtype), lens=tl), ref, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [16, 32, 64, 128])
@pytest.mark.parametrize("K", [16, 48, 96, 128])
@pytest.mark.parametrize("N,G", [(2, 2), (5, 1), (4, 2)])
def test_every_padded_key_and_value_size(K, V, N, G, dtype):
    torch_cuda()
    size = (1, 75 if K < 96 else 131, N, G, K, V)
    say("ssm variant", size, dtype)
    compare(size, dtype, seed=K + V + N)


def heads_per_workgroup(B, T, N, G, dtype):
    """The sizes of the parts that a query/key's heads are split into by the backward's plan."""
    src = os.path.join(os.path.dirname(m2.__file__), "csrc", "m2rnn_ssm.hip")
    with open(src) as f:
        aim = int(re.search(r"constexpr long kSsmBwdGroups = (\d+);", f.read()).group(1))
    groups, hpg = B * G * -(-T // (64 if dtype == "bf16" else 32)), N // G
    if groups >= aim or hpg == 1:
        return [hpg]
    per = -(-hpg // min(hpg, -(-aim // groups)))
    return [min(per, hpg - i) for i in range(0, hpg, per)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [
    (512, 7, 5, 1, 32, 16), (260, 66, 3, 1, 16, 16), (512, 5, 3, 1, 96, 16),   # 16 columns: the head loop one ahead
    (512, 5, 4, 1, 16, 32), (260, 66, 2, 1, 64, 32),                          # the next head's inputs in registers
    (512, 6, 3, 1, 32, 64), (512, 4, 3, 1, 64, 64), (512, 3, 4, 2, 128, 64),
    (512, 3, 2, 1, 16, 128), (512, 3, 3, 1, 48, 128),                         # two blocks of columns for each head
])
def test_several_heads_in_a_workgroup(size, dtype):
    torch_cuda()
    B, T, N, G, K, V = size
    say("ssm heads in a workgroup", size, dtype)
    assert heads_per_workgroup(B, T, N, G, dtype) == [N // G]
    compare(size, dtype, seed=sum(size))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,V", [(32, 16), (16, 32), (48, 64), (32, 128)])
def test_heads_split_unevenly(K, V, dtype):
    torch_cuda()
    size = (130, 9, 10, 1, K, V)
    say("ssm uneven split", size, dtype)
    assert heads_per_workgroup(130, 9, 10, 1, dtype) == [3, 3, 3, 1]
    compare(size, dtype, seed=K + V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,V", [(5, 32, 16), (3, 16, 32), (2, 32, 64)])
def test_several_heads_in_a_padded_batch(N, K, V, dtype):
    torch_cuda()
    B, T = 260, 66
    say("ssm heads in a workgroup, padded", N, K, V, dtype)
    assert heads_per_workgroup(B, T, N, 1, dtype) == [N]
    lens = np.random.default_rng(N).integers(0, T + 1, B)
    lens[:3] = (0, 64, 33)
    compare((B, T, N, 1, K, V), dtype, seed=N, lens=[int(x) for x in lens])


def test_partial_sums_through_the_tree_bf16():
    """64 sequences of 33 chunks: more rows of partial sums than one launch adds."""
    torch_cuda()
    size = (64, 2049, 1, 1, 16, 16)
    say("ssm tree", size)
    compare(size, "bf16", seed=1)
