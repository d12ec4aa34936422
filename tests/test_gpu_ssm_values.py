"""Values that are not finite within a sequence, in the selective scan's forward: outputs that do not depend on them
keep their bits, the outputs that do are not finite."""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from test_gpu_ssm import make, on_gpu, run

pytestmark = pytest.mark.gpu

SIZES = [  # B, T, N, Nqk, K, V: waves that share scores, heads that share them, one wave for itself, two blocks of columns
    (2, 150, 4, 2, 64, 64), (2, 150, 5, 1, 32, 16), (2, 150, 2, 2, 48, 16), (2, 150, 4, 4, 128, 32), (2, 150, 2, 1, 32, 128),
    (1, 700, 2, 1, 64, 16),  # time segments
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_earlier_steps_and_other_heads_keep_their_bits(size, dtype):
    torch = torch_cuda()
    B, T, N, G, K, V = size
    rep = N // G
    d = make(*size, dtype, seed=T + V)
    clean = run(on_gpu(d, dtype), back=False)
    b, n = B - 1, N - 1
    grp = n // rep
    for t in (0, 1, 17, 40, 63, 64, 77, 127, T - 1):
        for name, bad in (("v", np.nan), ("v", np.inf), ("v", -np.inf), ("k", np.nan), ("k", np.inf), ("a", np.nan),
                          ("q", np.nan), ("q", -np.inf)):
            say("ssm not finite", size, dtype, name, bad, "step", t)
            e = dict(d)
            e[name] = np.array(d[name])
            col = V // 2 + 3
            at = {"v": (b, t, n, col), "k": (b, t, grp, K // 2), "q": (b, t, grp, 5), "a": (b, t, n)}[name]
            e[name][at] = bad
            got = run(on_gpu(e, dtype), back=False)
            hit = torch.zeros(B, T, N, V, dtype=torch.bool, device="cuda")
            state = torch.zeros(B, N, K, V, dtype=torch.bool, device="cuda")
            if name == "v":
                hit[b, t:, n, col] = True
                state[b, n, :, col] = True
            elif name == "a":
                hit[b, t:, n] = True
                state[b, n] = True
            elif name == "k":
                hit[b, t:, grp * rep:(grp + 1) * rep] = True
                state[b, grp * rep:(grp + 1) * rep, K // 2] = True
            else:
                hit[b, t, grp * rep:(grp + 1) * rep] = True
            for x, was, h in ((got["y"], clean["y"], hit), (got["H_T"], clean["H_T"], state)):
                assert torch.equal(x[~h], was[~h])
                assert not bool(torch.isfinite(x[h]).any())


def test_two_values_of_one_chunk():
    """Each column is lost from its own first such step on."""
    torch = torch_cuda()
    say("ssm not finite, two steps")
    d = make(1, 64, 1, 1, 32, 32, "bf16", seed=9)
    clean = run(on_gpu(d, "bf16"), back=False)
    for t, c in ((20, 3), (5, 3), (50, 31), (37, 16)):
        d["v"][0, t, 0, c] = np.nan
    got = run(on_gpu(d, "bf16"), back=False)
    first = {3: 5, 31: 50, 16: 37}
    for c in range(32):
        t = first.get(c, 64)
        assert torch.equal(got["y"][0, :t, 0, c], clean["y"][0, :t, 0, c]), c
        assert bool(torch.isnan(got["y"][0, t:, 0, c]).all()), c
