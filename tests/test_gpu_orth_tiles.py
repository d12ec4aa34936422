"""Every instance of the orthogonalised update's product kernels (each tile shape for X X^T whole and split, b A + c A A, B X) against 64 bits.

Rows and columns have sizes over six orders of magnitude, and an error counts relative to its row and its column: as a norm of the
difference over both.  Tolerance: the definition itself with roundings put in at random where the kernels round, as in
test_gpu_orth.py (22 bits of what is multiplied, 2^-23; products 2^-24 sqrt(3 K / 16) of their typical value in their row and column, and
2^-22 for the pass that is left out); six times the difference that these make (the larger of two draws), and the output's rounding.
"""
import pytest

from _gpu import say, torch_cuda
from _orth import SIZES

pytestmark = pytest.mark.gpu

COEFS = (3.4445, -4.7750, 2.0315)


def definition(G, steps, seed=None):
    """In 64 bits, with roundings if there is a seed."""
    import torch
    gen = torch.Generator("cuda")
    gen.manual_seed(seed or 0)
    new = lambda x: torch.empty_like(x)  # noqa: E731

    def put(x, K):
        if seed is None:
            return x
        e = x * new(x).uniform_(-1, 1, generator=gen) * 2.0 ** -23
        if K:
            q = x.pow(2).mean(1, keepdim=True).sqrt() * x.pow(2).mean(0, keepdim=True).sqrt() / x.pow(2).mean().sqrt()
            e += new(x).normal_(generator=gen) * q * (2.0 ** -22 + 2.0 ** -24 * (3 * K / 16) ** 0.5)
        return x + e
    X = G.double()
    X = X.t().contiguous() if X.shape[0] > X.shape[1] else X
    X = put(X / (X.pow(2).sum().sqrt() + 1e-7), 0)
    for _ in range(steps):
        A = put(X @ X.t().contiguous(), X.shape[1])
        B = put(COEFS[1] * A + COEFS[2] * (A @ A), A.shape[0])
        X = put(COEFS[0] * X + put(B @ X, A.shape[0]), 0)
    return X.t() if G.shape[0] > G.shape[1] else X


@pytest.mark.parametrize("batch,m,n", SIZES)
def test_every_tile_shape(batch, m, n):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("orth tiles", batch, m, n)
    gen = torch.Generator("cuda")
    gen.manual_seed(m + n)
    new = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    g = new(batch, m, n).normal_(generator=gen) * 10 ** new(batch, m, 1).uniform_(-6, 0, generator=gen)
    g *= 10 ** new(batch, 1, n).uniform_(-6, 0, generator=gen)
    steps = 2
    out = m2.m2rnn_orthogonalize(g, steps)
    for b in {0, batch - 1}:
        ref = definition(g[b], steps)
        over = ref.pow(2).mean(1, keepdim=True).sqrt() * ref.pow(2).mean(0, keepdim=True).sqrt()
        tol = 6 * max(float(((definition(g[b], steps, s) - ref) / over).norm()) for s in (1, 2)) + 2.0 ** -24 * float((ref / over).norm())
        d = float(((out[b].double() - ref) / over).norm())
        assert d <= tol, (b, d, tol, float((ref / over).norm()))
    size = m2._size_query("m2rnn_orthogonalize_workspace_size", batch, m, n, m2._dtype_code(g))
    again = m2.m2rnn_orthogonalize(g, steps, workspace=torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, out)
