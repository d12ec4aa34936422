"""The orthogonalised update on the GPU against the fp64 oracle.

Tolerance: the oracle itself with roundings put in at random where the kernels round.  A stored matrix keeps 22 bits (an error
of up to 2^-23 of each value), and a product over K terms is accumulated in fp32 in K/16 partial sums of each of three
passes, which as a random walk is 2^-24 sqrt(3 K / 16) of its typical value, 2^-22 more for the pass that is left
out.  Six times the difference that such roundings make (the larger of two draws), as a norm, plus half a bf16 step.
"""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from oracle import layer

pytestmark = pytest.mark.gpu

COEFS = (3.4445, -4.7750, 2.0315)


def gradient(batch, m, n, seed, dtype):
    import torch
    r = np.random.default_rng(seed)
    k = max(1, min(m, n) // 8)
    g = (r.normal(0, 1, (batch, m, k)) * np.exp(-3.0 * np.arange(k) / k)) @ r.normal(0, 1, (batch, k, n)) + r.normal(0, 0.3, (batch, m, n))
    t = torch.tensor(g * 1e-3, dtype=torch.float32, device="cuda")
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def noisy(seed):
    r = np.random.default_rng(seed)

    def put(x, K):
        e = x * r.uniform(-1, 1, x.shape) * 2.0 ** -23
        if K:
            e = e + r.normal(0, 1, x.shape) * np.sqrt(np.mean(x * x)) * (2.0 ** -22 + 2.0 ** -24 * np.sqrt(3 * K / 16))
        return x + e
    return put


def check(g, out, steps=5, coefs=COEFS, eps=1e-7):
    import torch
    assert out.dtype == g.dtype and out.shape == g.shape
    G, O = g.double().cpu().numpy(), out.double().cpu().numpy()
    G, O = G.reshape(-1, *G.shape[-2:]), O.reshape(-1, *O.shape[-2:])
    for b in range(G.shape[0]):
        ref = layer.orthogonalize(G[b], steps, coefs, eps)
        tol = 6 * max(np.linalg.norm(layer.orthogonalize(G[b], steps, coefs, eps, noisy(s)) - ref) for s in (1, 2))
        tol += (2.0 ** -8 if g.dtype == torch.bfloat16 else 0.0) * np.linalg.norm(ref)
        d = np.linalg.norm(O[b] - ref)
        assert d <= tol, (b, d, tol, np.linalg.norm(ref))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("batch,m,n", [(1, 1, 1), (2, 1, 7), (3, 16, 16), (5, 33, 17), (2, 64, 64), (3, 63, 65), (1, 64, 130),
                                       (2, 128, 128), (1, 129, 515), (2, 300, 100), (1, 256, 1000), (1, 513, 400), (1, 1, 5000), (2, 16, 513),
                                       (1, 2000, 32), (3, 17, 700), (2, 3, 512), (1, 5, 40000)])
def test_against_the_oracle(batch, m, n, dtype):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("orth", batch, m, n, dtype)
    g = gradient(batch, m, n, m + n, dtype)
    out = m2.m2rnn_orthogonalize(g)
    check(g, out)
    size = m2._size_query("m2rnn_orthogonalize_workspace_size", batch, m, n, m2._dtype_code(g))
    again = m2.m2rnn_orthogonalize(g, workspace=torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, out)
    assert m2.m2rnn_orthogonalize(g, out=g) is g and torch.equal(g, out)


@pytest.mark.parametrize("m,n", [(16, 16), (12, 600), (64, 48), (40, 200), (128, 96), (140, 300)])
def test_steps_and_coefficients(m, n):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("orth coefs", m, n)
    g = gradient(2, m, n, 3, "fp32")
    check(g, m2.m2rnn_orthogonalize(g, 1), 1)
    check(g, m2.m2rnn_orthogonalize(g, 8, (1.5, -0.5, 0.0), 1e-6), 8, (1.5, -0.5, 0.0), 1e-6)
    rows = [(3.0, -3.5, 1.5), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)]
    check(g, m2.m2rnn_orthogonalize(g, 3, rows), 3, rows)
    # one matrix at a time, two leading axes: the same bits
    a = m2.m2rnn_orthogonalize(g)
    assert torch.equal(m2.m2rnn_orthogonalize(g[1].contiguous()), a[1])
    assert torch.equal(m2.m2rnn_orthogonalize(g.view(1, 2, m, n)), a.view(1, 2, m, n))


@pytest.mark.parametrize("m,n,dtype", [(1990, 2110, "fp32"), (2950, 2900, "bf16"), (2620, 2700, "fp32"), (600, 9000, "fp32")])
def test_large_tiles_that_end_inside(m, n, dtype):
    """Sizes whose products take each of the larger tiles, of which the last ones end past the matrix."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("orth tiles", m, n, dtype)
    g = gradient(1, m, n, m + n, dtype)
    out = m2.m2rnn_orthogonalize(g, 2)
    check(g, out, 2)
    size = m2._size_query("m2rnn_orthogonalize_workspace_size", 1, m, n, m2._dtype_code(g))
    again = m2.m2rnn_orthogonalize(g, 2, workspace=torch.full((size + 16,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, out)


def test_offsets_past_2_31():
    """A batch whose planes end past 2^31 elements: its first and last matrices."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    batch, m, n = 35200, 140, 300
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB")
    g = torch.empty(batch, m, n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(9))
    out = m2.m2rnn_orthogonalize(g)
    for part in (slice(0, 2), slice(batch - 2, batch)):
        check(g[part], out[part])
    del g, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,n", [(24, 40), (700, 8), (64, 64), (150, 90)])
def test_scales_and_values_that_are_not_finite(m, n):
    """Any scale of the gradient gives the same result; zeros give zeros; one matrix that is not finite leaves the
    others of the batch their bits."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    g = gradient(4, m, n, 5, "fp32")
    a = m2.m2rnn_orthogonalize(g, eps=0.0)
    for k in (-80, 60):  # squares far outside fp32
        assert torch.equal(m2.m2rnn_orthogonalize(g * 2.0 ** k, eps=0.0), a)
    b = g.clone()
    b[0] = 0.0
    b[2, m // 2, n // 2] = float("nan")
    o, ref = m2.m2rnn_orthogonalize(b), m2.m2rnn_orthogonalize(g)
    assert not o[0].any() and torch.equal(o[1], ref[1]) and torch.equal(o[3], ref[3])
    assert not torch.isfinite(o[2]).any()
    one = torch.zeros(1, m, n, device="cuda")
    one[0, 3, 5] = -2e-3  # a single entry: rank one, all of the norm
    check(one, m2.m2rnn_orthogonalize(one))


@pytest.mark.parametrize("m,n", [(64, 64), (100, 128), (160, 200)])
def test_past_the_bound_is_not_finite(m, n):
    """A product that fp16 cannot hold gives no number that could be taken for a result; thin matrices have no such bound."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    g = torch.zeros(1, m, n, device="cuda")
    g[0, 1, 2] = 1.0  # one singular value, 1: B has an entry of 1000
    assert not torch.isfinite(m2.m2rnn_orthogonalize(g, 1, (1.0, 1000.0, 0.0))).all()
    thin = g[:, :16].contiguous()
    assert float(m2.m2rnn_orthogonalize(thin, 1, (1.0, 1000.0, 0.0))[0, 1, 2]) == pytest.approx(1001.0, rel=1e-5)


def test_empty_and_refusals():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        assert m2.m2rnn_orthogonalize(torch.zeros(shape, device="cuda")).shape == shape
    g = torch.randn(8, 12, device="cuda")
    for kw, err in ((dict(steps=0), ValueError), (dict(coefs=(1.0, 2.0)), ValueError), (dict(coefs=[COEFS] * 4), ValueError),
                    (dict(steps=65), m2.M2RNNError), (dict(eps=-1.0), m2.M2RNNError), (dict(out=g.bfloat16()), TypeError)):
        with pytest.raises(err):
            m2.m2rnn_orthogonalize(g, **kw)
    for bad, err in ((g.half(), TypeError), (g.t(), ValueError), (g[0], ValueError)):
        with pytest.raises(err):
            m2.m2rnn_orthogonalize(bad)


@pytest.mark.parametrize("m,n", [(30, 40), (48, 60), (120, 128), (60, 250), (150, 300), (400, 260)])
def test_coefficients_within_their_bounds(m, n):
    """Steps that grow X many times over and cubic ones with large factors, at singular values where they are within the bounds."""
    torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("orth bounds", m, n)
    g = gradient(1, m, n, 6, "fp32")
    norm = float(g.double().norm())
    for rows, over in (([(6.0, -14.0, 9.0), (1.5, -0.5, 0.0)], 1), ([(30.0, 0.0, 0.0), (2.0, -1.5, 0.5)], 25),
                       ([(1.5, -6000.0, 0.0)], 70), ([(40.0, -200000.0, 0.0), (1.5, -0.5, 0.0)], 400), ([(0.0, 1.0, 2.0)], 1),
                       ([(1.0, 0.0, 20.0), (0.5, 0.0, 0.0)], 2), ([(1.0, 0.0, 3e8)], 70)):
        eps = (over - 1) * norm  # no singular value above 1 / over
        check(g, m2.m2rnn_orthogonalize(g, len(rows), rows, eps), len(rows), rows, eps)


def test_coefficients_that_can_be_read_once():
    """An iterator of coefficients gives what a list of them gives, on the current stream and on another."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    g = gradient(1, 20, 30, 7, "fp32")
    rows = [(3.0, -3.5, 1.5), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for given, steps in ((lambda: rows, 3), (lambda: COEFS, 5)):
        ref = m2.m2rnn_orthogonalize(g, steps, given())
        assert torch.equal(m2.m2rnn_orthogonalize(g, steps, iter(given())), ref)
        out = m2.m2rnn_orthogonalize(g, steps, iter(given()), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def noisy_by_rows_and_columns(seed):
    """As noisy, but a product's roundings are relative to its row and its column: their root mean squares over the whole's take the
    place of the matrix's."""
    r = np.random.default_rng(seed)

    def put(x, K):
        e = x * r.uniform(-1, 1, x.shape) * 2.0 ** -23
        if K:
            q = np.sqrt(np.mean(x * x, 1, keepdims=True)) * np.sqrt(np.mean(x * x, 0, keepdims=True)) / np.sqrt(np.mean(x * x))
            e = e + r.normal(0, 1, x.shape) * q * (2.0 ** -22 + 2.0 ** -24 * np.sqrt(3 * K / 16))
        return x + e
    return put


@pytest.mark.parametrize("size", [1e-3, 1e-7, 1e-14])
@pytest.mark.parametrize("m,n,dtype", [(20, 700, "fp32"), (700, 16, "fp32"), (48, 60, "fp32"), (64, 100, "bf16"), (120, 100, "fp32"),
                                       (60, 250, "fp32"), (150, 300, "fp32"), (500, 260, "fp32"), (256, 512, "bf16")])
def test_rows_and_columns_far_smaller_than_the_others(m, n, dtype, size):
    """Rows (of tokens that are rare, of heads hardly used), columns, and both, far smaller than the others: each keeps the digits
    that it has by itself.  The update takes them as they are, and so do products in fp32."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("orth sizes", m, n, dtype, size)
    r = np.random.default_rng(m + n)
    for what in ("rows", "columns", "both"):
        rows, cols = r.permutation(m)[: m // 2], r.permutation(n)[: n // 2]
        G = r.normal(0, 1e-3, (m, n))
        if what != "columns":
            G[rows] *= size
        if what != "rows":
            G[:, cols] *= size
        g = torch.tensor(G, dtype=torch.float32, device="cuda")
        g = g.bfloat16() if dtype == "bf16" else g
        G = g.double().cpu().numpy()
        for steps, coefs in ((5, COEFS), (9, (1.5, -0.5, 0.0))):
            O = m2.m2rnn_orthogonalize(g, steps, coefs).double().cpu().numpy()
            ref = layer.orthogonalize(G, steps, coefs, 1e-7)
            off = [layer.orthogonalize(G, steps, coefs, 1e-7, noisy_by_rows_and_columns(s)) - ref for s in (1, 2)]
            small_r, small_c = np.zeros(m, bool), np.zeros(n, bool)
            small_r[rows], small_c[cols] = what != "columns", what != "rows"
            for a in {False, what != "columns"}:
                for b in {False, what != "rows"}:
                    part = np.ix_(small_r == a, small_c == b)
                    tol = 6 * max(np.linalg.norm(x[part]) for x in off)
                    tol += (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.linalg.norm(ref[part])
                    d = np.linalg.norm((O - ref)[part])
                    assert d <= tol, (what, steps, a, b, d, tol, np.linalg.norm(ref[part]))
