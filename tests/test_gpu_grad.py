"""The gradient norm over many tensors and the clipping, on the GPU against sums in fp64.

Tolerances: squares of fp32 values are exact in fp64 up to 2^-53 and their sum's error is below
n 2^-53, so the norm is off by its last rounding, 2^-24 of it, plus 2^-30 for what is left.  A clipped
value meets the norm's rounding, the factor's and the product's: 3 * 2^-24, and half a bf16 step (2^-8)
where it is stored in bf16.
"""
import math

import numpy as np
import pytest

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu


def tensors(sizes, dtypes, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = torch.bfloat16 if dtypes == "bf16" or (dtypes == "mixed" and i % 2) else torch.float32
        out.append((torch.randn(n, generator=g, device="cuda") * scale * 10.0 ** -(i % 4)).to(dt))
    return out


def norm64(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def check(ts, max_norm, norm, out):
    import torch
    n = norm64(ts)
    assert abs(float(norm) - n) <= (2.0 ** -24 + 2.0 ** -30) * n, (float(norm), n)
    c = min(1.0, max_norm / n) if n > 0 else 1.0
    for i, (t, o) in enumerate(zip(ts, out)):
        ref = t.double() * c
        tol = 3 * 2.0 ** -24 * ref.abs() + 1e-44
        if t.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * ref.abs()
        assert o.dtype == t.dtype and bool(((o.double() - ref).abs() <= tol).all()), i
        if c == 1.0:
            assert torch.equal(o, t), i


SIZES = {"one": [1], "odd": [0, 1, 2, 3, 5, 7, 8, 9, 255, 257, 1023, 4095, 4096, 4097, 12289], "many": [33] * 300 + [100000],
         "large": [3_000_001, 17, 1_048_576], "none": [0, 0]}


@pytest.mark.parametrize("dtypes", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_norm_and_clip(sizes, dtypes):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("clip", sizes, dtypes)
    ts = tensors(SIZES[sizes], dtypes, 5)
    n = norm64(ts)
    for max_norm in (0.3 * n, n * 1.01 + 1.0, 0.0):
        out = [torch.full_like(t, 7.0) for t in ts]
        norm = m2.m2rnn_grad_clip(ts, max_norm, out=out)
        check(ts, max_norm, norm, out)
        place = [t.clone() for t in ts]
        norm2 = m2.m2rnn_grad_clip(place, max_norm)
        assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(place, out))
    assert torch.equal(m2.m2rnn_grad_norm(ts), norm)


def test_views_at_every_alignment():
    """Tensors that start at every element within 16 bytes, with outputs at the same and at other ones;
    the elements around them stay as they are."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    for dt, step in ((torch.float32, 4), (torch.bfloat16, 8)):
        for a in range(step):
            for b in (0, a, step - 1):
                say("alignment", dt, a, b)
                src = torch.randn(6000, device="cuda").to(dt)
                dst = torch.full_like(src, 3.0)
                g, o = src[a:a + 5000], dst[b:b + 5000]
                norm = m2.m2rnn_grad_clip([g], 1.0, out=[o])
                check([g], 1.0, norm, [o])
                assert bool((dst[:b] == 3.0).all()) and bool((dst[b + 5000:] == 3.0).all())
                before = src.clone()
                m2.m2rnn_grad_clip([g], 1.0)
                assert torch.equal(src[:a], before[:a]) and torch.equal(src[a + 5000:], before[a + 5000:])
                assert torch.equal(g, o)


@pytest.mark.parametrize("scale", [1e-30, 1e25])
def test_gradients_whose_squares_leave_fp32(scale):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    ts = tensors([1000, 77], "fp32", 6, scale)
    for max_norm in (scale, 1e30):
        out = [torch.empty_like(t) for t in ts]
        check(ts, max_norm, m2.m2rnn_grad_clip(ts, max_norm, out=out), out)


@pytest.mark.parametrize("scale,max_norm", [(1e30, 1e-12), (1e25, 1e-14), (1e36, 1e-3), (1e30, 3e-1), (1.0, 1e-36)])
@pytest.mark.parametrize("dtypes", ["fp32", "bf16"])
def test_factors_near_the_smallest_number(scale, max_norm, dtypes):
    """max_norm / norm near or below 2^-126: the clipped values are ordinary numbers and keep their bits.  (The
    bound of values that are themselves below fp32's normal numbers is their spacing, 2^-149, once for each rounding.)"""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("clip factor", scale, max_norm, dtypes)
    ts = tensors([1000, 77, 4099], dtypes, 16, scale)
    out = [torch.empty_like(t) for t in ts]
    norm = m2.m2rnn_grad_clip(ts, max_norm, out=out)
    n = norm64(ts)
    assert abs(float(norm) - n) <= (2.0 ** -24 + 2.0 ** -30) * n
    step = 2.0 ** -8 if dtypes == "bf16" else 0.0
    for t, o in zip(ts, out):
        ref = t.double() * (float(np.float32(max_norm)) / n)
        # bf16's own smallest numbers are 2^-133 apart
        least = 2 * 2.0 ** -149 + (2.0 ** -134 if dtypes == "bf16" else 0.0)
        assert bool(((o.double() - ref).abs() <= (3 * 2.0 ** -24 + step) * ref.abs() + least).all())
    m2.m2rnn_grad_clip(ts, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(ts, out))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    ts = tensors([5000, 33], "mixed", 7)
    ts[0][4321] = bad
    keep = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts]
    norm = m2.m2rnn_grad_clip(ts, 1e-3, out=out)
    m2.m2rnn_grad_clip(ts, 1e-3)
    assert not bool(torch.isfinite(norm))
    for k, t, o in zip(keep, ts, out):
        assert torch.equal(k.nan_to_num(1.0, 2.0, 3.0), t.nan_to_num(1.0, 2.0, 3.0))
        assert torch.equal(k.nan_to_num(1.0, 2.0, 3.0), o.nan_to_num(1.0, 2.0, 3.0))


def test_a_given_norm_and_refusals():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    ts = tensors([1000, 50], "fp32", 8)
    total = torch.tensor(4.0 * norm64(ts), dtype=torch.float32, device="cuda")  # e.g. over 16 ranks
    out = [torch.empty_like(t) for t in ts]
    assert m2.m2rnn_grad_clip(ts, 1.0, norm=total, out=out) is total
    for t, o in zip(ts, out):
        ref = t.double() / float(total)
        assert bool(((o.double() - ref).abs() <= 3 * 2.0 ** -24 * ref.abs()).all())
    with pytest.raises(m2.M2RNNError):  # the same tensor twice would be scaled twice
        m2.m2rnn_grad_clip([ts[0], ts[0]], 1.0)
    with pytest.raises(m2.M2RNNError):
        m2.m2rnn_grad_clip(ts, 1.0, out=[ts[1].new_empty(2000)[:1000], ts[0][:50]])
    with pytest.raises(m2.M2RNNError):  # an output that covers a part of its own tensor
        m2.m2rnn_grad_clip([ts[0][:500]], 1.0, out=[ts[0][100:600]])
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError):
            m2.m2rnn_grad_clip(ts, bad)
    with pytest.raises(ValueError):
        m2.m2rnn_grad_clip([ts[0].view(10, 100).t()], 1.0)
    with pytest.raises(TypeError):
        m2.m2rnn_grad_norm([ts[0].half()])
    with pytest.raises(ValueError):
        m2.m2rnn_grad_norm([])


def test_empty_lists():
    """A rank without gradients: norm 0, nothing to clip."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    norm = torch.full((), 7.0, device="cuda")
    assert m2.m2rnn_grad_norm([], norm=norm) is norm and float(norm) == 0.0
    norm.fill_(3.0)  # combined over ranks
    for out in (None, []):
        assert m2.m2rnn_grad_clip([], 1.0, norm=norm, out=out) is norm and float(norm) == 3.0
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    m2.m2rnn_grad_norm([], norm=norm, stream=s)
    torch.cuda.synchronize()
    assert float(norm) == 0.0
    for bad in (lambda: m2.m2rnn_grad_norm([]), lambda: m2.m2rnn_grad_clip([], 1.0),
                lambda: m2.m2rnn_grad_clip([], 1.0, norm=norm, out=[norm]), lambda: m2.m2rnn_grad_clip([norm], 1.0, out=[]),
                lambda: m2.m2rnn_grad_norm([], norm=norm.cpu()), lambda: m2.m2rnn_grad_norm([], norm=norm.double())):
        with pytest.raises(ValueError):
            bad()


def test_graph_and_stream():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    ts = tensors([70000] + [19] * 200, "mixed", 9)
    out = [torch.empty_like(t) for t in ts]
    ref_norm = m2.m2rnn_grad_clip(ts, 1.0, out=out).clone()
    ref = [o.clone() for o in out]
    norm = torch.zeros((), device="cuda")
    ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def work():
        m2.m2rnn_grad_norm(ts, norm=norm, workspace=ws, stream=s)
        m2.m2rnn_grad_clip(ts, 1.0, norm=norm, out=out, stream=s)
    work()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    assert torch.equal(norm, ref_norm)
    with torch.cuda.graph(graph, stream=s):
        work()
    for _ in range(3):
        for o in out:
            o.fill_(float("nan"))
        norm.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, ref_norm) and all(torch.equal(a, b) for a, b in zip(out, ref))
