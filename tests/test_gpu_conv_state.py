"""The causal conv4 + SiLU with its window (prompts in pieces, padded batches, single tokens) on the GPU
against its fp64 oracle.

Tolerance: the sum of five terms is within 8 * 2^-24 of their magnitudes, SiLU's slope is at most 1.1,
and its own evaluation (2^x of a rounded x log2 e, a sum, a reciprocal, a product) within
(2 |pre| + 8) * 2^-24 of the value; bf16 outputs add half a step, 2^-8 of the value.
"""
import numpy as np
import pytest

from oracle import ssm

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(B, T, C, dtype, seed):
    import torch
    r = np.random.default_rng(seed)

    def rounded(x):
        t = torch.tensor(x, dtype=torch.float32)
        return (t.to(torch.bfloat16) if dtype == "bf16" else t).float().numpy()
    return (rounded(r.normal(0, 1, (B, T, C))), r.normal(0, 0.7, (C, 4)).astype(np.float32),
            r.normal(0, 0.3, C).astype(np.float32), rounded(r.normal(0, 1, (B, 3, C))))


def gpu(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def within(u, x, w, b, win, lens, dtype):
    ref, rwin = ssm.conv4_silu_window(x, w, b, win, lens)
    live = np.isfinite(x)
    mags = ssm._f64(np.where(live, np.abs(x), 0.0))
    B, T, C = x.shape
    seen = np.concatenate([np.zeros((B, 3, C)) if win is None else np.abs(win), mags], 1)
    S = sum(np.abs(w[:, i]) * seen[:, i:i + T] for i in range(4)) + (0.0 if b is None else np.abs(b))
    tol = U * (8 * 1.1 * S + (2 * S + 8) * np.abs(ref)) + 1e-37
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    got = u.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    worst = float(np.max(np.abs(got - ref) / tol)) if ref.size else 0.0
    say("worst error over its bound: %.3g" % worst)
    assert worst <= 1.0
    return rwin


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,bias,win", [(1, 1, 4, True, True), (2, 2, 8, False, True), (3, 3, 260, True, False),
                                            (2, 5, 64, True, True), (1, 200, 12, True, True), (4, 131, 1024, False, False)])
def test_pieces(B, T, C, bias, win, dtype):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("conv window", B, T, C, dtype)
    x, w, b, wn = make(B, T, C, dtype, 3 + T)
    b, wn = b if bias else None, wn if win else None
    tx, tw, tb = gpu(x, dtype), gpu(w), None if b is None else gpu(b)
    u, wout = m2.m2rnn_conv4_silu_fwd_state(tx, tw, tb, None if wn is None else gpu(wn, dtype))
    rwin = within(u, x, w, b, wn, None, dtype)
    assert np.array_equal(wout.float().cpu().numpy(), rwin)
    # a prompt in two pieces and then token by token is the same, bit for bit
    cut = T // 2
    u0, w0 = m2.m2rnn_conv4_silu_fwd_state(tx[:, :cut].contiguous(), tw, tb, None if wn is None else gpu(wn, dtype))
    parts = [u0]
    for t in range(cut, min(T, cut + 6)):
        u1, w1 = m2.m2rnn_conv4_silu_step(tx[:, t].contiguous(), tw, tb, w0)
        u2, w2 = m2.m2rnn_conv4_silu_step(tx[:, t].contiguous(), tw, tb, w0, win_out=w0)
        assert w2 is w0 and torch.equal(w1, w0) and torch.equal(u1, u2)
        parts.append(u2[:, None])
    end = min(T, cut + 6)
    u3, w3 = m2.m2rnn_conv4_silu_fwd_state(tx[:, end:].contiguous(), tw, tb, w0)
    parts.append(u3)
    assert torch.equal(torch.cat(parts, 1), u) and torch.equal(w3, wout)
    if wn is None:  # without a window: the training forward
        assert torch.equal(m2.m2rnn_conv4_silu_fwd(tx, tw, tb), u)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_batch(dtype):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    lens = [70, 0, 1, 2, 33, -5, 500]
    x, w, b, wn = make(7, 70, 36, dtype, 9)
    past = np.arange(70)[None] >= np.clip(lens, 0, 70)[:, None]
    x[past] = np.nan
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    u, wout = m2.m2rnn_conv4_silu_fwd_state(gpu(x, dtype), gpu(w), gpu(b), gpu(wn, dtype), lens=tl)
    rwin = within(u, x, w, b, wn, np.array(lens), dtype)
    assert np.array_equal(wout.float().cpu().numpy(), rwin)
    assert not u[torch.from_numpy(past).cuda()].any()


def test_refusals_and_empty():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    x, w, b, wn = (gpu(z) for z in make(2, 4, 8, "f32", 1))
    with pytest.raises(m2.M2RNNError):  # the prompt's windows must not overlap
        m2.m2rnn_conv4_silu_fwd_state(x, w, b, wn, win_out=wn)
    with pytest.raises(ValueError):
        m2.m2rnn_conv4_silu_fwd_state(x, w, b, wn[:1])
    with pytest.raises(ValueError):
        m2.m2rnn_conv4_silu_step(x, w, b, wn)
    u, wo = m2.m2rnn_conv4_silu_fwd_state(x[:, :0].contiguous(), w, b, wn)
    assert u.shape == (2, 0, 8) and torch.equal(wo, wn)
    u, wo = m2.m2rnn_conv4_silu_fwd_state(x[:, :0].contiguous(), w, b)
    assert not wo.any()
