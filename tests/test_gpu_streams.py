"""Calls on a stream of their own (stream=): inputs that the caller drops while the call still waits for earlier work
of that stream, and results dropped while the caller's stream still waits to read them, keep their memory."""
import pytest

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu

N = 1 << 20  # elements of the largest tensors: 4 MiB, in segments of the allocator's own


def calls():
    """name -> a function of a random source that gives (call, its inputs)."""
    import torch
    import matrix_state_nonlinear_m2rnn_amd as m2

    def x(r, *shape):
        return torch.empty(shape, device="cuda").normal_(generator=r)
    gate = lambda r, n, V: (x(r, n).abs(), x(r, n) - 3.0, x(r, n, V))  # noqa: E731

    def scan(r):
        q, k, v, a = x(r, 1, 1024, 16, 64), x(r, 1, 1024, 16, 64), x(r, 1, 1024, 16, 64), x(r, 1, 1024, 16)
        return m2.m2rnn_ssm_fwd, [q, k, v, a, *gate(r, 16, 64)]

    def back(r):
        _, args = scan(r)
        ckpt = m2.m2rnn_ssm_fwd_ckpt(*args)[2]
        return m2.m2rnn_ssm_bwd, [*args, ckpt, x(r, 1, 1024, 16, 64)]

    def step(r):
        return m2.m2rnn_ssm_step, [x(r, 64, 16, 64), x(r, 64, 16, 64), x(r, 64, 16, 64), x(r, 64, 16), *gate(r, 16, 64),
                                   x(r, 64, 16, 64, 64)]

    def conv(r):
        return m2.m2rnn_conv4_silu_fwd_state, [x(r, 1, 1024, 1024), x(r, 1024, 4)]

    def conv_step(r):
        return m2.m2rnn_conv4_silu_step, [x(r, 1024, 1024), x(r, 1024, 4)]

    def rope(r):
        pos = torch.arange(1024, device="cuda", dtype=torch.int32)[None].contiguous()
        return m2.m2rnn_qk_norm_rope_fwd, [x(r, 1, 1024, 16, 64), x(r, 1, 1024, 16, 64), x(r, 64), x(r, 64), pos,
                                           torch.rand(32, device="cuda", dtype=torch.float64, generator=r)]

    def rope_back(r):
        _, args = rope(r)
        return m2.m2rnn_qk_norm_rope_bwd, [*args, x(r, 1, 1024, 16, 64), x(r, 1, 1024, 16, 64)]

    def norm(r):
        return m2.m2rnn_grad_norm, [[x(r, N), x(r, N)]]

    def clip(r):
        return (lambda g, o, stream=None: (m2.m2rnn_grad_clip(g, 1.0, out=o, stream=stream), *o)), [
            [x(r, N), x(r, N)], [x(r, N), x(r, N)]]
    return dict(scan=scan, back=back, step=step, conv=conv, conv_step=conv_step, rope=rope, rope_back=rope_back, norm=norm,
                clip=clip)


def recurrence_calls():
    """The same for the M²RNN recurrence and its block's steps."""
    import torch
    import matrix_state_nonlinear_m2rnn_amd as m2

    def x(r, *shape):
        return torch.empty(shape, device="cuda").normal_(generator=r)

    def fwd_args(r):
        q, k, v = (x(r, 2, 512, 8, 64) * 0.2 for _ in range(3))
        return [q, k, v, torch.sigmoid(x(r, 2, 512, 8)), x(r, 8, 64, 64) * 0.05, x(r, 8, 64)]

    def back(r):
        args = fwd_args(r)
        ckpt = m2.m2rnn_fwd_ckpt(*args)[2]
        return m2.m2rnn_bwd_ckpt, [*args, ckpt, x(r, 2, 512, 8, 64)]

    def bwd(r):
        def f(*args, stream=None):
            return m2.m2rnn_bwd(*args[:6], None, args[6], stream=stream)
        return f, [*fwd_args(r), x(r, 2, 512, 8, 64)]

    def decode(r):
        return m2.m2rnn_decode_step, [x(r, 32, 16, 64), x(r, 32, 16, 64), x(r, 32, 16, 64), torch.sigmoid(x(r, 32, 16)),
                                      x(r, 16, 64, 64) * 0.05, x(r, 16, 64), x(r, 32, 16, 64, 64)]

    def block(r):
        q, k, v, f, W, w_r = fwd_args(r)
        return m2.m2rnn_fwd_block, [q, k, v, x(r, 2, 512, 8), x(r, 8).abs(), x(r, 8), W, w_r, x(r, 2, 512, 8, 64), x(r, 8, 64)]

    def finish(r):
        args = fwd_args(r)

        def f(*args, stream=None):
            y, H, ws = m2.m2rnn_scan_fwd(*args, stream=stream)
            return m2.m2rnn_scan_fwd_finish(*args, y=y, H_T=H, workspace=ws, stream=stream), H
        return f, args

    def scan_bwd(r):
        args = fwd_args(r)
        dims = m2.Dims(2, 512, 8, 64, 64, 8)
        ws = torch.empty(m2.m2rnn_bwd_ckpt_workspace_size(dims, m2.DTYPE_F32), dtype=torch.uint8, device="cuda")
        ckpt = m2.m2rnn_fwd_ckpt(*args)[2]

        def f(*args, stream=None):
            out = m2.m2rnn_scan_bwd(*args, workspace=ws, stream=stream)
            return m2.m2rnn_scan_bwd_finish(*args, workspace=ws, stream=stream, out=out)
        return f, [*args, ckpt, x(r, 2, 512, 8, 64)]
    return dict(
        m2_fwd=lambda r: (m2.m2rnn_fwd, fwd_args(r)), m2_ckpt=lambda r: (m2.m2rnn_fwd_ckpt, fwd_args(r)),
        m2_noalloc=lambda r: (m2.m2rnn_fwd_noalloc, fwd_args(r)), m2_back=back, m2_bwd=bwd, m2_decode=decode,
        m2_block=block, m2_finish=finish, m2_scan_bwd=scan_bwd,
        gate=lambda r: (m2.m2rnn_gate_fwd, [x(r, 4, 4096, 64), x(r, 64), x(r, 64)]),
        gate_back=lambda r: (m2.m2rnn_gate_bwd, [x(r, 4, 4096, 64), x(r, 64), x(r, 64), x(r, 4, 4096, 64)]),
        out_norm=lambda r: (m2.m2rnn_out_norm_fwd, [x(r, 1024, 1024), x(r, 1024, 1024), x(r, 1024)]),
        out_norm_back=lambda r: (m2.m2rnn_out_norm_bwd, [x(r, 1024, 1024), x(r, 1024, 1024), x(r, 1024), x(r, 1024, 1024)]),
        conv_train=lambda r: (m2.m2rnn_conv4_silu_fwd, [x(r, 1, 1024, 1024), x(r, 1024, 4), x(r, 1024)]),
        conv_back=lambda r: (m2.m2rnn_conv4_silu_bwd, [x(r, 1, 1024, 1024), x(r, 1024, 4), x(r, 1024), x(r, 1, 1024, 1024)]))


def flat(t):
    import torch
    if isinstance(t, torch.Tensor):
        return [t]
    return [x for u in (t.values() if isinstance(t, dict) else t) if u is not None for x in flat(u)]


def busy(m):
    """Some milliseconds of work on the current stream."""
    for _ in range(20):
        m @ m


NAMES = ["scan", "back", "step", "conv", "conv_step", "rope", "rope_back", "norm", "clip"]
NAMES += ["m2_fwd", "m2_ckpt", "m2_noalloc", "m2_back", "m2_bwd", "m2_decode", "m2_block", "m2_finish", "m2_scan_bwd",
          "gate", "gate_back", "out_norm", "out_norm_back", "conv_train", "conv_back"]


@pytest.mark.parametrize("name", NAMES)
def test_dropped_inputs_and_results(name):
    torch = torch_cuda()
    say("own stream", name)
    r = torch.Generator(device="cuda")
    m = torch.zeros(4096, 4096, device="cuda")
    s = torch.cuda.Stream()

    def made():
        r.manual_seed(5)
        return {**calls(), **recurrence_calls()}[name](r)
    f, args = made()
    ref = [t.clone() for t in flat(f(*args))]
    shapes = [(t.shape, t.dtype) for t in flat(args)]
    del args
    torch.cuda.synchronize()
    for _ in range(2):  # the second time round the allocator holds blocks of these sizes
        f, args = made()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            busy(m)
        got = f(*args, stream=s)
        del args
        other = [torch.empty(shape, dtype=dt, device="cuda").fill_(77) for shape, dt in shapes]
        torch.cuda.synchronize()
        for a, b in zip(flat(got), ref):
            assert torch.equal(a, b), "an input's memory was handed out while the call still read it"
        # the results, read late by the caller's stream
        busy(m)
        copies = [t.clone() for t in flat(got)]
        sizes = [(t.shape, t.dtype) for t in flat(got)]
        del got, a
        with torch.cuda.stream(s):
            mine = [torch.empty(shape, dtype=dt, device="cuda").fill_(77) for shape, dt in sizes]
        torch.cuda.synchronize()
        for a, b in zip(copies, ref):
            assert torch.equal(a, b), "a result's memory was handed out while the caller's stream still read it"
        del other, mine, copies, a, b
