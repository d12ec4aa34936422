"""Refusals of the selective scan's entry points: every invalid call returns its documented status
before anything is enqueued (so they run without a GPU, on pointers that lead nowhere)."""
import ctypes

import pytest

import matrix_state_nonlinear_m2rnn_amd as m2

P = ctypes.c_void_p
D = m2.Dims


def call(name, dims, dtype=0, bad=None, ptr=256, nbytes=1 << 40, ws=True):
    """The entry point with every pointer at `ptr` (lens, H0, dH_T NULL), the argument `bad` replaced."""
    names = {"fwd": "q k v a alpha beta w_r lens H0 y H_T", "fwd_ckpt": "q k v a alpha beta w_r lens H0 y H_T ckpt",
             "bwd": "q k v a alpha beta w_r lens ckpt dy dH_T dq dk dv da dalpha dbeta dw_r dH0",
             "step": "q k v a alpha beta w_r H_in H_out y"}[name].split()
    args = {n: None if n in ("lens", "H0", "dH_T") else P(ptr) for n in names}
    args.update(bad or {})
    tail = [] if name == "step" else [P(256) if ws else None, nbytes]
    return getattr(m2.lib(), "m2rnn_ssm_" + name)(None if dims is None else ctypes.byref(dims), dtype,
                                                  *[args[n] for n in names], *tail, None)


@pytest.mark.parametrize("name", ["fwd", "fwd_ckpt", "bwd", "step"])
def test_dims_and_pointers(name):
    T = 1 if name == "step" else 4
    assert call(name, None) == m2.M2RNN_EINVAL
    assert call(name, D(-1, T, 2, 16, 16)) == m2.M2RNN_EINVAL
    assert call(name, D(1, T, 2, 16, 16), dtype=7) == m2.M2RNN_EINVAL
    assert call(name, D(1, T, 4, 16, 16, 3)) == m2.M2RNN_EINVAL          # Nqk must divide N
    assert call(name, D(1, T, 4, 16, 16, 8)) == m2.M2RNN_EINVAL
    assert call(name, D(1, T, 4, 16, 16, -1)) == m2.M2RNN_EINVAL
    assert call(name, D(1, T, 2, 16, 48)) == m2.M2RNN_EUNSUPPORTED       # V
    assert call(name, D(1, T, 2, 24, 16)) == m2.M2RNN_EUNSUPPORTED       # K not a multiple of 16
    assert call(name, D(1, T, 2, 144, 16)) == m2.M2RNN_EUNSUPPORTED      # K > 128
    assert call(name, D(1 << 20, T, 1 << 10, 16, 16)) == m2.M2RNN_EUNSUPPORTED  # too many pairs
    big = {"q": "q", "k": "q", "v": "q", "y": "q", "H_out": "q", "ckpt": "q", "dy": "q", "dq": "q", "dv": "q"}
    names = {"fwd": "qkvy", "fwd_ckpt": ("q", "v", "y", "ckpt"), "bwd": ("q", "v", "ckpt", "dy", "dq", "dv"),
             "step": ("q", "v", "y", "H_out")}[name]
    for n in names:
        assert n in big
        assert call(name, D(1, T, 2, 16, 16), bad={n: None}) == m2.M2RNN_EINVAL, n
        assert call(name, D(1, T, 2, 16, 16), bad={n: P(264)}) == m2.M2RNN_EINVAL, n   # 16-byte alignment
    for n in ("a", "alpha", "beta"):
        assert call(name, D(1, T, 2, 16, 16), bad={n: None}) == m2.M2RNN_EINVAL, n
        assert call(name, D(1, T, 2, 16, 16), bad={n: P(258)}) == m2.M2RNN_EINVAL, n
    assert call(name, D(0, T, 0, 16, 16)) == m2.M2RNN_OK


def test_steps_and_state_overlap():
    assert call("step", D(2, 2, 2, 16, 16)) == m2.M2RNN_EINVAL           # T must be 1
    assert call("step", D(2, 0, 2, 16, 16)) == m2.M2RNN_EINVAL
    assert call("step", D(2, 1, 2, 16, 16), bad={"H_in": P(1 << 20), "H_out": P((1 << 20) + 256)}) == m2.M2RNN_EINVAL


def test_workspaces():
    n = ctypes.c_size_t(0)
    L = m2.lib()
    one = D(16, 4096, 64, 64, 64)      # enough pairs to fill the chip: no segments, no workspace
    assert L.m2rnn_ssm_fwd_workspace_size(ctypes.byref(one), 1, ctypes.byref(n)) == 0 and n.value == 0
    few = D(1, 4096, 2, 64, 64)       # time segments, whose entering states need room
    assert L.m2rnn_ssm_fwd_workspace_size(ctypes.byref(few), 1, ctypes.byref(n)) == 0
    assert n.value >= 2 * 2 * 64 * 64 * 4
    assert call("fwd", few, 1, nbytes=n.value - 1) == m2.M2RNN_EWORKSPACE
    assert call("fwd", few, 1, ws=False) == m2.M2RNN_EWORKSPACE
    assert L.m2rnn_ssm_bwd_workspace_size(ctypes.byref(few), 1, ctypes.byref(n)) == 0
    assert n.value >= 2 * 64 * 64 * 64 * 4
    assert call("bwd", few, 1, nbytes=n.value - 1) == m2.M2RNN_EWORKSPACE
    assert call("bwd", few, 1, ws=False) == m2.M2RNN_EWORKSPACE
    assert L.m2rnn_ssm_bwd_workspace_size(ctypes.byref(few), 1, None) == m2.M2RNN_EINVAL
    assert L.m2rnn_ssm_fwd_workspace_size(None, 1, ctypes.byref(n)) == m2.M2RNN_EINVAL


def test_sizes_that_no_launch_holds():
    n = ctypes.c_size_t(0)
    L = m2.lib()
    size = lambda *d, dt=1: L.m2rnn_ssm_bwd_workspace_size(ctypes.byref(D(*d)), dt, ctypes.byref(n))  # noqa: E731
    # 2^24 workgroups of the backward, one for each query/key head and chunk
    assert call("bwd", D(1 << 8, 1 << 16, 64, 16, 16), 1) == m2.M2RNN_EUNSUPPORTED
    assert size(1 << 8, 1 << 16, 64, 16, 16) == m2.M2RNN_EUNSUPPORTED
    assert size(1 << 8, 1 << 16, 32, 16, 16) == m2.M2RNN_OK
    assert size(1 << 8, 1 << 16, 32, 16, 16, dt=0) == m2.M2RNN_EUNSUPPORTED  # chunks of half the length
    assert size(1 << 8, 1 << 16, 64, 16, 16, 32) == m2.M2RNN_OK
    # rows of its partial sums
    assert size(1 << 11, 1 << 17, 1, 16, 16) == m2.M2RNN_EUNSUPPORTED
    assert size((1 << 11) - 1, 1 << 17, 1, 16, 16) == m2.M2RNN_OK
    assert L.m2rnn_ssm_fwd_workspace_size(ctypes.byref(D(1 << 11, 1 << 17, 1, 16, 16)), 1, ctypes.byref(n)) == 0
    assert L.m2rnn_ssm_fwd_workspace_size(ctypes.byref(D(1, 1, (1 << 20) + 1, 16, 16)), 1,
                                          ctypes.byref(n)) == m2.M2RNN_EUNSUPPORTED


def test_checkpoint_interval():
    assert m2.ssm_checkpoint_interval(m2.DTYPE_BF16) == 64 and m2.ssm_checkpoint_interval(m2.DTYPE_F32) == 32
    n = ctypes.c_int64(0)
    assert m2.lib().m2rnn_ssm_checkpoint_interval(9, ctypes.byref(n)) == m2.M2RNN_EINVAL


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    q, v, a = torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 4, 16), torch.zeros(1, 4, 4)
    n = torch.zeros(4)
    with pytest.raises(ValueError):  # on the CPU
        m2.m2rnn_ssm_fwd(q, q, v, a, n, n, torch.zeros(4, 16))
    with pytest.raises(ValueError):  # 3 query/key heads for 4 heads
        m2.m2rnn_ssm_fwd(torch.zeros(1, 4, 3, 16), torch.zeros(1, 4, 3, 16), v, a, n, n, torch.zeros(4, 16))
    with pytest.raises(ValueError):
        m2.m2rnn_ssm_step(q, q, v, a, n, n, torch.zeros(4, 16))


def test_binding_refuses_foreign_streams_and_workspaces():
    torch = pytest.importorskip("torch")

    class Stream:
        device = torch.device("cuda", 0)
        cuda_stream = 0
    with pytest.raises(ValueError):  # a stream of another device than the inputs'
        m2._call_on(torch.device("cuda", 1), Stream())
    cpu = torch.device("cpu")
    assert m2._workspace(0, cpu, None) is None
    assert m2._workspace(16, cpu, torch.empty(16, dtype=torch.uint8)).numel() == 16
    for bad in (torch.empty(15, dtype=torch.uint8), torch.empty(1).expand(100), torch.empty(64, 2)[:, 0]):
        with pytest.raises(ValueError):  # too small, or more elements than bytes behind them
            m2._workspace(16, cpu, bad)
    with pytest.raises(ValueError):  # on the host, for inputs on a GPU
        m2._workspace(16, torch.device("cuda", 0), torch.empty(64))
