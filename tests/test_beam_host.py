"""The beam search entry points without a GPU: arguments that the library and
the binding refuse, workspace sizes, and how the binding describes a state."""

import ctypes
import itertools

import numpy as np
import pytest
import torch

import top_logits_filtering_amd as tk
from tests import beam_ref
from top_logits_filtering_amd.binding import BeamState, _state_layout

NULLPTR, INVALID = 1, 2
FAKE = 1 << 40  # a device-looking address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    import os

    from top_logits_filtering_amd.binding import LIB_PATH

    if not os.path.exists(LIB_PATH):
        from top_logits_filtering_amd.build import build

        build()
    return tk.load_library()


def select(lib, **kw):
    a = dict(x=FAKE, ld=100, dt=0, N=2, K=3, V=100, c=FAKE + (1 << 30), done=None, end=0, w=None, n=4,
             s=FAKE + (1 << 31), p=FAKE + (1 << 32), t=FAKE + (1 << 33), ws=FAKE + (1 << 34), size=1 << 20)
    a.update(kw)
    return lib.beam_search_select(a["x"], a["ld"], a["dt"], a["N"], a["K"], a["V"], a["c"], a["done"], a["end"],
                                  a["w"], a["n"], a["s"], a["p"], a["t"], a["ws"], a["size"], None)


def test_select_refusals(lib):
    for name, word in (("x", "logits"), ("c", "scores"), ("s", "out_scores"), ("p", "out_parents"),
                       ("t", "out_tokens"), ("ws", "workspace")):
        assert select(lib, **{name: None}) == NULLPTR
        assert word in tk.last_error()
    for kw, word in (
        (dict(dt=3), "dtype"), (dict(N=-1), "negative"), (dict(K=0), "beams"), (dict(K=129), "beams"),
        (dict(N=1 << 31), "maximum"), (dict(N=1 << 62, K=128), "maximum"), (dict(V=-1), "negative"),
        (dict(V=(1 << 20) + 1, ld=1 << 21), "maximum"), (dict(n=0), "n=0"), (dict(n=257), "n=257"),
        (dict(ld=99), "stride"), (dict(ld=1 << 40), "stride"), (dict(done=FAKE + (1 << 35), end=-1), "end_token"),
        (dict(x=FAKE + 2), "aligned"), (dict(ws=FAKE + (1 << 34) + 8), "aligned"), (dict(size=15), "workspace"),
        (dict(s=FAKE + 400), "overlap"), (dict(p=FAKE + (1 << 31) + 28), "overlap"),
        (dict(t=FAKE + (1 << 34) + 4), "overlap"), (dict(ws=FAKE + (1 << 30)), "overlap"),
        (dict(w=FAKE + (1 << 33)), "overlap"),
        (dict(done=FAKE + (1 << 32) + 31), "overlap"),
    ):
        assert select(lib, **kw) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    need = lib.beam_search_select_workspace(0, 2, 3, 100, 4)
    assert select(lib, size=need - 1) == INVALID and str(need) in tk.last_error()
    assert select(lib, N=0, x=None, c=None, s=None, p=None, t=None, ws=None) == 0
    assert select(lib, N=0, dt=9) == INVALID


def test_select_workspace(lib):
    f = lib.beam_search_select_workspace
    for bad in ((7, 1, 1, 10, 1), (0, -1, 1, 10, 1), (0, 1, 0, 10, 1), (0, 1, 1, 1 << 21, 1), (0, 1, 1, 10, 0)):
        assert f(*bad) == -1 and tk.last_error()
    assert f(0, 0, 1, 10, 1) >= 16
    assert tk.beam_search_select_workspace(torch.bfloat16, 64, 4, 151936, 8) == f(2, 64, 4, 151936, 8)
    assert tk.beam_search_select_workspace(torch.bfloat16, 64, 4, 151936) == f(2, 64, 4, 151936, 4)
    with pytest.raises(tk.TopKTopPError):
        tk.beam_search_select_workspace(torch.float32, 1, 200, 10)
    # the largest sizes stay within an int64 and grow with n
    assert 0 < f(0, (1 << 31) // 128 - 1, 128, 1 << 20, 1) < f(0, (1 << 31) // 128 - 1, 128, 1 << 20, 256)


def state(**kw):
    a = dict(data=FAKE, row_stride=4096, size=(1, 1, 2), stride=(1, 1, 2048), positions=8, position_stride=256,
             run=256)
    a.update(kw)
    s = BeamState()
    for k, v in a.items():
        if k in ("size", "stride"):
            getattr(s, k)[:] = v
        else:
            setattr(s, k, v)
    return s


def reorder(lib, states, parents=FAKE + (1 << 36), N=2, K=4, lengths=None, count=None):
    arr = (BeamState * max(1, len(states)))(*states)
    return lib.beam_reorder_states(arr, len(states) if count is None else count, parents, N, K, lengths, None)


def test_reorder_refusals(lib):
    assert lib.beam_reorder_states(None, 1, FAKE, 2, 4, None, None) == NULLPTR
    assert reorder(lib, [state()], parents=None) == NULLPTR
    assert reorder(lib, [state(data=None)]) == NULLPTR and "state 0" in tk.last_error()
    for kw, word in (
        (dict(run=-1), "negative"), (dict(size=(1, -1, 2)), "negative"), (dict(positions=-2), "negative"),
        (dict(row_stride=4095), "share memory"), (dict(row_stride=0), "share memory"),
        (dict(row_stride=-4096), "share memory"), (dict(stride=(1, 1, 2047)), "share memory"),
        (dict(position_stride=255), "share memory"), (dict(size=(2, 1, 2), stride=(0, 1, 2048)), "share memory"),
        (dict(row_stride=1 << 50), "2^46"), (dict(size=(1, 1 << 40, 2), stride=(1, 1 << 20, 2048)), "2^46"),
        (dict(data=FAKE + (1 << 36) - 100), "overlaps parents"),
    ):
        assert reorder(lib, [state(), state(**kw)]) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    # single bytes: too many columns in a row
    assert reorder(lib, [state(run=1, positions=1, size=(1, 1, 1 << 32), stride=(1, 1, 3), row_stride=1 << 40)],
                   parents=FAKE - 64) == INVALID and "columns" in tk.last_error()
    assert reorder(lib, [state()], lengths=FAKE + 64) == INVALID and "lengths" in tk.last_error()
    assert reorder(lib, [state()], K=0) == INVALID and reorder(lib, [state()], K=129) == INVALID
    assert reorder(lib, [state()], N=-1) == INVALID and reorder(lib, [state()], N=1 << 31) == INVALID
    assert reorder(lib, [state()], count=-1) == INVALID
    # nothing to do
    assert reorder(lib, []) == 0 and reorder(lib, [state()], N=0, parents=None) == 0
    assert reorder(lib, [state(positions=0), state(run=0), state(size=(1, 0, 2), data=None), BeamState()]) == 0


def test_backtrace_refusals(lib):
    def call(tok=FAKE, par=FAKE + (1 << 32), T=10, N=2, K=4, beams=None, lengths=None, M=4, out=FAKE + (1 << 33)):
        return lib.beam_backtrace(tok, par, T, N, K, beams, lengths, M, -1, out, None)

    assert call(tok=None) == NULLPTR and call(par=None) == NULLPTR and call(out=None) == NULLPTR
    for kw, word in ((dict(T=-1), "T=-1"), (dict(T=1 << 31), "T="), (dict(N=-1), "negative"), (dict(K=0), "beams"),
                     (dict(K=129), "beams"), (dict(M=-1), "M=-1"), (dict(M=5), "exceed"),
                     (dict(M=(1 << 20) + 1, beams=FAKE + (1 << 34)), "M="), (dict(out=FAKE + 316), "overlap"),
                     (dict(lengths=FAKE + (1 << 33) + 319), "overlap")):
        assert call(**kw) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    for kw in (dict(T=0), dict(N=0), dict(M=0)):
        assert call(tok=None, par=None, out=None, **kw) == 0


def test_binding_refusals():
    x = torch.zeros(6, 10, dtype=torch.float16)
    c = torch.zeros(2, 3)
    i32 = dict(dtype=torch.int32)
    ok_out = (torch.zeros(2, 4), torch.zeros(2, 4, **i32), torch.zeros(2, 4, **i32))
    for err, args, kw in (
        (ValueError, (x[0], c), {}), (ValueError, (x, c[0]), {}), (ValueError, (x[:5], c), {}),
        (TypeError, (x, c.half()), {}), (TypeError, (x.int(), c), {}), (ValueError, (x, c.t().contiguous().t()), {}),
        (TypeError, (x, c), dict(finished=c, end_token=1)),
        (ValueError, (x, c), dict(finished=torch.zeros(2, 3, dtype=torch.bool))),
        (ValueError, (x, c), dict(finished=torch.zeros(3, 2, dtype=torch.bool), end_token=1)),
        (ValueError, (x, c), dict(finished=torch.zeros(2, 3, dtype=torch.bool), end_token=2 ** 31)),
        (ValueError, (x, c), dict(finished=torch.zeros(2, 3, dtype=torch.bool), end_token=-1)),
        (TypeError, (x, c), dict(weights=c.double())), (ValueError, (x, c), dict(weights=torch.zeros(2, 4))),
    ):
        with pytest.raises(err):
            tk.beam_search_select(*args, 4, out=ok_out, **kw)
    with pytest.raises(ValueError, match="GPU"):
        tk.beam_search_select(x, c, 4, out=ok_out)

    s, p = torch.zeros(6, 5, 2), torch.zeros(2, 3, **i32)
    for err, args, kw in (
        (TypeError, (s, p.long()), {}), (ValueError, (s, p[0]), {}),
        (ValueError, (s, p), dict(lengths=torch.zeros(2, **i32))),
        (TypeError, (s, p), dict(lengths=torch.zeros(2), seq_dim=1)),
        (ValueError, (s, p), dict(lengths=torch.zeros(3, **i32), seq_dim=1)),
    ):
        with pytest.raises(err):
            tk.beam_reorder_states(*args, **kw)
    with pytest.raises(ValueError, match="GPU"):
        tk.beam_reorder_states(s, p)

    h = torch.zeros(5, 2, 3, **i32)
    for err, args, kw in (
        (ValueError, (h[0], h[0]), {}), (TypeError, (h.long(), h), {}), (ValueError, (h, h[:4]), {}),
        (ValueError, (h, h), dict(beams=torch.zeros(2, **i32))),
        (ValueError, (h, h), dict(beams=torch.zeros(2, 4, **i32), lengths=torch.zeros(2, 3, **i32))),
        (TypeError, (h, h), dict(lengths=torch.zeros(2, 4))),
        (ValueError, (h, h), dict(pad=2 ** 31)), (ValueError, (h, h), dict(pad=-2 ** 31 - 1)),
    ):
        with pytest.raises(err):
            tk.beam_backtrace(*args, **kw)
    with pytest.raises(ValueError, match="GPU"):
        tk.beam_backtrace(h, h)


@pytest.mark.parametrize("shape,view", [
    ((6, 4, 7, 8), lambda t: t),
    ((6, 4, 7, 8), lambda t: t[:, 1:3, :5, 2:6]),
    ((3, 6, 4, 7, 8), lambda t: t.permute(1, 0, 3, 2, 4)),
    ((6, 9, 5), lambda t: t.transpose(1, 2)),
    ((6, 2, 3, 4, 5), lambda t: t[:, :, ::2, :, ::2]),
    ((6, 1, 1, 1), lambda t: t),
])
@pytest.mark.parametrize("seq", [None, 2])
def test_state_layout_addresses_every_element(shape, view, seq):
    """The description's bytes are exactly the view's, each at its own row and position."""
    t = view(torch.arange(int(np.prod(shape)), dtype=torch.int32).view(shape))
    row_stride, size, stride, positions, position_stride, run = _state_layout(tuple(t.shape), t.stride(), 4, 0, seq)
    flat = torch.arange(int(np.prod(shape)))
    for r in range(t.shape[0]):
        seen = []
        for pos in range(positions):
            here = []
            for i in itertools.product(*(range(n) for n in size)):
                at = r * row_stride + sum(a * b for a, b in zip(i, stride)) + pos * position_stride
                assert at % 4 == 0 and run % 4 == 0
                here += flat[t.storage_offset() + at // 4:][:run // 4].tolist()
            if seq is not None:
                assert sorted(here) == sorted(t[r].select(seq - 1, pos).reshape(-1).tolist())
            seen += here
        assert sorted(seen) == sorted(t[r].reshape(-1).tolist())
    real = [s for s, n in zip(stride, size) if n != 1]
    assert real == sorted(real, reverse=True) and list(size)[:3 - len(real)] == [1] * (3 - len(real))


def test_state_layout_joins_axes():
    # [rows, heads, positions, dim] without lengths is one run; with them, heads stay apart
    assert _state_layout((8, 4, 16, 32), (2048, 512, 32, 1), 2, 0, None)[-1] == 4096
    row, size, stride, positions, step, run = _state_layout((8, 4, 16, 32), (2048, 512, 32, 1), 2, 0, 2)
    assert (row, size[2], stride[2], positions, step, run) == (4096, 4, 1024, 16, 64, 64)
    with pytest.raises(ValueError, match="separate axes"):
        _state_layout((2, 3, 3, 3, 3, 3), (10 ** 6, 10 ** 5, 10 ** 4, 10 ** 3, 100, 10), 4, 0, None)


def test_plain_forms_by_hand():
    """The tests' own reference on a case small enough to follow."""
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.1, 0.8]]))
    c = np.log(np.array([[0.6, 0.4]]))
    s, p, t = beam_ref.select(x, c, 4)
    assert p.tolist() == [[1, 0, 0, 0]] and t.tolist() == [[2, 0, 1, 2]]
    assert np.allclose(np.exp(s), [[0.32, 0.3, 0.15, 0.15]])
    s, p, t = beam_ref.select(x, c, 3, finished=np.array([[False, True]]), end_token=9)
    assert p.tolist() == [[1, 0, 0]] and t.tolist() == [[9, 0, 1]] and np.allclose(np.exp(s), [[0.4, 0.3, 0.15]])
    parents = np.array([[[0, 1, 2]], [[0, 0, 1]], [[2, 0, 2]]], np.int32)
    tokens = np.arange(9, dtype=np.int32).reshape(3, 1, 3)
    assert beam_ref.backtrace(tokens, parents).tolist() == [[[1, 5, 6], [0, 3, 7], [1, 5, 8]]]
    assert beam_ref.reorder(np.array([[1], [2], [3]]), np.array([[2, 0, -1]]), 0).tolist() == [[3], [1], [3]]
    assert ctypes.sizeof(BeamState) == 88


def test_reorder_refuses_states_that_record_gradients():
    leaf = torch.zeros(6, 5, requires_grad=True)
    parents = torch.zeros(2, 3, dtype=torch.int32)
    for state in (leaf, leaf[:, :3], leaf * 2, [torch.zeros(6, 2), leaf]):
        with pytest.raises(ValueError, match="requires grad"):
            tk.beam_reorder_states(state, parents)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # that of tensors on the CPU
            tk.beam_reorder_states(state, parents)
