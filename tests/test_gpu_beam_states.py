"""beam_reorder_states and beam_backtrace against plain indexing: copies, so
every bit must be equal (needs an MI355X)."""

import numpy as np
import pytest

from tests import beam_ref
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


def filled(torch, shape, dtype, seed):
    g = np.random.default_rng(seed)
    n = int(np.prod(shape))
    es = torch.empty(0, dtype=dtype).element_size()
    raw = torch.from_numpy(g.integers(0, 256, n * es, dtype=np.uint8))
    return raw.cuda().view(dtype).view(shape)


def bits(t):
    es = t.element_size()
    import torch

    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[es]).cpu().numpy()


def parents_of(N, K, seed, invalid=True):
    rng = np.random.default_rng(seed)
    p = rng.integers(0, K, (N, K)).astype(np.int32)
    if invalid and K > 1:
        p[rng.random((N, K)) < 0.15] = -1
        p[0, 0] = K
    return p


CASES = [
    # N, K, shape around the rows (R), dtype, batch_dim, seq_dim
    (1, 2, ("R", 1), "float32", 0, None),
    (3, 4, ("R", 2, 33, 64), "bfloat16", 0, 2),
    (2, 3, ("R", 17, 5, 40), "float16", 0, 1),
    (2, 5, (3, "R", 19, 3, 75), "float32", 1, 2),
    (1, 8, (2, 3, "R", 2, 9, 8), "bfloat16", 2, -2),
    (2, 16, ("R", 50, 24), "float32", 0, 1),
    (1, 17, ("R", 31, 2, 16), "bfloat16", 0, 1),
    (2, 32, ("R", 6, 10, 32), "float16", 0, 2),
    (1, 33, ("R", 12, 16), "float32", 0, 1),
    (1, 128, ("R", 40, 8), "bfloat16", 0, 1),
    (2, 4, ("R", 7, 3), "bfloat16", 0, 1),  # runs of 6 bytes
    (2, 4, ("R", 13, 5), "uint8", 0, 1),  # of 5 bytes
    (1, 70, ("R", 9, 3), "uint8", 0, 1),
    (2, 6, (11, "R", 7), "int64", 1, 0),  # positions in front of the rows
    (2, 4, (5, 8, "R"), "int32", 2, 0),  # the rows lie side by side
    (40, 3, ("R", 300), "float32", 0, 1),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_reorder(case):
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, shape, dtype, bd, sd = case
    shape = tuple(N * K if s == "R" else s for s in shape)
    parents = parents_of(N, K, 1)
    dev_p = torch.from_numpy(parents).cuda()
    for lengths in ([None] if sd is None else [None, "ragged"]):
        if lengths is not None:
            T = shape[sd]
            lengths = np.random.default_rng(3).integers(0, T + 1, N).astype(np.int32)
            lengths[0] = T - 1
            lengths[-1] = T + 5
        state = filled(torch, shape, getattr(torch, dtype), 7)
        want = beam_ref.reorder(bits(state), parents, bd, sd, lengths)
        dev_l = None if lengths is None else torch.from_numpy(lengths).cuda()
        got = tk.beam_reorder_states(state, dev_p, batch_dim=bd, seq_dim=sd, lengths=dev_l)
        torch.cuda.synchronize()
        assert got is state
        assert np.array_equal(bits(state), want)
    say(f"reorder {case}")


def test_reorder_views_and_lists():
    """Views of padded and fused buffers: only the views change. More states
    than a launch takes, of several shapes; a state given twice is moved twice."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K = 2, 4
    R = N * K
    parents = parents_of(N, K, 5)
    dev_p = torch.from_numpy(parents).cuda()
    lengths = np.array([5, 9], np.int32)
    dev_l = torch.from_numpy(lengths).cuda()
    buf = filled(torch, (R + 2, 2, 3, 12, 40), torch.bfloat16, 1)
    raw = bits(buf).copy()
    views = [buf[1:R + 1, 0, :, :11, 3:35], buf[1:R + 1, 1, :, :11, 3:35]]  # keys and values in one buffer
    want = raw.copy()
    for j in range(2):
        want[1:R + 1, j, :, :11, 3:35] = beam_ref.reorder(raw[1:R + 1, j, :, :11, 3:35], parents, 0, 2, lengths)
    tk.beam_reorder_states(views, dev_p, seq_dim=2, lengths=dev_l)
    torch.cuda.synchronize()
    assert np.array_equal(bits(buf), want)

    base = filled(torch, (R, 3, 10, 8), torch.float32, 2)
    flipped = base.permute(3, 0, 2, 1)  # any order of axes
    want = beam_ref.reorder(bits(base), parents, 0)
    tk.beam_reorder_states(flipped, dev_p, batch_dim=1)
    torch.cuda.synchronize()
    assert np.array_equal(bits(base), want)

    states = [filled(torch, (R, 2, 11, 8 * (1 + i % 3)), torch.float16, i) for i in range(53)]
    states.append(torch.empty((R, 2, 0, 8), dtype=torch.float16, device="cuda"))
    want = [beam_ref.reorder(bits(s), parents, 0, 2, lengths) for s in states]
    tk.beam_reorder_states(states, dev_p, seq_dim=-2, lengths=dev_l)
    torch.cuda.synchronize()
    assert all(np.array_equal(bits(s), w) for s, w in zip(states, want))

    one = filled(torch, (R, 500), torch.float32, 9)
    twice = beam_ref.reorder(beam_ref.reorder(bits(one), parents, 0), parents, 0)
    tk.beam_reorder_states([one, one], dev_p)
    torch.cuda.synchronize()
    assert np.array_equal(bits(one), twice)


def test_reorder_graph_and_streams():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K = 3, 5
    parents = torch.zeros((N, K), dtype=torch.int32, device="cuda")
    state = filled(torch, (N * K, 4, 33, 16), torch.bfloat16, 1)
    now = bits(state).copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tk.beam_reorder_states(state, parents)
    for i in range(4):
        p = parents_of(N, K, i)
        parents.copy_(torch.from_numpy(p))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        now = beam_ref.reorder(now, p, 0)
        assert np.array_equal(bits(state), now)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    tk.beam_reorder_states(state, parents, stream=st)
    st.synchronize()
    assert np.array_equal(bits(state), beam_ref.reorder(now, p, 0))


TRACES = [
    # T, N, K, M
    (1, 1, 1, 1),
    (2, 3, 2, 5),
    (31, 2, 4, 4),
    (32, 1, 3, 2),
    (33, 2, 5, 7),
    (100, 4, 4, 4),
    (700, 3, 8, 33),
    (2048, 2, 8, 8),
    (2500, 1, 128, 40),  # more than one piece
    (40000, 1, 2, 3),
    (5, 70, 6, 1),
]


@pytest.mark.parametrize("shape", TRACES, ids=[str(s) for s in TRACES])
def test_backtrace(shape):
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    T, N, K, M = shape
    rng = np.random.default_rng(T)
    tokens = rng.integers(0, 50000, (T, N, K)).astype(np.int32)
    parents = rng.integers(0, K, (T, N, K)).astype(np.int32)
    beams = rng.integers(0, K, (N, M)).astype(np.int32)
    lengths = rng.integers(0, T + 1, (N, M)).astype(np.int32)
    lengths[0, 0] = T + 3
    d = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    broken = parents.copy()
    broken[rng.random((T, N, K)) < 0.5 / T] = -1
    broken[0] = 1000000  # not followed
    wild = beams.copy()
    wild[0, 0], wild[-1, -1] = -1, K
    for p, b, le in ((parents, beams, lengths), (parents, beams, None), (broken, wild, lengths),
                     (broken, None, None), (broken, None, lengths[:, :K] if M >= K else lengths)):
        pad = -1 if le is None else 7
        got = tk.beam_backtrace(d(tokens), d(p), d(b), d(np.ascontiguousarray(le) if le is not None else None), pad)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), beam_ref.backtrace(tokens, p, b, le, pad))
    say(f"backtrace {shape}")


def test_backtrace_ends_around_pieces():
    """A history longer than a workgroup holds is taken in pieces from its end;
    paths that end at every step near where one piece meets the next."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    T, N, K = 1267, 2, 86
    rng = np.random.default_rng(4)
    tokens = rng.integers(0, 50000, (T, N, K)).astype(np.int32)
    parents = rng.integers(0, K, (T, N, K)).astype(np.int32)
    lengths = np.stack([np.r_[140:220, 690:780], np.r_[1097:1267]]).astype(np.int32)
    beams = rng.integers(0, K, lengths.shape).astype(np.int32)
    got = tk.beam_backtrace(*(torch.from_numpy(a).cuda() for a in (tokens, parents, beams, lengths)))
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), beam_ref.backtrace(tokens, parents, beams, lengths))


def test_backtrace_out_and_graph():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    T, N, K = 90, 3, 4
    rng = np.random.default_rng(1)
    tokens, parents = (torch.from_numpy(rng.integers(0, K, (T, N, K)).astype(np.int32)).cuda() for _ in range(2))
    big = torch.full((N * K * T + 64,), 5, dtype=torch.int32, device="cuda")
    out = big[32:-32].view(N, K, T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tk.beam_backtrace(tokens, parents, out=out)
    for i in range(3):
        out.fill_(0)
        tokens.add_(1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), beam_ref.backtrace(tokens.cpu().numpy(), parents.cpu().numpy()))
    assert bool((big[:32] == 5).all()) and bool((big[-32:] == 5).all())


def test_backtrace_of_many_prompts():
    """More prompts than one grid holds workgroups."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    T, N, K = 2, (1 << 21) + 5, 2
    rng = np.random.default_rng(6)
    tokens = rng.integers(0, 50000, (T, N, K)).astype(np.int32)
    parents = rng.integers(-1, K, (T, N, K)).astype(np.int32)
    got = tk.beam_backtrace(torch.from_numpy(tokens).cuda(), torch.from_numpy(parents).cuda())
    torch.cuda.synchronize()
    first = np.take_along_axis(tokens[0], np.maximum(parents[1], 0), 1)
    want = np.stack([np.where(parents[1] < 0, -1, first), tokens[1]], 2)
    assert np.array_equal(got.cpu().numpy(), want)


def test_reorder_counts_as_a_modification():
    """A state saved for a backward pass must not change unnoticed; a parameter
    may be reordered under no_grad, as may tensors of inference mode."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K = 2, 3
    parents = torch.tensor([[1, 0, 2], [0, 0, 0]], dtype=torch.int32, device="cuda")
    x = torch.ones((N * K, 4), device="cuda", requires_grad=True)
    states = [torch.rand((N * K, 4), device="cuda"), torch.rand((N * K, 4), device="cuda")]
    before = [s._version for s in states]
    y = (x * states[1]).sum()
    tk.beam_reorder_states(states, parents)
    assert all(s._version > v for s, v in zip(states, before))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    base = torch.rand((N * K, 8), device="cuda")
    seen = base._version
    tk.beam_reorder_states(base[:, :4], parents)
    assert base._version > seen  # a view's memory is its base's
    tk.beam_reorder_states([], parents)

    leaf = torch.rand((N * K, 4), device="cuda", requires_grad=True)
    now, want = leaf._version, beam_ref.reorder(leaf.detach().cpu().numpy(), parents.cpu().numpy(), 0)
    with pytest.raises(ValueError, match="requires grad"):
        tk.beam_reorder_states(leaf, parents)
    with torch.no_grad():
        tk.beam_reorder_states(leaf, parents)
    assert leaf._version > now and np.array_equal(leaf.detach().cpu().numpy(), want)
    with torch.inference_mode():
        cache = torch.rand((N * K, 4), device="cuda")
        want = beam_ref.reorder(cache.cpu().numpy(), parents.cpu().numpy(), 0)
        tk.beam_reorder_states(cache, parents)
    assert np.array_equal(cache.cpu().numpy(), want)
    tk.beam_reorder_states(cache, parents)  # and outside of it
    torch.cuda.synchronize()
    assert np.array_equal(cache.cpu().numpy(), beam_ref.reorder(want, parents.cpu().numpy(), 0))


@pytest.mark.parametrize("K", [4, 8, 12, 128])
def test_backtrace_of_unaligned_histories(K):
    """Numbers of beams that are read four at a time, in histories that begin at
    any multiple of 4 bytes."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    T, N, M = 75, 3, 9
    rng = np.random.default_rng(K)
    tokens = rng.integers(0, 50000, (T, N, K)).astype(np.int32)
    parents = rng.integers(-1, K + 1, (T, N, K)).astype(np.int32)
    parents[rng.random((T, N, K)) < 0.8] = 1
    beams = rng.integers(0, K, (N, M)).astype(np.int32)
    lengths = rng.integers(0, T + 1, (N, M)).astype(np.int32)
    want = beam_ref.backtrace(tokens, parents, beams, lengths)
    for shift in range(5):
        buf = torch.full((2, T * N * K + 8), 10 ** 9, dtype=torch.int32, device="cuda")
        history = [b[shift:shift + T * N * K].view(T, N, K) for b in buf]
        for view, a in zip(history, (tokens, parents)):
            view.copy_(torch.from_numpy(a))
        assert history[1].data_ptr() % 16 == 4 * shift % 16
        got = tk.beam_backtrace(*history, *(torch.from_numpy(a).cuda() for a in (beams, lengths)))
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), want)


NARROW = [
    # N, K, shape around the rows (R), bytes, seq_dim
    (3, 4, ("R", 4, 64, 515), 2, 3),  # keys held transposed, an odd number of positions
    (3, 4, ("R", 4, 64, 512), 2, 3),
    (3, 4, ("R", 2, 64, 513), 1, 3),
    (3, 4, ("R", 4, 300, 75), 2, 2),  # an odd head size
    (3, 6, ("R", 300, 3, 75), 2, 1),
    (3, 40, ("R", 999, 6), 2, 1),
    (3, 5, ("R", 70001), 2, 1),  # words by position
    (3, 5, ("R", 4, 200, 33), 4, 2),
]


@pytest.mark.parametrize("case", NARROW, ids=[str(c) for c in NARROW])
def test_reorder_of_narrow_runs(case):
    """States whose positions are a few bytes that follow each other, at more
    than a workgroup's size, with lengths that end at every byte of a word."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, shape, es, sd = case
    shape = tuple(N * K if s == "R" else s for s in shape)
    dtype = {1: torch.uint8, 2: torch.bfloat16, 4: torch.float32}[es]
    parents = parents_of(N, K, 2)
    dev_p = torch.from_numpy(parents).cuda()
    T = shape[sd]
    start = filled(torch, shape, dtype, 11)
    for least in range(0, 18, 3):
        lengths = np.array([T - 1 - least, T // 2 + least, least], np.int32)
        state = start.clone()
        want = beam_ref.reorder(bits(state), parents, 0, sd, lengths)
        tk.beam_reorder_states(state, dev_p, seq_dim=sd, lengths=torch.from_numpy(lengths).cuda())
        torch.cuda.synchronize()
        assert np.array_equal(bits(state), want), lengths
    say(f"reorder {case}")
