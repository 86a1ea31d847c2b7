"""beam_search_select against the plain implementation in 64 bits (needs an
MI355X). Parents and tokens must be equal. Scores: a sum of exp is off by at most
3.5e-7 of itself (hardware exp2 8.5e-8, measured over all arguments that occur;
three additions in fp32 at 2^-24 = 6.0e-8 each, and a multiply-add at as much or,
for 16-bit logits, 1e-8 of a series that is cut short; everything else is in 64
bits and below 1e-9), so its logarithm is by less than 3.6e-7; the score is
rounded once to fp32, by at most 2^-24 of its value."""

import numpy as np
import pytest

from tests import beam_ref
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu

SUM_ERROR = 3.6e-7
DTYPES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def make(torch, rows, V, dtype, seed, ld=None, offset=0, scale=3.0):
    """Logits [rows, V] as a view with row stride ld that starts `offset`
    elements into its buffer; the buffer's other elements are NaN."""
    ld = V if ld is None else ld
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((rows, V)) * scale).astype(np.float32)).to(getattr(torch, DTYPES[dtype]))
    buf = torch.full((offset + rows * ld + 16,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :V] if rows * ld else buf[:0].view(rows, V)
    view.copy_(x)
    return view


def check(torch, logits, scores, n, finished=None, end=0, weights=None, **kw):
    import top_logits_filtering_amd as tk

    dev = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t)  # noqa: E731
    got = tk.beam_search_select(logits, dev(scores, torch.float32), n, finished=dev(finished, torch.bool),
                                end_token=end, weights=dev(weights, torch.float32), **kw)
    torch.cuda.synchronize()
    ref = beam_ref.select(logits.double().cpu().numpy(), scores, n, finished, end, weights)
    s, p, t = (v.cpu().numpy() for v in got)
    assert np.array_equal(p, ref[1]), (p, ref[1])
    assert np.array_equal(t, ref[2]), (t, ref[2])
    gone = np.isneginf(ref[0])
    assert np.array_equal(np.isneginf(s[gone]), np.ones(gone.sum(), bool))
    with np.errstate(over="ignore"):
        want = ref[0].astype(np.float32)
    inf = np.isinf(want) & ~gone  # rounds to -inf in fp32
    assert np.array_equal(s[inf], want[inf])
    fine = ~gone & ~inf
    err = np.abs(s[fine].astype(np.float64) - ref[0][fine])
    assert np.all(err <= 2.0 ** -24 * np.abs(ref[0][fine]) + SUM_ERROR), err.max()
    return got


def beam_scores(N, K, seed):
    rng = np.random.default_rng(seed + 1000)
    return -(5 + np.cumsum(rng.exponential(0.7, (N, K)), 1)).astype(np.float32)


SHAPES = [
    # N, K, V, n, ld - V, offset
    (1, 1, 1, 1, 0, 0),
    (2, 3, 1, 4, 0, 1),
    (2, 3, 5, 4, 0, 0),
    (3, 2, 7, 20, 1, 3),  # fewer continuations than ranks
    (1, 4, 1000, 8, 0, 0),
    (4, 4, 2048, 8, 0, 0),
    (2, 5, 2049, 3, 6, 1),
    (3, 7, 4099, 13, 0, 5),  # rows at every alignment
    (1, 2, 40001, 16, 3, 2),
    (130, 1, 517, 2, 0, 0),
    (2, 128, 300, 256, 0, 0),  # the widest beams
    (1, 3, 151936, 6, 0, 0),
    (90, 4, 33000, 8, 0, 0),  # enough rows for whole-register chunks
    (1, 1, 1 << 20, 5, 0, 0),
]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_shapes(shape, dtype):
    torch = need_gpu()
    N, K, V, n, more, offset = shape
    x = make(torch, N * K, V, dtype, seed=V + n, ld=V + more, offset=offset)
    check(torch, x, beam_scores(N, K, V), n)
    say(f"select {shape} {dtype}")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_finished_weights_and_dead_beams(dtype):
    torch = need_gpu()
    N, K, V, n = 6, 5, 3001, 12
    rng = np.random.default_rng(5)
    x = make(torch, N * K, V, dtype, seed=9)
    scores = beam_scores(N, K, 3)
    finished = rng.random((N, K)) < 0.4
    finished[0] = True  # nothing but finished beams
    finished[1] = False
    weights = (0.2 + rng.random((N, K))).astype(np.float32)
    x[finished.reshape(-1).nonzero()[0]] = float("nan")  # not read
    check(torch, x, scores, n, finished, end=2, weights=weights)
    scores[2, 1:] = -np.inf  # a search's first step: one live beam
    scores[3] = -np.inf
    scores[4, 0], scores[4, 3] = np.nan, np.inf
    weights[5] = [0.0, -1.0, np.inf, np.nan, 1.0]
    check(torch, x, scores, n, finished, end=2, weights=weights)
    check(torch, x, scores, n, finished, end=V + 7)  # the end token may lie outside the vocabulary
    scores[2, 1:] = -1e9
    scores[3] = np.finfo(np.float32).min
    scores[3, 2] = -1.0
    check(torch, x, scores, n)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [50, 3001, 40000])
def test_masked_logits(V, dtype):
    """Rows that a mask leaves nothing, one token or a few of; masks of -inf
    and of the type's lowest value; NaN and infinities."""
    torch = need_gpu()
    N, K, n = 3, 4, 9
    low = torch.finfo(getattr(torch, DTYPES[dtype])).min
    for fill in (float("-inf"), low):
        x = make(torch, N * K, V, dtype, seed=V)
        rng = np.random.default_rng(V)
        for r, left in enumerate([0, 1, 3, 8, 9, 10, V]):
            gone = torch.from_numpy(rng.permutation(V)[left:]).cuda()
            x[r, gone] = fill
        x[7] = 0.0
        x[8, V // 2] = float("nan")
        x[9, V - 1] = float("inf")
        x[10, 0] = -float("nan")
        check(torch, x, beam_scores(N, K, 1), n)
    x = make(torch, N * K, V, dtype, seed=V, scale=0.01)
    x[0] = float("-inf")
    x[0, V - 1] = low
    x[1] = torch.finfo(x.dtype).max
    x[2, 3] = torch.finfo(x.dtype).max
    x[3] = low
    x[4] -= 20000.0
    x[5] += 20000.0
    x[6, : V // 2] = float("-inf")
    x[6, V // 2:] = low
    x[7] = x[7].abs() * 0 - 0.0
    x[7, ::2] = 0.0  # -0 and +0 are equal
    check(torch, x, beam_scores(N, K, 1), n)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_ties(dtype):
    """Equal logits, equal beams, and values in orders that defeat a bound from
    the threads' maxima."""
    torch = need_gpu()
    for N, K, V, n in [(2, 4, 20000, 16), (1, 1, 9000, 256), (1, 128, 600, 256), (300, 1, 40000, 33)]:
        rows = N * K
        scores = beam_scores(N, K, 2)
        x = make(torch, rows, V, dtype, seed=1)
        x[:] = 1.5  # every continuation of a beam ties
        check(torch, x, scores, n)
        scores[:] = -3.0  # and the beams with each other
        check(torch, x, scores, n)
        x[:] = make(torch, 1, V, dtype, seed=4, scale=0.02)  # equal beams
        check(torch, x, scores, n)
        ramp = torch.linspace(-5, 5, V).to(x.dtype).cuda()
        x[:] = ramp
        check(torch, x, scores, n)
        x[:] = ramp.flip(0)
        check(torch, x, scores, n)
        # all large values in the elements of one thread, many of them equal
        P = 16 // x.element_size()
        at = torch.arange(V, device="cuda")
        mine = (at // P) % 256 == 77
        x[:] = torch.where(mine, 9.0 - (at % 13).float(), -4.0).to(x.dtype)
        check(torch, x, scores, n)
        say(f"ties {N, K, V, n} {dtype}")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [777, 20000])
def test_beams_closer_than_a_32_bit_sum(V, dtype):
    """Candidates of different beams 1e-8 apart, far below what sums in fp32
    tell apart: scores near 0, where fp32 has steps below 1e-9, are chosen so
    that all beams' best candidates lie on a grid of 1e-8 in a random order."""
    torch = need_gpu()
    N, K = 24, 4
    rng = np.random.default_rng(V)
    base = rng.standard_normal(V) * 2
    rows = np.stack([rng.permutation(base) for _ in range(N * K)])
    if dtype == "f32":
        rows += 1e-3 * rng.standard_normal(rows.shape)
    x = make(torch, N * K, V, dtype, seed=0)
    x.copy_(torch.from_numpy(rows.astype(np.float32)))
    xd = x.double().cpu().numpy()
    top = xd.max(1)
    logp = -np.log(np.exp(xd - top[:, None]).sum(1)).reshape(N, K)
    grid = np.stack([rng.permutation(K) for _ in range(N)]) * 1e-8
    scores = (logp.mean() - logp + grid).astype(np.float32)
    assert np.abs(scores).max() < 0.01  # steps of 2^-31
    weights = np.ones((N, K), np.float32)
    for n in (1, 3, 40):
        check(torch, x, scores, n)
        check(torch, x, scores, n, weights=weights * 0.125)
    finished = np.zeros((N, K), bool)
    finished[:, 1] = True
    scores[:, 1] = (logp.mean() + grid[:, 1]).astype(np.float32) * 0  # exact, and close to no other
    check(torch, x, scores, 5, finished, end=3)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_equal_beams_at_unequal_addresses(dtype):
    """Beams with the same logits and scores tie, also where their rows begin at
    different offsets from 16 bytes and are summed in another order."""
    torch = need_gpu()
    N, K, V = 2, 9, 30001
    x = make(torch, N * K, V, dtype, seed=1, ld=V + 6)
    x[:] = x[:1].clone()
    scores = np.full((N, K), -1.25, np.float32)
    check(torch, x, scores, 40)
    x[:] = torch.linspace(-9, 9, V, device="cuda").to(x.dtype)
    check(torch, x, scores, 40)
    scores[:, 4] += 1e-7  # and with one that is a step of fp32 better
    check(torch, x, scores, 40)


def test_outputs_stay_inside():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, V, n = 3, 4, 1111, 7
    x = make(torch, N * K, V, "bf16", seed=2)
    big = [torch.full((N * n + 64,), 77, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    out = tuple(b[32:32 + N * n].view(N, n) for b in big)
    size = tk.beam_search_select_workspace(torch.bfloat16, N, K, V, n)
    ws = torch.full((size + 64,), 77, dtype=torch.uint8, device="cuda")
    got = check(torch, x, beam_scores(N, K, 0), n, out=out, workspace=ws[32:32 + size])
    assert got[0].data_ptr() == out[0].data_ptr()
    for b in big + [ws]:
        edge = torch.cat([b[:32], b[-32:]])
        assert bool((edge == 77).all())


def test_streams_and_graphs():
    """Concurrent calls on several streams; a captured call replayed between
    other work and on new inputs, beside a second graph."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, V, n = 4, 4, 50000, 8
    xs = [make(torch, N * K, V, "bf16", seed=i) for i in range(4)]
    sc = [torch.from_numpy(beam_scores(N, K, i)).cuda() for i in range(4)]
    want = [[t.clone() for t in tk.beam_search_select(x, s, n)] for x, s in zip(xs, sc)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(5):
        for i, st in enumerate(streams):
            got[i].append(tk.beam_search_select(xs[i], sc[i], n, stream=st if i % 2 else st.cuda_stream))
    torch.cuda.synchronize()
    for i in range(4):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))

    graphs, outs = [], []
    x, s = xs[0].clone(), sc[0].clone()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tk.beam_search_select(x, s, n))
        graphs.append(g)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        s.copy_(sc[i])
        torch.cuda.synchronize()
        for g, o in zip(graphs, outs):
            g.replay()
            tk.beam_search_select(xs[3], sc[3], n)
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want[i]))


def test_handle_of_the_default_stream():
    """A stream handle of 0 is the default stream, whichever stream is current."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk
    from top_logits_filtering_amd.binding import _scope

    N, K, V = 2, 3, 5000
    x = make(torch, N * K, V, "f16", seed=8)
    c = torch.from_numpy(beam_scores(N, K, 8)).cuda()
    want = [t.clone() for t in tk.beam_search_select(x, c)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert _scope(None, x.device)[0] == side.cuda_stream != 0
        handle, scope = _scope(0, x.device)
        with scope:
            assert handle == 0 and torch.cuda.current_stream() == torch.cuda.default_stream()
        got = tk.beam_search_select(x, c, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_workspace_for_successive_calls():
    """It holds nothing between calls: calls of several shapes take the same one in turn."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    shapes = [(3, 4, 9001, 8, "bf16"), (1, 2, 40001, 16, "f32"), (2, 20, 600, 100, "f16"), (3, 4, 9001, 8, "bf16")]
    size = max(tk.beam_search_select_workspace(getattr(torch, DTYPES[d]), N, K, V, n) for N, K, V, n, d in shapes)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for i, (N, K, V, n, d) in enumerate(shapes):
        fin = np.random.default_rng(i).random((N, K)) < 0.3
        check(torch, make(torch, N * K, V, d, seed=i), beam_scores(N, K, i), n, finished=fin, end=3, workspace=ws)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_subnormal_logits(dtype):
    """Values that differ by subnormal steps are ranked as they are."""
    torch = need_gpu()
    N, K, V, n = 1, 2, 12000, 12
    step = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}[dtype]
    rng = np.random.default_rng(5)
    for low, high in ((-40, 40), (-40, -1), (-3, -1), (-1, 0)):
        k = rng.integers(low, high + 1, (N * K, V)).astype(np.float64)
        x = torch.from_numpy((k * step).astype(np.float32)).to(getattr(torch, DTYPES[dtype])).cuda()
        assert np.array_equal(x.double().cpu().numpy(), k * step)
        check(torch, x, np.array([[-1.0, -1.5]], np.float32), n)


@pytest.mark.parametrize("equal", [False, True])
def test_widest_beams_and_rows(equal):
    """128 beams of 2^20 tokens: as many lists as a prompt can have."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    K, V, n = 128, 1 << 20, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.zeros((K, V), device="cuda") if equal else torch.randn((K, V), generator=g, device="cuda")
    # beams that lie well apart (equal: the first has all ranks), or all within reach of each other
    c = torch.arange(K, device="cuda", dtype=torch.float32).neg().view(1, K) * (1.0 if equal else 0.001)
    scores, parents, tokens = tk.beam_search_select(x, c, n)
    torch.cuda.synchronize()
    best, beam, token = [], [], []
    for b in range(K):
        row = x[b].double()
        if equal:
            val, tok = row[:n], torch.arange(n, device="cuda")
        else:
            val, tok = row.topk(n)  # distinct enough: equal ones do not matter below
        best.append((val - torch.logsumexp(row, 0) + c[0, b].double()).cpu().numpy())
        beam.append(np.full(n, b))
        token.append(tok.cpu().numpy())
    best, beam, token = (np.concatenate(v) for v in (best, beam, token))
    pick = np.lexsort((token, beam, -best))[:n]
    assert np.array_equal(parents[0].cpu().numpy(), beam[pick])
    assert np.array_equal(tokens[0].cpu().numpy(), token[pick])
    err = np.abs(scores[0].double().cpu().numpy() - best[pick])
    assert np.all(err <= 2.0 ** -24 * np.abs(best[pick]) + SUM_ERROR)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_logits_far_from_zero(dtype):
    """Rows that lie high or low, up to and past where the sums are formed less
    their maximum; few tokens have most of the weight, so that scores are small
    and show the sum's error."""
    torch = need_gpu()
    N, K, V = 6, 5, 30001
    rng = np.random.default_rng(9)
    x = rng.standard_normal((N * K, V)) - 14.0
    x[:, 100:104] += rng.uniform(9.0, 16.0, (N * K, 4))
    x += np.repeat([-30.0, -8.0, 12.0, 40.0, 74.0, 100.0], K)[:, None]
    x = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, DTYPES[dtype])).cuda()
    check(torch, x, np.tile(-np.arange(K, dtype=np.float32) / 64, (N, 1)), 2 * K)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [3, 40, 30001])
def test_beams_alike_but_for_one_logit(V, dtype):
    """Rows that differ in one small logit, the first, last or any other: their
    sums differ by less than a 32-bit one shows, and rank the beams."""
    torch = need_gpu()
    N, K = 2, 8
    x = make(torch, N * K, V, dtype, seed=12, ld=V + 5, offset=1, scale=1.0)
    x[:] = x[:1].clone()
    for i, at in enumerate((0, V - 1, V // 2, 1, V - 2, V - 1)):
        for row in (i + 1, K + (i * 3) % K):
            x[row, at] = -9.0 - 0.25 * i
    check(torch, x, np.full((N, K), -0.5, np.float32), min(3 * K, K * V))


def unlike_rows(torch, dtype, V, at, value):
    """Rows [len(value), V] that differ in one logit: element `at` + 1 of a row
    is its `value`, which lies 18 or more below the row's largest logit, `at`, in
    the same 16 bytes. What it adds to their sum is lost in fp32 but not in 64
    bits, in which it ranks the beams."""
    x = make(torch, 1, V, dtype, seed=21, scale=1.0).repeat(len(value), 1)
    assert at % 4 == 0 and x.data_ptr() % 16 == 0 and V * x.element_size() % 16 == 0
    x[:, at] = 15.0
    x[:, at + 1] = torch.tensor(value, device="cuda").to(x.dtype)
    return x


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("V", [8, 40, 1600, 40000])
def test_unlike_beams_whose_32_bit_sums_agree(V, dtype):
    """Beams of equal scores whose rows differ by one logit far below the
    largest of its 16 bytes: 32-bit sums are the same to the last bit, 64-bit
    ones rank the beams, the one that has a token banned first."""
    torch = need_gpu()
    inf = float("inf")
    at = V // 2 // 8 * 8
    value = [-4.5, -3.0, -inf, -6.0, -3.0, -inf, -9.0, -4.5]
    K = len(value)
    one = np.full((1, K), -1.5, np.float32)
    for order in (list(range(K)), list(range(K))[::-1], [0, 2], [1, 5, 0]):
        x = unlike_rows(torch, dtype, V, at, [value[b] for b in order])
        k = len(order)
        for n in (1, k, min(3 * k + 1, k * V)):
            check(torch, x, one[:, :k], n)
            check(torch, x, one[:, :k], n, weights=np.full((1, k), 0.375, np.float32))
    # pairs of like rows, and with the same rows in several prompts, one of them like throughout
    x = torch.cat([unlike_rows(torch, dtype, V, at, v) for v in ([-4.5, -6.0] * 4, [-6.0] * 8, sorted(value))])
    for n in (1, 5, 20):
        check(torch, x, np.full((3, K), -0.25, np.float32), n)


@pytest.mark.parametrize("K", [2, 5])
def test_finished_beam_that_32_bits_tie_with_another(K):
    """A finished beam's score is exact. An unfinished one whose best token has
    all but 1.5e-8 of the weight scores less, which only 64 bits show."""
    torch = need_gpu()
    V = 4096
    x = torch.full((K, V), float("-inf"), device="cuda")
    x[:, 400] = 0.0
    x[:, 401] = -18.0
    scores = np.full((1, K), -0.125, np.float32)
    finished = np.zeros((1, K), bool)
    finished[0, K - 1] = True
    for n in (1, 2, K + 3):
        check(torch, x, scores, n, finished, end=7)
        check(torch, x, scores, n, finished[:, ::-1], end=7)
        check(torch, x, scores, n, np.ones((1, K), bool), end=7)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("score", [-3e7, -1e9, -1e10, -3e12, 2e10])
def test_scores_whose_steps_exceed_a_sum_s_error(score, dtype):
    """Scores so large that ranks have coarse steps even in 64 bits: rows with
    the same logits in another order tie there, and their 32-bit sums, which
    differ, may round to different steps."""
    torch = need_gpu()
    N, K, V = 60, 4, 24
    rng = np.random.default_rng(17)
    base = (rng.standard_normal((N, 1, V)) * 3).astype(np.float32)
    x = make(torch, N * K, V, dtype, seed=0)
    x.copy_(torch.from_numpy(rng.permuted(np.broadcast_to(base, (N, K, V)), axis=2).reshape(N * K, V)))
    scores = np.full((N, K), score, np.float32)
    for n in (1, 7, 60):
        check(torch, x, scores, n)
        check(torch, x, scores, n, weights=np.full((N, K), 0.75, np.float32))
