"""The beam search operators together, as a search uses them, and at sizes past
4 GiB (needs an MI355X)."""

import numpy as np
import pytest

from tests import beam_ref
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


class Search:
    """A search over a table model: the logits of a row are the table's row of
    its last token. States that follow the beams: the tokens so far, and one
    vector per token, as a cache holds them."""

    N, K, V, T, D, end = 3, 4, 601, 26, 24, 5

    def __init__(self, torch, seed):
        rng = np.random.default_rng(seed)
        N, K, V, T, D = self.N, self.K, self.V, self.T, self.D
        table = rng.standard_normal((V, V)).astype(np.float32) * 2
        table[:, self.end] += 4.5  # answers end now and then
        self.table = torch.from_numpy(table).cuda().bfloat16()
        self.embed = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)).cuda().half()
        self.topk = torch.full((N * K,), 40, dtype=torch.int32, device="cuda")
        self.last = torch.from_numpy(rng.integers(0, V, N).repeat(K).astype(np.int32)).cuda()
        self.scores = torch.full((N, K), float("-inf"), device="cuda")
        self.scores[:, 0] = 0.0  # one live beam at first
        self.finished = torch.zeros((N, K), dtype=torch.bool, device="cuda")
        self.steps = torch.zeros((N, K), device="cuda")
        self.words = torch.full((N * K, T), -1, dtype=torch.int32, device="cuda")
        self.cache = torch.zeros((2, N * K, 3, T, D), dtype=torch.float16, device="cuda")
        self.tokens = torch.zeros((T, N, K), dtype=torch.int32, device="cuda")
        self.parents = torch.zeros((T, N, K), dtype=torch.int32, device="cuda")
        self.at = torch.zeros((), dtype=torch.int64, device="cuda")
        self.time = torch.arange(T, device="cuda")
        self.lengths = torch.zeros(N, dtype=torch.int32, device="cuda")

    def step(self, torch, tk, checked=False):
        """One step; nothing in it waits for the host (unless `checked`)."""
        N, K = self.N, self.K
        logits = self.table[self.last.long()]
        logits = tk.apply_top_k_top_p(logits, k=self.topk)
        weights = ((6.0 + self.steps) / 6.0) ** -0.7
        scores, parents, tokens = tk.beam_search_select(logits, self.scores, K, finished=self.finished,
                                                        end_token=self.end, weights=weights)
        if checked:
            self.check(logits, weights, scores, parents, tokens)
        tk.beam_reorder_states([self.words], parents, seq_dim=1, lengths=self.lengths)
        tk.beam_reorder_states(self.cache, parents, batch_dim=1, seq_dim=3, lengths=self.lengths)
        up = parents.long()
        self.finished.copy_(self.finished.gather(1, up) | (tokens == self.end))
        self.steps.copy_(self.steps.gather(1, up) + (~self.finished))
        self.scores.copy_(scores)
        self.last.copy_(tokens.view(-1))
        here = self.time == self.at
        self.words.copy_(torch.where(here, self.last[:, None], self.words))
        self.cache.copy_(torch.where(here[:, None], self.embed[self.last.long()][:, None, None, :], self.cache))
        self.tokens.copy_(torch.where(here[:, None, None], tokens, self.tokens))
        self.parents.copy_(torch.where(here[:, None, None], parents, self.parents))
        self.at.add_(1)
        self.lengths.add_(1)

    def check(self, logits, weights, scores, parents, tokens):
        ref = beam_ref.select(logits.double().cpu().numpy(), self.scores.cpu().numpy(), self.K,
                              self.finished.cpu().numpy(), self.end, weights.cpu().numpy())
        assert np.array_equal(parents.cpu().numpy(), ref[1])
        assert np.array_equal(tokens.cpu().numpy(), ref[2])


def test_search():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    s = Search(torch, 3)
    for _ in range(s.T):
        s.step(torch, tk, checked=True)
    torch.cuda.synchronize()
    assert bool(s.finished.any())
    sequences = tk.beam_backtrace(s.tokens, s.parents)
    torch.cuda.synchronize()
    # the reordered history and the one read out of the parents are the same
    assert torch.equal(sequences.view(s.N * s.K, s.T), s.words)
    want = beam_ref.backtrace(s.tokens.cpu().numpy(), s.parents.cpu().numpy())
    assert np.array_equal(sequences.cpu().numpy(), want)
    # and the cache holds the vectors of those words
    vectors = s.embed[s.words.long()]  # [rows, T, D]
    assert torch.equal(s.cache, vectors[None, :, None].expand_as(s.cache))
    say(f"search: {int(s.finished.sum())} of {s.N * s.K} beams finished")


def test_search_in_a_graph():
    """A whole step captured once and replayed for the length of the search,
    with eager work in between, against the eager search."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    eager, replayed = Search(torch, 8), Search(torch, 8)
    keep = {k: v.clone() for k, v in vars(replayed).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        replayed.step(torch, tk)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.step(torch, tk)
    for k, v in keep.items():
        getattr(replayed, k).copy_(v)
    torch.cuda.synchronize()
    for _ in range(eager.T):
        graph.replay()
        eager.step(torch, tk)
        torch.cuda.synchronize()
        for k in keep:
            assert torch.equal(getattr(eager, k), getattr(replayed, k)), k


def test_select_past_4_gib():
    """Rows that begin past 2^32 bytes, and 2^32 elements, into the logits."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, V, n = 4097, 8, 151936, 5
    rows = N * K  # 4.98e9 elements, 9.96 GB
    x = torch.empty((rows, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x.normal_(generator=g)
    c = -torch.rand((N, K), generator=g, device="cuda")
    scores, parents, tokens = tk.beam_search_select(x, c, n)
    torch.cuda.synchronize()
    for i in (0, 1767, 1768, 3533, 3534, N - 1):
        ref = beam_ref.select(x[i * K:(i + 1) * K].double().cpu().numpy(), c[i:i + 1].cpu().numpy(), n)
        assert np.array_equal(parents[i].cpu().numpy(), ref[1][0]), i
        assert np.array_equal(tokens[i].cpu().numpy(), ref[2][0]), i
    assert int(tokens.min()) >= 0 and int(tokens.max()) < V
    say("select past 4 GiB")


@pytest.mark.parametrize("K", [3, 4, 7, 16, 21])
def test_reorder_more_than_the_cache(K):
    """Calls on more memory than the last-level cache holds take reads that go
    past it; the last state spans more than 4 GiB."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N = 2
    rng = np.random.default_rng(K)
    p = rng.integers(-1, K + 1, (N, K)).astype(np.int32)
    parents = torch.from_numpy(p).cuda()
    ok = (p >= 0) & (p < K)
    source = torch.from_numpy((np.where(ok, p, np.arange(K)) + K * np.arange(N)[:, None]).reshape(-1)).cuda()
    T = 4100
    lengths = torch.tensor([T - 3, 1001], dtype=torch.int32, device="cuda")
    D = (1 << 32) // (N * K * T * 2) // 8 * 8 + 64
    states = [torch.randint(-2 ** 15, 2 ** 15, (N * K, 3, 257, 24), dtype=torch.int16, device="cuda"),
              torch.empty((N * K, T, D), dtype=torch.int16, device="cuda").random_(-2 ** 15, 2 ** 15)]
    assert states[1].numel() * 2 > 1 << 32
    for state, axis in zip(states, (2, 1)):
        state = [state]
        if axis == 2:  # the small one beside the large one's bulk
            state.append(torch.zeros((N * K, 1, 300, (1 << 29) // (N * K * 600) // 8 * 8), dtype=torch.int16,
                                     device="cuda"))
        keep = state[0].clone()
        tk.beam_reorder_states(state, parents, seq_dim=axis, lengths=lengths)
        torch.cuda.synchronize()
        position = torch.arange(keep.shape[axis], device="cuda")
        moved = (position[None] < lengths.repeat_interleave(K)[:, None])
        moved = moved[:, None, :, None] if axis == 2 else moved[:, :, None]
        for r in range(N * K):  # row by row: the whole would need several copies
            want = torch.where(moved[r], keep[source[r]], keep[r])
            assert torch.equal(state[0][r], want), (axis, r)
        del keep


def test_given_outputs_count_as_modified():
    """Outputs that the caller gives are written in place: what was saved of
    them for a backward pass must not change unnoticed."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, V, T = 2, 3, 50, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    logits = torch.randn((N * K, V), generator=g, device="cuda", requires_grad=True)
    scores = torch.zeros((N, K), device="cuda")
    want = tk.beam_search_select(logits, scores)
    assert not any(t.requires_grad for t in want)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = (torch.zeros((N, K), device="cuda"), torch.zeros((N, K), **i32), torch.zeros((N, K), **i32))
    seen = [t._version for t in out]
    x = torch.ones((N, K), device="cuda", requires_grad=True)
    y = (x * out[0]).sum() + torch.index_select(x, 1, out[1].view(-1)).sum()
    got = tk.beam_search_select(logits, scores, out=out)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(t._version > v for t, v in zip(out, seen))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()

    leaf = torch.zeros((N, K), device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="require grad"):
        tk.beam_search_select(logits, scores, out=(leaf, *out[1:]))
    with torch.no_grad():
        tk.beam_search_select(logits, scores, out=(leaf, *out[1:]))
    assert torch.equal(leaf.detach(), want[0])

    tokens, parents = (torch.zeros((T, N, K), **i32) for _ in range(2))
    paths = torch.ones((N, K, T), **i32)
    seen = paths._version
    assert tk.beam_backtrace(tokens, parents, out=paths) is paths and paths._version > seen
    with torch.inference_mode():
        paths = torch.ones((N, K, T), **i32)
    tk.beam_backtrace(tokens, parents, out=paths)
    assert not bool(paths.any())
