"""The paged cache operators against plain simulations, entry by entry: whole numbers and copies, so every bit must be
equal (needs an MI355X)."""

import numpy as np
import pytest

from tests import spec_ref
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


class Pool:
    """A page table on the GPU and its numpy twin."""

    def __init__(self, torch, R, C, P, S, ld=None):
        self.torch, self.S = torch, S
        full = torch.full((R, ld or C), -1, dtype=torch.int32, device="cuda")
        self.full, self.tables = full, full[:, :C]
        self.lengths = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.uses = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.t, self.n, self.u = np.full((R, C), -1, np.int32), np.zeros(R, np.int32), np.zeros(P, np.int32)

    def same(self, note=""):
        assert (self.lengths.cpu().numpy() == self.n).all(), note
        assert (self.uses.cpu().numpy() == self.u).all(), note
        assert (self.tables.cpu().numpy() == self.t).all(), note
        assert bool((self.full[:, self.t.shape[1]:] == -1).all()), note

    def sound(self):
        """Uses are the held entries."""
        held = [self.t[r, c] for r in range(len(self.n)) for c in range(spec_ref.pages(self.n[r], self.S))]
        assert (np.bincount(held, minlength=len(self.u)) == self.u).all()

    def fork(self, parents):
        import top_logits_filtering_amd as tk

        p = self.torch.from_numpy(parents.astype(np.int32)).cuda()
        assert tk.cache_pages_fork(self.tables, self.lengths, p, self.uses, self.S) is self.tables
        spec_ref.fork(self.t, self.n, parents, self.u, self.S)

    def resize(self, new, caches=None, twins=None, **kw):
        import top_logits_filtering_amd as tk

        new = np.asarray(new, np.int32)
        got = tk.cache_pages_resize(self.tables, self.lengths, self.torch.from_numpy(new).cuda(), self.uses, self.S,
                                    caches=caches, **kw)
        assert got is self.lengths
        spec_ref.resize(self.t, self.n, new, self.u, self.S, twins)


def cache(torch, rng, P, S, inner, dtype, layout):
    """A cache and its numpy twin [P, S, ...] of bytes. layout: slots first, heads first, or a strided view."""
    es = torch.empty(0, dtype=dtype).element_size()
    if layout == "slots":
        shape, view = (P, S) + inner, lambda t: t
    elif layout == "heads":
        shape, view = (P, inner[0], S) + inner[1:], lambda t: t.transpose(1, 2)
    else:  # inside a wider buffer, layers in front
        shape, view = (P, S + 1) + inner[:-1] + (inner[-1] + 3,), lambda t: t[:, :S, ..., 1:-2]
    raw = torch.from_numpy(rng.integers(0, 256, int(np.prod(shape)) * es, dtype=np.uint8)).cuda()
    t = raw.view(dtype).view(shape)
    return view(t), t


def bits(t):
    import torch

    whole = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()]
    return t.contiguous().view(whole).cpu().numpy()


@pytest.mark.parametrize("N,K,C,S,P", [
    (1, 1, 1, 1, 3), (1, 4, 8, 16, 60), (3, 5, 40, 7, 700), (2, 8, 130, 16, 2200), (70, 3, 64, 4, 14000),
    (2, 128, 65, 5, 17000), (1, 33, 200, 3, 7000), (300, 4, 3, 16, 4000),
])
def test_fork_and_resize(N, K, C, S, P):
    """Random forks and resizes one after the other, bad parents and lengths among them."""
    torch = need_gpu()
    say("fork and resize", N, K, C, S, P)
    rng = np.random.default_rng(N * K + C)
    pool = Pool(torch, N * K, C, P, S, ld=C + N % 3)
    inner, dtype = (2, 8), torch.float32
    c, _ = cache(torch, rng, P, S, inner, dtype, "slots")
    twin = bits(c)
    most = C * S
    for turn in range(8):
        kind = turn % 4
        if kind == 0:
            new = rng.integers(0, most + 1, N * K)
        elif kind == 1:  # a step's growth
            new = np.minimum(pool.n + rng.integers(0, 6, N * K), most)
        elif kind == 2:
            new = np.where(rng.random(N * K) < 0.5, pool.n // 2, np.minimum(pool.n + 3 * S, most))
        else:
            new = pool.n + rng.integers(-2, 3, N * K)
        if turn > 3:
            new = np.where(rng.random(N * K) < 0.05, rng.choice([-1, most + 1, -2 ** 31, 2 ** 31 - 1], N * K), new)
        pool.resize(new, c, [twin])
        pool.same((turn, "resize"))
        pool.sound()
        assert (bits(c) == twin).all(), turn
        parents = rng.integers(0, K, (N, K))
        if turn > 1:
            parents[rng.random((N, K)) < 0.2] = -1
            parents[rng.random((N, K)) < 0.05] = K
        pool.fork(parents)
        pool.same((turn, "fork"))
        pool.sound()


@pytest.mark.parametrize("dtype,inner,layout,S", [
    ("bfloat16", (8, 128), "slots", 16), ("bfloat16", (3, 64), "heads", 16), ("float16", (2, 75), "heads", 5),
    ("float32", (1, 33), "view", 8), ("uint8", (2, 5), "slots", 3), ("uint8", (3, 64), "heads", 32),
    ("bfloat16", (2, 3), "view", 1), ("float64", (2, 2, 9), "view", 4), ("float32", (5,), "slots", 40),
])
def test_pages_are_copied_before_they_are_written(dtype, inner, layout, S):
    torch = need_gpu()
    say("copies", dtype, inner, layout, S)
    rng = np.random.default_rng(S)
    N, K, C = 5, 4, 6
    P = N * K * C + 9
    pool = Pool(torch, N * K, C, P, S)
    made = [cache(torch, rng, P, S, inner, getattr(torch, dtype), layout) for _ in range(3)]
    caches, fulls = [m[0] for m in made], [m[1] for m in made]
    other, other_full = cache(torch, rng, P, S, (2, 4), torch.float32, "slots")
    dims = dict(page_dim=0, slot_dim=1)
    if layout == "heads":
        given, dims["slot_dim"] = fulls, 2
    else:
        given = caches + [other]
    twins = [bits(c) for c in caches] + ([bits(other)] if layout != "heads" else [])
    first = np.zeros(N * K, np.int64)
    first[::K] = rng.integers(1, C * S - 3, N)
    pool.resize(first, given, twins, **dims)
    for turn in range(6):
        pool.fork(rng.integers(0, K, (N, K)) if turn else np.zeros((N, K), np.int64))
        step = rng.integers(0, 3, N * K)
        pool.resize(np.minimum(pool.n + step, C * S), given, twins, **dims)
        pool.same(turn)
        pool.sound()
        now = [bits(c) for c in caches] + ([bits(other)] if layout != "heads" else [])
        assert all((a == b).all() for a, b in zip(now, twins)), turn
    before = [f.clone() for f in fulls]
    pool.resize(np.zeros(N * K), given, twins, **dims)
    assert (pool.uses == 0).all() and (pool.tables == -1).all()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, fulls))


def test_growth_without_caches_and_without_pages():
    torch = need_gpu()
    S = 4
    pool = Pool(torch, 6, 4, 9, S)
    pool.resize([6, 4, 3, 0, 1, 16])  # 2, 1, 1, 0, 1 pages, and 4 that are the last ones
    pool.same()
    assert pool.n.tolist() == [6, 4, 3, 0, 1, 16]
    pool.resize([8, 4, 4, 1, 2, 16])  # row 3 needs a page: it and row 4 stay, though that needs none
    pool.same()
    assert pool.n.tolist() == [8, 4, 4, 0, 1, 16]
    pool.resize([8, 0, 4, 1, 2, 13])  # row 1 gives one back
    pool.same()
    assert pool.n.tolist() == [8, 0, 4, 1, 2, 13]
    # shared last pages that nobody can copy: the first that would have to is the end
    pool = Pool(torch, 4, 4, 20, S)
    pool.resize([6, 0, 0, 0])
    pool.fork(np.array([[0, 0, 0, 3]]))
    pool.resize([6, 7, 6, 5])
    pool.same()
    assert pool.n.tolist() == [6, 6, 6, 0]
    pool.resize([0, 0, 7, 5])  # the only one left writes into it
    pool.same()
    assert pool.n.tolist() == [0, 0, 7, 5]


def test_all_that_share_a_page_grow():
    """All but the last copy; with too few pages for that, those behind stay and the page stays shared."""
    torch = need_gpu()
    S, P = 4, 5
    rng = np.random.default_rng(0)
    for free, want in ((4, [3, 3, 3, 3]), (3, [3, 3, 3, 3]), (2, [3, 3, 2, 2]), (0, [2, 2, 2, 2])):
        pool = Pool(torch, 4, 2, 1 + free, S)
        c, _ = cache(torch, rng, 1 + free, S, (2, 4), torch.float32, "slots")
        twin = bits(c)
        pool.resize([2, 0, 0, 0], c, [twin])
        pool.fork(np.zeros((1, 4), np.int64))
        assert pool.u.max() == 4
        pool.resize([3] * 4, c, [twin])
        pool.same(free)
        pool.sound()
        assert pool.n.tolist() == want and (bits(c) == twin).all()


@pytest.mark.parametrize("R,C,P", [(1500, 30, 30000), (5000, 3, 9000), (1, 20000, 300000), (1024, 1, 1024),
                                   (2, 70000, 100003)])
def test_many_rows_and_pages(R, C, P):
    torch = need_gpu()
    rng = np.random.default_rng(R)
    S = 2
    pool = Pool(torch, R, C, P, S)
    for turn in range(4):
        pool.resize(rng.integers(0, C * S + 1, R) if turn != 1 else np.full(R, C * S))
        pool.same((R, turn))
    if R % 4 == 0:
        pool.fork(rng.integers(0, 4, (R // 4, 4)))
        pool.same()
    pool.sound()


def test_entries_that_name_no_page():
    """Tables that hold numbers outside the pool: nothing outside it is touched."""
    torch = need_gpu()
    rng = np.random.default_rng(1)
    S, P, C = 4, 40, 5
    pool = Pool(torch, 6, C, P, S)
    c, full = cache(torch, rng, P, S, (2, 4), torch.float32, "slots")
    pool.resize([9, 7, 12, 6, 15, 3])
    for r, col, page in ((0, 2, -5), (1, 1, P), (2, 0, 2 ** 31 - 1), (3, 1, -2 ** 31), (4, 3, P + 3)):
        pool.tables[r, col] = page
        if 0 <= pool.t[r, col] < P:  # as if it had been given back
            pool.u[pool.t[r, col]] -= 1
            pool.uses[int(pool.t[r, col])] -= 1
        pool.t[r, col] = page
    twin = bits(c)
    pool.fork(np.array([[1, 0, 2], [0, 0, 1]]))
    pool.same()
    pool.resize([10, 10, 10, 9, 9, 20], c, [twin])
    pool.same()
    pool.resize([1, 0, 13, 2, 2, 2], c, [twin])
    pool.same()
    assert (bits(c) == twin).all()


COMPACT = [
    # N, D, C, S, inner, dtype, layout, caches
    (1, 1, 1, 1, (1, 1), "uint8", "slots", 1), (3, 12, 5, 16, (4, 64), "bfloat16", "heads", 4),
    (9, 39, 6, 16, (8, 128), "bfloat16", "slots", 3), (4, 20, 12, 5, (3, 75), "float16", "heads", 2),
    (2, 255, 40, 7, (2, 9), "float32", "view", 2), (5, 30, 60, 1, (2, 5), "uint8", "slots", 2),
    (70, 8, 3, 16, (1, 40), "float32", "slots", 130), (2, 63, 3, 40, (2, 3, 8), "float64", "view", 1),
]


@pytest.mark.parametrize("case", COMPACT, ids=[str(c) for c in COMPACT])
def test_compact(case):
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, D, C, S, inner, dtype, layout, count = case
    say("compact", case)
    rng = np.random.default_rng(N + D)
    P = N * C + 3
    tables = np.argsort(rng.random(P))[:N * C].reshape(N, C).astype(np.int32)
    if N > 2:
        tables[1, C // 2], tables[2, 0] = -1, P
    made = [cache(torch, rng, P, S, inner, getattr(torch, dtype), layout) for _ in range(count)]
    views = [m[0] for m in made]
    given, slot = ([m[1] for m in made], 2) if layout == "heads" else (views, 1)
    twins = [bits(v) for v in views]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    for turn in range(3):
        starts = rng.integers(0, max(1, C * S - D), N)
        path = np.sort(np.stack([rng.permutation(2 * D)[:D] for _ in range(N)]), 1)
        counts = rng.integers(-1, D + 2, N)
        if turn == 1:  # all of it, some in place already
            path, counts = np.broadcast_to(np.arange(D), (N, D)).copy(), np.full(N, D)
            path[:, D // 2:] += 1
        if turn == 2:  # paths that end early
            path[rng.random((N, D)) < 0.1] = -1
            starts[rng.random(N) < 0.3] = -3
            starts[-1] = C * S - 2
        got = tk.cache_pages_compact(given, i32(tables), i32(starts), i32(path), i32(counts), slot_dim=slot)
        assert got is given or got == given
        spec_ref.compact(twins, tables, starts, path, counts)
        assert all((bits(v) == w).all() for v, w in zip(views, twins)), turn


def test_compact_past_four_gigabytes():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    P, S, H, E = 1100, 16, 64, 1024  # 2 MiB a page in bf16
    c = torch.zeros(P, S, H, E, dtype=torch.bfloat16, device="cuda")
    assert c.numel() * 2 > 2 ** 31
    big = torch.zeros(P * 2 + 50, S, H, E, dtype=torch.bfloat16, device="cuda")
    assert big.numel() * 2 > 2 ** 32
    tables = torch.tensor([[big.shape[0] - 1, 0]], dtype=torch.int32, device="cuda")
    big[-1, 9], big[0, 3] = 5.0, 7.0
    i32 = dict(dtype=torch.int32, device="cuda")
    tk.cache_pages_compact(big, tables, torch.tensor([6], **i32), torch.tensor([[3, 13]], **i32), torch.tensor([2], **i32))
    assert (big[-1, 6] == 5).all() and (big[-1, 7] == 7).all() and (big[-1, 8] == 0).all()


def test_speculative_steps():
    """The operators together as they are used: room for a tree of drafts, verification, the accepted entries moved to
    their places, the rest given back; cache entries hold what the token at their position was."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    rng = np.random.default_rng(6)
    N, D, V, S, C, H = 4, 12, 200, 4, 40, 3
    P = N * C
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lengths = torch.full((N, C), -1, **i32), torch.zeros(N, **i32)
    uses = torch.zeros(P, **i32)
    caches = [torch.full((P, S, H), -1.0, device="cuda"), torch.full((P, H, S), -1.0, device="cuda").transpose(1, 2)]
    parents = (torch.arange(D, **i32) // 3 - 1).expand(N, D).contiguous()
    g = torch.Generator(device="cuda").manual_seed(2)
    said = [[int(rng.integers(V))] for _ in range(N)]  # the first token, not in the cache yet

    def write(positions, tokens):
        page = torch.gather(tables, 1, (positions // S)).long()
        for c in caches:
            c[page, (positions % S).long()] = tokens[..., None].float()

    for step in range(6):
        # the last token and the drafts behind it go into the cache
        tk.cache_pages_resize(tables, lengths, lengths + 1 + D, uses, S)
        before = torch.tensor([len(s) - 1 for s in said], device="cuda")
        logits = torch.randn(N * (D + 1), V, device="cuda", generator=g) * 2
        drafts = torch.topk(logits.view(N, D + 1, V), 3).indices[:, :, torch.randperm(3)].to(torch.int32)
        drafts = torch.stack([drafts[:, j // 3, j % 3] for j in range(D)], 1)
        last = torch.tensor([s[-1] for s in said], **i32)
        write(before[:, None] + torch.arange(D + 1, device="cuda"), torch.cat([last[:, None], drafts], 1))
        u = torch.rand(N, D + 1, device="cuda", generator=g)
        tokens, accepted, path = tk.speculative_verify(logits, drafts, u, parents=parents)
        tk.cache_pages_compact(caches, tables, (before + 1).to(torch.int32), path, accepted)
        tk.cache_pages_resize(tables, lengths, (before + 1 + accepted).to(torch.int32), uses, S)
        for i in range(N):
            said[i] += tokens[i, :int(accepted[i]) + 1].tolist()
            held = torch.arange(len(said[i]) - 1, device="cuda")
            assert int(lengths[i]) == len(held)
            for c in caches:
                got = c[tables[i, held // S].long(), held % S]
                assert (got == torch.tensor(said[i][:-1], device="cuda")[:, None].float()).all(), (step, i)
        assert int(uses.sum()) == sum(spec_ref.pages(len(s) - 1, S) for s in said)
    assert max(len(s) for s in said) > 8


def test_beam_steps():
    """A beam search on pages beside one on whole rows (beam_reorder_states): the same entries at every step."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, V, S, C, E = 3, 4, 50, 4, 8, 8
    R, P, T = N * K, 3 * 4 * 8, 20
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lengths, uses = torch.full((R, C), -1, **i32), torch.zeros(R, **i32), torch.zeros(P, **i32)
    paged = torch.zeros(P, S, E, device="cuda")
    whole = torch.zeros(R, C * S, E, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    scores = torch.zeros(N, K, device="cuda")
    for t in range(T):
        tk.cache_pages_resize(tables, lengths, lengths + 1, uses, S, caches=paged)
        assert (lengths == t + 1).all()
        entry = torch.randn(R, E, device="cuda", generator=g)
        paged[tables[:, t // S].long(), t % S] = entry
        whole[:, t] = entry
        logits = torch.randn(R, V, device="cuda", generator=g)
        scores, parents, _ = tk.beam_search_select(logits, scores)
        tk.cache_pages_fork(tables, lengths, parents, uses, S)
        tk.beam_reorder_states(whole, parents)
        at = torch.arange(t + 1, device="cuda")
        assert torch.equal(paged[tables[:, at // S].long(), (at % S).expand(R, -1)], whole[:, :t + 1]), t
    assert int((uses > 0).sum()) < R * 5  # the beams of a prompt share their beginning


def test_fork_of_a_long_row():
    """More columns than one launch's threads; only the last ones and the first hold pages."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    C = (1 << 28) + 77
    tables = torch.full((2, C), -1, dtype=torch.int32, device="cuda")
    uses = torch.zeros(200, dtype=torch.int32, device="cuda")
    at = torch.cat([torch.arange(3, device="cuda"), torch.arange(C - 150, C, device="cuda")])
    tables[0, at] = torch.arange(153, dtype=torch.int32, device="cuda")
    uses[:153] = 1
    lengths = torch.tensor([C, 5], dtype=torch.int32, device="cuda")
    tk.cache_pages_fork(tables, lengths, torch.zeros(1, 2, dtype=torch.int32, device="cuda"), uses, 1)
    assert bool((tables[1] == tables[0]).all()) and bool((lengths == C).all())
    assert bool((tables[0, at] == torch.arange(153, device="cuda")).all()) and int((tables[0] >= 0).sum()) == 153
    assert bool((uses[:153] == 2).all()) and bool((uses[153:] == 0).all())


def test_captured_steps():
    """Resize, compact and fork in a graph, replayed between eager work on the same pool."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, K, S, C, E = 2, 3, 4, 6, 16
    R, P = N * K, 64
    i32 = dict(dtype=torch.int32, device="cuda")

    def fresh():
        tables, lengths, uses = torch.full((R, C), -1, **i32), torch.zeros(R, **i32), torch.zeros(P, **i32)
        caches = [torch.arange(P * S * E, device="cuda", dtype=torch.float32).view(P, S, E) * (1 + k) for k in range(3)]
        return tables, lengths, uses, caches

    new, parents = torch.zeros(R, **i32), torch.zeros(N, K, **i32)
    path, counts, starts = torch.zeros(R, 2, **i32), torch.zeros(R, **i32), torch.zeros(R, **i32)
    ws = torch.empty(tk.cache_pages_resize_workspace(R, P), dtype=torch.uint8, device="cuda")

    def step(pool, **kw):
        tables, lengths, uses, caches = pool
        tk.cache_pages_resize(tables, lengths, new, uses, S, caches=caches, **kw)
        tk.cache_pages_compact(caches, tables, starts, path, counts)
        tk.cache_pages_fork(tables, lengths, parents, uses, S)

    def inputs(turn):
        rng = np.random.default_rng(turn)
        new.copy_(torch.from_numpy(rng.integers(4, C * S, R).astype(np.int32)))
        parents.copy_(torch.from_numpy(rng.integers(0, K, (N, K)).astype(np.int32)))
        starts.copy_((new // S * S - 4).clamp(min=0))
        path.copy_(torch.tensor([[1, 3]], **i32).expand(R, 2))
        counts.zero_()  # rows of a fork share pages, which compact must not write

    live, twin = fresh(), fresh()
    inputs(0)
    step(live, workspace=ws)  # warm
    step(twin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(live, workspace=ws)
    for turn in range(1, 6):
        inputs(turn)
        graph.replay()
        torch.cuda.synchronize()
        step(twin)
        for a, b in zip(live[:3] + tuple(live[3]), twin[:3] + tuple(twin[3])):
            assert torch.equal(a, b), turn
