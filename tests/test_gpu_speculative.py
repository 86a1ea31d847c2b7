"""speculative_verify against a plain reference in 64 bits: tokens, counts and paths are whole numbers and have to be
equal (needs an MI355X).

Only where a decision lies closer to its border than the roundings of 64 bits in the reference and in the kernel can
either outcome stand: sums of V terms, each off by a few 2^-53, are taken to be within 1e-12 here (V 2^-53 for V = 2^13;
larger rows' errors are random, and stay below that)."""

import numpy as np
import pytest

from tests import spec_ref
from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu

TYPES = ("float32", "float16", "bfloat16")
BORDER = 1e-12


def head(rng, shape, spikes=6, scale=2.5, high=9.0):
    """Rows as a model's head gives them: a wide body and a few tokens that stand out."""
    x = rng.standard_normal(shape) * scale
    flat = x.reshape(-1, shape[-1])
    if shape[-1] > 0:
        for _ in range(spikes):
            flat[np.arange(len(flat)), rng.integers(0, shape[-1], len(flat))] = high + 3 * rng.standard_normal(len(flat))
    return x


def on_gpu(torch, a, dtype, pad=0, offset=0):
    """A [rows, V] array as a view of a wider buffer that begins `offset` elements in."""
    rows, V = a.shape
    full = torch.full((rows * (V + pad) + offset,), 7.0, dtype=dtype, device="cuda")
    view = full[offset:].view(rows, V + pad)[:, :V]
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype))
    return view


def back(t):
    return t.double().cpu().numpy()


def plan_uniforms(rng, x, drafts, y, parents, u):
    """Half of the uniforms are set so that the draft behind them is likelier to stand than by chance."""
    u = u.copy()
    u[rng.random(u.shape) < 0.5] *= 0.1
    return u


def check(torch, x, drafts, uniforms=None, y=None, parents=None, lengths=None, say_name="", **kw):
    import top_logits_filtering_amd as tk

    N, D = drafts.shape
    V = x.shape[1]
    i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    gu = None if uniforms is None else torch.from_numpy(np.ascontiguousarray(uniforms, np.float32)).cuda()
    tokens, accepted, path = tk.speculative_verify(x, i32(drafts), gu, draft_logits=y, parents=i32(parents),
                                                   lengths=i32(lengths), **kw)
    torch.cuda.synchronize()
    rt, ra, rp, margin = spec_ref.verify(back(x).reshape(N, D + 1, V), drafts,
                                         None if uniforms is None else np.float32(uniforms),
                                         None if y is None else back(y).reshape(N, D, V), parents, lengths)
    sure = margin > BORDER
    got_t, got_a = tokens.cpu().numpy(), accepted.cpu().numpy()
    assert (got_a[sure] == ra[sure]).all(), (say_name, np.nonzero(got_a != ra), got_a, ra)
    assert (got_t[sure] == rt[sure]).all(), (say_name, np.argwhere(got_t != rt)[:5], got_t[got_t != rt][:5],
                                             rt[got_t != rt][:5], margin[(got_t != rt).any(1)][:5])
    if parents is not None:
        assert (path.cpu().numpy()[sure] == rp[sure]).all(), say_name
    else:
        assert path is None
    return ra, int((~sure).sum())


def drafts_for(rng, x, D):
    """Drafts of which about half are among the likeliest tokens."""
    N, V = x.shape[0], x.shape[2]
    drafts = rng.integers(0, V, (N, D)).astype(np.int32)
    for i in range(N):
        for j in range(D):
            if rng.random() < 0.6:
                row = x[i, j]
                p = spec_ref.softmax(row)
                if p is not None:
                    drafts[i, j] = rng.choice(V, p=p) if V <= 5000 else int(np.argsort(-row)[rng.integers(0, min(V, 3))])
    return drafts


CASES = [
    # N, D, V, pad, offset
    (1, 0, 1, 0, 0), (3, 0, 100, 0, 0), (2, 1, 1, 0, 0), (2, 1, 2, 0, 1), (4, 2, 7, 3, 1), (5, 3, 100, 0, 0),
    (8, 4, 1000, 0, 0), (3, 7, 2049, 5, 3), (16, 2, 5000, 8, 0), (2, 8, 32003, 1, 1), (3, 3, 65536, 0, 0),
    (1, 5, 151936, 0, 0), (40, 1, 257, 0, 0),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", ["draft", "lookup", "greedy"])
@pytest.mark.parametrize("case", CASES, ids=[str(c) for c in CASES])
def test_chain(case, mode, dtype):
    torch = need_gpu()
    N, D, V, pad, offset = case
    say("chain", case, mode, dtype)
    t = getattr(torch, dtype)
    rng = np.random.default_rng(sum(case) + len(mode) + len(dtype))
    for turn in range(2):
        base = head(rng, (N, D + 1, V))
        y = base[:, :D] + 0.5 * rng.standard_normal((N, D, V))
        x = on_gpu(torch, base.reshape(-1, V), t, pad, offset)
        gy = on_gpu(torch, y.reshape(-1, V), t, pad + 1, 0) if mode == "draft" else None
        drafts = drafts_for(rng, base, D)
        if turn == 1 and D:
            drafts[rng.random(drafts.shape) < 0.1] = -1
            drafts[rng.random(drafts.shape) < 0.1] = V
        lengths = rng.integers(-1, D + 2, N) if turn == 1 else None
        u = None if mode == "greedy" else plan_uniforms(rng, base, drafts, y, None, rng.random((N, D + 1)))
        check(torch, x, drafts, u, gy, None, lengths, (case, mode, dtype))


TREES = [
    # N, D, V, branches
    (3, 1, 50, 1), (4, 6, 300, 2), (2, 12, 1000, 3), (5, 39, 2000, 3), (2, 60, 5000, 4), (3, 64, 500, 9),
    (2, 255, 300, 16), (2, 255, 120, 255), (3, 9, 32003, 3),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("case", TREES, ids=[str(c) for c in TREES])
def test_tree(case, greedy, dtype):
    torch = need_gpu()
    N, D, V, branch = case
    say("tree", case, greedy, dtype)
    rng = np.random.default_rng(1000 + sum(case) + len(dtype))
    for turn in range(3):
        base = head(rng, (N, D + 1, V), spikes=3)
        if turn == 2:  # parents of any kind, some not there
            parents = np.stack([rng.integers(-1, np.arange(1, D + 1)) - 1 for _ in range(N)])
            parents = np.maximum(parents, -1)
            wrong = rng.random(parents.shape) < 0.05
            parents[wrong] = np.where(rng.random(int(wrong.sum())) < 0.5, -2, np.broadcast_to(np.arange(D), (N, D))[wrong])
        else:
            parents = np.broadcast_to(np.arange(D) // branch - 1, (N, D)).copy()
        drafts = np.empty((N, D), np.int32)
        for i in range(N):
            for j in range(D):
                row = base[i, max(parents[i, j], -1) + 1]
                order = np.argsort(-row)
                drafts[i, j] = order[min(V - 1, j % branch + (0 if turn == 0 else int(rng.integers(0, 2))))]
        x = on_gpu(torch, base.reshape(-1, V), getattr(torch, dtype), turn, turn)
        lengths = rng.integers(0, D + 1, N) if turn == 1 else None
        u = None if greedy else rng.random((N, D + 1))
        check(torch, x, drafts, u, None, parents, lengths, (case, greedy, dtype, turn))


@pytest.mark.parametrize("dtype", TYPES)
def test_chain_is_a_tree_of_single_branches(dtype):
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    rng = np.random.default_rng(5)
    N, D, V = 6, 7, 3001
    base = head(rng, (N, D + 1, V))
    x = on_gpu(torch, base.reshape(-1, V), getattr(torch, dtype))
    drafts = torch.from_numpy(drafts_for(rng, base, D)).cuda()
    parents = (torch.arange(D, dtype=torch.int32, device="cuda") - 1).expand(N, D).contiguous()
    for u in (None, torch.rand(N, D + 1, device="cuda")):
        a, b = tk.speculative_verify(x, drafts, u), tk.speculative_verify(x, drafts, u, parents=parents)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        want = torch.where(torch.arange(D, device="cuda") < a[1][:, None], torch.arange(D, device="cuda"), -1)
        assert torch.equal(b[2].long(), want)


# More logits than are worth reading whole: the path is followed row by row.
LARGE = [
    # N, D, V, mode, branch, pad
    (1200, 3, 4001, "draft", 0, 0), (150, 10, 20003, "draft", 0, 5), (3, 8, 1000003, "draft", 0, 0),
    (2500, 2, 5000, "lookup", 0, 3), (40, 30, 30000, "lookup", 0, 0), (500, 39, 3001, "lookup", 3, 0),
    (90, 255, 1500, "lookup", 4, 1), (2, 60, 400000, "lookup", 5, 0), (2000, 5, 3000, "greedy", 0, 0),
    (600, 39, 1501, "greedy", 3, 2), (1, 255, 260000, "lookup", 255, 0), (20000, 1, 800, "draft", 0, 0),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", LARGE, ids=[str(c) for c in LARGE])
def test_large(case, dtype):
    torch = need_gpu()
    N, D, V, mode, branch, pad = case
    say("large", case, dtype)
    t = getattr(torch, dtype)
    assert N * (D + 1) * V * t.itemsize >= 2 ** 25
    g = torch.Generator(device="cuda").manual_seed(N + D)
    rng = np.random.default_rng(N + D)
    x = torch.empty(N * (D + 1), V + pad, dtype=t, device="cuda")
    x.normal_(generator=g).mul_(3)
    x = x[:, :V]
    y = None
    if mode == "draft":
        y = (x.view(N, D + 1, V)[:, :D].float() + 0.4 * torch.randn(N, D, V, device="cuda", generator=g)).to(t)
        y = y.view(N * D, V)
    # drafts that stand more often than not
    width = max(1, branch)
    best = torch.topk(x.float(), min(width, V), dim=1).indices.view(N, D + 1, -1)
    node = torch.arange(D, device="cuda") // width if branch else torch.arange(D, device="cuda")
    drafts = best[:, node, torch.arange(D, device="cuda") % best.shape[2]]
    drafts = torch.where(torch.rand(N, D, device="cuda", generator=g) < 0.2, 7 % V, drafts).to(torch.int32).cpu().numpy()
    parents = np.broadcast_to(node.cpu().numpy() - 1, (N, D)).copy() if branch else None
    lengths = rng.integers(-1, D + 2, N) if N > 3 else None
    u = None if mode == "greedy" else rng.random((N, D + 1)) * rng.choice([1.0, 0.05, 0.01], (N, D + 1))
    at = np.unique(np.concatenate([np.arange(min(N, 40)), rng.integers(0, N, 60), np.arange(max(0, N - 20), N)]))
    import top_logits_filtering_amd as tk

    i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    gu = None if u is None else torch.from_numpy(np.float32(u)).cuda()
    for turn in range(2):
        if turn == 1 and N > 1:  # rows that hold nothing, or too much
            x.view(N, D + 1, V)[0, 0] = -float("inf")
            x.view(N, D + 1, V)[N - 1, min(1, D), V // 2] = float("nan")
            if y is not None:
                y.view(N, D, V)[N // 2, 0, V - 1] = float("inf")
        tokens, accepted, path = tk.speculative_verify(x, i32(drafts), gu, draft_logits=y, parents=i32(parents),
                                                       lengths=i32(lengths))
        torch.cuda.synchronize()
        assert int(accepted.min()) >= 0 and int(accepted.max()) <= D
        sel = torch.from_numpy(at).cuda()
        pick = lambda m: None if m is None else m[at]
        rt, ra, rp, margin = spec_ref.verify(
            Rows(x.view(N, D + 1, V), sel), drafts[at], None if u is None else np.float32(u)[at],
            None if y is None else Rows(y.view(N, D, V), sel), pick(parents), pick(lengths))
        sure = margin > BORDER
        assert (accepted.cpu().numpy()[at][sure] == ra[sure]).all(), turn
        assert (tokens.cpu().numpy()[at][sure] == rt[sure]).all(), turn
        if parents is not None:
            assert (path.cpu().numpy()[at][sure] == rp[sure]).all(), turn


class Rows:
    """Some sequences' rows, fetched one at a time."""

    def __init__(self, t, at):
        self.t, self.at, self.shape = t, at, (len(at),) + tuple(t.shape[1:])

    def __getitem__(self, key):
        return self.t[self.at[key[0]], key[1]].double().cpu().numpy()


def odd_rows(kind, V, rng):
    x = head(rng, (V,), spikes=4)
    if kind == "filtered":
        x[np.argsort(-x)[min(5, V):]] = -np.inf
    elif kind == "one":
        x[:] = -np.inf
        x[V // 2] = 3.0
    elif kind == "none":
        x[:] = -np.inf
    elif kind == "nan":
        x[V // 3] = np.nan
    elif kind == "inf":
        x[V - 1] = np.inf
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "lowest":  # masks of the type's lowest value
        x[3:] = -65504.0
    elif kind == "all lowest":
        x[:] = -65504.0
    elif kind == "high":
        x += 600.0
    elif kind == "low":
        x -= 900.0
    elif kind == "wide":
        x *= 400.0
    elif kind == "zeros":
        x[:] = np.where(np.arange(V) % 2, 0.0, -0.0)
    return x


KINDS = ("plain", "filtered", "one", "none", "nan", "inf", "equal", "lowest", "all lowest", "high", "low", "wide",
         "zeros")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [11, 3000])
@pytest.mark.parametrize("kind", KINDS)
def test_odd_rows(kind, V, dtype):
    """Each kind of row as a target row, with every kind as the draft's row."""
    torch = need_gpu()
    say("odd", kind, V, dtype)
    rng = np.random.default_rng(len(kind) + V)
    N, D = 2 * len(KINDS), 2
    base, y = np.empty((N, D + 1, V)), np.empty((N, D, V))
    for i in range(N):
        at = (i // len(KINDS)) % 2
        base[i] = [odd_rows(kind if w == at else "plain", V, rng) for w in range(D + 1)]
        y[i] = [odd_rows(KINDS[i % len(KINDS)], V, rng) for _ in range(D)]
    t = getattr(torch, dtype)
    x, gy = on_gpu(torch, base.reshape(-1, V), t, 1, 1), on_gpu(torch, y.reshape(-1, V), t)
    drafts = rng.integers(0, V, (N, D)).astype(np.int32)
    drafts[:, 0] = V // 2
    for u in (rng.random((N, D + 1)), np.zeros((N, D + 1)), np.full((N, D + 1), 1 - 2.0 ** -24)):
        check(torch, x, drafts, u, gy, say_name=(kind, V, dtype, "draft"))
        check(torch, x, drafts, u, say_name=(kind, V, dtype, "lookup"))
        check(torch, x, drafts, u, parents=np.full((N, D), -1), say_name=(kind, V, dtype, "tree"))
    check(torch, x, drafts, say_name=(kind, V, dtype, "greedy"))


@pytest.mark.parametrize("dtype", TYPES)
def test_same_rows(dtype):
    """Where the draft model is the target model, every draft that has any weight stands; one without is replaced by a
    token from p, whatever the rows' offsets are."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    rng = np.random.default_rng(8)
    N, D, V = 5, 4, 20001
    base = head(rng, (N, D + 1, V))
    base[:, :, 17] = -np.inf
    t = getattr(torch, dtype)
    x = on_gpu(torch, base.reshape(-1, V), t, 3, 1)
    y = on_gpu(torch, back(x).reshape(N, D + 1, V)[:, :D].reshape(-1, V), t, 0, 0)
    drafts = rng.integers(20, V, (N, D)).astype(np.int32)
    u = np.full((N, D + 1), 1 - 2.0 ** -24)
    u[:, D] = rng.random(N)
    acc, _ = check(torch, x, drafts, u, y)
    assert (acc == D).all()
    drafts[:, 2] = 17
    acc, _ = check(torch, x, drafts, u, y)
    assert (acc == 2).all()
    # a row moved by a constant is the same distribution up to what roundings of the logits leave
    y2 = on_gpu(torch, base[:, :D].reshape(-1, V) + 0.25, torch.float32)
    x2 = on_gpu(torch, base.reshape(-1, V), torch.float32)
    tokens, accepted, _ = tk.speculative_verify(x2, torch.from_numpy(drafts).cuda(),
                                                torch.from_numpy(np.float32(u * 0.999)).cuda(), draft_logits=y2)
    assert (accepted.cpu().numpy() == 2).all() and (tokens[:, 2] >= 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [500, 50000])
def test_close_decisions(V, dtype):
    """Uniforms next to the border on either side: decisions that sums in 32 bits cannot make."""
    torch = need_gpu()
    rng = np.random.default_rng(V)
    N, D = 48, 1
    base = head(rng, (N, D + 1, V))
    y = base[:, :D] + rng.standard_normal((N, D, V))
    t = getattr(torch, dtype)
    x, gy = on_gpu(torch, base.reshape(-1, V), t), on_gpu(torch, y.reshape(-1, V), t)
    xs, ys = back(x).reshape(N, D + 1, V), back(gy).reshape(N, D, V)
    drafts, u1, u2 = np.empty((N, D), np.int32), rng.random((N, 2)), rng.random((N, 2))
    for i in range(N):
        p, q = spec_ref.softmax(xs[i, 0]), spec_ref.softmax(ys[i, 0])
        drafts[i, 0] = rng.choice(V, p=np.maximum(q - p, 0) / np.maximum(q - p, 0).sum())
        steps = i % 5 - 2
        for u, border in ((u1, p[drafts[i, 0]] / q[drafts[i, 0]]), (u2, p[drafts[i, 0]])):
            near = np.float32(border)
            for _ in range(abs(steps)):
                near = np.nextafter(near, np.float32(steps), dtype=np.float32)
            u[i, 0] = min(max(near, 0), 1 - 2.0 ** -24)
    a, _ = check(torch, x, drafts, u1, gy)
    b, _ = check(torch, x, drafts, u2)
    assert 0 < a.sum() < N and 0 < b.sum() < N


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [3, 600])
@pytest.mark.parametrize("mode", ["far", "alike"])
def test_uniforms_at_the_ends(mode, N, dtype):
    """Uniforms of 0, next to 1 and of 1, where the row begins and ends with tokens of next to no weight (far), or
    where p and q are the same but for two tokens, so that the others' residuals are nothing but roundings. The token
    has to be there, and its piece of [0, 1) to reach the uniform but for roundings: terms are off by up to 4e-14,
    those of both rows together by 8e-14 of 1, of which the residual is a part m only: 1e-13 / m. The reference's sums
    of 20000 terms are within 20000 2^-53 < 1e-11."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    rng = np.random.default_rng(N)
    V, D = 20000, 1
    base = head(rng, (N, D + 1, V), high=4.0)
    drafts, y = np.zeros((N, D), np.int32), None
    u = np.tile(np.array([[0.0, 0.0], [1 - 2.0 ** -24, 1 - 2.0 ** -24], [1.0, 1.0]]), (N // 3, 1))
    lengths = None
    t = getattr(torch, dtype)
    if mode == "far":
        base[:, :, :9000] = -100.0
        base[:, :, -4000:] = -100.0
        lengths = torch.zeros(N, dtype=torch.int32, device="cuda")
    else:
        # two of forty tokens swap their weights; the draft, the one that q has more of, is rejected
        keep = np.argpartition(-base[:, 0] + 20 * (rng.random((N, V)) < 0.5), 40, axis=1)[:, :40]
        few = np.full((N, V), -np.inf)
        np.put_along_axis(few, keep, np.take_along_axis(base[:, 0], keep, 1), 1)
        few[np.arange(N), keep[:, 5]] = 4.0
        few[np.arange(N), keep[:, 6]] = 2.0
        base[:, 0] = few
        other = few.copy()
        other[np.arange(N), keep[:, 5]] = 2.0
        other[np.arange(N), keep[:, 6]] = 4.0
        drafts[:, 0] = keep[:, 6]
        u[:, 0] = 1 - 2.0 ** -24
        y = on_gpu(torch, other, t)
    x = on_gpu(torch, base.reshape(-1, V), t)
    tokens, accepted, _ = tk.speculative_verify(x, torch.from_numpy(drafts).cuda(),
                                                torch.from_numpy(np.float32(u)).cuda(), draft_logits=y, lengths=lengths)
    got = tokens.cpu().numpy()
    assert (accepted == 0).all() and (got[:, 0] >= 0).all() and (got[:, 0] < V).all()
    xs = back(x).reshape(N, D + 1, V)[:, 0]
    e = np.exp(xs - xs.max(1, keepdims=True))
    r, m = e / e.sum(1, keepdims=True), np.ones(N)
    if y is not None:
        ys = back(y)
        q = np.exp(ys - ys.max(1, keepdims=True))
        r = np.maximum(r - q / q.sum(1, keepdims=True), 0.0)
        m = r.sum(1)
        assert m.min() > 1e-6
        r /= m[:, None]
    upto = np.cumsum(r, 1)
    at = np.minimum(np.float32(u[:, D]).astype(np.float64), 1.0)
    i = np.arange(N)
    end, off = upto[i, got[:, 0]], 1e-11 + 1e-13 / m
    assert (end - r[i, got[:, 0]] <= at + off).all() and (end >= at - off).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [4, 400])
@pytest.mark.parametrize("count", [5, 5000])
def test_residuals_of_alike_rows(count, N, dtype):
    """Rows p and q that are the same in `count` tokens and permuted in 40 others, so that the ratio of their sums is 1
    but for roundings and no sum in 32 bits tells which of the equal tokens is larger; uniforms anywhere and next to the
    borders of the residual's tokens."""
    torch = need_gpu()
    rng = np.random.default_rng(count + N)
    V, D = 20000, 1
    t = getattr(torch, dtype)
    p = np.full((N, D + 1, V), -np.inf)
    q = np.full((N, D, V), -np.inf)
    drafts = np.empty((N, D), np.int32)
    for i in range(N):
        at = rng.choice(V, count + 40, replace=False)
        p[i, 0, at] = rng.standard_normal(count + 40) * 2
        q[i, 0, at] = p[i, 0, at]
        few = at[:40]
        p[i, 0, few] += 4.0
        q[i, 0, few] = np.roll(p[i, 0, few], 1)
        drafts[i, 0] = few[np.argmax(q[i, 0, few] - p[i, 0, few])]
    x, y = on_gpu(torch, p.reshape(-1, V), t), on_gpu(torch, q.reshape(-1, V), t)
    u = rng.random((N, D + 1))
    u[:, 0] = 1 - 2.0 ** -24
    xs, ys = back(x).reshape(N, D + 1, V), back(y)
    for i in range(0, N, 2):
        r = np.maximum(spec_ref.softmax(xs[i, 0]) - spec_ref.softmax(ys[i]), 0)
        edges = np.cumsum(r) / r.sum()
        edge = np.float32(edges[rng.choice(np.nonzero(r > 1e-6)[0])])
        u[i, D] = min(np.nextafter(edge, np.float32(i % 4), dtype=np.float32) if i % 8 < 4 else edge, 1 - 2.0 ** -24)
    acc, _ = check(torch, x, drafts, u, y)
    assert (acc == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_what_is_left_may_be_little(dtype):
    """Proposals that have next to all of their row are rejected: the token comes from the rest, of which most lies far
    below the row's largest."""
    torch = need_gpu()
    rng = np.random.default_rng(11)
    N, D, V = 700, 1, 12000
    base = np.empty((N, D + 1, V))
    base[:, :, : V // 2] = -26.0 - 3.0 * rng.random((N, D + 1, V // 2))
    base[:, :, V // 2:] = -52.0 - rng.random((N, D + 1, V - V // 2))
    base[:, :, 7] = 0.0
    x = on_gpu(torch, base.reshape(-1, V), getattr(torch, dtype))
    u = rng.random((N, D + 1))
    u[:, 0] = 1.0  # not below p(7), which no uniform below 1 reaches here
    u[: N // 2, D] = 1 - 2.0 ** -24
    u[: N // 4, D] = 0.0
    drafts = np.full((N, D), 7, np.int32)
    acc, _ = check(torch, x, drafts, u)
    assert (acc == 0).all()


def test_no_vocabulary():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    for D in (0, 3):
        x, drafts = torch.zeros(2 * (D + 1), 0, device="cuda"), torch.zeros(2, D, dtype=torch.int32, device="cuda")
        u = torch.rand(2, D + 1, device="cuda")
        for kw in ({}, dict(uniforms=u), dict(uniforms=u, draft_logits=torch.zeros(2 * D, 0, device="cuda")),
                   dict(uniforms=u, parents=torch.full((2, D), -1, dtype=torch.int32, device="cuda"))):
            tokens, accepted, _ = tk.speculative_verify(x, drafts, **kw)
            assert (tokens == -1).all() and (accepted == 0).all()


def test_every_token_is_drawn_in_its_place():
    """One row, uniforms over all of [0, 1): each token's share, at the borders as well."""
    torch = need_gpu()
    rng = np.random.default_rng(3)
    V, N = 600, 4000
    row = head(rng, (V,), spikes=3, scale=1.0, high=2.0)
    x = on_gpu(torch, row[None], torch.float32).expand(N, V).contiguous()
    p = spec_ref.softmax(back(x[:1])[0])
    edges = np.float32(np.cumsum(p)[:-1])
    u = np.concatenate([np.linspace(0, 1, N - 2 * (V - 1), endpoint=False), np.nextafter(edges, np.float32(0)),
                        np.nextafter(edges, np.float32(2))])
    check(torch, x, np.zeros((N, 0), np.int32), np.minimum(u, 1 - 2.0 ** -24)[:, None])


@pytest.mark.parametrize("dtype", TYPES)
def test_longest_rows(dtype):
    torch = need_gpu()
    rng = np.random.default_rng(2)
    N, D, V = 2, 1, 1 << 20
    base = head(rng, (N, D + 1, V))
    y = base[:, :D] + rng.standard_normal((N, D, V))
    t = getattr(torch, dtype)
    x, gy = on_gpu(torch, base.reshape(-1, V), t, 1, 1), on_gpu(torch, y.reshape(-1, V), t)
    drafts = base[:, :D].argmax(2).astype(np.int32)
    for turn in range(3):
        u = rng.random((N, D + 1))
        check(torch, x, drafts, u, gy)
        check(torch, x, drafts, u)
    check(torch, x, drafts)


def test_many_sequences():
    """More workgroups than one launch holds, and rows of four tokens."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, D, V = 2_200_000, 1, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(N * (D + 1), V, device="cuda", generator=g)
    drafts = torch.randint(0, V, (N, D), device="cuda", generator=g, dtype=torch.int32)
    u = torch.rand(N, D + 1, device="cuda", generator=g)
    tokens, accepted, _ = tk.speculative_verify(x, drafts, u)
    at = torch.cat([torch.arange(1000), torch.arange(N // 2 - 500, N // 2 + 500), torch.arange(N - 1000, N)])
    xs = x.view(N, D + 1, V)[at.cuda()].double().cpu().numpy()
    rt, ra, _, margin = spec_ref.verify(xs, drafts.cpu().numpy()[at], u.cpu().numpy()[at])
    ok = margin > BORDER
    assert (tokens.cpu().numpy()[at][ok] == rt[ok]).all() and (accepted.cpu().numpy()[at][ok] == ra[ok]).all()


def test_rows_past_four_gigabytes():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    V, D, ld = 1000, 1, 1 << 20
    N = 700  # 1400 rows of 4 MiB
    x = torch.zeros(N * (D + 1), ld, device="cuda")[:, :V]
    g = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randn(N * (D + 1), V, device="cuda", generator=g) * 3)
    y = torch.zeros(N * D, ld, device="cuda", dtype=torch.float32)[:, 5:5 + V]
    y.copy_(x.view(N, 2, V)[:, 0] + torch.randn(N, V, device="cuda", generator=g))
    drafts = y.argmax(1).view(N, 1).to(torch.int32)
    u = torch.rand(N, D + 1, device="cuda", generator=g)
    tokens, accepted, _ = tk.speculative_verify(x, drafts, u, draft_logits=y)
    rt, ra, _, margin = spec_ref.verify(back(x).reshape(N, 2, V), drafts.cpu().numpy(), u.cpu().numpy(),
                                        back(y).reshape(N, 1, V))
    ok = margin > BORDER
    assert (tokens.cpu().numpy()[ok] == rt[ok]).all() and (accepted.cpu().numpy()[ok] == ra[ok]).all()


def test_outputs_streams_and_workspaces():
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    rng = np.random.default_rng(4)
    N, D, V = 3, 4, 5000
    base = head(rng, (N, D + 1, V))
    x = on_gpu(torch, base.reshape(-1, V), torch.bfloat16)
    y = on_gpu(torch, (base[:, :D] + rng.standard_normal((N, D, V))).reshape(-1, V), torch.bfloat16)
    drafts = torch.from_numpy(drafts_for(rng, base, D)).cuda()
    u = torch.rand(N, D + 1, device="cuda")
    want = tk.speculative_verify(x, drafts, u, draft_logits=y)
    out = (torch.full((N, D + 1), 9, dtype=torch.int32, device="cuda"),
           torch.full((N,), 9, dtype=torch.int32, device="cuda"), None)
    size = tk.speculative_verify_workspace(torch.bfloat16, N, D, V, draft_logits=True)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # holds nothing of use
    versions = out[0]._version, out[1]._version
    got = tk.speculative_verify(x, drafts, u, draft_logits=y, out=out, workspace=ws)
    assert got is out and out[0]._version > versions[0] and out[1]._version > versions[1]
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a = tk.speculative_verify(x, drafts, u, draft_logits=y, stream=s1)
    b = tk.speculative_verify(x, drafts, u, draft_logits=y, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for r in (a, b):
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])
    with pytest.raises(tk.TopKTopPError, match="workspace"):
        tk.speculative_verify(x, drafts, u, draft_logits=y, workspace=ws[:size - 16].clone())


def test_captured():
    """Calls in a graph, replayed with other inputs between eager work."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, D, V = 4, 3, 4000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(N * (D + 1), V, device="cuda", generator=g) * 3
    y = x.view(N, D + 1, V)[:, :D].reshape(-1, V) + torch.randn(N * D, V, device="cuda", generator=g)
    drafts = torch.randint(0, V, (N, D), device="cuda", dtype=torch.int32, generator=g)
    parents = torch.full((N, D), -1, dtype=torch.int32, device="cuda")
    u = torch.rand(N, D + 1, device="cuda", generator=g)

    def step():
        return (*tk.speculative_verify(x, drafts, u, draft_logits=y)[:2],
                *tk.speculative_verify(x, drafts, u, parents=parents), *tk.speculative_verify(x, drafts)[:2])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(4):
        x.normal_(generator=g).mul_(3)
        y.copy_(x.view(N, D + 1, V)[:, :D].reshape(-1, V) + torch.randn(N * D, V, device="cuda", generator=g))
        drafts.copy_(y.view(N, D, V).argmax(2))
        u.copy_(torch.rand(N, D + 1, device="cuda", generator=g))
        want = [t.clone() for t in step()]
        for t in held:
            t.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), turn
