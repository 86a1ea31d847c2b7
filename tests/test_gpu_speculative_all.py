"""speculative_verify on odd rows, every sequence of it: also where roundings may decide, what comes has to be one of the
outcomes that they can give (needs an MI355X).

Terms are within 2e-14 of themselves, so a draw's cumulative sums are within 1e-13 of the row, and those of what q leaves of
p, 1 / m of it, within m 1e-13; the reference's sums of V = 3000 terms are within 1e-12. Where p and q of a token are the
same to 1e-12, only roundings tell whether anything is left of it."""

import numpy as np
import pytest

from tests.gpu_util import need_gpu, say
from tests.spec_ref import LEAST, softmax
from tests.test_gpu_speculative import KINDS, back, odd_rows, on_gpu

pytestmark = pytest.mark.gpu

BORDER = 1e-12


class Close(Exception):
    """An acceptance that roundings may decide."""


def accepts(a, b):
    """a < b."""
    if a != b and abs(a - b) <= BORDER * max(a, b):
        raise Close
    return a < b


def outcome(x, y, drafts, u, siblings):
    """(accepted drafts' numbers, p, what the token is drawn from, whether only roundings tell if a token has weight)."""
    D, path, row = len(drafts), [], 0
    while True:
        p = softmax(x[row])
        if p is None:
            return path, None, None, None
        none = np.zeros(len(p), bool)
        kids = ([] if path else list(range(D))) if siblings else ([row] if row < D else [])
        if not kids:
            return path, p, p, none
        r, noise, go = p.copy(), none, None
        if y is not None:
            q = softmax(y[row])
            q = np.zeros(len(p)) if q is None else q
            d = drafts[row]
            if accepts(u[row] * q[d], p[d]):
                go = row
            else:
                noise = (np.abs(p - q) <= BORDER * np.maximum(p, q)) & (p > 0)
                r = np.maximum(p - q, 0.0)
        else:
            low, seen = 0.0, set()
            for j in kids:
                d = int(drafts[j])
                if d in seen:
                    continue
                seen.add(d)
                high = low + p[d]
                if accepts(u[row], high) and go is None:
                    go = j
                low, r[d] = high, 0.0
        if go is None:
            if r.sum() <= LEAST * (1 - BORDER):
                return path, p, p, none
            if r.sum() <= LEAST * (1 + BORDER) or (noise.any() and p[noise].sum() * BORDER >= LEAST):
                raise Close
            return path, p, r, noise
        path.append(go)
        row = go + 1


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("V,times", [(11, 1), (11, 20), (3000, 1), (3000, 11)])  # few workgroups, and many
@pytest.mark.parametrize("kind", KINDS)
def test_every_sequence(kind, V, times, dtype):
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    say("all", kind, V, times, dtype)
    rng = np.random.default_rng(len(kind) + V)
    kinds, D = 2 * len(KINDS), 2
    base, other = np.empty((kinds, D + 1, V)), np.empty((kinds, D, V))
    for i in range(kinds):
        base[i] = [odd_rows(kind if w == i // len(KINDS) else "plain", V, rng) for w in range(D + 1)]
        other[i] = [odd_rows(KINDS[i % len(KINDS)], V, rng) for _ in range(D)]
    drafts = rng.integers(0, V, (kinds, D)).astype(np.int32)
    drafts[:, 0] = V // 2
    tile = lambda a: np.concatenate([a] * times)
    t = getattr(torch, dtype)
    x, y = on_gpu(torch, tile(base).reshape(-1, V), t, 1, 1), on_gpu(torch, tile(other).reshape(-1, V), t)
    xs, ys = back(x).reshape(-1, D + 1, V)[:kinds], back(y).reshape(-1, D, V)[:kinds]
    gd = torch.from_numpy(tile(drafts)).cuda()
    parents = torch.full((kinds * times, D), -1, dtype=torch.int32, device="cuda")
    certain = total = 0
    for u in (rng.random((kinds, D + 1)), np.zeros((kinds, D + 1)), np.full((kinds, D + 1), 1 - 2.0 ** -24)):
        u = np.float32(u)
        gu = torch.from_numpy(tile(u)).cuda()
        for kw in (dict(draft_logits=y), {}, dict(parents=parents)):
            got = [a.cpu().numpy() if a is not None else None for a in tk.speculative_verify(x, gd, gu, **kw)]
            tokens, accepted = got[0].reshape(times, kinds, D + 1), got[1].reshape(times, kinds)
            assert (tokens == tokens[0]).all() and (accepted == accepted[0]).all()
            for i in range(kinds):
                row, n = tokens[0, i], int(accepted[0, i])
                total += 1
                assert 0 <= n <= D and (row[n + 1:] == -1).all() and -1 <= row[n] < V
                try:
                    path, p, r, noise = outcome(xs[i], ys[i] if "draft_logits" in kw else None, drafts[i],
                                                u[i].astype(np.float64), "parents" in kw)
                except Close:
                    continue
                assert n == len(path) and (row[:n] == drafts[i, path]).all(), (i, row, path)
                if got[2] is not None:
                    assert (got[2].reshape(times, kinds, D)[0, i] == path + [-1] * (D - n)).all()
                if p is None:
                    assert row[n] == -1
                    certain += 1
                    continue
                v, upto = int(row[n]), np.cumsum(r)
                m, at = upto[-1], float(u[i, D]) * upto[-1]
                off = BORDER * m + 1e-13 * p.sum()
                assert v >= 0 and (r[v] > 0 or noise[v]), (i, v)
                assert upto[v] - r[v] <= at + off and at - off <= upto[v], (i, v, at, upto[v])
                if u[i, D] == 0:  # nothing that has weight for certain lies before it
                    assert not ((r[:v] > 0) & ~noise[:v]).any(), (i, v)
                    certain += not noise[:v + 1].any()
                else:
                    certain += bool(upto[v] - r[v] <= at - off and at + off < upto[v])
    assert certain >= 0.8 * total, (certain, total)
