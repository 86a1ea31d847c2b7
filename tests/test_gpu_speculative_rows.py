"""Rows at the ends of what speculative_verify takes, against their weights in 64 bits (needs an MI355X)."""

import numpy as np
import pytest

from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu

TYPES = ("float32", "float16", "bfloat16")
LOWEST = {"float32": -3.4028234663852886e38, "float16": -65504.0, "bfloat16": -3.3895313892515355e38}


def drawn(torch, x, u, y=None, drafts=None, parents=None):
    """Tokens behind the last accepted draft, of rows x [N * (D + 1), V]; u [N, D + 1]."""
    import top_logits_filtering_amd as tk

    N = u.shape[0]
    D = u.shape[1] - 1
    i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    drafts = np.zeros((N, D), np.int32) if drafts is None else drafts
    tokens, accepted, _ = tk.speculative_verify(x, i32(drafts), torch.from_numpy(np.float32(u)).cuda(), draft_logits=y,
                                                parents=i32(parents))
    torch.cuda.synchronize()
    accepted = accepted.cpu().numpy()
    return tokens.cpu().numpy()[np.arange(N), accepted], accepted


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,N", [(5, 3), (20001, 3), (20001, 700), (151936, 2)])  # few workgroups and many
@pytest.mark.parametrize("kind", ["lowest", "largest", "one above", "far apart"])
def test_rows_of_the_largest_sizes(kind, V, N, dtype):
    """Logits so large that 70 less is the same number: rows all at the type's lowest or largest value are even ones, and
    one token above all others has all the weight. Even rows' borders are multiples of 1 / V: uniforms (k + 1/2) / V, off by
    2^-24 of themselves, are at least (1/2 - 2^-24 V) / V > 0.4 / V away."""
    torch = need_gpu()
    say("sizes", kind, V, N, dtype)
    rng = np.random.default_rng(V + N)
    low = LOWEST[dtype]
    k = rng.integers(0, V, N)
    u = ((k + 0.5) / V)[:, None]
    base = np.full((N, V), low if kind == "lowest" else -low)
    want = k
    if kind in ("one above", "far apart"):
        base[:] = low if kind == "one above" else -1e4
        want = rng.integers(0, V, N)
        base[np.arange(N), want] = low / 2 if kind == "one above" else -low
    x = torch.from_numpy(base).cuda().to(getattr(torch, dtype))
    assert torch.isfinite(x).all()
    got, accepted = drawn(torch, x, u)
    assert (accepted == 0).all() and (got == want).all()
    # with a draft that the target gives nothing, out of a row of its own: what is left is the target row
    if V > 5 and kind != "far apart":
        out = (want + 1) % V
        rows = np.repeat(base[:, None], 2, 1)
        rows[np.arange(N), 0, out] = -np.inf
        other = np.full((N, V), -np.inf)
        other[np.arange(N), out] = -low
        x = torch.from_numpy(rows.reshape(-1, V)).cuda().to(getattr(torch, dtype))
        y = torch.from_numpy(other).cuda().to(getattr(torch, dtype))
        if kind != "one above":  # one token fewer
            k = rng.integers(0, V - 1, N)
            u = ((k + 0.5) / (V - 1))[:, None]
            want = k + (k >= out)
        got, accepted = drawn(torch, x, np.repeat(u, 2, 1), y, out[:, None])
        assert (accepted == 0).all() and (got == want).all()


FAR = (0.0, 1e-45, 1.1e-30, 2.5e-29, 0.3, 1 - 2.0 ** -24, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [7, 700])  # few workgroups and many
@pytest.mark.parametrize("far", [-64.0, -100.0, -600.0])
@pytest.mark.parametrize("mode", ["plain", "proposal", "tree", "drawn", "drawn from masked"])
def test_tokens_far_below_the_others(mode, far, N, dtype):
    """Rows that begin and end with tokens far below the others, which no sum in 64 bits of the whole row shows, and
    uniforms that fall on them: 0 on the first token of any weight, 1 on the last, and others between.

    Weights are within 2e-14 of themselves and those of a draw within m 4e-14 of what is left, 1 / m of the row (m < 2000
    here: the drafts' share is above 1 / 2000): cumulative sums are sure to 1e-10 of themselves."""
    torch = need_gpu()
    say("far", mode, far, N, dtype)
    rng = np.random.default_rng(N + int(-far) + len(mode))
    V, D, t = 20000, 0 if mode == "plain" else 1, getattr(torch, dtype)
    base = rng.random((N, D + 1, V)).astype(np.float64)
    base[:, :, :9000] = base[:, :, -4000:] = far
    base[:, 0, 3] = base[:, 0, V - 2] = -np.inf
    base[1::2, 0, :2] = -np.inf  # the first token of any weight is another one
    draft = rng.integers(9000, V - 4000, N)
    i = np.arange(N)
    if D:
        base[i, 0, draft] = 4.0
    x = torch.from_numpy(base.reshape(-1, V)).cuda().to(t)
    xs = x.double().cpu().numpy().reshape(N, D + 1, V)[:, 0].astype(np.longdouble)
    softmax = lambda a: (lambda e: e / e.sum(1, keepdims=True))(np.exp(a - a.max(1, keepdims=True)))
    r = softmax(xs)
    u = np.full((N, D + 1), 1 - 2.0 ** -24)
    u[:, D] = np.resize(FAR, N)
    y = None
    if mode in ("proposal", "tree"):
        r[i, draft] = 0
    elif D:
        other = base[:, 0].copy()
        other[i, draft] = 7.0
        if mode == "drawn from masked":
            other[other < 0] = -np.inf
        y = torch.from_numpy(other).cuda().to(t)
        q = softmax(y.double().cpu().numpy().astype(np.longdouble))
        assert (q[i, draft] > r[i, draft]).all()
        r = np.maximum(r - q, 0)
        r[i, draft] = 0
        assert (r.sum(1) > 1 / 2000).all()
    got, accepted = drawn(torch, x, u, y, draft[:, None] if D else None, np.full((N, 1), -1) if mode == "tree" else None)
    assert (accepted == 0).all()
    upto = np.cumsum(r, 1)
    for k in range(N):
        uk = np.longdouble(np.float32(u[k, D]))
        weight = np.nonzero(r[k] > 0)[0]
        if uk >= 1:
            assert got[k] == weight[-1], k
            continue
        at = uk * upto[k, -1]
        want = weight[upto[k, weight] > at][0]
        if uk > 0:
            near = np.abs(upto[k, weight] - at) <= 1e-10 * at
            if near.any():
                continue
        assert got[k] == want, (k, float(uk), got[k], want)
