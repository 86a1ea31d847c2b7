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
