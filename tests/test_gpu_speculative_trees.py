"""speculative_verify of trees that are large enough to be read step by step, with parents of any kind, against the
reference in 64 bits (needs an MI355X).

Decisions within 1e-12 of a border may go either way: the reference's sums of V = 20001 terms are within V 2^-53 = 2.3e-12
at the very most and, as their roundings are random, within 1e-13."""

import numpy as np
import pytest

from tests import spec_ref
from tests.gpu_util import need_gpu, say
from tests.test_gpu_speculative import Rows

pytestmark = pytest.mark.gpu

BORDER = 1e-12
KINDS = ("self", "later", "huge", "negative", "constant")


def odd_parents(kind, N, D, branch, rng):
    """Trees of `branch` drafts behind each, where some drafts' parents are none; what follows these stays."""
    j = np.arange(D)
    good = np.broadcast_to(j // branch - 1, (N, D)).astype(np.int64)
    if kind == "constant":
        return np.broadcast_to(rng.integers(0, 8, (N, 1)), (N, D)).astype(np.int32)
    wrong = rng.random((N, D)) < 0.15
    wrong[:, : 2 * branch: 2] = False  # paths go on for a while
    value = {
        "self": np.broadcast_to(j, (N, D)),
        "later": j + rng.integers(1, 300, (N, D)),
        "huge": rng.choice([255, 256, 1000, 2 ** 31 - 1], (N, D)),
        "negative": rng.choice([-2, -300, -2 ** 31], (N, D)),
    }[kind]
    return np.where(wrong, value, good).astype(np.int32)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("mib", [100, 200])  # one step behind the first rows, and two
@pytest.mark.parametrize("kind", KINDS)
def test_parents_that_are_not_there(kind, mib, greedy, dtype):
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    say("parents", kind, mib, greedy, dtype)
    t = getattr(torch, dtype)
    D, V, branch = 39, 20001, 3
    N = -(-mib * 2 ** 20 // ((D + 1) * V * t.itemsize))
    seed = mib + len(kind)
    rng, g = np.random.default_rng(seed), torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N * (D + 1), V, device="cuda", generator=g).mul_(3).to(t)
    parents = odd_parents(kind, N, D, branch, rng)
    # drafts out of the likeliest tokens of the rows that they follow, or would follow
    best = torch.topk(x.float(), branch, dim=1).indices.view(N, D + 1, branch).cpu().numpy()
    rows = np.where((parents >= -1) & (parents < np.arange(D)), parents + 1, np.arange(D) // branch)
    drafts = best[np.arange(N)[:, None], rows, np.arange(D) % branch].astype(np.int32)
    if kind == "constant":  # drafts up to the parent are not there; the token that the first row takes leads nowhere
        parents[: N // 2, 0] = -1
        parents[: N // 2, 1:] = 0
        drafts[: N // 2, 0] = best[: N // 2, 0, 0]
        drafts[: N // 2, 1:] = best[: N // 2, 1:2, 0]
    lengths = rng.integers(D - 9, D + 1, N).astype(np.int32)
    u = None if greedy else np.float32(rng.random((N, D + 1)) * rng.choice([0.02, 0.3], (N, D + 1)))
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()
    size = tk.speculative_verify_workspace(t, N, D, V)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    tokens, accepted, path = tk.speculative_verify(x, dev(drafts), dev(u), parents=dev(parents), lengths=dev(lengths),
                                                   workspace=ws)
    torch.cuda.synchronize()
    rt, ra, rp, margin = spec_ref.verify(Rows(x.view(N, D + 1, V), torch.arange(N, device="cuda")), drafts, u, None,
                                         parents, lengths)
    sure = margin > BORDER
    assert sure.mean() > 0.9
    # paths go on past the rows of each step
    assert (ra >= 1).sum() >= 3 and (kind == "constant" or (ra >= 2).sum() >= 2), ra
    assert (accepted.cpu().numpy()[sure] == ra[sure]).all()
    assert (tokens.cpu().numpy()[sure] == rt[sure]).all()
    assert (path.cpu().numpy()[sure] == rp[sure]).all()
