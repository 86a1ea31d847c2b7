"""speculative_verify without drafts, a draw from every row, against cumulative sums in 64 bits (needs an MI355X)."""

import numpy as np
import pytest

from tests.gpu_util import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_more_sequences_than_a_launch_holds(dtype):
    """N > 2^22 rows of 4 tokens. The sums of four terms are within 4 2^-53, the kernel's terms of 3e-14 of them: where a
    uniform is no closer than 1e-12 to a border, the token is certain."""
    torch = need_gpu()
    import top_logits_filtering_amd as tk

    N, V = (1 << 22) + 1037, 4
    say("many draws", dtype, N)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(N, V, device="cuda", generator=g).mul_(2).to(getattr(torch, dtype))
    u = torch.rand(N, 1, device="cuda", generator=g)
    none = torch.empty(N, 0, dtype=torch.int32, device="cuda")
    tokens, accepted, path = tk.speculative_verify(x, none, u)
    best, _, _ = tk.speculative_verify(x, none)
    torch.cuda.synchronize()
    xs = x.double().cpu().numpy()
    e = np.exp(xs - xs.max(1, keepdims=True))
    upto = np.cumsum(e, 1)
    at = u.double().cpu().numpy() * upto[:, -1:]
    want = (upto <= at).sum(1)
    sure = (np.abs(upto[:, :-1] - at) > 1e-12 * upto[:, -1:]).all(1)
    assert sure.mean() > 0.999
    assert (tokens.cpu().numpy()[:, 0][sure] == want[sure]).all()
    assert (best.cpu().numpy()[:, 0] == xs.argmax(1)).all()
    assert (accepted == 0).all() and path is None
