"""Cases of the beam search operators and their plain forms.

Three operators that a beam search runs at each step, next to the logits filter:
beam_search_select (the n best continuations over beams and vocabulary),
beam_reorder_states (the caches' rows follow the chosen parents, in place) and
beam_backtrace (the sequences read out of the steps' tokens and parents).
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_IDX_BITS = 20  # tokens are below 2^20


def listed():
    return [
        # one prompt on a toy vocabulary: the smallest call, nothing but latency
        dict(name="select N1 K4 V1000 f32", op="select", N=1, K=4, V=1000, pad=0, n=8, dtype="f32", done=0,
             weights=False),
        # one prompt being served with four beams, a large vocabulary: a few long rows for the whole chip
        dict(name="select N1 K4 V151936 bf16", op="select", N=1, K=4, V=151936, pad=0, n=8, dtype="bf16", done=0,
             weights=False),
        # 16 prompts, length-normalised, a quarter of the beams finished already
        dict(name="select N16 K4 V32000 f16 done", op="select", N=16, K=4, V=32000, pad=0, n=4, dtype="f16", done=1,
             weights=True),
        # odd everything: rows that start at any 2-byte address, views of a padded buffer
        dict(name="select N5 K7 V32003 bf16 padded", op="select", N=5, K=7, V=32003, pad=22, n=13, dtype="bf16",
             done=0, weights=False),
        # a serving batch: 64 prompts of four beams, 2K candidates each
        dict(name="select N64 K4 V151936 bf16", op="select", N=64, K=4, V=151936, pad=0, n=8, dtype="bf16", done=0,
             weights=False),
        # wide beams (retrieval, translation n-best lists)
        dict(name="select N2 K64 V151936 bf16 wide", op="select", N=2, K=64, V=151936, pad=0, n=128, dtype="bf16",
             done=0, weights=False),
        # the largest batch, fp32 logits
        dict(name="select N128 K8 V128256 f32", op="select", N=128, K=8, V=128256, pad=0, n=16, dtype="f32", done=0,
             weights=False),
        # one prompt's small cache, two layers
        dict(name="reorder N1 K4 T64", op="reorder", N=1, K=4, count=4, outer=0, H=4, T=64, D=64, layout="htd",
             lengths=True, dtype="bf16"),
        # eight prompts, the caches of 16 layers as separate tensors [rows, heads, positions, dim]
        dict(name="reorder N8 K4 T1024 layers", op="reorder", N=8, K=4, count=32, outer=0, H=8, T=1024, D=128,
             layout="htd", lengths=True, dtype="bf16"),
        # one tensor for all layers [layers, rows, positions, heads, dim], an odd head size, fp32
        dict(name="reorder N5 K6 T300 stacked", op="reorder", N=5, K=6, count=1, outer=24, H=3, T=300, D=75,
             layout="thd", lengths=True, dtype="f32"),
        # a short answer's history
        dict(name="backtrace T100 N4 K4", op="backtrace", T=100, N=4, K=4, M=4),
        # a batch of long answers
        dict(name="backtrace T2048 N64 K8", op="backtrace", T=2048, N=64, K=8, M=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "reorder", "backtrace"])
    if op == "select":
        dtype = rng.choice(["f32", "f16", "bf16"])
        K = _log_int(rng, 1, 64)
        V = _log_int(rng, 500, 262144)
        N = _log_int(rng, 1, max(1, min(128, 131_000_000 // (K * V))))
        n = rng.choice([K, 2 * K, _log_int(rng, 1, 128)])
        return dict(op=op, N=N, K=K, V=V, pad=rng.choice([0, 0, rng.randint(1, 64)]), n=n, dtype=dtype,
                    done=rng.choice([0, 0, rng.randint(0, K)]), weights=rng.random() < 0.3)
    if op == "reorder":
        dtype = rng.choice(["f32", "f16", "bf16"])
        N, K = _log_int(rng, 1, 16), _log_int(rng, 2, 16)
        H, D, T = rng.choice([1, 2, 3, 8]), rng.choice([64, 128, rng.randint(40, 200)]), _log_int(rng, 16, 1024)
        layout = rng.choice(["htd", "thd"])
        one = N * K * H * T * D * (4 if dtype == "f32" else 2)
        most = max(1, min(32, 2_100_000_000 // one))
        stacked = rng.random() < 0.4
        c = _log_int(rng, 1, most)
        return dict(op=op, N=N, K=K, count=1 if stacked else c, outer=c if stacked else 0, H=H, T=T, D=D,
                    layout=layout, lengths=rng.random() < 0.7, dtype=dtype)
    K = _log_int(rng, 1, 16)
    return dict(op=op, T=_log_int(rng, 16, 2048), N=_log_int(rng, 1, 64), K=K, M=rng.choice([1, K, _log_int(rng, 1, 16)]))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _spread(count, lo, hi, g):
    """`count` whole numbers from lo to hi, evenly apart, in an order made from the seed: their sum is always the same."""
    v = torch.linspace(lo, hi, count, dtype=torch.float64, device="cuda").round().to(torch.int32)
    return v[torch.randperm(count, generator=g, device="cuda")]


def _lengths_range(T):
    return max(1, T // 2), T


def _chain(K):
    """Parents before the beams are renamed: about six in ten beams go on, the best ones twice; beam 0 stays."""
    u = max(1, min(K - 1, math.ceil(0.6 * K)))
    return [b * u // K for b in range(K)]


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "select":
        N, K, V, pad = case["N"], case["K"], case["V"], case["pad"]
        # what a language model's head gives: a wide body and a few tokens that stand out
        x = torch.randn((N * K, V + pad), generator=g, device="cuda") * 2.5
        at = torch.randint(0, V, (N * K, 12), generator=g, device="cuda")
        x.scatter_(1, at, 9.0 + 3.0 * torch.randn((N * K, 12), generator=g, device="cuda"))
        x = x.to(_DTYPES[case["dtype"]])
        # sums of log-probabilities after some steps, the best beam first
        gaps = torch.empty((N, K), device="cuda").exponential_(2.0, generator=g)
        scores = -(12.0 + torch.cumsum(gaps, 1))
        done = None
        if case["done"]:
            order = torch.argsort(torch.rand((N, K), generator=g, device="cuda"), dim=1)
            done = order < case["done"]
        weights = None
        if case["weights"]:
            steps = torch.randint(5, 60, (N, K), generator=g, device="cuda").float()
            weights = ((5.0 + steps) / 6.0) ** -0.6
        out = (torch.empty((N, case["n"]), device="cuda"),
               torch.empty((N, case["n"]), dtype=torch.int32, device="cuda"),
               torch.empty((N, case["n"]), dtype=torch.int32, device="cuda"))
        return dict(case=case, logits=x[:, :V], scores=scores, done=done, end=min(2, V - 1), weights=weights, out=out)
    N, K = case["N"], case["K"]
    if case["op"] == "reorder":
        H, T, D = case["H"], case["T"], case["D"]
        inner = (H, T, D) if case["layout"] == "htd" else (T, H, D)
        shape = ((case["outer"],) if case["outer"] else ()) + (N * K,) + inner
        states = [torch.empty(shape, dtype=_DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
                  for _ in range(case["count"])]
        name = torch.argsort(torch.rand((N, K), generator=g, device="cuda"), dim=1)
        chain = torch.tensor(_chain(K), device="cuda").expand(N, K)
        parents = torch.empty((N, K), dtype=torch.int64, device="cuda")
        parents.scatter_(1, name, torch.gather(name, 1, chain))
        batch_dim = 1 if case["outer"] else 0
        seq_dim = batch_dim + (2 if case["layout"] == "htd" else 1)
        lengths = _spread(N, *_lengths_range(T), g) if case["lengths"] else None
        return dict(case=case, states=states, parents=parents.to(torch.int32), batch_dim=batch_dim, seq_dim=seq_dim,
                    lengths=lengths)
    T, M = case["T"], case["M"]
    tokens = torch.randint(0, 32000, (T, N, K), generator=g, dtype=torch.int32, device="cuda")
    # the best beams are parents more often
    u = torch.rand((T, N, K), generator=g, device="cuda")
    parents = (u * u * K).to(torch.int32).clamp_(max=K - 1)
    beams = torch.randint(0, K, (N, M), generator=g, dtype=torch.int32, device="cuda")
    lengths = _spread(N * M, *_lengths_range(T), g).view(N, M)
    out = torch.empty((N, M, T), dtype=torch.int32, device="cuda")
    return dict(case=case, tokens=tokens, parents=parents, beams=beams, lengths=lengths, out=out)


def run(state):
    op = state["case"]["op"]
    if own:
        import top_logits_filtering_amd as tk

        if op == "select":
            return tk.beam_search_select(state["logits"], state["scores"], state["case"]["n"], finished=state["done"],
                                         end_token=state["end"], weights=state["weights"], out=state["out"])
        if op == "reorder":
            return tk.beam_reorder_states(state["states"], state["parents"], batch_dim=state["batch_dim"],
                                          seq_dim=state["seq_dim"], lengths=state["lengths"])
        return tk.beam_backtrace(state["tokens"], state["parents"], beams=state["beams"], lengths=state["lengths"],
                                 out=state["out"])
    if op == "select":
        return _plain_select(state)
    if op == "reorder":
        return _plain_reorder(state)
    return _plain_backtrace(state)


def _plain_select(state):
    x, scores, n = state["logits"], state["scores"], state["case"]["n"]
    (N, K), V = scores.shape, x.shape[1]
    xf = x.float() + 0.0  # -0 counts as +0
    # the n largest logits of each beam, the lower token first among equal ones: value and token in one whole number
    bits = xf.view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) << _IDX_BITS
    key += (1 << _IDX_BITS) - 1 - torch.arange(V, device=x.device)
    m = min(n, V)
    token = (1 << _IDX_BITS) - 1 - (torch.topk(key, m, dim=1).values & ((1 << _IDX_BITS) - 1))
    # log of the sum of exp, in 64 bits: the order between beams hangs on it
    xd = xf.double()
    top = xd.amax(1, keepdim=True)
    total = (top + torch.log(torch.exp(xd - top).sum(1, keepdim=True)))
    value = torch.gather(xd, 1, token)
    c = scores.double().view(N * K, 1)
    w = torch.ones_like(c) if state["weights"] is None else state["weights"].double().view(N * K, 1)
    score = c + (value - total)
    alive = torch.isfinite(c) & torch.isfinite(w) & (w > 0)
    valid = alive & torch.isfinite(total) & (value > -math.inf)
    if state["done"] is not None:  # a finished beam goes on as itself and as nothing else
        done, first = state["done"].view(N * K, 1), torch.arange(m, device=x.device) == 0
        score = torch.where(done, c, score)
        token = torch.where(done, state["end"], token)
        valid = torch.where(done, alive & first, valid)
    rank = torch.where(valid, score * w, -math.inf).view(N, K * m)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :n]
    valid = torch.gather(valid.view(N, K * m), 1, order)
    score = torch.where(valid, torch.gather(score.view(N, K * m), 1, order), -math.inf).float()
    parent = torch.where(valid, order // m, -1).to(torch.int32)
    token = torch.where(valid, torch.gather(token.view(N, K * m), 1, order), -1).to(torch.int32)
    short = n - order.shape[1]
    if short > 0:
        score = torch.nn.functional.pad(score, (0, short), value=-math.inf)
        parent = torch.nn.functional.pad(parent, (0, short), value=-1)
        token = torch.nn.functional.pad(token, (0, short), value=-1)
    return score, parent, token


def _plain_reorder(state):
    parents, dim = state["parents"].long(), state["batch_dim"]
    N, K = parents.shape
    beam = torch.arange(K, device=parents.device).expand(N, K)
    parents = torch.where((parents >= 0) & (parents < K), parents, beam)
    source = (parents + K * torch.arange(N, device=parents.device)[:, None]).view(-1)
    keep = None
    if state["lengths"] is not None:
        s = state["states"][0]
        position = torch.arange(s.shape[state["seq_dim"]], device=s.device)
        keep = position[None, :] < state["lengths"].repeat_interleave(K)[:, None]
        keep = keep.view([s.shape[d] if d in (dim, state["seq_dim"]) else 1 for d in range(s.dim())])
    for s in state["states"]:
        moved = s.index_select(dim, source)
        s.copy_(moved if keep is None else torch.where(keep, moved, s))
    return state["states"]


def _plain_backtrace(state, pad=-1):
    tokens, parents = state["tokens"], state["parents"].long()
    (T, N, K), M = tokens.shape, state["case"]["M"]
    dev = tokens.device
    end, beams = state["lengths"].long() - 1, state["beams"].long()
    # Where a path is before step t+1, as a map of where it is after it: at a beam (0..K-1), not begun (K+m), or nowhere
    # (K+M). The maps of all steps after t, one after the other, are put together by doubling.
    nowhere = K + M
    at_beam = torch.where((parents >= 0) & (parents < K), parents, nowhere)
    at_beam = torch.cat([at_beam[1:], torch.arange(K, device=dev).expand(1, N, K)])
    begins = torch.arange(T, device=dev)[:, None, None] == end
    ok = (beams >= 0) & (beams < K)
    waiting = torch.where(begins, torch.where(ok, beams, nowhere), K + torch.arange(M, device=dev))
    where = torch.cat([at_beam, waiting, torch.full((T, N, 1), nowhere, device=dev)], 2)
    step = 1
    while step < T:
        where = torch.cat([torch.gather(where[:-step], 2, where[step:]), where[T - step:]])
        step *= 2
    path = where[:, :, K:K + M]
    found = torch.gather(tokens, 2, path.clamp(max=K - 1))
    return torch.where(path < K, found, pad).permute(1, 2, 0).contiguous()


def work(case):
    if case["op"] == "select":
        N, K, V, n = case["N"], case["K"], case["V"], case["n"]
        es = 4 if case["dtype"] == "f32" else 2
        rows = N * (K - case["done"])
        small = N * K * (4 + (1 if case["done"] else 0) + (4 if case["weights"] else 0))
        # an exponential, a sum and a comparison for each logit
        return {"bytes": rows * V * es + small + N * n * 12, "flops": rows * V * 3}
    if case["op"] == "reorder":
        N, K, T = case["N"], case["K"], case["T"]
        es = 4 if case["dtype"] == "f32" else 2
        lo, hi = _lengths_range(T)
        positions = sum(round(lo + (hi - lo) * i / max(1, N - 1)) for i in range(N)) if case["lengths"] else N * T
        chain = _chain(K)
        moved = [b for b in range(K) if chain[b] != b]
        rows = len(moved) + len({chain[b] for b in moved})  # written, and read
        one = case["H"] * case["D"] * es * positions * rows
        return {"bytes": one * max(1, case["outer"]) * case["count"] + N * K * 4, "flops": 0}
    T, N, M = case["T"], case["N"], case["M"]
    lo, hi = _lengths_range(T)
    steps = sum(round(lo + (hi - lo) * i / max(1, N * M - 1)) for i in range(N * M))
    return {"bytes": steps * 8 + N * M * (T * 4 + 8), "flops": 0}


def exact(case, seed):
    if case["op"] == "reorder":
        return None  # a copy: there is nothing that is computed
    s = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(case, s)
    tokens, parents = s["tokens"].cpu().numpy(), s["parents"].cpu().numpy()
    beams, lengths = s["beams"].cpu().numpy(), s["lengths"].cpu().numpy()
    T, N, M = case["T"], case["N"], case["M"]
    out = np.full((N, M, T), -1, dtype=np.int64)
    item = np.arange(N)[:, None]
    at = beams.copy()
    for t in range(T - 1, -1, -1):
        on = t < lengths
        out[:, :, t] = np.where(on, tokens[t][item, at], -1)
        at = np.where(on, parents[t][item, at], at)
    return torch.from_numpy(out.astype(np.int32))


def _exact_select(case, s):
    N, K, n = case["N"], case["K"], case["n"]
    if N * K * case["V"] > 300_000_000:
        return None
    c = s["scores"].cpu().numpy().astype(np.float64)
    w = np.ones((N, K)) if s["weights"] is None else s["weights"].cpu().numpy().astype(np.float64)
    done = np.zeros((N, K), bool) if s["done"] is None else s["done"].cpu().numpy()
    score, parent, token = np.full((N, n), -np.inf), np.full((N, n), -1, np.int32), np.full((N, n), -1, np.int32)
    for i in range(N):
        x = s["logits"][i * K:(i + 1) * K].double().cpu().numpy()
        found = []  # (rank, beam, logit, token, score)
        for b in range(K):
            if not np.isfinite(c[i, b]) or not 0 < w[i, b] < np.inf:
                continue
            if done[i, b]:
                found.append((-c[i, b] * w[i, b], b, 0.0, s["end"], c[i, b]))
                continue
            row = x[b]
            top = row.max()
            if not np.isfinite(top):
                continue
            total = top + np.log(np.exp(row - top).sum())
            least = np.partition(row, -n)[-n] if n < row.size else -np.inf
            for v in np.nonzero(row >= least)[0]:
                if row[v] > -np.inf:
                    own_score = c[i, b] + (row[v] - total)
                    found.append((-own_score * w[i, b], b, -row[v], int(v), own_score))
        found.sort()
        for r, f in enumerate(found[:n]):
            score[i, r], parent[i, r], token[i, r] = f[4], f[1], f[3]
    return score, torch.from_numpy(parent), torch.from_numpy(token)
