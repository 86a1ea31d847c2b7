"""Cases of the speculative decoding and paged cache operators and their plain forms.

speculative_verify decides how many drafted tokens stand and picks the token behind them; cache_pages_fork lets the
rows of a page table follow their beams, cache_pages_resize gives rows the pages that they need and takes back those
that they do not, and cache_pages_compact moves the cache entries of an accepted path behind one another.
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_LEAST = 2.0 ** -40  # a residual of no more mass than this counts as none


def listed():
    return [
        # one prompt on a toy vocabulary, greedy: the smallest call, nothing but latency
        dict(name="verify N1 D3 V1000 f32 greedy", op="verify", N=1, D=3, V=1000, pad=0, dtype="f32", mode="greedy",
             branch=0, keep=0, ragged=False),
        # one conversation being served, five tokens drafted by a small model
        dict(name="verify N1 D5 V151936 bf16", op="verify", N=1, D=5, V=151936, pad=0, dtype="bf16", mode="draft",
             branch=0, keep=0, ragged=False),
        # tokens looked up in the prompt, as many as were found, logits filtered to the 50 best; odd rows of a padded buffer
        dict(name="verify N17 D8 V32003 f16 lookup filtered", op="verify", N=17, D=8, V=32003, pad=22, dtype="f16",
             mode="lookup", branch=0, keep=50, ragged=True),
        # a serving batch with a draft model
        dict(name="verify N64 D4 V151936 bf16", op="verify", N=64, D=4, V=151936, pad=0, dtype="bf16", mode="draft",
             branch=0, keep=0, ragged=False),
        # trees of 39 drafted tokens, three behind each
        dict(name="verify N32 D39 V151936 bf16 tree", op="verify", N=32, D=39, V=151936, pad=0, dtype="bf16",
             mode="lookup", branch=3, keep=0, ragged=False),
        # the largest batch, fp32 logits
        dict(name="verify N128 D3 V128256 f32", op="verify", N=128, D=3, V=128256, pad=0, dtype="f32", mode="draft",
             branch=0, keep=0, ragged=False),
        # one prompt of four beams, a short answer
        dict(name="fork N1 K4 C64", op="fork", N=1, K=4, C=64, S=16),
        # a batch of long answers
        dict(name="fork N64 K8 C2048", op="fork", N=64, K=8, C=2048, S=16),
        # a speculative step of a serving batch: room for five more tokens, then all of it given back
        dict(name="resize R64 C256 P16384", op="resize", N=64, K=1, C=256, S=16, P=16384, grow=5, count=0, H=0, D=0,
             layout="", dtype=""),
        # a step of a beam search: fork, room for one more token (shared last pages are copied), and back
        dict(name="resize N16 K4 C64 copies", op="resize", N=16, K=4, C=64, S=16, P=2304, grow=1, count=32, H=8, D=128,
             layout="shd", dtype="bf16"),
        # one conversation's accepted path, two layers
        dict(name="compact N1 D12", op="compact", N=1, D=12, C=16, S=16, count=4, H=4, E=64, layout="hsd",
             dtype="bf16"),
        # a serving batch, the caches of 32 layers
        dict(name="compact N64 D39 layers", op="compact", N=64, D=39, C=16, S=16, count=64, H=8, E=128, layout="shd",
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["verify", "verify", "verify", "fork", "resize", "compact"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "verify":
        mode = rng.choice(["draft", "draft", "lookup", "greedy"])
        branch = rng.choice([0, 1, 2, 3, 4]) if mode != "draft" else 0
        D = _log_int(rng, 1, 48 if branch > 1 else 10)
        V = _log_int(rng, 500, 262144)
        rows = 2 * D + 1 if mode == "draft" else D + 1
        N = _log_int(rng, 1, max(1, min(128, 110_000_000 // (rows * V))))
        return dict(op=op, N=N, D=D, V=V, pad=rng.choice([0, 0, rng.randint(1, 64)]), dtype=dtype, mode=mode,
                    branch=branch, keep=rng.choice([0, 0, rng.randint(20, 200)]), ragged=rng.random() < 0.4)
    S = rng.choice([8, 16, 16, 32, rng.randint(1, 40)])
    if op == "fork":
        return dict(op=op, N=_log_int(rng, 1, 64), K=_log_int(rng, 1, 16), C=_log_int(rng, 4, 1024), S=S)
    layout = rng.choice(["shd", "hsd"])
    H, E = rng.choice([1, 2, 3, 8]), rng.choice([64, 128, rng.randint(40, 200)])
    if op == "resize":
        C = _log_int(rng, 4, 256)
        if rng.random() < 0.5:
            N = _log_int(rng, 1, 128)
            return dict(op=op, N=N, K=1, C=C, S=S, P=_log_int(rng, N * C + 64, N * C + 16384), grow=rng.randint(1, 12),
                        count=0, H=0, D=0, layout="", dtype="")
        N, K, C = _log_int(rng, 1, 16), rng.randint(2, 6), min(C, 32)
        P = N * K * C + 64
        one = P * S * H * E * (4 if dtype == "f32" else 2)
        return dict(op=op, N=N, K=K, C=C, S=S, P=P, grow=rng.randint(1, 3),
                    count=_log_int(rng, 1, max(1, min(32, 1_000_000_000 // one))), H=H, D=E, layout=layout, dtype=dtype)
    N, D = _log_int(rng, 1, 64), _log_int(rng, 3, 48)
    C = (2 * D + 20) // S + 2
    one = N * C * S * H * E * (4 if dtype == "f32" else 2)
    return dict(op=op, N=N, D=D, C=C, S=S, count=_log_int(rng, 1, max(1, min(64, 1_000_000_000 // one))), H=H, E=E,
                layout=layout, dtype=dtype)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _evenly(count, lo, hi):
    """`count` whole numbers from lo to hi, evenly apart; one alone lies in the middle."""
    return [round(lo + (hi - lo) * i / (count - 1)) for i in range(count)] if count > 1 else [(lo + hi + 1) // 2]


def _spread(count, lo, hi, g):
    """Whole numbers evenly apart, in an order made from the seed: their sum is always the same."""
    v = torch.tensor(_evenly(count, lo, hi), dtype=torch.int32, device="cuda")
    return v[torch.randperm(count, generator=g, device="cuda")]


def _spread_sum(count, lo, hi, f):
    return sum(f(v) for v in _evenly(count, lo, hi))


def _full_levels(D, branch):
    """Levels that are full in a tree of D drafts with `branch` behind each: paths that long exist along every branch."""
    levels, width, held = 0, branch, 0
    while held + width <= D:
        held += width
        width *= branch
        levels += 1
    return levels


def _draft_counts(case):
    """Fewest drafts of a sequence; they are spread from there to D."""
    return (case["D"] // 2 if case["branch"] <= 1 else case["D"]) if case["ragged"] else case["D"]


def _rand(shape, g, dtype=torch.float64):
    return torch.rand(shape, generator=g, device="cuda", dtype=dtype)


def _pick(weights, g):
    """A token of each row, drawn by its weight."""
    noise = torch.empty(weights.shape, device="cuda", dtype=torch.float64).exponential_(generator=g)
    return (weights / noise.clamp_(min=1e-300)).argmax(-1)


def _largest(x):
    """The largest value's index in each row, the lowest among equal ones."""
    index = torch.arange(x.shape[-1], device=x.device, dtype=torch.int32)
    found = torch.where(x == x.amax(-1, keepdim=True), index, x.shape[-1] - 1)
    return found.amin(-1).long()


def _head_logits(rows, V, g):
    """What a language model's head gives: a wide body and a few tokens that stand out."""
    x = torch.randn((rows, V), generator=g, device="cuda") * 2.5
    at = torch.randint(0, V, (rows, 12), generator=g, device="cuda")
    out = 9.0 + 3.0 * torch.randn((rows, 12), generator=g, device="cuda")
    return x.scatter_reduce_(1, at, out, "amax")


def _filtered(x, keep):
    if keep == 0:
        return x
    least = torch.topk(x, min(keep, x.shape[1]), dim=1).values[:, -1:]
    return torch.where(x >= least, x, -math.inf)


def _prepare_verify(case, g):
    N, D, V, dtype = case["N"], case["D"], case["V"], _DTYPES[case["dtype"]]
    dev = "cuda"
    lengths = _spread(N, _draft_counts(case), D, g)
    drafts = torch.randint(0, V, (N, D), generator=g, device=dev)
    uniforms = _rand((N, D + 1), g)
    x = torch.empty((N, D + 1, V + case["pad"]), dtype=dtype, device=dev)
    y = torch.empty((N, D, V), dtype=dtype, device=dev) if case["mode"] == "draft" else None
    parents = None
    if case["branch"]:
        parents = (torch.arange(D, device=dev) // case["branch"] - 1).to(torch.int32).expand(N, D).contiguous()
    # as many drafts as these stand, whatever the seed
    if case["branch"]:
        accepted = _spread(N, 0, min(_full_levels(D, case["branch"]), 6), g)
    else:
        accepted = (lengths * _spread(N, 0, 100, g).double() / 100).round().to(torch.int32)
    accepted = torch.minimum(accepted, lengths)
    depth = torch.zeros((N, D + 1), dtype=torch.int32, device=dev)
    item = torch.arange(N, device=dev)
    for w in range(D + 1):
        row = _head_logits(N, V, g)
        if y is not None and w < D:
            y[:, w] = _filtered(row, case["keep"]).to(dtype)
            row = row + 0.7 * torch.randn(row.shape, generator=g, device=dev)
        x[:, w].normal_(generator=g)
        x[:, w, :V] = _filtered(row, case["keep"]).to(dtype)
        p = torch.softmax(x[:, w, :V].double(), 1)
        room = 0.02 + 0.96 * _rand((N,), g)
        if case["branch"]:
            if w > 0:
                depth[:, w] = depth[:, (w - 1) // case["branch"]] + 1
            first, last = w * case["branch"], min(D, (w + 1) * case["branch"])
            if first >= last:
                continue
            on = depth[:, w] < accepted
            noise = torch.empty(p.shape, device=dev, dtype=torch.float64).exponential_(generator=g)
            found = torch.topk(p / noise, last - first, dim=1).indices
            if case["mode"] == "greedy":  # the child that goes on, if any, is the largest logit
                top = _largest(x[:, w, :V])
                found = torch.where(found == top[:, None], (found + 1) % V, found)
                child = torch.randint(0, last - first, (N,), generator=g, device=dev)
                found[item, child] = torch.where(on, top, found[item, child])
            drafts[:, first:last] = found
            chance = torch.gather(p, 1, found)
            upto = torch.cumsum(chance, 1)
            child = _pick(chance, g)
            low, width = (upto - chance)[item, child], chance[item, child]
            total = upto[:, -1]
            uniforms[:, w] = torch.where(on, low + width * room, total + (1 - total) * room)
            continue
        if w == D:
            continue
        on = w < accepted
        if case["mode"] == "greedy":
            top = _largest(x[:, w, :V])
            drafts[:, w] = torch.where(on, top, (top + 1 + drafts[:, w] % (V - 1)) % V)
            continue
        if y is not None:  # accepted tokens follow min(p, q), rejected ones max(q - p, 0)
            q = torch.softmax(y[:, w].double(), 1)
            token = torch.where(on, _pick(torch.minimum(p, q), g), _pick((q - p).clamp_(min=0), g))
            ratio = (p[item, token] / q[item, token]).nan_to_num(1.0)
        else:
            token = torch.where(on, _pick(p, g), _pick(p * (1 - p), g))
            ratio = p[item, token]
        drafts[:, w] = token
        uniforms[:, w] = torch.where(on, ratio.clamp(max=1) * room, ratio + (1 - ratio) * room)
    out = (torch.empty((N, D + 1), dtype=torch.int32, device=dev), torch.empty((N,), dtype=torch.int32, device=dev),
           torch.empty((N, D), dtype=torch.int32, device=dev) if case["branch"] else None)
    return dict(case=case, logits=x.view(N * (D + 1), -1)[:, :V], drafts=drafts.to(torch.int32),
                uniforms=None if case["mode"] == "greedy" else uniforms.float().clamp_(max=1 - 2.0 ** -24),
                draft_logits=None if y is None else y.view(N * D, V), parents=parents,
                lengths=lengths if case["ragged"] else None, out=out)


def _chain(K):
    """Parents before the beams are renamed: about six in ten beams go on, the best ones twice; beam 0 stays."""
    u = max(1, min(K - 1, math.ceil(0.6 * K)))
    return [b * u // K for b in range(K)]


def _parents(N, K, g):
    name = torch.argsort(_rand((N, K), g), dim=1)
    chain = torch.tensor(_chain(K), device="cuda").expand(N, K)
    parents = torch.empty((N, K), dtype=torch.int64, device="cuda")
    parents.scatter_(1, name, torch.gather(name, 1, chain))
    return parents.to(torch.int32)


def _tokens_range(case):
    """Tokens that a row holds: from half of its table to all but what it is going to grow by."""
    most = case["C"] * case["S"] - case.get("grow", 0)
    return max(1, most // 2), most


def _pool(N, K, lengths, C, S, P, g):
    """Tables and uses of N prompts of K beams; the beams of a prompt share the first half of their pages."""
    dev = "cuda"
    held = (lengths + S - 1) // S  # [N]
    shared = held // 2 if K > 1 else held * 0
    column = torch.arange(C, device=dev)
    beam = torch.arange(K, device=dev)
    mine = (column >= shared[:, None, None]) | (beam == 0)[None, :, None]
    mine = mine & (column < held[:, None, None])
    number = torch.cumsum(mine.view(-1), 0).view(N, K, C) - 1
    pages = torch.randperm(P, generator=g, device=dev)  # a pool that has been in use for a while
    table = torch.where(mine, pages[number.clamp(min=0)], -1)
    table = torch.where((column < shared[:, None])[:, None], table[:, :1], table)
    table = torch.where(column < held[:, None, None], table, -1).view(N * K, C).to(torch.int32)
    uses = torch.zeros(P + 1, dtype=torch.int32, device=dev)
    uses.scatter_add_(0, torch.where(table >= 0, table, P).view(-1).long(),
                      torch.ones(N * K * C, dtype=torch.int32, device=dev))
    return table, uses[:P].clone()


def _caches(case, P, dim, g):
    S, H = case["S"], case["H"]
    shape = (P, S, H, dim) if case["layout"] == "shd" else (P, H, S, dim)
    return [torch.empty(shape, dtype=_DTYPES[case["dtype"]], device="cuda").normal_(generator=g)
            for _ in range(case["count"])]


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    N, C, S = case["N"], case["C"], case["S"]
    slot_dim = 1 if case.get("layout", "") != "hsd" else 2
    if case["op"] == "compact":
        D, P = case["D"], N * C
        table, _ = _pool(N, 1, torch.full((N,), C * S, device="cuda"), C, S, P, g)
        starts = _spread(N, 0, C * S - D, g)
        # paths as a tree of three behind each gives them; how many entries of them move does not depend on the seed
        counts = _spread(N, 0, _path_length(D), g)
        path = torch.full((N, D), -1, dtype=torch.int32, device="cuda")
        at = torch.full((N,), -1, dtype=torch.int64, device="cuda")
        for k in range(_path_length(D)):
            at = 3 * (at + 1) + (1 if k == 0 else torch.randint(0, 3, (N,), generator=g, device="cuda"))
            path[:, k] = torch.where(k < counts, at, -1)
        return dict(case=case, caches=_caches(case, P, case["E"], g), table=table, starts=starts, path=path,
                    counts=counts, slot_dim=slot_dim)
    K = case["K"]
    held = _spread(N, *_tokens_range(case), g)
    P = case.get("P", N * K * C + 64)
    table, uses = _pool(N, K, held, C, S, P, g)
    lengths = held.repeat_interleave(K)
    state = dict(case=case, table=table, uses=uses, lengths=lengths, parents=_parents(N, K, g))
    if case["op"] == "resize":
        state["before"], state["after"] = lengths.clone(), lengths + case["grow"]
        state["caches"] = _caches(case, P, case["D"], g) if case["count"] else None
        state["slot_dim"] = slot_dim
    return state


def _path_length(D):
    """Levels of three behind each that D drafts fill."""
    return _full_levels(D, 3) if D >= 3 else 0


def run(state):
    op = state["case"]["op"]
    if own:
        import top_logits_filtering_amd as tk

        if op == "verify":
            return tk.speculative_verify(state["logits"], state["drafts"], state["uniforms"],
                                         draft_logits=state["draft_logits"], parents=state["parents"],
                                         lengths=state["lengths"], out=state["out"])
        S = state["case"]["S"]
        if op == "compact":
            return tk.cache_pages_compact(state["caches"], state["table"], state["starts"], state["path"],
                                          state["counts"], slot_dim=state["slot_dim"])
        if op == "fork" or state["caches"] is not None:
            tk.cache_pages_fork(state["table"], state["lengths"], state["parents"], state["uses"], S)
        if op == "resize":
            for new in (state["after"], state["before"]):
                tk.cache_pages_resize(state["table"], state["lengths"], new, state["uses"], S, caches=state["caches"],
                                      slot_dim=state["slot_dim"])
            return state["table"], state["lengths"], state["uses"], state["caches"] or []
        return state["table"], state["lengths"], state["uses"]
    if op == "verify":
        return _plain_verify(state)
    if op == "compact":
        return _plain_compact(state)
    if op == "fork" or state["caches"] is not None:
        _plain_fork(state)
    if op == "resize":
        for new in (state["after"], state["before"]):
            _plain_resize(state, new)
        return state["table"], state["lengths"], state["uses"], state["caches"] or []
    return state["table"], state["lengths"], state["uses"]


def _distribution(x):
    """softmax of each row in 64 bits; a row with a NaN or +inf, or with nothing above -inf, has none: all zeros."""
    x = x.double()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    return torch.where(torch.isfinite(top), e / e.sum(-1, keepdim=True), 0.0)


def _plain_verify(state):
    drafts = state["drafts"].long()
    N, D = drafts.shape
    x = state["logits"].view(N, D + 1, -1)
    V, dev = x.shape[2], x.device
    index = torch.arange(D, device=dev)
    live = index < (D if state["lengths"] is None else state["lengths"].clamp(0, D)[:, None])
    live = live & (drafts >= 0) & (drafts < V)
    token = drafts.clamp(0, V - 1)
    parent = (index - 1).expand(N, D) if state["parents"] is None else state["parents"].long()
    live = live & (parent >= -1) & (parent < index)
    node = (parent + 1).clamp(0, D)  # the row that a draft follows
    item = torch.arange(N, device=dev)
    greedy = state["uniforms"] is None
    # drafts that follow the same row, earlier ones, and which of them have the same token
    sibling = (node[:, :, None] == node[:, None, :]) & (index[:, None] > index) & live[:, None, :]
    first = live & ~(sibling & (token[:, :, None] == token[:, None, :])).any(2)
    if greedy:
        best = torch.where(torch.isfinite(x.amax(-1)), _largest(x), -1)
        taken = first & (torch.gather(best, 1, node) == token)
    else:
        p = _distribution(x)
        u = state["uniforms"].double()
        chance = p[item[:, None], node, token]
        if state["draft_logits"] is None:
            chance = torch.where(first, chance, 0.0)
            low = (chance[:, None, :] * sibling).sum(2)
            of = torch.gather(u, 1, node)
            taken = first & (of >= low) & (of < low + chance)
        else:
            q = _distribution(state["draft_logits"].view(N, D, V))
            taken = live & (u[:, :D] * torch.gather(q, 2, token[:, :, None])[:, :, 0] < chance)
    # on the path: taken, as are all drafts before it
    on, up = taken, torch.where(parent >= 0, parent, D)
    one, end = torch.ones((N, 1), dtype=torch.bool, device=dev), torch.full((N, 1), D, device=dev)
    for _ in range(max(1, D).bit_length()):
        on = on & torch.gather(torch.cat([on, one], 1), 1, up)
        up = torch.gather(torch.cat([up, end], 1), 1, up)
    count = on.sum(1)
    order = torch.sort((~on).to(torch.int8), dim=1, stable=True).indices
    standing = index < count[:, None]
    path = torch.where(standing, order, -1)
    stop = torch.where(on, index + 1, 0).amax(1) if D else torch.zeros(N, dtype=torch.int64, device=dev)
    if greedy:
        final = best[item, stop]
    else:
        r = p[item, stop]
        if state["draft_logits"] is not None:
            ends = stop < live.cumprod(1).sum(1)  # a draft was rejected here
            less = torch.where(ends[:, None], q[item, stop.clamp(max=max(D - 1, 0))], 0.0)
            residual = (r - less).clamp_(min=0)
        else:
            out = first & (node == stop[:, None])
            residual = r.clone()
            residual.scatter_reduce_(1, token, torch.where(out, 0.0, math.inf).double(), "amin")
        r = torch.where(residual.sum(1, keepdim=True) > _LEAST, residual, r)
        upto = torch.cumsum(r, 1)
        at = upto[:, -1:] * u[:, D:]
        final = torch.where(upto[:, -1] > 0, (upto <= at).sum(1).clamp_(max=V - 1), -1)
    tokens = torch.full((N, D + 1), -1, dtype=torch.int64, device=dev)
    tokens[:, :D] = torch.where(standing, torch.gather(token, 1, order), -1)
    tokens.scatter_(1, count[:, None], final[:, None])
    path = None if state["parents"] is None else path.to(torch.int32)
    return tokens.to(torch.int32), count.to(torch.int32), path


def _plain_fork(state):
    table, lengths, uses, parents = state["table"], state["lengths"], state["uses"], state["parents"].long()
    (N, K), C = parents.shape, table.shape[1]
    beam = torch.arange(K, device=table.device).expand(N, K)
    parents = torch.where((parents >= 0) & (parents < K), parents, beam)
    source = (parents + K * torch.arange(N, device=table.device)[:, None]).view(-1)
    spare = torch.zeros(len(uses) + 1, dtype=torch.int32, device=table.device)
    moved = table[source]
    for t, step in ((moved, 1), (table, -1)):
        spare.scatter_add_(0, torch.where(t >= 0, t, len(uses)).view(-1).long(),
                           torch.full((N * K * C,), step, dtype=torch.int32, device=table.device))
    uses += spare[:-1]
    table.copy_(moved)
    lengths.copy_(lengths[source])


def _plain_resize(state, new):
    table, lengths, uses, S = state["table"], state["lengths"], state["uses"], state["case"]["S"]
    (R, C), P, dev = table.shape, len(uses), table.device
    column = torch.arange(C, device=dev)
    old_pages, new_pages = (lengths + S - 1) // S, (new + S - 1) // S
    ok = (new >= 0) & (new_pages <= C)
    spare = torch.zeros(P + 1, dtype=torch.int32, device=dev)  # one more for what is none
    spare[:P] = uses
    # pages behind the new end
    gone = (ok & (new < lengths))[:, None] & (column >= new_pages[:, None]) & (column < old_pages[:, None]) & (table >= 0)
    spare.scatter_add_(0, torch.where(gone, table, P).view(-1).long(),
                       torch.full((R * C,), -1, dtype=torch.int32, device=dev))
    table.masked_fill_(gone, -1)
    # rows that write into a page that others use too: all copy it, but the last one if they are all that use it
    grows = ok & (new > lengths)
    tail = torch.gather(table, 1, (old_pages - 1).clamp(min=0)[:, None].long())[:, 0]
    has = grows & (lengths % S != 0) & (tail >= 0)
    tail = torch.where(has, tail, P).long()
    row = torch.arange(R, device=dev)
    writers = torch.zeros(P + 1, dtype=torch.int32, device=dev).scatter_add_(0, tail, has.to(torch.int32))
    last = torch.full((P + 1,), -1, device=dev).scatter_reduce_(0, tail, row, "amax")
    copies = has & ~((writers[tail] == spare[tail]) & (last[tail] == row))
    need = torch.where(grows, new_pages - old_pages + copies, 0)
    upto = torch.cumsum(need, 0)
    free = (spare[:P] == 0).sum()
    grows = grows & (upto <= free)
    if state["caches"] is None:  # nobody could copy
        grows = grows & ~(torch.cumsum(copies, 0) > 0)
    copies = copies & grows
    pages = torch.sort((spare[:P] != 0).to(torch.int8), stable=True).indices.to(torch.int32)
    first = upto - need
    new_tail = pages[first.clamp(max=P - 1).long()]
    number = first[:, None] + copies[:, None] + column - old_pages[:, None]
    added = grows[:, None] & (column >= old_pages[:, None]) & (column < new_pages[:, None])
    table.copy_(torch.where(added, pages[number.clamp(0, P - 1).long()], table))
    at_tail = copies[:, None] & (column == (old_pages - 1)[:, None])
    table.copy_(torch.where(at_tail, new_tail[:, None], table))
    spare.scatter_add_(0, torch.where(added | at_tail, table, P).view(-1).long(),
                       torch.ones(R * C, dtype=torch.int32, device=dev))
    spare.scatter_add_(0, torch.where(copies, tail, P), torch.full((R,), -1, dtype=torch.int32, device=dev))
    uses.copy_(spare[:P])
    if state["caches"] is not None:
        # rows that copy nothing repeat the first copy, or put page 0 onto itself if there is none
        some = copies.to(torch.int8).argmax()
        source = torch.where(copies, tail, torch.where(copies[some], tail[some], 0))
        target = torch.where(copies, new_tail, torch.where(copies[some], new_tail[some], 0)).long()
        kept = torch.where(copies, lengths % S, torch.where(copies[some], (lengths % S)[some], 0))
        for c in state["caches"]:
            keep = torch.arange(S, device=dev) < kept[:, None]
            shape = [R] + [S if d == state["slot_dim"] else 1 for d in range(1, c.dim())]
            c[target] = torch.where(keep.view(shape), c[source.clamp(max=P - 1)], c[target])
    lengths.copy_(torch.where(grows | (ok & (new < lengths)), new, lengths))


def _plain_compact(state):
    table, starts, path, counts = state["table"], state["starts"], state["path"].long(), state["counts"]
    S, D = state["case"]["S"], path.shape[1]
    step = torch.arange(D, device=table.device)
    moves = step < counts[:, None]
    source = starts[:, None] + torch.where(moves, path, 0)
    target = starts[:, None] + torch.where(moves, step, 0)

    def place(position):
        page = torch.gather(table, 1, (position // S).long())
        return page.long().view(-1), (position % S).long().view(-1)

    (page_from, slot_from), (page_to, slot_to) = place(source), place(target)
    # entries that do not move put the sequence's first one, wherever it comes from, to where it belongs
    stay = ~moves.view(-1)
    head = torch.arange(len(starts), device=table.device).repeat_interleave(D) * D
    source_of = torch.where(stay & (counts.repeat_interleave(D) > 0), head,
                            torch.arange(len(stay), device=table.device))
    page_from, slot_from = page_from[source_of], slot_from[source_of]
    for c in state["caches"]:
        v = c if state["slot_dim"] == 1 else c.transpose(1, 2)
        v[page_to, slot_to] = v[page_from, slot_from]
    return state["caches"]


def work(case):
    if case["op"] == "verify":
        N, D, V, es = case["N"], case["D"], case["V"], 4 if case["dtype"] == "f32" else 2
        # rows up to the one at which the sequence ends; the draft's row of a rejected token is needed too
        if case["branch"]:
            rows = _spread_sum(N, 0, min(_full_levels(D, case["branch"]), 6), lambda a: a + 1)
        else:
            mean = (_draft_counts(case) + D) / 2  # lengths and the share of them that stands are drawn apart
            rows = _spread_sum(N, 0, 100, lambda s: round(mean * s / 100) + 1)
            if case["mode"] == "draft":
                rows += _spread_sum(N, 0, 100, lambda s: min(round(mean * s / 100) + 1, mean))
        small = N * (D * 4 + (D + 1) * 8 + 4 + (D * 8 if case["branch"] else 0))
        # an exponential, a sum and a comparison for each logit
        return {"bytes": rows * V * es + small, "flops": rows * V * 3}
    if case["op"] == "compact":
        es = 4 if case["dtype"] == "f32" else 2
        moved = _spread_sum(case["N"], 0, _path_length(case["D"]), lambda a: a)
        return {"bytes": 2 * moved * case["count"] * case["H"] * case["E"] * es + case["N"] * (case["D"] * 4 + 8),
                "flops": 0}
    N, K, S = case["N"], case["K"], case["S"]
    pages = _spread_sum(N, *_tokens_range(case), lambda t: -(-t // S))
    fork = pages * (len(set(_chain(K))) + K) * 4 + N * K * 12
    if case["op"] == "fork":
        return {"bytes": fork, "flops": 0}
    es = 4 if case["dtype"] == "f32" else 2
    grown = _spread_sum(N, *_tokens_range(case), lambda t: -(-(t + case["grow"]) // S) - -(-t // S)) * K
    small = case["P"] * 4 + grown * 4 * 4 + N * K * 16
    if not case["count"]:
        return {"bytes": small, "flops": 0}
    kids = [_chain(K).count(b) for b in range(K)]
    one = sum(k for k in kids if k > 1)  # each parent with several children read once and written for all but one
    slots = _spread_sum(N, *_tokens_range(case), lambda t: t % S)
    return {"bytes": small + fork + slots * one * case["H"] * case["D"] * es * case["count"], "flops": 0}


def exact(case, seed):
    if case["op"] == "compact":
        return None  # a copy: there is nothing that is computed
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    table, uses = s["table"].cpu().numpy(), s["uses"].cpu().numpy()
    lengths, parents, S = s["lengths"].cpu().numpy(), s["parents"].cpu().numpy(), case["S"]
    if case["op"] == "fork" or case["count"]:
        N, K = parents.shape
        source = (parents + K * np.arange(N)[:, None]).reshape(-1)
        table, lengths = table[source], lengths[source]
        uses = np.bincount(table[table >= 0], minlength=len(uses)).astype(np.int32)
    if case["op"] == "resize":
        for new in (s["after"].cpu().numpy(), s["before"].cpu().numpy()):
            _exact_resize(table, lengths, new, uses, S)
    out = tuple(torch.from_numpy(a.astype(np.int32)) for a in (table, lengths, uses))
    return out if case["op"] == "fork" else out + ([None] * case["count"],)


def _exact_resize(table, lengths, new, uses, S):
    """One row after the other; the pools of these cases have room for all."""
    for r in np.nonzero(new < lengths)[0]:
        for c in range(-(-new[r] // S), -(-lengths[r] // S)):
            uses[table[r, c]] -= 1
            table[r, c] = -1
    grown = np.nonzero(new > lengths)[0]
    free = iter(np.nonzero(uses == 0)[0])
    for r in grown:
        held = -(-lengths[r] // S)
        if lengths[r] % S and uses[table[r, held - 1]] > 1:  # the last one that is left keeps the page
            uses[table[r, held - 1]] -= 1
            table[r, held - 1] = next(free)
            uses[table[r, held - 1]] = 1
        for c in range(held, -(-new[r] // S)):
            table[r, c] = next(free)
            uses[table[r, c]] = 1
    lengths[:] = new


def _softmax64(row):
    row = row.double().cpu().numpy()
    e = np.exp(row - row.max())
    return e / e.sum()


def _exact_verify(case, s):
    N, D, V = case["N"], case["D"], case["V"]
    x, drafts = s["logits"].view(N, D + 1, V), s["drafts"].tolist()
    lengths = [D] * N if s["lengths"] is None else s["lengths"].tolist()
    parents = [list(range(-1, D - 1))] * N if s["parents"] is None else s["parents"].tolist()
    u = None if s["uniforms"] is None else s["uniforms"].double().tolist()
    y = None if s["draft_logits"] is None else s["draft_logits"].view(N, D, V)
    tokens, counts = np.full((N, D + 1), -1, np.int32), np.zeros(N, np.int32)
    paths = np.full((N, D), -1, np.int32)
    for i in range(N):
        at, path = -1, []
        while True:  # at the token of draft `at`
            children = [j for j in range(lengths[i]) if parents[i][j] == at]
            taken = None
            if u is None:
                row = x[i, at + 1].double().cpu().numpy()
                final = int(row.argmax())
                taken = next((j for j in children if drafts[i][j] == final), None)
            else:
                p = _softmax64(x[i, at + 1])
                r = p
                if y is not None and children:
                    q, d = _softmax64(y[i, at + 1]), drafts[i][at + 1]
                    if u[i][at + 1] * q[d] < p[d]:
                        taken = at + 1
                    else:
                        r = np.maximum(p - q, 0)
                elif children:
                    r, sofar = p.copy(), 0.0
                    for j in children:
                        d = drafts[i][j]
                        if taken is None and sofar <= u[i][at + 1] < sofar + r[d]:
                            taken = j
                        sofar, r[d] = sofar + r[d], 0.0
                if taken is None:
                    r = r if r.sum() > _LEAST else p
                    upto = np.cumsum(r)
                    final = int(np.searchsorted(upto, u[i][D] * upto[-1], side="right"))
            if taken is None:
                break
            path.append(taken)
            at = taken
        counts[i] = len(path)
        tokens[i, :len(path)] = [drafts[i][j] for j in path]
        tokens[i, len(path)] = min(final, V - 1)
        paths[i, :len(path)] = path
    path = None if s["parents"] is None else torch.from_numpy(paths)
    return torch.from_numpy(tokens), torch.from_numpy(counts), path
