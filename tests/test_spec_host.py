"""The speculative decoding and paged cache entry points without a GPU: arguments that the library and the binding
refuse, workspace sizes, and the tests' own references by hand."""

import os

import numpy as np
import pytest
import torch

import top_logits_filtering_amd as tk
from tests import spec_ref
from top_logits_filtering_amd.binding import BeamState

NULLPTR, INVALID = 1, 2
FAKE = 1 << 40  # a device-looking address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from top_logits_filtering_amd.binding import LIB_PATH

    if not os.path.exists(LIB_PATH):
        from top_logits_filtering_amd.build import build

        build()
    return tk.load_library()


def verify(lib, **kw):
    a = dict(x=FAKE, ld=100, dt=0, N=2, D=3, V=100, d=FAKE + (1 << 30), u=FAKE + (1 << 31), y=None, ldy=100, p=None,
             n=None, t=FAKE + (1 << 32), a=FAKE + (1 << 33), path=None, ws=FAKE + (1 << 34), size=1 << 20)
    a.update(kw)
    return lib.speculative_verify(a["x"], a["ld"], a["dt"], a["N"], a["D"], a["V"], a["d"], a["u"], a["y"], a["ldy"],
                                  a["p"], a["n"], a["t"], a["a"], a["path"], a["ws"], a["size"], None)


def test_verify_refusals(lib):
    for name, word in (("x", "logits"), ("d", "drafts"), ("t", "out_tokens"), ("a", "out_accepted"),
                       ("ws", "workspace")):
        assert verify(lib, **{name: None}) == NULLPTR
        assert word in tk.last_error()
    y = FAKE + (1 << 35)
    for kw, word in (
        (dict(dt=3), "dtype"), (dict(N=-1), "negative"), (dict(D=-1), "drafts"), (dict(D=256), "drafts"),
        (dict(N=1 << 31), "maximum"), (dict(N=1 << 62), "maximum"), (dict(V=-1), "negative"),
        (dict(V=(1 << 20) + 1, ld=1 << 21), "maximum"), (dict(ld=99), "stride"), (dict(ld=1 << 40), "stride"),
        (dict(y=y, ldy=99), "draft_logits"), (dict(y=y, u=None), "uniforms"), (dict(y=y, p=FAKE + (1 << 36)), "parents"),
        (dict(x=FAKE + 2), "aligned"), (dict(y=y + 1, dt=1), "aligned"), (dict(ws=FAKE + (1 << 34) + 8), "aligned"),
        (dict(size=15), "workspace"), (dict(t=FAKE + 400), "overlap"), (dict(a=FAKE + (1 << 31) + 28), "overlap"),
        (dict(path=FAKE + (1 << 32) + 31), "overlap"), (dict(path=FAKE + (1 << 30) + 20), "overlap"),
        (dict(y=FAKE + (1 << 34) - 8), "overlap"), (dict(n=FAKE + (1 << 33) + 4), "overlap"),
    ):
        assert verify(lib, **kw) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    need = lib.speculative_verify_workspace(0, 2, 3, 100, 0)
    assert verify(lib, size=need - 1) == INVALID and str(need) in tk.last_error()
    assert verify(lib, N=0, x=None, d=None, t=None, a=None, ws=None) == 0
    assert verify(lib, N=0, dt=9) == INVALID


def test_verify_workspace(lib):
    f = lib.speculative_verify_workspace
    for bad in ((7, 1, 1, 10, 0), (0, -1, 1, 10, 0), (0, 1, -1, 10, 0), (0, 1, 256, 10, 0), (0, 1, 1, 1 << 21, 0)):
        assert f(*bad) == -1 and tk.last_error()
    assert f(0, 0, 1, 10, 0) >= 16 and f(0, 1, 0, 0, 0) >= 16
    assert tk.speculative_verify_workspace(torch.bfloat16, 64, 4, 151936, True) == f(2, 64, 4, 151936, 1)
    assert f(2, 64, 4, 151936, 0) > 16 and f(2, 64, 4, 151936, 1) > f(2, 63, 4, 151936, 1)
    with pytest.raises(tk.TopKTopPError):
        tk.speculative_verify_workspace(torch.float32, 1, 300, 10)
    # the largest sizes stay within an int64
    assert f(0, (1 << 31) // 511 - 1, 255, 1 << 20, 0) > 1 << 32 and f(0, (1 << 31) // 511 - 1, 255, 1 << 20, 1) > 1 << 32


def fork(lib, **kw):
    a = dict(t=FAKE, ld=10, C=10, n=FAKE + (1 << 30), p=FAKE + (1 << 31), N=2, K=4, u=FAKE + (1 << 32), P=100, S=16)
    a.update(kw)
    return lib.cache_pages_fork(a["t"], a["ld"], a["C"], a["n"], a["p"], a["N"], a["K"], a["u"], a["P"], a["S"], None)


def resize(lib, caches=(), count=None, **kw):
    a = dict(t=FAKE, ld=10, R=8, C=10, n=FAKE + (1 << 30), new=FAKE + (1 << 31), u=FAKE + (1 << 32), P=100, S=16,
             ws=FAKE + (1 << 33), size=1 << 20)
    a.update(kw)
    arr = (BeamState * max(1, len(caches)))(*caches)
    return lib.cache_pages_resize(a["t"], a["ld"], a["R"], a["C"], a["n"], a["new"], a["u"], a["P"], a["S"], arr,
                                  len(caches) if count is None else count, a["ws"], a["size"], None)


def compact(lib, caches=None, count=None, **kw):
    a = dict(t=FAKE, ld=10, N=8, C=10, s=FAKE + (1 << 30), p=FAKE + (1 << 31), D=4, c=FAKE + (1 << 32), P=100, S=16)
    a.update(kw)
    caches = [page_cache()] if caches is None else caches
    arr = (BeamState * max(1, len(caches)))(*caches)
    return lib.cache_pages_compact(arr, len(caches) if count is None else count, a["P"], a["S"], a["t"], a["ld"], a["N"],
                                   a["C"], a["s"], a["p"], a["D"], a["c"], None)


def page_cache(**kw):
    a = dict(data=FAKE + (1 << 36), row_stride=16 * 256, size=(1, 1, 2), stride=(1, 1, 128), positions=16,
             position_stride=256, run=128)
    a.update(kw)
    s = BeamState()
    for k, v in a.items():
        if k in ("size", "stride"):
            getattr(s, k)[:] = v
        else:
            setattr(s, k, v)
    return s


def test_fork_refusals(lib):
    for name, word in (("t", "tables"), ("n", "lengths"), ("p", "parents"), ("u", "uses")):
        assert fork(lib, **{name: None}) == NULLPTR and word in tk.last_error()
    for kw, word in (
        (dict(N=-1), "negative"), (dict(K=0), "beams"), (dict(K=129), "beams"), (dict(N=1 << 31), "maximum"),
        (dict(C=-1), "negative"), (dict(P=-1), "negative"), (dict(P=1 << 31), "maximum"), (dict(S=0), "page_size"),
        (dict(S=1 << 31), "page_size"), (dict(C=1 << 20, ld=1 << 20, S=1 << 11), "2^31"), (dict(ld=9), "stride"),
        (dict(n=FAKE + 300), "overlap"), (dict(u=FAKE + (1 << 30) - 396), "overlap"),
        (dict(p=FAKE + (1 << 32) + 396), "overlap"),
    ):
        assert fork(lib, **kw) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    assert fork(lib, N=0, t=None, n=None, p=None, u=None) == 0


def test_resize_refusals(lib):
    for name, word in (("t", "tables"), ("n", "lengths"), ("new", "new_lengths"), ("u", "uses"), ("ws", "workspace")):
        assert resize(lib, **{name: None}) == NULLPTR and word in tk.last_error()
    for kw, word in (
        (dict(R=-1), "negative"), (dict(C=-1), "negative"), (dict(S=0), "page_size"), (dict(ld=9), "stride"),
        (dict(ws=FAKE + (1 << 33) + 4), "aligned"), (dict(size=100), "workspace"), (dict(n=FAKE + 300), "overlap"),
        (dict(new=FAKE + (1 << 30) + 28), "overlap"), (dict(count=-1), "count"),
        (dict(caches=[page_cache(positions=8)]), "slots"), (dict(caches=[page_cache(row_stride=100)]), "share memory"),
        (dict(caches=[page_cache(data=FAKE + (1 << 33) - 16)]), "overlaps workspace"),
        (dict(caches=[page_cache(), page_cache(data=FAKE + (1 << 36) + 4096)]), "two caches overlap"),
        (dict(caches=[page_cache(run=1, stride=(1, 1, 3), size=(1, 1, 1 << 28), position_stride=1 << 30,
                                 row_stride=1 << 35, data=FAKE - (1 << 43))]), "columns"),
    ):
        assert resize(lib, **kw) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    assert resize(lib, caches=[page_cache(data=None)]) == NULLPTR
    assert lib.cache_pages_resize(FAKE, 10, 8, 10, FAKE + (1 << 30), FAKE + (1 << 31), FAKE + (1 << 32), 100, 16, None, 1,
                                  FAKE + (1 << 33), 1 << 20, None) == NULLPTR
    need = lib.cache_pages_resize_workspace(8, 100)
    assert resize(lib, size=need - 1) == INVALID and str(need) in tk.last_error()
    assert resize(lib, R=0, t=None, n=None, new=None, u=None, ws=None) == 0
    for bad in ((-1, 5), (5, -1), (1 << 31, 5), (5, 1 << 31)):
        assert lib.cache_pages_resize_workspace(*bad) == -1 and tk.last_error()
    with pytest.raises(tk.TopKTopPError):
        tk.cache_pages_resize_workspace(-1, 3)
    assert 0 < tk.cache_pages_resize_workspace(0, 0) < tk.cache_pages_resize_workspace(2 ** 31 - 1, 2 ** 31 - 2)


def test_compact_refusals(lib):
    for name, word in (("t", "tables"), ("s", "starts"), ("p", "path"), ("c", "counts")):
        assert compact(lib, **{name: None}) == NULLPTR and word in tk.last_error()
    for kw, word in (
        (dict(N=-1), "negative"), (dict(D=-1), "drafts"), (dict(D=256), "drafts"), (dict(S=0), "page_size"),
        (dict(S=15), "slots"), (dict(count=-1), "count"), (dict(p=FAKE + (1 << 36) - 4), "overlaps path"),
        (dict(caches=[page_cache(), page_cache()]), "two caches overlap"),
    ):
        assert compact(lib, **kw) == INVALID, kw
        assert word in tk.last_error(), (kw, tk.last_error())
    assert compact(lib, N=0, t=None) == 0 and compact(lib, D=0, p=None) == 0 and compact(lib, caches=[]) == 0


def test_binding_refusals():
    i32 = dict(dtype=torch.int32)
    x, d, u = torch.zeros(8, 10, dtype=torch.float16), torch.zeros(2, 3, **i32), torch.zeros(2, 4)
    y = torch.zeros(6, 10, dtype=torch.float16)
    out = (torch.zeros(2, 4, **i32), torch.zeros(2, **i32), None)
    for err, args, kw in (
        (ValueError, (x[0], d), {}), (ValueError, (x, d[0]), {}), (ValueError, (x[:7], d), {}),
        (TypeError, (x.int(), d), {}), (TypeError, (x, d.long()), {}), (ValueError, (x.t().contiguous().t(), d), {}),
        (TypeError, (x, d, u.double()), {}), (ValueError, (x, d, u[:, :3]), {}),
        (ValueError, (x, d), dict(draft_logits=y)), (TypeError, (x, d, u), dict(draft_logits=y.float())),
        (ValueError, (x, d, u), dict(draft_logits=y[:5])), (ValueError, (x, d, u), dict(draft_logits=y, parents=d)),
        (TypeError, (x, d, u), dict(parents=d.long())), (ValueError, (x, d, u), dict(parents=d[:, :2])),
        (TypeError, (x, d, u), dict(lengths=torch.zeros(2))), (ValueError, (x, d, u), dict(lengths=torch.zeros(3, **i32))),
    ):
        with pytest.raises(err):
            tk.speculative_verify(*args, out=out, **kw)
    with pytest.raises(ValueError, match="GPU"):
        tk.speculative_verify(x, d, u, out=out)

    t, n, uses, p = torch.zeros(6, 5, **i32), torch.zeros(6, **i32), torch.zeros(20, **i32), torch.zeros(2, 3, **i32)
    for err, args in (
        (ValueError, (t[0], n, p, uses, 16)), (TypeError, (t.long(), n, p, uses, 16)), (ValueError, (t, n[:5], p, uses, 16)),
        (ValueError, (t.t().contiguous().t(), n, p, uses, 16)), (TypeError, (t, n, p.long(), uses, 16)),
        (ValueError, (t, n, p[0], uses, 16)), (ValueError, (t, n, p, uses.view(4, 5), 16)),
        (ValueError, (t, n, p, uses[::2], 16)),
    ):
        with pytest.raises(err):
            tk.cache_pages_fork(*args)
    with pytest.raises(ValueError, match="GPU"):
        tk.cache_pages_fork(t, n, p, uses, 16)

    c = torch.zeros(20, 16, 2, 4)
    for err, args, kw in (
        (ValueError, (t, n.view(2, 3), n, uses, 16), {}), (TypeError, (t, n, n.long(), uses, 16), {}),
        (ValueError, (t, n, n[:5], uses, 16), {}), (ValueError, (t, n, n, uses, 8), dict(caches=c)),
        (ValueError, (t, n, n, uses[:19], 16), dict(caches=c)), (ValueError, (t, n, n, uses, 16), dict(caches=c, slot_dim=2)),
        (ValueError, (t, n, n, uses, 16), dict(caches=c, slot_dim=0)), (ValueError, (t, n, n, uses, 16), dict(caches=c, slot_dim=4)),
        (ValueError, (t, n, n, uses, 16), dict(caches=c.clone().requires_grad_())),
    ):
        with pytest.raises(err):
            tk.cache_pages_resize(*args, **kw)
    with pytest.raises(ValueError, match="GPU"):
        tk.cache_pages_resize(t, n, n.clone(), uses, 16, caches=[c])

    s, path = torch.zeros(6, **i32), torch.zeros(6, 3, **i32)
    for err, args, kw in (
        (ValueError, (c, t, s, path[0], s), {}), (TypeError, (c, t, s, path.long(), s), {}),
        (ValueError, (c, t, s[:5], path, s), {}), (ValueError, (c, t[:5], s, path, s), {}),
        (ValueError, ([c, c[:10]], t, s, path, s), {}), (ValueError, ([c, c[:, :8]], t, s, path, s), {}),
        (ValueError, (c, t, s, path, s), dict(page_dim=1)), (ValueError, (c, t, s, path, s), dict(page_dim=7)),
        (ValueError, (c.clone().requires_grad_(), t, s, path, s), {}),
    ):
        with pytest.raises(err):
            tk.cache_pages_compact(*args, **kw)
    with pytest.raises(ValueError, match="GPU"):
        tk.cache_pages_compact((c for _ in range(1)), t, s, path, s)
    assert tk.cache_pages_compact([], t, s, path, s) == []


def test_references_by_hand():
    lg = lambda *p: np.log(np.maximum(np.array(p), 1e-300))
    x = np.stack([lg(0.5, 0.3, 0.2), lg(0.1, 0.6, 0.3), lg(0.25, 0.25, 0.5)])[None]
    y = np.stack([lg(0.25, 0.5, 0.25), lg(0.2, 0.3, 0.5)])[None]
    d = np.array([[1, 2]])
    # 0.5 * 0.5 < 0.3 stands, 0.7 * 0.5 >= 0.3 does not; max(p - q, 0) = (0, 0.3, 0)
    assert [a.tolist() for a in spec_ref.verify(x, d, np.array([[0.5, 0.7, 0.9]]), y)[:3]] == [[[1, 1, -1]], [1], [[0, -1]]]
    assert spec_ref.verify(x, d, np.array([[0.5, 0.5, 0.6]]), y)[0].tolist() == [[1, 2, 2]]
    # proposals: 0.29 < 0.3 stands, 0.31 does not; then p without token 1, (0.5, 0, 0.2)
    assert spec_ref.verify(x, d, np.array([[0.29, 0.31, 0.1]]))[0].tolist() == [[1, 0, -1]]
    assert spec_ref.verify(x, d, np.array([[0.31, 0.0, 0.72]]))[0].tolist() == [[2, -1, -1]]
    # two drafts behind the last token: pieces [0, 0.3) and [0.3, 0.5)
    both = np.array([[-1, -1]])
    for u, want in ((0.2, [[1, 0, -1]]), (0.4, [[2, 0, -1]]), (0.6, [[0, -1, -1]])):
        assert spec_ref.verify(x, d, np.array([[u, 0.5, 0.0]]), parents=both)[0].tolist() == want
    assert spec_ref.verify(x, np.array([[0, 1]]))[0].tolist() == [[0, 1, 2]]

    t, n, u = np.array([[3, 5], [4, -1]], np.int32), np.array([5, 2], np.int32), np.array([0, 0, 0, 1, 1, 1], np.int32)
    spec_ref.fork(t, n, np.array([[0, 0]]), u, 4)
    assert t.tolist() == [[3, 5], [3, 5]] and n.tolist() == [5, 5] and u.tolist() == [0, 0, 0, 2, 0, 2]
    c = np.arange(24).reshape(6, 4)
    spec_ref.resize(t, n, np.array([6, 6]), u, 4, [c])
    assert t.tolist() == [[3, 0], [3, 5]] and u.tolist() == [1, 0, 0, 2, 0, 1] and c[0].tolist() == [20, 1, 2, 3]
    spec_ref.resize(t, n, np.array([4, 0]), u, 4)
    assert t.tolist() == [[3, -1], [-1, -1]] and u.tolist() == [0, 0, 0, 1, 0, 0]
    spec_ref.compact([c], np.array([[1, 2]]), np.array([2]), np.array([[1, 3]]), np.array([2]))
    assert c[1].tolist() == [4, 5, 7, 9]
