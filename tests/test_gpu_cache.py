"""The paged cache's calls against their plain statements: whole numbers and copied bytes, all exact."""
import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


def pools(layers, pages, ps, heads, dim, order="token", dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pages, ps, heads, dim) if order == "token" else (layers, pages, heads, ps, dim)
    out = [torch.randn(shape, generator=g, device="cuda", dtype=dtype) for _ in range(2)]
    return [t if order == "token" else t.transpose(2, 3) for t in out]


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def tables(g, N, width, pages, ps, share=0.0):
    """Random tables over distinct pages, and with `share` rows that repeat their neighbour's full pages."""
    lens = g.integers(0, width * ps + 1, N).astype(np.int32)
    ids = g.permutation(pages).astype(np.int32)
    table, refs, at = np.full((N, width), -1, np.int32), np.zeros(pages, np.int32), 0
    for n in range(N):
        lens[n] = min(lens[n], (pages - at) * ps)
        used = -(-lens[n] // ps)
        table[n, :used] = ids[at:at + used]
        at += used
        if n and g.random() < share:
            full = min(lens[n], lens[n - 1]) // ps
            table[n, :full] = table[n - 1, :full]
    for n in range(N):
        np.add.at(refs, table[n, :-(-lens[n] // ps)], 1)
    return table, lens, refs


SIZES = [(1, 1, 1, 1), (1, 4, 9, 16), (5, 7, 40, 4), (33, 20, 700, 16), (8, 3, 30, 5),
         (1500, 6, 9500, 8), (300, 130, 40000, 20)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("share", [0.0, 0.6])
def test_resize(size, inplace, share):
    N, width, pages, ps = size
    g = np.random.default_rng(N * width + ps)
    table, lens, refs = tables(g, N, width, pages, ps, share)
    new = np.clip(lens + g.integers(-2 * ps, 2 * ps + 1, N), 0, width * ps).astype(np.int32)
    k, v = pools(1, pages, ps, 1, 8)
    c = xp.Cache(k, v)
    t, n, r, want_len = cu(table), cu(lens), cu(refs), cu(new)
    outs = (t, n, r) if inplace else tuple(torch.full_like(x, 55) for x in (t, n, r))
    xp.xp_cache_resize(c.handle, t, n, want_len, r, *outs)
    err = xp.xp_cache_get_error(c.handle)
    want = S.resize(table, lens, new, refs, ps)
    for got, w in zip(outs, want):
        assert np.array_equal(got.cpu().numpy(), w)
    if not share:
        assert err in (xp.XP_OK, xp.XP_ENOPAGES) and (err == xp.XP_OK) == np.array_equal(want[1], new)


def test_resize_flags():
    ps, pages = 4, 6
    k, v = pools(1, pages, ps, 1, 8)
    c = xp.Cache(k, v)
    table = np.array([[0, 1, -1, -1], [0, 2, -1, -1]], np.int32)
    lens, refs = np.array([7, 8], np.int32), np.array([2, 1, 1, 0, 0, 0], np.int32)

    def run(new, tab=table, lens=lens, refs=refs):
        outs = cu(tab), cu(lens), cu(refs)
        xp.xp_cache_resize(c.handle, outs[0], outs[1], cu(new), outs[2], *outs)
        return xp.xp_cache_get_error(c.handle), [o.cpu().numpy().tolist() for o in outs]

    # into the shared page: refused, the other row still served
    assert run([3, 9]) == (xp.XP_ESHARED, [[[0, 1, -1, -1], [0, 2, 3, -1]], [7, 9], [2, 1, 1, 1, 0, 0]])
    # to its edge: allowed
    assert run([4, 0]) == (xp.XP_OK, [[[0, -1, -1, -1], [-1] * 4], [4, 0], [1, 0, 0, 0, 0, 0]])
    # more than the columns hold, more than the pool holds
    assert run([99, 8])[0] == xp.XP_ELENGTH
    assert run([16, 16]) == (xp.XP_ENOPAGES, [[[0, 1, 3, 4], [0, 2, 5, -1]], [16, 12], [2, 1, 1, 1, 1, 1]])
    # a page freed twice, an id outside the pool
    assert run([7, 0], refs=np.array([2, 1, 0, 0, 0, 0], np.int32))[0] == xp.XP_EBADPAGE
    assert run([0, 8], tab=np.array([[0, 9, -1, -1], [0, 2, -1, -1]], np.int32))[0] == xp.XP_EBADPAGE


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("form", ["token", "head", "odd", "f32"])
@pytest.mark.parametrize("cuts", [False, True])
def test_fork(size, form, cuts):
    N, width, pages, ps = size
    g = np.random.default_rng(N + width + ps)
    table, lens, refs = tables(g, N, width, pages, ps, 0.3)
    M = min(2 * N + 1, 400)
    parent = g.integers(0, N, M).astype(np.int32)
    cut = g.integers(0, width * ps + 1, M).astype(np.int32) if cuts else None
    layers, heads, dim = (1, 1, 8) if pages > 5000 else (3, 2, 5 if form == "odd" else 16)
    k, v = pools(layers, pages, ps, heads, dim, "head" if form == "head" else "token",
                 torch.float32 if form == "f32" else torch.bfloat16)
    wk, wv = k.clone(), v.clone()
    c = xp.Cache(k, v)
    outs = [torch.full((M, width), 55, dtype=torch.int32, device="cuda"),
            torch.full((M,), 55, dtype=torch.int32, device="cuda"), torch.full_like(cu(refs), 55)]
    xp.xp_cache_fork(c.handle, cu(table), cu(lens), cu(parent), None if cut is None else cu(cut),
                     cu(refs), *outs)
    assert xp.xp_cache_get_error(c.handle) in (xp.XP_OK, xp.XP_ENOPAGES)
    child, clens, crefs, moves = S.fork(table, lens, parent, cut, refs, ps)
    for got, w in zip(outs, (child, clens, crefs)):
        assert np.array_equal(got.cpu().numpy(), w)
    if moves:
        src, dst, toks = (torch.tensor(x, device="cuda") for x in zip(*moves))
        live = (torch.arange(ps, device="cuda")[None, :] < toks[:, None])[None, :, :, None, None]
        for w in (wk, wv):
            w[:, dst] = torch.where(live, w[:, src], w[:, dst])
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_fork_rows_of_the_same_table():
    k, v = pools(2, 12, 4, 2, 8)
    c = xp.Cache(k, v)
    table = np.full((4, 3), -1, np.int32)
    table[0, :2] = [7, 3]
    refs = np.zeros(12, np.int32)
    refs[[7, 3]] = 1
    t, n, r = cu(table), cu([6, 0, 0, 0]), cu(refs)
    xp.xp_cache_fork(c.handle, t, n, cu([0, 0, 5]), None, r, t[1:], n[1:], r)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_ELENGTH       # parent 5 does not exist
    assert t.cpu().tolist() == [[7, 3, -1], [7, 0, -1], [7, 1, -1], [-1, -1, -1]]
    assert n.cpu().tolist() == [6, 6, 6, 0]
    assert r.cpu().tolist() == [1, 1, 0, 1, 0, 0, 0, 3, 0, 0, 0, 0]
    assert torch.equal(k[:, 0, :2], k[:, 3, :2]) and torch.equal(v[:, 1, :2], v[:, 3, :2])


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("order", ["token", "head"])
def test_compact(size, inplace, order):
    N, width, pages, ps = size
    g = np.random.default_rng(N + width * ps)
    table, lens, refs = tables(g, N, width, pages, ps, 0.4)
    refs[g.integers(0, pages, 2)] += 1        # pages that tables kept elsewhere hold
    k, v = pools(2, pages, ps, 1, 8, order)
    wk, wv = k.clone(), v.clone()
    c = xp.Cache(k, v)
    t, r = cu(table), cu(refs)
    to, ro = (t, r) if inplace else (torch.full_like(t, 55), torch.full_like(r, 55))
    new, live = (None, None) if inplace else (torch.full_like(r, 55), torch.zeros_like(r[:1]))
    xp.xp_cache_compact(c.handle, t, cu(lens), r, to, ro, new, live)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    wt, wr, wm, wl, moves = S.compact(table, lens, refs, ps)
    assert np.array_equal(to.cpu().numpy(), wt) and np.array_equal(ro.cpu().numpy(), wr)
    if not inplace:
        assert np.array_equal(new.cpu().numpy(), wm) and int(live) == wl
    if moves:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        wk[:, dst], wv[:, dst] = wk[:, src], wv[:, src]
    assert torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.parametrize("form", ["token", "head", "odd", "interleaved"])
def test_copy(form):
    if form == "interleaved":      # K and V of a page side by side
        both = torch.randn(3, 20, 2, 8, 2, 16, device="cuda").bfloat16()
        k, v = both[:, :, 0], both[:, :, 1]
    else:
        k, v = pools(3, 20, 8, 2, 5 if form == "odd" else 16, "head" if form == "head" else "token")
    wk, wv = k.clone(), v.clone()
    c = xp.Cache(k, v)
    src, dst = [3, 19, -1, 3, 0], [4, 0, 7, 18, -5]
    xp.xp_cache_copy(c.handle, cu(src), cu(dst))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    # 19 -> 0 reads before 0 -> nowhere: pairs do not depend on each other
    for a, b in ((3, 4), (19, 0), (3, 18)):
        wk[:, b], wv[:, b] = wk[:, a], wv[:, a]
    assert torch.equal(k, wk) and torch.equal(v, wv)
    xp.xp_cache_copy(c.handle, cu([20]), cu([1]))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_EBADPAGE and torch.equal(k, wk)
    xp.xp_cache_copy(c.handle, cu([]), cu([]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("T,ps,dim", [(1, 16, 64), (5, 4, 128), (16, 7, 24), (3, 1, 5)])
def test_append(dtype, order, T, ps, dim):
    N, H, width = 6, 3, 9
    k, v = pools(2, N * width, ps, H, dim, order, dtype)
    wk, wv = k.clone(), v.clone()
    c = xp.Cache(k, v)
    g = np.random.default_rng(T)
    table = g.permutation(N * width).reshape(N, width).astype(np.int32)
    lens = np.array([0, 1, T, width * ps, T + 2, 2], np.int32)
    qkv = torch.randn(N, T, 3 * H, dim, device="cuda").to(dtype)       # a fused projection's K and V
    nk, nv = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    xp.xp_cache_append(c.handle, 1, nk, nv, cu(table), cu(lens))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    for n in range(N):
        for t in range(T):
            pos = lens[n] - T + t
            if pos >= 0:
                wk[1, table[n, pos // ps], pos % ps] = nk[n, t]
                wv[1, table[n, pos // ps], pos % ps] = nv[n, t]
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_append_flags():
    k, v = pools(1, 4, 4, 1, 8)
    before = k.clone()
    c = xp.Cache(k, v)
    new = torch.randn(1, 1, 1, 8, device="cuda").bfloat16()
    xp.xp_cache_append(c.handle, 0, new, new, cu([[1, 9]]), cu([6]))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_EBADPAGE
    xp.xp_cache_append(c.handle, 0, new, new, cu([[1, 2]]), cu([9]))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_ELENGTH
    assert torch.equal(k, before)


def test_large_pool_offsets():
    # a layer stride beyond 2^31 elements: pages at the far end of a 9 GB pool
    k, v = (torch.empty(2, 70000, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = xp.Cache(k, v)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k, v):
        t[:, 69990:] = torch.randn(2, 10, 16, 8, 128, generator=g, device="cuda").bfloat16()
    xp.xp_cache_copy(c.handle, cu([69999, 69991]), cu([69995, 3]))
    assert torch.equal(k[1, 69995], k[1, 69999]) and torch.equal(v[:, 3], v[:, 69991])


def test_refusals():
    k, v = pools(1, 8, 4, 2, 8)
    for bad in (lambda: xp.Cache(k[:, :, :, :, :4], v[:, :, :, :, :4]),             # pages not dense
                lambda: xp.Cache(*[t.expand(1, 8, 4, 2, 8)[:, :, ::2] for t in (k, v)])):
        with pytest.raises((xp.XPError, ValueError)):
            bad()
    with pytest.raises(ValueError):
        xp.Cache(k, v.float())
    with pytest.raises(xp.XPError):
        xp.Cache(torch.zeros(1, 2, 4, 1, 264, device="cuda"), torch.zeros(1, 2, 4, 1, 264, device="cuda"))
    c = xp.Cache(k, v, max_seqs=2)
    t, n, r = cu([[0, 1], [2, -1]]), cu([8, 3]), cu([1, 1, 1, 0, 0, 0, 0, 0])

    def code(f, *a):
        with pytest.raises(xp.XPError) as e:
            f(*a)
        return e.value.code

    three = cu(np.full((3, 2), -1)), cu([0, 0, 0])
    assert code(xp.xp_cache_resize, c.handle, three[0], three[1], three[1], r, *three, r) == xp.XP_ECAPACITY
    assert code(xp.xp_cache_resize, c.handle, t, n, n, r[:7], t, n, r[:7]) == xp.XP_EINVAL
    assert code(xp.xp_cache_fork, c.handle, t, n, cu([0, 0, 0]), None, r, *three, r) == xp.XP_ECAPACITY
    assert code(xp.xp_cache_compact, c.handle, t, n, r[:7], t, r[:7]) == xp.XP_EINVAL
    assert code(xp.xp_cache_append, c.handle, 1, k[0, :2, :1], v[0, :2, :1], t, n) == xp.XP_EINVAL
    assert code(xp.xp_cache_append, c.handle, 0, k[0, :2, :1].float(), v[0, :2, :1].float(), t, n) == xp.XP_EINVAL
    with pytest.raises(ValueError):
        xp.xp_cache_resize(c.handle, t.long(), n, n, r, t, n, r)
    with pytest.raises(ValueError):
        xp.xp_cache_resize(c.handle, t, n[:1], n, r, t, n, r)
    # nothing above was launched
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK and t.cpu().tolist() == [[0, 1], [2, -1]]
