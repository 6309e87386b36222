"""The calls around a drafted block at the edges of what they accept."""
import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import step_oracle as S
from test_gpu_attention import Case as Attention
from test_gpu_verify import Case, make_head

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


@pytest.mark.parametrize("first", [0, 3])
def test_append_keeps_to_the_columns_of_its_table(first):
    # columns `first`.. of a wider table: a length past them is flagged and writes nothing, though the
    # wider table names pages there (and, in the last row, its storage may end there)
    ps, width = 4, 3
    k, v = (torch.zeros(1, 12, ps, 1, 8, device="cuda") for _ in range(2))
    cache = xp.Cache(k, v)
    wide = ints([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]])
    table = wide[:, first:first + width]
    new = torch.randn(2, 2, 1, 8, device="cuda")
    want_k, want_v = k.clone(), v.clone()
    xp.xp_cache_append(cache.handle, 0, new, new, table, ints([width * ps + 1, 5]))
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_ELENGTH
    last, row = int(table[0, width - 1]), table[1].tolist()
    for pool in (want_k, want_v):
        pool[0, last, ps - 1] = new[0, 0]              # the token that still fits
        pool[0, row[0], ps - 1] = new[1, 0]
        pool[0, row[1], 0] = new[1, 1]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def beams(g, rows, width, ps):
    """A table of `rows` filled rows over shuffled pages, lengths, counts and an fp32 pool for it."""
    lens = g.integers(0, width * ps + 1, rows).astype(np.int32)
    used = -(-lens // ps)
    pages = int(used.sum()) + 2 * rows + 3
    ids, at = g.permutation(pages).astype(np.int32), 0
    table, refs = np.full((rows, width), -1, np.int32), np.zeros(pages, np.int32)
    for n, u in enumerate(used):
        table[n, :u] = ids[at:at + u]
        at += u
    refs[ids[:at]] = 1
    return table, lens, refs, torch.arange(pages * ps * 4, device="cuda").view(1, pages, ps, 1, 4).float()


@pytest.mark.parametrize("rows,width,ps", [(2, 1, 3), (4, 3, 4), (33, 20, 5), (40, 400, 2), (1500, 7, 4)])
@pytest.mark.parametrize("first", [0, 1])
def test_fork_over_its_own_parents(rows, width, ps, first):
    # a beam's reorder: children take the places of rows that are parents of others, in a table that
    # is some columns of a wider one
    g = np.random.default_rng(rows + width + first)
    table, lens, refs, k = beams(g, rows, width, ps)
    M = rows - first
    parent = g.integers(0, rows, M).astype(np.int32)
    parent[:M // 2] = (np.arange(M // 2) + 1) % rows
    cut = g.integers(0, width * ps + 1, M).astype(np.int32)
    v = k + 0.5
    want_k, want_v = k.clone(), v.clone()
    cache = xp.Cache(k, v)
    wide = torch.full((rows, width + 5), 99, dtype=torch.int32, device="cuda")
    t = wide[:, 2:2 + width]
    t.copy_(ints(table))
    n, r = ints(lens), ints(refs)
    xp.xp_cache_fork(cache.handle, t, n, ints(parent), ints(cut), r, t[first:], n[first:], r)
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
    child, child_lens, want_refs, moves = S.fork(table, lens, parent, cut, refs, ps)
    assert np.array_equal(t[first:].cpu().numpy(), child)
    assert np.array_equal(t[:first].cpu().numpy(), table[:first])
    assert np.array_equal(n[first:].cpu().numpy(), child_lens)
    assert np.array_equal(r.cpu().numpy(), want_refs)
    assert (wide[:, :2] == 99).all() and (wide[:, 2 + width:] == 99).all()
    for s, d, count in moves:
        want_k[:, d, :count], want_v[:, d, :count] = want_k[:, s, :count], want_v[:, s, :count]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_fork_between_tables_that_lie_among_each_other():
    # columns side by side and rows in turn share no entry; a shift by a column is refused
    k = torch.zeros(1, 16, 4, 1, 4, device="cuda")
    cache = xp.Cache(k, k.clone())
    refs = ints([1, 1, 1] + [0] * 13)
    both = ints(np.full((4, 6), -1))
    for parents, children in ((both[:2, :3], both[:2, 3:]), (both[::2, :3], both[1::2, :3])):
        both.fill_(-1)
        parents.copy_(ints([[2, 0, -1], [1, -1, -1]]))
        lens, out_lens, out_refs = ints([8, 4]), ints([0, 0]), refs.clone()
        xp.xp_cache_fork(cache.handle, parents, lens, ints([1, 0]), None, refs, children, out_lens,
                         out_refs)
        assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
        assert children.tolist() == [[1, -1, -1], [2, 0, -1]] and out_lens.tolist() == [4, 8]
        assert parents.tolist() == [[2, 0, -1], [1, -1, -1]]
        assert out_refs.tolist()[:4] == [2, 2, 2, 0]
    before = both.clone()
    for parents, children in ((both[:2, :3], both[:2, 1:4]), (both[:2, :3], both[1:3, 2:5]),
                              (both[:1, :3], both[:1, 1:4]),
                              (both.view(-1)[:20].view(5, 4)[:3, :3], both[:2, :3])):
        with pytest.raises(xp.XPError) as e:
            xp.xp_cache_fork(cache.handle, parents, ints([4] * len(parents)), ints([0] * len(children)),
                             None, refs, children, ints([0] * len(children)), refs.clone())
        assert e.value.code == xp.XP_EINVAL
    assert torch.equal(both, before)


@pytest.mark.parametrize("drafts", [True, False])
def test_noise_that_lets_no_id_win(drafts):
    # a row of NaN or infinite noise: no token, not an id outside the vocabulary
    c = Case(N=6, B=4, V=600, seed=3, dtype="f32", drafts=drafts)
    c.u[:3] = np.float32(1 - 2 ** -24)
    c.noise[0], c.noise[1], c.noise[4] = np.nan, np.inf, np.nan
    tokens, counts, _ = c.run()
    assert c.error == xp.XP_EEMPTY
    want, want_counts, _, _ = c.want()
    for n in range(c.N):
        accepted = want_counts[n] - 1
        if n in (0, 1, 4):
            assert counts[n] == accepted and (tokens[n, accepted:] == -1).all()
            assert np.array_equal(tokens[n, :accepted], want[n, :accepted])
        else:
            assert np.array_equal(tokens[n], want[n]) and counts[n] == want_counts[n]


def test_empty_batches():
    # no rows, sequences or children: nothing to do, and an empty tensor has no address
    k = torch.randn(1, 6, 4, 2, 64, device="cuda")
    cache = xp.Cache(k, k.clone())
    none = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    no = torch.empty(0, dtype=torch.int32, device="cuda")
    refs = ints([0, 2, 0, 1, 0, 0])
    new = torch.empty(0, 5, 2, 64, device="cuda")
    xp.xp_cache_append(cache.handle, 0, new, new, none, no)
    out = ints([9] * 6)
    xp.xp_cache_resize(cache.handle, none, no, no, refs, none, no, out)
    assert torch.equal(out, refs)
    table, lens = ints([[1, 3, -1], [1, -1, -1]]), ints([6, 4])
    out.fill_(9)
    xp.xp_cache_fork(cache.handle, table, lens, no, None, refs, none, no, out)
    assert torch.equal(out, refs)
    child, child_lens = ints([[7, 7, 7]]), ints([7])
    xp.xp_cache_fork(cache.handle, none, no, ints([0]), None, refs, child, child_lens, out)
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_ELENGTH         # there is no row 0
    assert child.tolist() == [[-1, -1, -1]] and child_lens.tolist() == [0] and torch.equal(out, refs)
    # packing without tables moves what refs hold
    want = k.clone()
    want[:, 0] = want[:, 3]
    new_id = ints([9] * 6)
    xp.xp_cache_compact(cache.handle, none, no, refs, none, out, new_id)
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
    assert out.tolist() == [1, 2, 0, 0, 0, 0] and new_id.tolist() == [-1, 1, -1, 0, -1, -1]
    assert torch.equal(k, want)
    q = torch.empty(0, 5, 4, 64, device="cuda")
    for prefix_len in (0, 8):
        a = xp.make_attn(q, q, 0, prefix_len, 12, 0.1)
        xp.xp_prefix_attention(cache.handle, a, q, ints([1, 3]), none, no, q, None,
                               cache.attention_workspace(a))
    c = Case(N=2, B=4, V=64, seed=1)
    head = make_head(64, 4, 2, "bf16")
    xp.xp_verify_drafts(head.handle, c.target[:0], torch.empty(0, 64, device="cuda"),
                        torch.empty(0, 4, dtype=torch.int64, device="cuda"), no,
                        torch.empty(0, device="cuda"), torch.empty(0, 3, device="cuda"),
                        torch.empty(0, 64, device="cuda"),
                        torch.empty(0, 4, dtype=torch.int64, device="cuda"), no,
                        torch.empty(0, 3, device="cuda"), head.verify_workspace(0))
    assert xp.xp_get_error(head.handle) == xp.XP_OK and xp.xp_cache_get_error(cache.handle) == xp.XP_OK


def test_sizes_whose_products_pass_32_and_64_bits():
    # host arithmetic only: what is refused and what a plan asks for
    k = torch.zeros(1, 2, 4, 1, 4, device="cuda")
    cache = xp.Cache(k, k.clone())

    def bytes_of(N, T, heads, prefix_len, max_len=0):
        a = xp.xp_attn(0, N, T, heads, 4, xp.XP_F32, prefix_len, max_len, 1.0, 4, 4, 4, 4, 4, 4)
        return xp.xp_attention_workspace_bytes(cache.handle, a)

    assert bytes_of(1 << 22, 1 << 22, 1 << 22, 4) == 0             # 2^66 rows
    assert bytes_of(1 << 30, 4, 1, 4) == 0                         # 2^32
    # one range over 2^31 - 2000 keys: a partial result a row
    assert bytes_of(20000, 1, 1, (1 << 31) - 2000) == 20000 * 8 + 20000 * 16
    assert bytes_of(20000, 1, 1, 0, (1 << 31) - 2000) == 20000 * 8 + 20000 * 16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinite_value_shows_where_its_weight_underflows(dtype):
    # the first 128 keys score 400 below the others, a whole range of them: their weights are 0 in 32
    # bits, but a row that sees an infinite or NaN value does not come out finite there
    D, n = 64, 600
    k, v = (torch.randn(1, 40, 16, 1, D, device="cuda").to(xp.torch_dtype(dtype)) for _ in range(2))
    q = torch.zeros(2, 1, 1, D, device="cuda", dtype=k.dtype)
    q[..., 0] = 1
    k[:, :8, :, :, 0], k[:, 8:, :, :, 0] = -200, 200
    v[0, 0, 3, 0, 5], v[0, 7, 15, 0, 9], v[0, 2, 0, 0, 63] = torch.inf, torch.nan, -torch.inf
    cache = xp.Cache(k, v)
    table = torch.arange(40, dtype=torch.int32, device="cuda").repeat(2, 1)
    out = torch.empty_like(q)
    for prefix_len, lens in ((0, [n, 0]), (n, [0, 0])):
        a = xp.make_attn(q, out, 0, prefix_len, max(lens), 1.0)
        xp.xp_prefix_attention(cache.handle, a, q, table[0], table, ints(lens), out, None,
                               cache.attention_workspace(a))
        odd = torch.zeros(D, dtype=torch.bool, device="cuda")
        odd[[5, 9, 63]] = True
        assert torch.equal(~out[0, 0, 0].isfinite(), odd)
        if prefix_len:
            assert torch.equal(~out[1, 0, 0].isfinite(), odd)
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK


@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_of_the_prefix_leaves_the_rest_of_a_row_as_it_was(D):
    # every row sees it: its dim is NaN, and nothing is summed anew for the others (another way of
    # summing, a thread a row, would show in their last bits, and in a call of many rows take seconds)
    c = Attention([40, 300, 7, 130, 0], T=5, H=2, G=4, D=D, P=200, seed=6)
    out, lse = c.run()
    page, row = int(c.prefix_table[9]), 3
    c.v[0, page, row, 1, 6] = torch.nan
    c.v[0, page, row, 1, D - 1] = torch.inf
    got, got_lse = c.run()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:, :, 4:, [6, D - 1]] = True
    assert torch.equal(got.isnan(), hit & (torch.arange(D, device="cuda") == 6))
    assert (got[:, :, 4:, D - 1] == torch.inf).all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(got_lse, lse)
    # a hidden value on top of it still reaches only the rows that see it
    c.v[0, int(c.table[1, 299 // 16]), 299 % 16, 1, 7] = torch.nan
    again, _ = c.run()
    hit[1, 4, 4:, 7] = True
    assert torch.equal(again.isnan(), hit & (torch.arange(D, device="cuda") != D - 1))
    assert xp.xp_cache_get_error(c.cache.handle) == xp.XP_OK


@pytest.mark.parametrize("page", [16, 1])
def test_strides_that_are_never_used_do_not_count(page):
    # one layer, head, page or token may come with any stride (a view's): the same form of every call
    # runs, to the bit, as the workspace that it asks for tells
    D, n, pages = 128, 48, 48 // page
    k, v = (torch.randn(1, pages, page, 1, D, device="cuda").bfloat16() for _ in range(2))
    odd = [t.as_strided(t.shape, (0, page * D, 7 if page == 1 else D, 5, 1)) for t in (k, v)]
    assert odd[0].stride() != k.stride() and torch.equal(odd[0], k)
    q = torch.randn(1, 1, 1, D, device="cuda").bfloat16()
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    got = []
    for (a, b), x in (((k, v), q), (odd, q.as_strided(q.shape, (3, 1, 9, 1)))):
        cache = xp.Cache(a, b)
        out = torch.empty_like(q)
        attn = xp.make_attn(x, out, 0, 0, n, 0.1)
        ws = cache.attention_workspace(attn)
        xp.xp_prefix_attention(cache.handle, attn, x, None, table, ints([n]), out, None, ws)
        xp.xp_cache_append(cache.handle, 0, x, x, table, ints([n - 1]))
        if page == 16:
            xp.xp_cache_copy(cache.handle, ints([0]), ints([1]))
        assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
        got.append((ws.numel(), out, k.clone(), v.clone()))
        assert out.isfinite().all() and torch.equal(k[0, (n - 2) // page, (n - 2) % page], q[0, 0])
        k[0, (n - 2) // page, (n - 2) % page], v[0, (n - 2) // page, (n - 2) % page] = 0.5, 0.25
    assert got[0][0] == got[1][0]
    one_page = torch.randn(3, 1, 16, 2, 64, device="cuda").bfloat16()
    view = one_page.as_strided(one_page.shape, (2048, 2049, 128, 64, 1))
    a = xp.make_attn(torch.empty(1, 1, 2, 64, device="cuda").bfloat16(),
                     torch.empty(1, 1, 2, 64, device="cuda").bfloat16(), 2, 0, 16, 0.1)
    sizes = [xp.Cache(t, t).attention_workspace(a).numel() for t in (one_page, view)]
    assert sizes[0] == sizes[1]


def test_fork_of_more_rows_than_a_cluster_holds_over_its_own_parents():
    rows, width, ps = 70001, 2, 3
    g = np.random.default_rng(8)
    table, lens, refs, k = beams(g, rows, width, ps)
    parent = np.concatenate([np.arange(1, rows), [0]]).astype(np.int32)
    cache = xp.Cache(k, k + 0.5, max_seqs=rows)
    t, n, r = ints(table), ints(lens), ints(refs)
    xp.xp_cache_fork(cache.handle, t, n, ints(parent), None, r, t, n, r)
    assert xp.xp_cache_get_error(cache.handle) == xp.XP_OK
    # worked out at once: every row's full pages are held twice, partly filled last pages are copied to
    # the lowest free ids in child order
    lens = lens[parent]
    full, part = lens // ps, lens % ps
    child = np.where(np.arange(width) < full[:, None], table[parent], -1)
    np.add.at(refs, child[child >= 0], 1)
    free = np.nonzero(refs == 0)[0][:(part > 0).sum()]
    child[np.nonzero(part)[0], full[part > 0]] = free
    refs[free] = 1
    assert np.array_equal(t.cpu().numpy(), child) and np.array_equal(n.cpu().numpy(), lens)
    assert np.array_equal(r.cpu().numpy(), refs)
    some = np.nonzero(part)[0][::997]
    src, dst = table[parent[some], full[some]], child[some, full[some]]
    for s, d, count in zip(src.tolist(), dst.tolist(), part[some].tolist()):
        assert torch.equal(cache.k[:, d, :count], cache.k[:, s, :count])
