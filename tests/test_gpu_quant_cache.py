"""Writing a cache of 8 or 4 bits, reading caches back, and the table calls on quantised pools: codes,
scales and copied bytes are whole numbers and equal, read values are exact but for the rounding to the
rows' type (half a step of bf16, 2^-8)."""
import numpy as np
import pytest
import torch

from jacobi_speculative_decode_gb300 import xp
from oracle import quant_oracle as Q

pytestmark = pytest.mark.gpu


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def make(bits, layers, pages, ps, heads, dim, fill=0xAA):
    k, v = (xp.QuantCache.pool(layers, pages, ps, heads, dim, bits) for _ in range(2))
    k.fill_(fill), v.fill_(fill)
    return xp.QuantCache(k, v, ps, dim, bits)


def rows_of(g, N, T, heads, dim, dtype):
    x = g.normal(size=(N, T, heads, dim)) * np.exp(g.normal(size=(N, T, heads, 1)) * 3)
    return torch.from_numpy(x).to(dtype).cuda()


def written(pool, layer, x, table, lens, ps, bits, T):
    """The pool's bytes after an append of rows x to `layer`."""
    want = pool.copy()
    for n in range(x.shape[0]):
        for t in range(T):
            pos = int(lens[n]) - T + t
            if pos < 0:
                continue
            for h in range(x.shape[2]):
                codes, byte, _ = Q.quantise(x[n, t, h], bits)
                Q.put(want[layer, table[n, pos // ps], h], pos % ps, codes, byte, ps, bits)
    return want


SHAPES = [  # (sequences, tokens, heads, dim, page)
    (1, 1, 1, 16, 1), (3, 1, 8, 128, 16), (2, 5, 3, 80, 20), (5, 17, 2, 64, 8), (2, 33, 1, 256, 5),
    (1, 40, 2, 96, 7), (4, 3, 40, 112, 4)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_and_read(shape, bits, dtype):
    N, T, H, D, ps = shape
    g = np.random.default_rng(N * T + D + bits)
    lens = g.integers(0, 3 * T + 2, N).astype(np.int32)      # some shorter than the new tokens
    lens[0] = T
    width = -(-int(lens.max()) // ps) + 1
    pages = N * width + 2
    table = g.permutation(pages)[:N * width].reshape(N, width).astype(np.int32)
    c = make(bits, 2, pages, ps, H, D)
    before = [p.cpu().numpy() for p in (c.k, c.v)]
    # slices of a fused projection
    fused = rows_of(g, N, T, 3 * H, D, dtype)
    k, v = fused[:, :, :H], fused[:, :, 2 * H:]
    xp.xp_cache_append(c.handle, 1, k, v, cu(table), cu(lens))
    # a few rows are drawn too large to be held: the oracle says which cases have one
    live = torch.arange(T)[None, :] >= T - torch.from_numpy(lens)[:, None]
    over = any(Q.quantise(x.double().cpu().numpy()[live.numpy()], bits)[2] for x in (k, v))
    assert xp.xp_cache_get_error(c.handle) == (xp.XP_ERANGE if over else xp.XP_OK)
    want = [written(b, 1, x.double().cpu().numpy(), table, lens, ps, bits, T) for b, x in zip(before, (k, v))]
    for got, w in zip((c.k, c.v), want):
        assert (got.cpu().numpy() == w).all()
    # the newest tokens, and everything from the start, as either type
    for first, count in ((lens - T, T), (None, int(lens.max()) + 3), (np.full(N, 2, np.int32), 1)):
        for out_dtype in (torch.float32, torch.bfloat16):
            wide = torch.full((2, N, count, H + 1, D), 7.0, dtype=out_dtype, device="cuda")
            ko, vo = wide[0, :, :, :H], wide[1, :, :, :H]
            at = None if first is None else cu(first)
            short = np.where(lens > 0, lens, 0)
            # only written positions stand for numbers: the others hold what the pool was filled with
            xp.xp_cache_read(c.handle, 1, cu(table), cu(short), at, ko, vo)
            for got, w in zip((ko, vo), want):
                got = got.double().cpu().numpy()
                for n in range(N):
                    for t in range(count):
                        pos = (0 if first is None else int(first[n])) + t
                        if 0 <= pos < lens[n]:
                            if pos < lens[n] - T:
                                continue
                            x = np.stack([Q.get(w[1, table[n, pos // ps], h], pos % ps, ps, D, bits)
                                          for h in range(H)])
                            tol = 0.0 if out_dtype == torch.float32 or bits == 4 else 2.0 ** -8
                            assert (np.abs(got[n, t] - x) <= tol * np.abs(x)).all()
                        else:
                            assert (got[n, t] == 0).all()
            assert (wide[:, :, :, H:] == 7.0).all()
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK


@pytest.mark.parametrize("bits", [4, 8])
def test_borders(bits):
    """Ties, scales' borders, zeros, subnormals, the largest values and next to them."""
    most, s = Q.most_of(bits), Q.scale_values()
    g = np.random.default_rng(bits)
    x = []
    for b in (1, 5, 8, 9, 60, 120, 127, Q.top_byte(bits)):
        edge = np.float32(s[b] * most)
        for top in (edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(1e9))):
            if b == Q.top_byte(bits) and top > edge:
                continue
            ties = (g.integers(-most, most, 15) + 0.5) * s[b]
            for r in (ties, np.nextafter(ties.astype(np.float32), np.float32(0)),
                      np.nextafter(ties.astype(np.float32), np.float32(1e9))):
                x.append(np.concatenate([[top], np.clip(r, -top, top)]))
    x += [np.zeros(16), np.full(16, -0.0), np.full(16, 2.0 ** -126), np.full(16, 1e-40), np.full(16, 2.0 ** -18)]
    x = np.asarray(x, np.float32).reshape(1, -1, 1, 16)
    T = x.shape[1]
    c = make(bits, 1, 1, T, 1, 16, fill=0)
    rows = torch.from_numpy(x).cuda()
    xp.xp_cache_append(c.handle, 0, rows, rows, cu([[0]]), cu([T]))
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    want = written(np.zeros(c.k.shape, np.uint8), 0, x.astype(np.float64), np.zeros((1, 1), int), [T], T, bits, T)
    assert (c.k.cpu().numpy() == want).all() and (c.v.cpu().numpy() == want).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 1e38, 66000.0])
def test_what_does_not_fit_is_told(bits, bad):
    c = make(bits, 1, 2, 4, 2, 32, fill=0)
    x = np.random.default_rng(1).normal(size=(1, 2, 2, 32)).astype(np.float32)
    x[0, 1, 0, 20] = bad
    rows, fine = torch.from_numpy(x).cuda(), torch.zeros(1, 2, 2, 32, device="cuda")
    for k, v in ((rows, fine), (fine, rows)):
        xp.xp_cache_append(c.handle, 0, k, v, cu([[1]]), cu([2]))
        assert xp.xp_cache_get_error(c.handle) == xp.XP_ERANGE
        assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    got = torch.empty(1, 2, 2, 32, device="cuda")
    xp.xp_cache_read(c.handle, 0, cu([[1]]), cu([2]), None, got, torch.empty_like(got))
    assert (got == 0).all()                  # the last append's keys
    xp.xp_cache_append(c.handle, 0, rows, fine, cu([[1]]), cu([2]))
    xp.xp_cache_read(c.handle, 0, cu([[1]]), cu([2]), None, got, torch.empty_like(got))
    codes, byte, over = Q.quantise(x, bits)
    assert over and (got.double().cpu().numpy() == Q.values(codes, byte)).all()


@pytest.mark.parametrize("dtype,order", [(torch.bfloat16, "token"), (torch.float32, "head")])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 80, 7])
def test_read_of_plain_caches(dtype, order, out_dtype, dim):
    g = torch.Generator(device="cuda").manual_seed(dim)
    shape = (2, 9, 5, 3, dim) if order == "token" else (2, 9, 3, 5, dim)
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    if order == "head":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    c = xp.Cache(k, v)
    table = cu([[3, 8, 1], [0, 2, 5]])
    lens, first = [13, 4], [2, -3]
    ko, vo = (torch.empty(2, 20, 3, dim, dtype=out_dtype, device="cuda") for _ in range(2))
    xp.xp_cache_read(c.handle, 1, table, cu(lens), cu(first), ko, vo)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    for got, pool in ((ko, k), (vo, v)):
        for n in range(2):
            whole = pool[1, table[n].long()].reshape(15, 3, dim)[:lens[n]].to(out_dtype)
            for t in range(20):
                pos = first[n] + t
                assert (got[n, t] == (whole[pos] if 0 <= pos < lens[n] else 0)).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_bad_pages_columns_and_empty_batches(bits):
    c = make(bits, 1, 3, 4, 2, 32, fill=0)
    x = torch.ones(1, 6, 2, 32, device="cuda")
    out = torch.full_like(x, 9.0)
    codes, byte, _ = Q.quantise(np.ones(16), bits)
    one = float(Q.values(codes, byte)[0])       # what a one is held as
    for table, lens, code in (([[7, 1]], [6], xp.XP_EBADPAGE), ([[-1, 1]], [6], xp.XP_EBADPAGE),
                              ([[1]], [6], xp.XP_ELENGTH)):
        xp.xp_cache_append(c.handle, 0, x, x, cu(table), cu(lens))
        assert xp.xp_cache_get_error(c.handle) == code
        xp.xp_cache_read(c.handle, 0, cu(table), cu(lens), None, out, torch.empty_like(out))
        assert xp.xp_cache_get_error(c.handle) == code
        # what has no page reads as zeros, the rest as written
        bad = [0, 1, 2, 3] if code == xp.XP_EBADPAGE else [4, 5]
        assert (out[0, bad] == 0).all() and (out[0, [t for t in range(6) if t not in bad]] == one).all()
    none = torch.empty(0, 3, 2, 32, device="cuda")
    xp.xp_cache_append(c.handle, 0, none, none, cu(np.zeros((1, 2))), cu(np.zeros(1)))
    xp.xp_cache_read(c.handle, 0, cu(np.zeros((1, 2))), cu(np.zeros(1)), None, none, none)
    empty = torch.empty(1, 0, 2, 32, device="cuda")
    xp.xp_cache_read(c.handle, 0, cu([[0, 1]]), cu([3]), None, empty, empty)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK


@pytest.mark.parametrize("bits,dim,heads,ps", [(4, 128, 8, 16), (8, 80, 3, 5)])
def test_table_calls_on_quantised_pools(bits, dim, heads, ps):
    layers, pages = 3, 40
    c = make(bits, layers, pages, ps, heads, dim)
    g = torch.Generator(device="cuda").manual_seed(3)
    for pool in (c.k, c.v):
        pool.copy_(torch.randint(0, 256, pool.shape, generator=g, device="cuda", dtype=torch.uint8))
    k, v = c.k.clone(), c.v.clone()
    xp.xp_cache_copy(c.handle, cu([1, -1, 5]), cu([2, 3, 39]))
    k[:, 2], k[:, 39], v[:, 2], v[:, 39] = k[:, 1], k[:, 5], v[:, 1], v[:, 5]
    assert (c.k == k).all() and (c.v == v).all()
    # two sequences, the second forked twice: full pages are shared, the partial one is copied whole
    table, lens, refs = cu(np.full((4, 6), -1)), cu(np.zeros(4)), cu(np.zeros(pages))
    xp.xp_cache_resize(c.handle, table, lens, cu([3 * ps, 2 * ps + 1, 0, 0]), refs, table, lens, refs)
    xp.xp_cache_fork(c.handle, table, lens, cu([1, 1]), None, refs, table[2:], lens[2:], refs)
    assert lens.tolist() == [3 * ps, 2 * ps + 1, 2 * ps + 1, 2 * ps + 1]
    assert table[2, :3].tolist() == [3, 4, 6] and table[3, :3].tolist() == [3, 4, 7]
    for p in (6, 7):
        assert (c.k[:, p] == k[:, 5]).all() and (c.v[:, p] == v[:, 5]).all()
    k, v = c.k.clone(), c.v.clone()
    old = table.clone()
    xp.xp_cache_resize(c.handle, table, lens, cu([0, 2 * ps + 1, 2 * ps + 1, 2 * ps + 1]), refs, table, lens, refs)
    xp.xp_cache_compact(c.handle, table, lens, refs, table, refs)
    assert xp.xp_cache_get_error(c.handle) == xp.XP_OK
    for n in range(1, 4):
        for j in range(3):
            assert (c.k[:, table[n, j]] == k[:, old[n, j]]).all()
            assert (c.v[:, table[n, j]] == v[:, old[n, j]]).all()
    assert int(table.max()) == 4


def test_offsets_past_two_to_the_31(bits=4):
    ps, H, D = 64, 8, 128
    size = xp.xp_quant_head_bytes(ps, D, bits)
    pages = 2 ** 31 // (H * size) + 9
    c = make(bits, 1, pages, ps, H, D, fill=0)
    g = np.random.default_rng(5)
    x = rows_of(g, 1, 70, H, D, torch.bfloat16)
    table, lens = cu([[pages - 1, pages - 4]]), cu([70])
    xp.xp_cache_append(c.handle, 0, x, x, table, lens)
    out = torch.empty(1, 70, H, D, device="cuda")
    xp.xp_cache_read(c.handle, 0, table, lens, None, out, torch.empty_like(out))
    codes, byte, _ = Q.quantise(x.double().cpu().numpy(), bits)
    assert (out.double().cpu().numpy() == Q.values(codes, byte)).all()
    assert int(c.k[0, :pages - 4].max()) == 0


def test_a_stream_and_a_graph():
    c = make(4, 1, 8, 16, 2, 64, fill=0)
    g = np.random.default_rng(6)
    x = rows_of(g, 2, 4, 2, 64, torch.bfloat16)
    table, lens = cu([[0, 1], [2, 3]]), cu([9, 20])
    first = lens - 4
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        xp.xp_cache_append(c.handle, 0, x, x, table, lens)
        xp.xp_cache_read(c.handle, 0, table, lens, first, ko, vo)
    for seed in (1, 2):
        y = rows_of(np.random.default_rng(seed), 2, 4, 2, 64, torch.bfloat16)
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        codes, byte, _ = Q.quantise(y.double().cpu().numpy(), 4)
        assert (ko.double().cpu().numpy() == Q.values(codes, byte)).all() and (ko == vo).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_off_their_types_boundary_are_refused(dtype):
    c = make(8, 1, 2, 16, 1, 64, fill=0)
    x = torch.ones(1, 3, 1, 64, device="cuda", dtype=dtype)
    table, lens = cu([[0, 1]]), cu([3])
    code = xp.XP_BF16 if dtype == torch.bfloat16 else xp.XP_F32
    for dk, dv in ((1, 0), (0, 1)):
        k, v = x.data_ptr() + dk, x.data_ptr() + dv
        assert xp.lib().xp_cache_append(c.handle, 0, k, v, 192, 64, 64, 1, 64, code, table.data_ptr(), 2,
                                        lens.data_ptr(), 1, 2, None) == xp.XP_EINVAL
        assert xp.lib().xp_cache_read(c.handle, 0, table.data_ptr(), 2, 2, lens.data_ptr(), None, 1, 2, k, v, 192, 64,
                                      64, 1, 64, code, None) == xp.XP_EINVAL
    if dtype == torch.bfloat16:
        q = torch.ones(1, 1, 1, 64, device="cuda", dtype=dtype)
        a = xp.make_attn(q, q, 0, 0, 16, 0.1)
        ws = c.attention_workspace(a)
        for dq, do in ((1, 0), (0, 1)):
            with pytest.raises(xp.XPError) as e:
                xp._check("attention", xp.lib().xp_prefix_attention(
                    c.handle, a, q.data_ptr() + dq, None, 0, table.data_ptr(), 2, 2, lens.data_ptr(),
                    q.data_ptr() + do, None, ws.data_ptr(), ws.numel() * ws.element_size(), None))
            assert e.value.code == xp.XP_EINVAL
    assert int(c.k.max()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [4, 8])
def test_magnitudes_around_the_greatest_that_is_held(bits, dtype):
    """The range ends at 127*512 and 7*7680, though larger scales would have finite values too: above it a group is
    held at the end and told, up to it nothing is."""
    end = Q.most_of(bits) * Q.scale_values()[Q.top_byte(bits)]
    g = np.random.default_rng(3)
    c = make(bits, 1, 1, 1, 1, 16, fill=0)
    got = torch.empty(1, 1, 1, 16, device="cuda", dtype=dtype)
    for top in (0.9 * end, end * (1 - 2.0 ** -7), end, end * (1 + 2.0 ** -6), 1.1 * end, 1.2 * end, 65504.0, 3e38):
        x = g.uniform(-0.5, 0.5, 16) * end
        x[5] = -top
        x = torch.from_numpy(x).reshape(1, 1, 1, 16).to(dtype).cuda()
        codes, byte, over = Q.quantise(x.double().cpu().numpy(), bits)
        assert over == (abs(x[0, 0, 0, 5].item()) > end)
        xp.xp_cache_append(c.handle, 0, x, x, cu([[0]]), cu([1]))
        assert xp.xp_cache_get_error(c.handle) == (xp.XP_ERANGE if over else xp.XP_OK)
        xp.xp_cache_read(c.handle, 0, cu([[0]]), cu([1]), None, got, torch.empty_like(got))
        want = torch.from_numpy(Q.values(codes, byte)).to(dtype)      # both round to nearest
        assert torch.equal(got.cpu(), want)
