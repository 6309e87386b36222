"""What is measured of the operators around a drafted block: the shared-prefix attention that scores it,
its verification, and the paged cache behind both.

``prepare`` builds what a serving program holds before the call, ``run`` is one call.  The plain forms are
elementary torch operations in 32 bits; ``exact`` states the same definitions in 64 bits, one sequence or
block at a time.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # four short chats behind a system prompt, one new token each: latency counts
        dict(name="attention decode few", op="attention", dtype="bf16", seqs=4, tokens=1, kv_heads=8,
             group=4, dim=128, prefix=512, tail_min=1, tail_max=64, page=16, order="token"),
        # a full batch of single tokens behind one long document, 64-wide heads
        dict(name="attention decode many", op="attention", dtype="bf16", seqs=256, tokens=1,
             kv_heads=8, group=8, dim=64, prefix=16384, tail_min=100, tail_max=2000, page=32,
             order="token"),
        # the batched-decode draft blocks (32 blocks of 16 slots) scored against a shared prefix
        dict(name="attention draft blocks", op="attention", dtype="bf16", seqs=32, tokens=16,
             kv_heads=8, group=4, dim=128, prefix=8192, tail_min=17, tail_max=1500, page=64,
             order="token"),
        # many draft blocks, tails up to 2048 tokens, pages with the heads outside the tokens
        dict(name="attention many blocks", op="attention", dtype="bf16", seqs=128, tokens=16,
             kv_heads=8, group=4, dim=128, prefix=8192, tail_min=16, tail_max=2048, page=128,
             order="head"),
        # odd sizes in fp32: pages of 20 tokens, tails shorter than the block, 96-wide heads
        dict(name="attention fp32 odd", op="attention", dtype="f32", seqs=7, tokens=5, kv_heads=3,
             group=4, dim=96, prefix=1001, tail_min=0, tail_max=333, page=20, order="token"),
        # one request, seven drafts from the greedy refinement (one-hot): latency counts
        dict(name="verify one block", op="verify", dtype="bf16", seqs=1, slots=8, vocab=151936,
             drafts="onehot", accept=0.8, greedy_every=0),
        # 32 blocks with the drafter's logits, every eighth request greedy
        dict(name="verify draft logits", op="verify", dtype="bf16", seqs=32, slots=16, vocab=151936,
             drafts="logits", accept=0.8, greedy_every=8),
        # the largest batch of the refinement, one-hot drafts
        dict(name="verify large batch", op="verify", dtype="bf16", seqs=256, slots=16, vocab=151936,
             drafts="onehot", accept=0.7, greedy_every=8),
        # pages for the next block of every sequence, and back after verification: tables only
        dict(name="pages resize", op="resize", seqs=256, width=128, pages=16384, page=16, layers=1,
             kv_heads=1, dim=64, fill_min=100, fill_max=1500, grow=17),
        # one prompt continued four ways
        dict(name="pages fork few", op="fork", seqs=1, children=4, width=32, pages=256, page=16,
             layers=4, kv_heads=8, dim=128, fill_min=90, fill_max=90),
        # 64 prompts into 256 continuations
        dict(name="pages fork many", op="fork", seqs=64, children=256, width=32, pages=2048, page=64,
             layers=8, kv_heads=8, dim=128, fill_min=65, fill_max=1900),
        # a pool at 40% after many sequences ended, packed to its front
        dict(name="pages compact", op="compact", seqs=48, width=32, pages=2048, page=64, layers=8,
             kv_heads=8, dim=128, live=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "verify", "verify", "resize", "fork", "compact"])
    if op == "attention":
        f32 = rng.random() < 0.25
        seqs, tokens = _log(rng, 1, 16 if f32 else 200), rng.choice([1, 1, 2, 4, 5, 8, 13, 16])
        case = dict(op=op, dtype="f32" if f32 else "bf16", seqs=seqs, tokens=tokens,
                    kv_heads=rng.choice([1, 2, 3, 8]), group=rng.choice([1, 2, 3, 4, 7, 8]),
                    dim=rng.choice([64, 80, 96, 128] if f32 else [64, 128, 128]),
                    prefix=rng.choice([0, _log(rng, 1, 2000 if f32 else 16000)]),
                    tail_min=rng.randint(0, 40), tail_max=_log(rng, 41, 2000),
                    page=rng.choice([16, 20, 64] if f32 else [16, 24, 32, 64, 128, 256]),
                    order=rng.choice(["token", "head"]))
        while work(case)["flops"] > 1.5e11 or (f32 and work(case)["flops"] > 5e9):
            case["seqs"] = max(1, case["seqs"] // 2)
            case["prefix"] = case["prefix"] * 2 // 3
        return case
    if op == "verify":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        vocab = rng.choice([_log(rng, 500, 151936), 151936])
        slots = rng.randint(2, 16)
        seqs = max(1, min(_log(rng, 1, 256), int(3.0e8 / (slots * vocab))))
        return dict(op=op, dtype=dtype, seqs=seqs, slots=slots, vocab=vocab,
                    drafts=rng.choice(["onehot", "logits"]), accept=rng.choice([0.5, 0.7, 0.9]),
                    greedy_every=rng.choice([0, 3]))
    page, dim = rng.choice([8, 16, 20, 64]), rng.choice([64, 128])
    if op == "resize":
        seqs, width = _log(rng, 1, 500), _log(rng, 8, 256)
        return dict(op=op, seqs=seqs, width=width, pages=seqs * width + rng.randint(1, 999), page=page,
                    layers=1, kv_heads=1, dim=64, fill_min=0, fill_max=width * page - 1 - page,
                    grow=rng.randint(1, page))
    width, layers, kv_heads = _log(rng, 4, 40), rng.randint(1, 8), rng.choice([1, 3, 8])
    if op == "fork":
        seqs, children = _log(rng, 1, 50), _log(rng, 1, 250)
        return dict(op=op, seqs=seqs, children=children, width=width,
                    pages=seqs * width + children + rng.randint(0, 50), page=page, layers=layers,
                    kv_heads=kv_heads, dim=dim, fill_min=1, fill_max=width * page - 1)
    seqs = _log(rng, 1, 48)
    return dict(op=op, seqs=seqs, width=width, pages=_log(rng, 2 * seqs + 8, 2000), page=page,
                layers=layers, kv_heads=kv_heads, dim=dim, live=rng.choice([0.1, 0.4, 0.8]))


# ------------------------------------------------------------- the inputs ---

def _spread(lo, hi, count):
    """`count` lengths spread evenly over [lo, hi], both ends among them: the case alone fixes which."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32)
    return t[torch.randperm(len(values), generator=g)].to(DEVICE)


def _accept_sigma(accept):
    """Noise on the draft's logits for which sum_v min(p, q) is `accept`: 2 Phi(-sigma / 2) for a mass
    spread over many tokens."""
    lo, hi = 0.0, 8.0
    for _ in range(60):
        mid = 0.5 * (lo + hi)
        lo, hi = (mid, hi) if math.erfc(mid / (2 * math.sqrt(2.0))) > accept else (lo, mid)
    return lo


def _pools(case, g_dev, order="token"):
    """K and V pools, seen as [layer, page, token, head, dim]; order "head" keeps a page's heads outside."""
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    layers, heads = case["layers"], case["kv_heads"]
    shape = ((layers, case["pages"], case["page"], heads, case["dim"]) if order == "token" else
             (layers, case["pages"], heads, case["page"], case["dim"]))
    pools = []
    for _ in range(2):
        t = torch.randn(shape, generator=g_dev, device=DEVICE, dtype=dt)
        pools.append(t if order == "token" else t.transpose(2, 3))
    return pools


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    g_dev = torch.Generator(device=DEVICE).manual_seed(seed)
    if case["op"] == "attention":
        return _prepare_attention(case, g, g_dev)
    if case["op"] == "verify":
        return _prepare_verify(case, g, g_dev)
    return _prepare_pages(case, g, g_dev)


def _prepare_attention(case, g, g_dev):
    N, T, H, G, D = (case[k] for k in ("seqs", "tokens", "kv_heads", "group", "dim"))
    ps, P = case["page"], case["prefix"]
    lens = _shuffled(_spread(case["tail_min"], case["tail_max"], N), g)
    width = -(-case["tail_max"] // ps)
    used = (lens.long() + ps - 1) // ps                       # pages of each tail
    prefix_pages = -(-P // ps)
    pages = prefix_pages + int(used.sum()) + 3
    ids = torch.randperm(pages, generator=g).to(torch.int32).to(DEVICE)
    prefix_table = ids[:max(prefix_pages, 1)].contiguous()
    slot = torch.arange(width, device=DEVICE)
    has = slot[None, :] < used[:, None]
    rank = prefix_pages + torch.cumsum(has.flatten(), 0).view(N, width) - 1
    table = torch.where(has, ids[rank.clamp(min=0)], -1).to(torch.int32).contiguous()
    k, v = _pools(dict(case, layers=1, pages=pages), g_dev, case["order"])
    # a pool is never cleared: what no token was written to holds anything, NaN among it
    live = torch.zeros(pages, ps, dtype=torch.bool, device=DEVICE)
    at = torch.arange(ps, device=DEVICE)
    left = (lens.long()[:, None] - slot[None, :] * ps)        # tokens left from each page on
    live[table[has].long()] = at[None, :] < left[has][:, None]
    if P:
        left = P - torch.arange(prefix_pages, device=DEVICE) * ps
        live[prefix_table.long()] = at[None, :] < left[:, None]
    k[0][~live] = math.nan
    v[0][~live] = math.nan
    # queries come out of a fused projection: their tokens are (heads + 2 kv heads) rows apart
    qkv = torch.randn(N, T, (G + 2) * H, D, generator=g_dev, device=DEVICE, dtype=k.dtype)
    q = (qkv * 1.5)[:, :, :G * H]
    s = dict(case=case, q=q, k=k, v=v, prefix_table=prefix_table, table=table, lens=lens,
             scale=1.0 / math.sqrt(D))
    if own:
        from jacobi_speculative_decode_gb300 import xp
        s["cache"] = xp.Cache(k, v)
        s["out"] = torch.empty(N, T, G * H, D, dtype=k.dtype, device=DEVICE)
        s["lse"] = torch.empty(N, T, G * H, dtype=torch.float32, device=DEVICE)
        s["attn"] = xp.make_attn(q, s["out"], layer=0, prefix_len=P, max_len=case["tail_max"],
                                 scale=s["scale"])
        s["ws"] = s["cache"].attention_workspace(s["attn"])
    return s


def _prepare_verify(case, g, g_dev):
    N, B, V = case["seqs"], case["slots"], case["vocab"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    spread = 2.5
    target = torch.randn(N, B, V, generator=g_dev, device=DEVICE) * spread
    target[:, :, V - V // 100:] = -math.inf                    # ids past the tokenizer's end
    temperature = torch.empty(N, device=DEVICE).uniform_(0.9, 1.1, generator=g_dev)
    greedy = torch.zeros(N, dtype=torch.bool, device=DEVICE)
    if case["greedy_every"]:
        greedy[::case["greedy_every"]] = True
    temperature[greedy] = 0.0
    heat = torch.where(greedy, 1.0, temperature)[:, None, None]
    blk = torch.randint(0, V - V // 100, (N, B), generator=g_dev, device=DEVICE)
    draft = None
    if case["drafts"] == "onehot":
        # the drafted token holds `accept` of the mass
        rest = torch.logsumexp(target[:, :-1] / heat, -1)
        peak = (rest + math.log(case["accept"] / (1 - case["accept"]))) * heat[:, :, 0]
        target[:, :-1].scatter_(2, blk[:, 1:, None], peak[:, :, None])
    else:
        noise = torch.randn(N, B - 1, V, generator=g_dev, device=DEVICE)
        draft = target[:, :-1] + noise * (_accept_sigma(case["accept"]) * heat)
        race = torch.empty(N, B - 1, V, device=DEVICE).exponential_(generator=g_dev)
        race = torch.where(greedy[:, None, None], 1.0, race)
        blk[:, 1:] = (draft / heat - race.log()).argmax(-1)
        draft = draft.view(N * (B - 1), V)
        del noise, race
    target = target.to(dt)
    u = torch.rand(N, B - 1, generator=g_dev, device=DEVICE)
    noise = torch.empty(N, V, device=DEVICE).exponential_(generator=g_dev).clamp_(min=1e-20)
    s = dict(case=case, target=target, draft=draft, blk=blk, temperature=temperature, u=u, noise=noise)
    if own:
        from jacobi_speculative_decode_gb300 import xp
        s["head"] = _small_head(xp, case, dt, N, B, V)
        s["ws"] = s["head"].verify_workspace(N)
        s["tokens"] = torch.empty(N, B, dtype=torch.int64, device=DEVICE)
        s["counts"] = torch.empty(N, dtype=torch.int32, device=DEVICE)
        s["prob"] = torch.empty(N, B - 1, dtype=torch.float32, device=DEVICE)
    return s


def _small_head(xp, case, dt, N, B, V):
    """A refinement head of the case's vocabulary and block (its own weights play no part here)."""
    r = 8
    shapes = dict(w1=(V, r), down_h=(r, r), down_g=(r, r), in_proj=(r, 3 * r), mix_L=(r, B, B),
                  w_gate=(r, r), w_up=(r, r), w_down=(r, r), w2=(V, r))
    w = {k: torch.zeros(shape, dtype=dt, device=DEVICE) for k, shape in shapes.items()}
    return xp.Head(dict(V=V, hidden=r, r=r, H=r, B=B), w, case["dtype"], N)


def _prepare_pages(case, g, g_dev):
    N, width, pages, ps = (case[k] for k in ("seqs", "width", "pages", "page"))
    k, v = _pools(case, g_dev)
    s = dict(case=case, k=k, v=v)
    if case["op"] == "compact":
        moved, live = _moves(case)
        low = torch.randperm(live, generator=g)[:live - moved]
        high = live + torch.randperm(pages - live, generator=g)[:moved]
        ids = torch.cat([low, high])[torch.randperm(live, generator=g)].to(torch.int32).to(DEVICE)
        # the live pages dealt out to the rows; each of the others also reads the first row's first page
        each = _spread(live // N, live // N, N)
        each[0] += live - sum(each)
        width = max(each) + 1
        each = torch.tensor(each, dtype=torch.int64, device=DEVICE)
        slot = torch.arange(width, device=DEVICE)
        has = slot[None, :] < each[:, None]
        rank = torch.cumsum(has.flatten(), 0).view(N, width) - 1
        own_pages = torch.where(has, ids[rank.clamp(min=0)], -1)
        table = torch.full((N, width), -1, dtype=torch.int32, device=DEVICE)
        table[0] = own_pages[0]
        table[1:, 0] = ids[0]
        table[1:, 1:] = own_pages[1:, :-1]
        each[1:] += 1
        lens = (each * ps - torch.randint(0, ps, (N,), generator=g).to(DEVICE)).to(torch.int32)
    else:
        lens = _shuffled(_spread(case["fill_min"], case["fill_max"], N), g)
        used = (lens.long() + ps - 1) // ps
        ids = torch.randperm(pages, generator=g).to(torch.int32).to(DEVICE)
        slot = torch.arange(width, device=DEVICE)
        has = slot[None, :] < used[:, None]
        rank = torch.cumsum(has.flatten(), 0).view(N, width) - 1
        table = torch.where(has, ids[rank.clamp(min=0)], -1).to(torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEVICE)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), (table >= 0).flatten().to(torch.int32))
    s.update(table=table.contiguous(), lens=lens, refs=refs)
    rows = N
    if case["op"] == "resize":
        # half of the rows take room for the next block, the others give back their last tokens
        grow = case["grow"]
        up = torch.arange(N, device=DEVICE) % 2 == 0
        s["new_lens"] = torch.where(up, lens + grow, (lens - grow).clamp(min=0)).to(torch.int32)
    if case["op"] == "fork":
        rows = case["children"]
        s["parent"] = _shuffled([i % N for i in range(rows)], g)
    if own:
        from jacobi_speculative_decode_gb300 import xp
        s["cache"] = xp.Cache(k, v)
        s["table_out"] = torch.empty(rows, table.shape[1], dtype=torch.int32, device=DEVICE)
        s["lens_out"] = torch.empty(rows, dtype=torch.int32, device=DEVICE)
        s["refs_out"] = torch.empty(pages, dtype=torch.int32, device=DEVICE)
        s["map"] = torch.empty(pages, dtype=torch.int32, device=DEVICE)
        s["live"] = torch.empty(1, dtype=torch.int32, device=DEVICE)
    return s


def _moves(case):
    """(pages that compaction moves, pages in use)."""
    pages = case["pages"]
    live = max(case["seqs"], min(pages - 1, int(case["live"] * pages)))
    return min(pages - live, round(live * (1 - live / pages))), live


# ---------------------------------------------------------------- one pass ---

def run(s):
    op = s["case"]["op"]
    if own:
        from jacobi_speculative_decode_gb300 import xp
        return {"attention": _own_attention, "verify": _own_verify, "resize": _own_resize,
                "fork": _own_fork, "compact": _own_compact}[op](xp, s)
    return {"attention": _plain_attention, "verify": _plain_verify, "resize": _plain_resize,
            "fork": _plain_fork, "compact": _plain_compact}[op](s)


def _own_attention(xp, s):
    xp.xp_prefix_attention(s["cache"].handle, s["attn"], s["q"], s["prefix_table"], s["table"],
                           s["lens"], s["out"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_verify(xp, s):
    xp.xp_verify_drafts(s["head"].handle, s["target"], s["draft"], s["blk"], None, s["temperature"],
                        s["u"], s["noise"], s["tokens"], s["counts"], s["prob"], s["ws"])
    return {"tokens": s["tokens"], "counts": s["counts"], "prob": s["prob"]}


def _own_resize(xp, s):
    xp.xp_cache_resize(s["cache"].handle, s["table"], s["lens"], s["new_lens"], s["refs"],
                       s["table_out"], s["lens_out"], s["refs_out"])
    return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"]}


def _own_fork(xp, s):
    xp.xp_cache_fork(s["cache"].handle, s["table"], s["lens"], s["parent"], None, s["refs"],
                     s["table_out"], s["lens_out"], s["refs_out"])
    return {"table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "k": s["k"],
            "v": s["v"]}


def _own_compact(xp, s):
    xp.xp_cache_compact(s["cache"].handle, s["table"], s["lens"], s["refs"], s["table_out"],
                        s["refs_out"], s["map"], s["live"])
    return {"table": s["table_out"], "refs": s["refs_out"], "map": s["map"], "live": s["live"],
            "k": s["k"], "v": s["v"]}


# --------------------------------------------------------- the plain forms ---

def _plain_attention(s):
    c = s["case"]
    N, T, H, G, D = (c[k] for k in ("seqs", "tokens", "kv_heads", "group", "dim"))
    P = c["prefix"]
    k, v, lens = s["k"][0], s["v"][0], s["lens"]
    kp = k[s["prefix_table"].long()].float().reshape(-1, H, D)[:P]
    vp = v[s["prefix_table"].long()].float().reshape(-1, H, D)[:P]
    pages = s["table"].clamp(min=0).long()
    L = pages.shape[1] * c["page"]
    at = torch.arange(L, device=DEVICE)
    live = (at[None, :] < lens[:, None])[:, :, None, None]
    kt = torch.where(live, k[pages].float().reshape(N, L, H, D), 0.0)
    vt = torch.where(live, v[pages].float().reshape(N, L, H, D), 0.0)
    q = s["q"].float().view(N, T, H, G, D)
    by_head = q.permute(2, 0, 1, 3, 4).reshape(H, N * T * G, D)
    by_seq = q.permute(0, 2, 1, 3, 4).reshape(N, H, T * G, D)
    tail = torch.matmul(by_seq, kt.permute(0, 2, 3, 1)).view(N, H, T, G, L) * s["scale"]
    sees = lens[:, None] - T + 1 + torch.arange(T, device=DEVICE)[None, :]     # [N, T] tail tokens
    hidden = at[None, None, :] >= sees[:, :, None]
    tail = tail.masked_fill(hidden[:, None, :, None, :], -math.inf)
    tail = tail.permute(1, 0, 2, 3, 4).reshape(H, N * T * G, L)
    score = torch.cat([torch.matmul(by_head, kp.permute(1, 2, 0)) * s["scale"], tail], -1)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight[:, :, :P], vp.permute(1, 0, 2))
    wt = weight[:, :, P:].view(H, N, T * G, L).transpose(0, 1)
    out = out + torch.matmul(wt, vt.permute(0, 2, 1, 3)).transpose(0, 1).reshape(H, N * T * G, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + torch.log(total))[:, :, 0]
    out = out.view(H, N, T, G, D).permute(1, 2, 0, 3, 4).reshape(N, T, H * G, D)
    lse = lse.view(H, N, T, G).permute(1, 2, 0, 3).reshape(N, T, H * G)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _first_top(z):
    ids = torch.arange(z.shape[-1], device=DEVICE)
    return torch.where(z == z.amax(-1, keepdim=True), ids, z.shape[-1]).amin(-1)


def _plain_softmax(z, heat):
    z = z.float() * (1.0 / heat)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_verify(s):
    target, draft, blk, u = s["target"], s["draft"], s["blk"], s["u"]
    N, B, V = target.shape
    greedy = s["temperature"] == 0
    heat = torch.where(greedy, 1.0, s["temperature"])[:, None, None]
    x = blk[:, 1:]
    p = _plain_softmax(target, heat)
    px = p[:, :-1].gather(2, x[:, :, None])[:, :, 0]
    qx = torch.ones_like(px)
    if draft is not None:
        qx = _plain_softmax(draft.view(N, B - 1, V), heat).gather(2, x[:, :, None])[:, :, 0]
    top = _first_top(target.float())
    px = torch.where(greedy[:, None], (top[:, :-1] == x).float(), px)
    qx = torch.where(greedy[:, None], 1.0, qx)
    ok = u * qx < px
    slot = torch.arange(B, device=DEVICE)
    a = torch.where(ok, B - 1, slot[None, :-1]).amin(1)        # slots accepted
    block = torch.arange(N, device=DEVICE)
    pa = p[block, a]
    rejected = a < B - 1
    b = a.clamp(max=B - 2)
    if draft is None:
        qa = (torch.arange(V, device=DEVICE)[None, :] == x[block, b][:, None]).float()
    else:
        qa = _plain_softmax(draft.view(N, B - 1, V)[block, b], heat[:, :, 0])
    w = torch.where(rejected[:, None], (pa - qa).clamp(min=0), pa)
    w = torch.where(w.amax(1, keepdim=True) > 0, w, pa)
    last = _first_top(w / s["noise"])
    last = torch.where(greedy, top[block, a], last)
    tokens = torch.where(slot[None, :-1] < a[:, None], x, -1)
    tokens = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], 1)
    tokens[block, a] = last
    tested = slot[None, :-1] <= a[:, None]
    prob = torch.where(tested, (px / qx).clamp(max=1.0), 0.0)
    return {"tokens": tokens, "counts": (a + 1).to(torch.int32), "prob": prob}


def _free_first(refs):
    """Page ids with the unused ones first, ascending, and how many are unused."""
    return torch.sort((refs > 0).to(torch.int32), stable=True)[1], (refs == 0).sum()


def _plain_resize(s):
    table, lens, new, refs, ps = s["table"], s["lens"], s["new_lens"], s["refs"], s["case"]["page"]
    width = table.shape[1]
    have, want = (lens + ps - 1) // ps, (new + ps - 1) // ps
    slot = torch.arange(width, device=DEVICE)[None, :]
    page = table.clamp(min=0).long()
    drop = (slot >= want[:, None]) & (slot < have[:, None])
    refs = refs.clone().index_add_(0, page.flatten(), -drop.flatten().to(torch.int32))
    order, count = _free_first(refs)
    need = (slot >= have[:, None]) & (slot < want[:, None])
    rank = torch.cumsum(need.flatten(), 0).view_as(need) - 1
    got = need & (rank < count)
    taken = order[rank.clamp(0, refs.numel() - 1)]
    refs.index_add_(0, taken.flatten(), got.flatten().to(torch.int32))
    keep = (slot < have[:, None]) & (slot < want[:, None])
    out = torch.where(got, taken, torch.where(keep, table.long(), -1)).to(torch.int32)
    room = (out >= 0).sum(1) * ps
    return {"table": out, "lens": torch.minimum(new, room).to(torch.int32), "refs": refs}


def _plain_fork(s):
    table, refs, ps = s["table"], s["refs"].clone(), s["case"]["page"]
    parent = s["parent"].long()
    lens, rows = s["lens"][parent], table[parent]
    full, part = (lens // ps).long(), lens % ps
    slot = torch.arange(table.shape[1], device=DEVICE)[None, :]
    shared = slot < full[:, None]
    order, count = _free_first(refs)
    need = part > 0
    rank = torch.cumsum(need, 0) - 1
    got = need & (rank < count)
    taken = order[rank.clamp(0, refs.numel() - 1)]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().to(torch.int32))
    refs.index_add_(0, taken, got.to(torch.int32))
    out = torch.where(shared, rows, -1)
    out = torch.where(got[:, None] & (slot == full[:, None]), taken[:, None].to(torch.int32), out)
    child = torch.where(need & ~got, full.to(torch.int32) * ps, lens)
    which = torch.nonzero(got)[:, 0]
    src = rows[which, full[which]].long()
    dst = taken[which]
    live = (torch.arange(ps, device=DEVICE)[None, :] < part[which][:, None])[None, :, :, None, None]
    for pool in (s["k"], s["v"]):
        pool[:, dst] = torch.where(live, pool[:, src], pool[:, dst])
    return {"table": out, "lens": child.to(torch.int32), "refs": refs, "k": s["k"], "v": s["v"]}


def _plain_compact(s):
    table, refs, ps = s["table"], s["refs"], s["case"]["page"]
    pages = refs.numel()
    used = refs > 0
    live = used.sum()
    ids = torch.arange(pages, device=DEVICE)
    src = torch.nonzero(used & (ids >= live))[:, 0]
    dst = torch.nonzero(~used & (ids < live))[:, 0]
    new = torch.where(used, ids, -1)
    new[src] = dst
    out_refs = torch.zeros_like(refs)
    out_refs[new[used]] = refs[used]
    slot = torch.arange(table.shape[1], device=DEVICE)[None, :]
    held = slot < ((s["lens"] + ps - 1) // ps)[:, None]
    out = torch.where(held, new[table.clamp(min=0).long()], -1).to(torch.int32)
    for pool in (s["k"], s["v"]):
        pool[:, dst] = pool[:, src]
    return {"table": out, "refs": out_refs, "map": new.to(torch.int32),
            "live": live.to(torch.int32).view(1), "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------- work ---

def work(case):
    op = case["op"]
    if op == "attention":
        N, T, H, G, D, P = (case[k] for k in ("seqs", "tokens", "kv_heads", "group", "dim", "prefix"))
        es = 4 if case["dtype"] == "f32" else 2
        lens = _spread(case["tail_min"], case["tail_max"], N)
        seen = sum(max(0, n - T + 1 + t) for n in lens for t in range(T)) + N * T * P
        tables = 4 * (-(-P // case["page"]) + sum(-(-n // case["page"]) + 1 for n in lens))
        return {"bytes": 2 * N * T * H * G * D * es + 4 * N * T * H * G
                + 2 * (P + sum(lens)) * H * D * es + tables, "flops": 4 * D * G * H * seen}
    if op == "verify":
        # rows past the first rejection need not be read: what is expected at this acceptance
        N, B, V, a = (case[k] for k in ("seqs", "slots", "vocab", "accept"))
        es = 4 if case["dtype"] == "f32" else 2
        drafts = sum(a ** b for b in range(B - 1))
        rows = drafts + a ** (B - 1)
        each = rows * es + (drafts * 4 if case["drafts"] == "logits" else 0)
        return {"bytes": N * (V * (each + 4) + 12 * B + 8 * B + 12),
                "flops": N * V * (rows + (drafts if case["drafts"] == "logits" else 0)) * 4}
    token = case["layers"] * 2 * case["kv_heads"] * case["dim"] * 2        # bytes, bf16
    rows = case["children"] if op == "fork" else case["seqs"]
    tables = 8 * case["pages"] + 8 * rows
    if op == "compact":
        moved, live = _moves(case)
        return {"bytes": 2 * moved * case["page"] * token + tables + 4 * case["pages"]
                + 8 * (live + case["seqs"]), "flops": 0}
    lens = _spread(case["fill_min"], case["fill_max"], case["seqs"])
    if op == "fork":
        each = [lens[i % case["seqs"]] for i in range(rows)]
        copied = sum(n % case["page"] for n in each)
        return {"bytes": 2 * copied * token + tables + 8 * sum(-(-n // case["page"]) for n in each),
                "flops": 0}
    return {"bytes": tables + 8 * sum(-(-n // case["page"]) for n in lens), "flops": 0}


# ------------------------------------------------------------------ 64 bits ---

def exact(case, seed):
    if case["op"] not in ("attention", "verify"):
        return None                    # copies and whole numbers
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] == "attention" else _exact_verify(s)


def _exact_attention(s):
    c = s["case"]
    T, H, G, D, P, ps = (c[k] for k in ("tokens", "kv_heads", "group", "dim", "prefix", "page"))
    outs, lses = [], []

    def tokens_of(pool, ids, count):
        got = [pool[0, p, :max(0, min(ps, count - i * ps))] for i, p in enumerate(ids)]
        return torch.cat(got + [pool[0, 0, :0]]).double()

    prefix = s["prefix_table"].tolist()[:-(-P // ps)]
    kp, vp = tokens_of(s["k"], prefix, P), tokens_of(s["v"], prefix, P)
    for n, length in enumerate(s["lens"].tolist()):
        ids = s["table"][n].tolist()[:-(-length // ps)]
        k = torch.cat([kp, tokens_of(s["k"], ids, length)]).repeat_interleave(G, 1)
        v = torch.cat([vp, tokens_of(s["v"], ids, length)]).repeat_interleave(G, 1)
        out = torch.zeros(T, H * G, D, dtype=torch.float64, device=DEVICE)
        lse = torch.full((T, H * G), -math.inf, dtype=torch.float64, device=DEVICE)
        for t in range(T):
            sees = P + max(0, length - T + 1 + t)
            if sees:
                score = torch.einsum("hd,jhd->hj", s["q"][n, t].double(), k[:sees]) * s["scale"]
                lse[t] = torch.logsumexp(score, -1)
                out[t] = torch.einsum("hj,jhd->hd", torch.exp(score - lse[t][:, None]), v[:sees])
        outs.append(out)
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_verify(s):
    N, B, V = s["target"].shape
    prob = torch.zeros(N, B - 1, dtype=torch.float64, device=DEVICE)
    for n, heat in enumerate(s["temperature"].tolist()):
        for b in range(B - 1):
            x, row = int(s["blk"][n, b + 1]), s["target"][n, b].double()
            if heat == 0:
                p, q = float(int(torch.nonzero(row == row.max())[0]) == x), 1.0
            else:
                p = float(torch.exp(row[x] / heat - torch.logsumexp(row / heat, 0)))
                q = 1.0
                if s["draft"] is not None:
                    d = s["draft"][n * (B - 1) + b].double()
                    q = float(torch.exp(d[x] / heat - torch.logsumexp(d / heat, 0)))
            prob[n, b] = min(1.0, p / q)
            if not float(s["u"][n, b]) * q < p:
                break
    return {"tokens": None, "counts": None, "prob": prob}
