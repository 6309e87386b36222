"""What is measured of the cache held in 8 or 4 bits, and of log probabilities.

A quantised cache is written (and what was written read back), read, and attended over; the emitted
tokens' log probabilities come with the entropy, the rank and the best alternatives.  ``prepare`` builds
what a serving program holds before the call, ``run`` is one call (a write: two).  The plain forms are
elementary torch operations in 32 bits; ``exact`` states the same definitions in 64 bits, apart from them.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one new token of four chats goes into the cache: latency counts
        dict(name="write one token", op="write", bits=4, dtype="bf16", seqs=4, tokens=1, kv_heads=8, dim=128,
             page=16, len_min=100, len_max=900),
        # eight prompts of 4096 tokens at once, rows in fp32
        dict(name="write prompts", op="write", bits=8, dtype="f32", seqs=8, tokens=4096, kv_heads=8, dim=128,
             page=64, len_min=4096, len_max=5000),
        # odd sizes: one short sequence of 80-wide heads read back whole
        dict(name="read one sequence", op="read", bits=8, dtype="f32", seqs=1, kv_heads=3, dim=80, page=20,
             len_min=333, len_max=333),
        # the tails of 32 requests leave the 4-bit cache as bf16
        dict(name="read batch", op="read", bits=4, dtype="bf16", seqs=32, kv_heads=8, dim=128, page=64,
             len_min=17, len_max=3000),
        # four short chats behind a system prompt, one new token each: latency counts
        dict(name="attention decode few", op="attention", bits=4, seqs=4, tokens=1, kv_heads=8, group=4,
             dim=128, prefix=512, tail_min=1, tail_max=64, page=16),
        # odd sizes: blocks longer than some tails, 96-wide heads, pages of 20 tokens, 8 bits
        dict(name="attention odd", op="attention", bits=8, seqs=7, tokens=5, kv_heads=3, group=4, dim=96,
             prefix=1001, tail_min=0, tail_max=333, page=20),
        # 32 draft blocks of 16 slots scored against a shared prefix, 8 bits
        dict(name="attention draft blocks", op="attention", bits=8, seqs=32, tokens=16, kv_heads=8, group=4,
             dim=128, prefix=8192, tail_min=17, tail_max=1500, page=64),
        # a full batch of single tokens behind one long document, 64-wide heads
        dict(name="attention decode many", op="attention", bits=4, seqs=256, tokens=1, kv_heads=8, group=8,
             dim=64, prefix=16384, tail_min=100, tail_max=2000, page=32),
        # sixteen long contexts of their own, one token each: the cache's bytes are the cost
        dict(name="attention long contexts", op="attention", bits=4, seqs=16, tokens=1, kv_heads=8, group=4,
             dim=128, prefix=0, tail_min=1000, tail_max=32768, page=64),
        # the tokens of one verified block, with five alternatives: latency counts
        dict(name="logprobs one block", op="logprobs", dtype="bf16", seqs=1, slots=8, vocab=151936, emitted=1.0,
             top=5),
        # a batch of verified blocks, 20 alternatives; slots behind the emitted tokens hold none
        dict(name="logprobs blocks", op="logprobs", dtype="bf16", seqs=32, slots=16, vocab=151936, emitted=0.8,
             top=20),
        # every token of long prompts under their own logits in fp32, an odd vocabulary, no alternatives
        dict(name="logprobs prompts", op="logprobs", dtype="f32", seqs=4, slots=512, vocab=151647, emitted=1.0,
             top=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention", "logprobs", "logprobs"])
    if op == "logprobs":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        vocab = rng.choice([_log(rng, 500, 151936), 151936, 151647])
        slots = rng.choice([1, 2, 5, 8, 16, _log(rng, 17, 700)])
        seqs = max(1, min(_log(rng, 1, 200), int(3.0e8 / (slots * vocab))))
        return dict(op=op, dtype=dtype, seqs=seqs, slots=slots, vocab=vocab,
                    emitted=rng.choice([0.5, 0.8, 1.0]), top=rng.choice([0, 1, 3, 5, 20, 32]))
    case = dict(op=op, bits=rng.choice([4, 8]), seqs=_log(rng, 1, 100), kv_heads=rng.choice([1, 2, 3, 8]),
                dim=rng.choice([64, 80, 96, 128, 128, 256]), page=rng.choice([8, 16, 20, 32, 64, 128]))
    if op == "attention":
        case.update(tokens=rng.choice([1, 1, 2, 4, 5, 8, 13, 16]), group=rng.choice([1, 2, 3, 4, 7, 8]),
                    prefix=rng.choice([0, _log(rng, 1, 16000)]), tail_min=rng.randint(0, 40),
                    tail_max=_log(rng, 41, 9000))
        while work(case)["flops"] > 4e10 or work(case)["bytes"] > 3e8:
            case["seqs"] = max(1, case["seqs"] // 2)
            case["prefix"] = case["prefix"] * 2 // 3
            case["tail_max"] = max(41, case["tail_max"] * 4 // 5)
        return case
    case.update(dtype=rng.choice(["bf16", "f32"]), len_max=_log(rng, 1, 4000))
    case["len_min"] = rng.randint(0, case["len_max"])
    if op == "write":
        case["tokens"] = rng.randint(1, case["len_max"])
    while work(case)["bytes"] > 4e8:
        case["seqs"] = max(1, case["seqs"] // 2)
        case["kv_heads"] = max(1, case["kv_heads"] // 2)
    return case


# ------------------------------------------------- the quantised cache held ---
#
# A head of a page: the tokens' codes, dim*bits/8 bytes each, then their scales, one byte for 16 dims, padded
# to a multiple of 4 bytes a token; the whole padded to a multiple of 16 bytes.  A scale is the float of five
# exponent and three mantissa bits that is the upper half of a 16-bit float's magnitude (bits = byte << 7);
# it is the least for which no element needs a code beyond +-(2^(bits-1) - 1).  A code is the element over
# the scale, rounded to nearest even, plus 2^(bits-1); 4-bit codes of dims 8w + 2j + e are the
# bits from 4 (j + 4 e) on of word w.

def _sizes(case):
    """(bytes of a token's codes, of its scales, of a head of a page)"""
    codes, scales = case["dim"] * case["bits"] // 8, -(-case["dim"] // 64) * 4
    return codes, scales, -(-case["page"] * (codes + scales) // 16) * 16


def _scale_values():
    return (torch.arange(256, device=DEVICE, dtype=torch.int32) << 7).to(torch.int16).view(torch.float16)


def _quantise(x, bits):
    """(codes uint8, scale bytes) of rows [..., dim] in 32 bits; a quotient next to a border is 64 bits'."""
    most = 2 ** (bits - 1) - 1
    top = x.unflatten(-1, (-1, 16)).abs().amax(-1)
    grid = _scale_values()[:0xE2 if bits == 4 else 0xC1].double()
    byte = torch.searchsorted(grid * most, top.double()).clamp(max=grid.numel() - 1)
    step = grid[byte][..., None]
    code = torch.round(x.unflatten(-1, (-1, 16)).double() / torch.where(step == 0, 1.0, step))
    code = code.clamp(-most, most).flatten(-2)
    return (code + (most + 1)).to(torch.uint8), byte.to(torch.uint8)


def _dequantise(codes, scales, bits):
    value = codes.float() - 2 ** (bits - 1)
    return value * _scale_values().float()[scales.long()].repeat_interleave(16, -1)


def _pack(codes, bits):
    """Codes [..., dim] to bytes [..., dim*bits/8]."""
    if bits == 8:
        return codes
    words = codes.unflatten(-1, (-1, 4, 2)).transpose(-1, -2).reshape(codes.shape[:-1] + (-1, 2))
    return words[..., 0] | words[..., 1] << 4


def _unpack(packed, bits):
    if bits == 8:
        return packed
    words = torch.stack([packed & 15, packed >> 4], -1).unflatten(-2, (-1, 4)).flatten(-2)
    return words.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)


def _rows(pool, case):
    """Views of a layer's pool: the codes [page, head, token, bytes] and scales [page, head, token, dim/16]."""
    codes, scales, _ = _sizes(case)
    ps = case["page"]
    head = pool[..., ps * codes:ps * (codes + scales)].unflatten(-1, (ps, scales))
    return pool[..., :ps * codes].unflatten(-1, (ps, codes)), head[..., :case["dim"] // 16]


def _filled_pool(case, pages, live, g_dev):
    """A pool [1, pages, heads, bytes] whose live tokens [pages, page] hold quantised normal numbers; what no
    token was written to holds anything."""
    H, D, bits = case["kv_heads"], case["dim"], case["bits"]
    pool = torch.randint(0, 256, (1, pages, H, _sizes(case)[2]), generator=g_dev, device=DEVICE,
                         dtype=torch.uint8)
    each = max(1, 2 ** 25 // (case["page"] * H * D))
    for p in range(0, pages, each):
        part = pool[0, p:p + each]
        x = torch.randn(part.shape[0], H, case["page"], D, generator=g_dev, device=DEVICE)
        codes, scales = _quantise(x, bits)
        to_codes, to_scales = _rows(part, case)
        at = live[p:p + each, None, :, None]
        to_codes.copy_(torch.where(at, _pack(codes, bits), to_codes))
        to_scales.copy_(torch.where(at, scales, to_scales))
    return pool


# ------------------------------------------------------------- the inputs ---

def _spread(lo, hi, count):
    """`count` lengths spread evenly over [lo, hi], both ends among them: the case alone fixes which."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _shuffled(values, g):
    t = torch.tensor(values, dtype=torch.int32)
    return t[torch.randperm(len(values), generator=g)].to(DEVICE)


def _tables(case, lens, prefix, g):
    """(prefix table, table, pages, tokens that are live in them): scattered pages, a few unused."""
    ps, N = case["page"], case["seqs"]
    width = max(1, -(-int(lens.max()) // ps))
    used = (lens.long() + ps - 1) // ps
    prefix_pages = -(-prefix // ps)
    pages = prefix_pages + int(used.sum()) + 3
    ids = torch.randperm(pages, generator=g).to(torch.int32).to(DEVICE)
    prefix_table = ids[:max(prefix_pages, 1)].contiguous()
    slot = torch.arange(width, device=DEVICE)
    has = slot[None, :] < used[:, None]
    rank = prefix_pages + torch.cumsum(has.flatten(), 0).view(N, width) - 1
    table = torch.where(has, ids[rank.clamp(min=0)], -1).to(torch.int32).contiguous()
    live = torch.zeros(pages, ps, dtype=torch.bool, device=DEVICE)
    at = torch.arange(ps, device=DEVICE)
    left = lens.long()[:, None] - slot[None, :] * ps
    live[table[has].long()] = at[None, :] < left[has][:, None]
    if prefix:
        left = prefix - torch.arange(prefix_pages, device=DEVICE) * ps
        live[prefix_table.long()] = at[None, :] < left[:, None]
    return prefix_table, table, pages, live


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    g_dev = torch.Generator(device=DEVICE).manual_seed(seed)
    if case["op"] == "logprobs":
        return _prepare_logprobs(case, g, g_dev)
    if case["op"] == "attention":
        return _prepare_attention(case, g, g_dev)
    return _prepare_rows(case, g, g_dev)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _prepare_rows(case, g, g_dev):
    N, H, D = case["seqs"], case["kv_heads"], case["dim"]
    lens = _shuffled(_spread(case["len_min"], case["len_max"], N), g)
    _, table, pages, live = _tables(case, lens, 0, g)
    s = dict(case=case, table=table, lens=lens)
    s["k"], s["v"] = (_filled_pool(case, pages, live, g_dev) for _ in range(2))
    T = case["len_max"]
    if case["op"] == "write":
        T = case["tokens"]
        s["first"] = lens - T
        # keys and values are the last heads of a fused projection; a few channels are large
        heads = torch.randn(N, T, 4 * H, D, generator=g_dev, device=DEVICE)
        heads[..., ::37] *= 8.0
        heads = heads.to(_dtype(case))
        s["rows_k"], s["rows_v"] = heads[:, :, 2 * H:3 * H], heads[:, :, 3 * H:]
    if own:
        from jacobi_speculative_decode_gb300 import xp
        s["cache"] = xp.QuantCache(s["k"], s["v"], case["page"], D, case["bits"])
        out = torch.float32 if case["op"] == "write" else _dtype(case)
        s["k_out"], s["v_out"] = (torch.empty(N, T, H, D, dtype=out, device=DEVICE) for _ in range(2))
    return s


def _prepare_attention(case, g, g_dev):
    N, T, H, G, D, P = (case[k] for k in ("seqs", "tokens", "kv_heads", "group", "dim", "prefix"))
    lens = _shuffled(_spread(case["tail_min"], case["tail_max"], N), g)
    prefix_table, table, pages, live = _tables(case, lens, P, g)
    k, v = (_filled_pool(case, pages, live, g_dev) for _ in range(2))
    # queries come out of a fused projection: their tokens are (heads + 2 kv heads) rows apart
    qkv = torch.randn(N, T, (G + 2) * H, D, generator=g_dev, device=DEVICE, dtype=torch.bfloat16)
    q = (qkv * 1.5)[:, :, :G * H]
    s = dict(case=case, q=q, k=k, v=v, prefix_table=prefix_table, table=table, lens=lens,
             scale=1.0 / math.sqrt(D))
    if own:
        from jacobi_speculative_decode_gb300 import xp
        s["cache"] = xp.QuantCache(k, v, case["page"], D, case["bits"])
        s["out"] = torch.empty(N, T, G * H, D, dtype=q.dtype, device=DEVICE)
        s["lse"] = torch.empty(N, T, G * H, dtype=torch.float32, device=DEVICE)
        s["attn"] = xp.make_attn(q, s["out"], layer=0, prefix_len=P, max_len=case["tail_max"],
                                 scale=s["scale"])
        s["ws"] = s["cache"].attention_workspace(s["attn"])
    return s


def _emitted(case):
    """Tokens of each block, at least one: spread so that `emitted` of all slots hold one."""
    B = case["slots"]
    lo = max(1, min(B, round(B * (2 * case["emitted"] - 1))))
    return _spread(lo, B, case["seqs"])


def _prepare_logprobs(case, g, g_dev):
    N, B, V = case["seqs"], case["slots"], case["vocab"]
    logits = torch.randn(N, B, V, generator=g_dev, device=DEVICE) * 2.5
    logits[:, :, V - V // 100:] = -math.inf                    # ids past the tokenizer's end
    logits = logits.to(_dtype(case))
    temperature = torch.empty(N, device=DEVICE).uniform_(0.7, 1.3, generator=g_dev)
    tokens = torch.empty(N, B, dtype=torch.int64, device=DEVICE)
    for n in range(N):
        race = torch.empty(B, V, device=DEVICE).exponential_(generator=g_dev)
        tokens[n] = (logits[n].float() / temperature[n] - race.log()).argmax(-1)
    counts = _shuffled(_emitted(case), g)
    tokens[torch.arange(B, device=DEVICE)[None, :] >= counts[:, None]] = -1
    s = dict(case=case, logits=logits, temperature=temperature, tokens=tokens)
    if own:
        from jacobi_speculative_decode_gb300 import xp
        s["head"] = _small_head(xp, case, logits.dtype, N, B, V)
        s["ws"] = s["head"].logprobs_workspace(N * B, case["top"])
        s["logprob"], s["entropy"] = (torch.empty(N, B, device=DEVICE) for _ in range(2))
        s["rank"] = torch.empty(N, B, dtype=torch.int32, device=DEVICE)
        s["top_ids"] = torch.empty(N, B, case["top"], dtype=torch.int64, device=DEVICE)
        s["top_logprobs"] = torch.empty(N, B, case["top"], device=DEVICE)
    return s


def _small_head(xp, case, dt, N, B, V):
    """A refinement head of the case's vocabulary (its own weights play no part here)."""
    r, B = 8, max(2, min(B, 16))
    shapes = dict(w1=(V, r), down_h=(r, r), down_g=(r, r), in_proj=(r, 3 * r), mix_L=(r, B, B),
                  w_gate=(r, r), w_up=(r, r), w_down=(r, r), w2=(V, r))
    w = {k: torch.zeros(shape, dtype=dt, device=DEVICE) for k, shape in shapes.items()}
    return xp.Head(dict(V=V, hidden=r, r=r, H=r, B=B), w, case["dtype"], N)


# ---------------------------------------------------------------- one pass ---

def run(s):
    op = s["case"]["op"]
    if own:
        from jacobi_speculative_decode_gb300 import xp
        return {"write": _own_write, "read": _own_read, "attention": _own_attention,
                "logprobs": _own_logprobs}[op](xp, s)
    return {"write": _plain_write, "read": _plain_read, "attention": _plain_attention,
            "logprobs": _plain_logprobs}[op](s)


def _own_write(xp, s):
    xp.xp_cache_append(s["cache"].handle, 0, s["rows_k"], s["rows_v"], s["table"], s["lens"])
    xp.xp_cache_read(s["cache"].handle, 0, s["table"], s["lens"], s["first"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_read(xp, s):
    xp.xp_cache_read(s["cache"].handle, 0, s["table"], s["lens"], None, s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attention(xp, s):
    xp.xp_prefix_attention(s["cache"].handle, s["attn"], s["q"], s["prefix_table"], s["table"],
                           s["lens"], s["out"], s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_logprobs(xp, s):
    xp.xp_token_logprobs(s["head"].handle, s["logits"], s["tokens"], s["temperature"], s["logprob"],
                         s["entropy"], s["rank"], s["top_ids"], s["top_logprobs"], s["ws"])
    return {k: s[k] for k in ("logprob", "entropy", "rank", "top_ids", "top_logprobs")}


# --------------------------------------------------------- the plain forms ---

def _gathered(pool, case, page, token):
    """Values [..., head, dim] in 32 bits of the tokens (page, token) of a layer's pool."""
    codes, scales = _rows(pool, case)
    return _dequantise(_unpack(codes[page, :, token], case["bits"]), scales[page, :, token], case["bits"])


def _plain_read(s):
    c = s["case"]
    at = torch.arange(c["len_max"], device=DEVICE)
    live = at[None, :] < s["lens"][:, None]
    page = s["table"].long()[:, at // c["page"]].clamp(min=0)
    token = (at % c["page"]).expand_as(page)
    return {name: torch.where(live[:, :, None, None], _gathered(s[name][0], c, page, token), 0.0)
            .to(_dtype(c)) for name in ("k", "v")}


def _plain_write(s):
    c = s["case"]
    at = s["first"].long()[:, None] + torch.arange(c["tokens"], device=DEVICE)[None, :]
    live, at = at >= 0, at.clamp(min=0)
    page = s["table"].long().gather(1, at // c["page"])
    token = at % c["page"]
    out = {}
    for name in ("k", "v"):
        codes, scales = _quantise(s["rows_" + name].float(), c["bits"])
        to_codes, to_scales = _rows(s[name][0], c)
        to_codes[page[live], :, token[live]] = _pack(codes, c["bits"])[live]
        to_scales[page[live], :, token[live]] = scales[live]
        back = _gathered(s[name][0], c, page.clamp(min=0), token)
        out[name] = torch.where(live[:, :, None, None], back, 0.0)
    return out


def _plain_attention(s):
    c = s["case"]
    N, T, H, G, D = (c[k] for k in ("seqs", "tokens", "kv_heads", "group", "dim"))
    P, ps, lens = c["prefix"], c["page"], s["lens"]
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * ps
    at = torch.arange(L, device=DEVICE)
    live = (at[None, :] < lens[:, None])[:, :, None, None]
    shared = torch.arange(P, device=DEVICE)

    def tail(pool):
        return torch.where(live, _gathered(pool, c, table[:, at // ps], (at % ps).expand(N, L)), 0.0)

    def prefix(pool):
        return _gathered(pool, c, s["prefix_table"].long()[shared // ps], shared % ps)

    kt, kp = tail(s["k"][0]), prefix(s["k"][0])
    q = s["q"].float().view(N, T, H, G, D)
    by_head = q.permute(2, 0, 1, 3, 4).reshape(H, N * T * G, D)
    by_seq = q.permute(0, 2, 1, 3, 4).reshape(N, H, T * G, D)
    score = torch.matmul(by_seq, kt.permute(0, 2, 3, 1)).view(N, H, T, G, L) * s["scale"]
    sees = lens[:, None] - T + 1 + torch.arange(T, device=DEVICE)[None, :]     # [N, T] tail tokens
    hidden = at[None, None, :] >= sees[:, :, None]
    score = score.masked_fill(hidden[:, None, :, None, :], -math.inf)
    score = score.permute(1, 0, 2, 3, 4).reshape(H, N * T * G, L)
    score = torch.cat([torch.matmul(by_head, kp.permute(1, 2, 0)) * s["scale"], score], -1)
    del kt, kp
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    out = torch.matmul(weight[:, :, :P], prefix(s["v"][0]).permute(1, 0, 2))
    wt = weight[:, :, P:].view(H, N, T * G, L).transpose(0, 1)
    out = out + torch.matmul(wt, tail(s["v"][0]).permute(0, 2, 1, 3)).transpose(0, 1).reshape(H, N * T * G, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + torch.log(total))[:, :, 0]
    out = out.view(H, N, T, G, D).permute(1, 2, 0, 3, 4).reshape(N, T, H * G, D)
    lse = lse.view(H, N, T, G).permute(1, 2, 0, 3).reshape(N, T, H * G)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_logprobs(s):
    c = s["case"]
    tokens, heat = s["tokens"], s["temperature"][:, None, None]
    none = tokens < 0
    x = tokens.clamp(min=0)[:, :, None]
    logits = s["logits"].float()
    top = logits.amax(-1, keepdim=True)
    below = (logits - top) / heat
    weight = torch.exp(below)
    total = weight.sum(-1, keepdim=True)
    mean = torch.where(weight > 0, weight * below, 0.0).sum(-1)
    log_total = torch.log(total)
    mine = logits.gather(2, x)
    ids = torch.arange(c["vocab"], device=DEVICE)
    rank = ((logits > mine) | ((logits == mine) & (ids < x))).sum(-1) + 1
    out = {"logprob": torch.where(none, 0.0, ((mine - top) / heat - log_total)[:, :, 0]),
           "entropy": torch.where(none, 0.0, log_total[:, :, 0] - mean / total[:, :, 0]),
           "rank": torch.where(none, 0, rank).to(torch.int32)}
    best = torch.empty(tokens.shape + (c["top"],), dtype=torch.int64, device=DEVICE)
    left = logits.clone() if c["top"] else logits
    for i in range(c["top"]):                        # the first of the largest of what is left
        first = torch.where(left == left.amax(-1, keepdim=True), ids, c["vocab"]).amin(-1)
        best[:, :, i] = first
        left.scatter_(2, first[:, :, None], -math.inf)
    value = (logits.gather(2, best) - top) / heat - log_total
    out["top_ids"] = torch.where(none[:, :, None], -1, best)
    out["top_logprobs"] = torch.where(none[:, :, None], 0.0, value)
    return out


# ------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "logprobs":
        rows, top = sum(_emitted(case)), case["top"]
        each = case["vocab"] * (4 if case["dtype"] == "f32" else 2) + 12 * top + 12
        return {"bytes": rows * each + 8 * case["seqs"] * case["slots"], "flops": rows * case["vocab"] * 5}
    H, D, ps = case["kv_heads"], case["dim"], case["page"]
    held = 2 * H * (D * case["bits"] // 8 + D // 16)           # bytes of a token of the cache
    if case["op"] == "attention":
        N, T, G, P = (case[k] for k in ("seqs", "tokens", "group", "prefix"))
        lens = _spread(case["tail_min"], case["tail_max"], N)
        seen = sum(max(0, n - T + 1 + t) for n in lens for t in range(T)) + N * T * P
        tables = 4 * (-(-P // ps) + sum(-(-n // ps) + 1 for n in lens))
        return {"bytes": N * T * H * G * (4 * D + 4) + (P + sum(lens)) * held + tables,
                "flops": 4 * D * G * H * seen}
    lens = _spread(case["len_min"], case["len_max"], case["seqs"])
    tables = 4 * sum(-(-n // ps) + 1 for n in lens)
    row = 2 * H * D * (4 if case["dtype"] == "f32" else 2)
    if case["op"] == "read":
        return {"bytes": sum(lens) * held + case["seqs"] * case["len_max"] * row + tables, "flops": 0}
    # rows in, codes out; codes in, values out
    T = case["tokens"]
    new = sum(min(T, n) for n in lens)
    return {"bytes": new * (row + 2 * held) + case["seqs"] * T * 8 * H * D + 2 * tables, "flops": 0}


# ------------------------------------------------------------------ 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attention": _exact_attention,
            "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_scale(byte):
    """2^-17 m below the first binade, (1 + m/8) 2^(e-15) from it on."""
    e, m = byte >> 3, (byte & 7).double()
    return torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2(e.double() - 18))


def _exact_tokens(pool, case, ids, count):
    """The first `count` tokens [count, head, dim] of the pages `ids`, one page at a time."""
    ps, D, bits = case["page"], case["dim"], case["bits"]
    codes, scales, _ = _sizes(case)
    dims = torch.arange(D, device=DEVICE)
    got = [torch.zeros(0, case["kv_heads"], D, dtype=torch.float64, device=DEVICE)]
    for i, p in enumerate(ids):
        n = min(ps, count - i * ps)
        if n <= 0:
            break
        held = pool[0, p].long()
        at = torch.arange(n, device=DEVICE)[:, None]
        if bits == 4:
            nibble = dims % 8 // 2 + dims % 2 * 4
            code = (held[:, at * codes + dims // 8 * 4 + nibble // 2] >> nibble % 2 * 4) % 16 - 8
        else:
            code = held[:, at * codes + dims] - 128
        step = _exact_scale(held[:, ps * codes + at * scales + dims // 16])
        got.append((code.double() * step).transpose(0, 1))
    return torch.cat(got)


def _exact_read(s):
    c, out = s["case"], {}
    for name in ("k", "v"):
        out[name] = torch.zeros(c["seqs"], c["len_max"], c["kv_heads"], c["dim"], dtype=torch.float64,
                                device=DEVICE)
        for n, length in enumerate(s["lens"].tolist()):
            out[name][n, :length] = _exact_tokens(s[name], c, s["table"][n].tolist(), length)
    return out


def _exact_write(s):
    """What a written row stands for: its codes in steps of the least scale that reaches its largest."""
    c, out = s["case"], {}
    most = 2 ** (c["bits"] - 1) - 1
    for name in ("k", "v"):
        x = s["rows_" + name].double()
        shape = x.shape
        x = x.reshape(-1, 16)
        top = x.abs().amax(1)
        e = torch.floor(torch.log2(torch.clamp(top / most, min=2.0 ** -14)))
        unit = torch.exp2(e - 3)                              # the spacing of scales in that binade
        m = torch.ceil(top / most / unit)
        m = torch.where((m - 1) * unit * most >= top, m - 1, m)
        step = (torch.where(m * unit * most < top, m + 1, m) * unit)[:, None]
        code = torch.where(step > 0, x / torch.where(step > 0, step, 1.0), 0.0)
        low = torch.floor(code)
        up = (code - low > 0.5) | ((code - low == 0.5) & (low % 2 != 0))
        at = s["first"].long()[:, None] + torch.arange(c["tokens"], device=DEVICE)[None, :]
        value = ((low + up) * step).reshape(shape)
        out[name] = torch.where((at >= 0)[:, :, None, None], value, 0.0)
    return out


def _exact_attention(s):
    c = s["case"]
    T, H, G, D, P = (c[k] for k in ("tokens", "kv_heads", "group", "dim", "prefix"))
    outs, lses = [], []
    shared = [_exact_tokens(s[name], c, s["prefix_table"].tolist(), P) for name in ("k", "v")]
    for n, length in enumerate(s["lens"].tolist()):
        ids = s["table"][n].tolist()
        k, v = (torch.cat([p, _exact_tokens(s[name], c, ids, length)]) for p, name in zip(shared, ("k", "v")))
        out = torch.zeros(T, H, G, D, dtype=torch.float64, device=DEVICE)
        lse = torch.full((T, H, G), -math.inf, dtype=torch.float64, device=DEVICE)
        q = s["q"][n].double().view(T, H, G, D)
        for t in range(T):
            sees = P + max(0, length - T + 1 + t)
            if sees:
                score = torch.einsum("hgd,jhd->hgj", q[t], k[:sees]) * s["scale"]
                lse[t] = torch.logsumexp(score, -1)
                out[t] = torch.einsum("hgj,jhd->hgd", torch.exp(score - lse[t][..., None]), v[:sees])
        outs.append(out.view(T, H * G, D))
        lses.append(lse.view(T, H * G))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_logprobs(s):
    N, B, _ = s["logits"].shape
    K = s["case"]["top"]
    out = {"logprob": torch.zeros(N, B, dtype=torch.float64, device=DEVICE),
           "entropy": torch.zeros(N, B, dtype=torch.float64, device=DEVICE), "rank": None, "top_ids": None,
           "top_logprobs": torch.zeros(N, B, K, dtype=torch.float64, device=DEVICE)}
    for n, heat in enumerate(s["temperature"].tolist()):
        for b, x in enumerate(s["tokens"][n].tolist()):
            if x < 0:
                continue
            row = torch.log_softmax(s["logits"][n, b].double() / heat, 0)
            out["logprob"][n, b] = row[x]
            seen = row[row > -math.inf]
            out["entropy"][n, b] = -(torch.exp(seen) * seen).sum()
            out["top_logprobs"][n, b] = torch.sort(row, descending=True)[0][:K]
    return out
