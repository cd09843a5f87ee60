"""Workloads of the operators around drafted trees, forked sequences and many-token expert
layers: attention of a tree of drafted tokens over the 4-bit key/value cache, acceptance of a
path with the move of its rows, forks of block tables with the pages they copy, matrix products
grouped by expert, and the expert layer for any number of tokens.

Each case names one step as a serving program makes it.  run() computes it in a plain form
(elementary torch operations in float32, one rounding at the end) or, with `own` set, through
this repository's entry points; exact() computes it in float64, written apart from the plain
form.

Shared definitions
  codec      w = s * q + b per group of `group` consecutive values, q unsigned of `bits` bits;
             a row's codes are one little-endian bitstream of uint32 words; s, b in the
             call's dtype.
  cache      one K and one V row of `dim` values per (token slot, kv head), 4-bit codes; slot =
             page * page_size + offset; quantization in float32 steps: s = (max - min) / 15,
             q = clamp(rint((x - min) / s), 0, 15), q = 0 where s = 0, then s and b = min are
             rounded to the dtype.  A block table names each sequence's pages in order.
  tree       parents[i] < i is node i's parent, -1 a root, less: no node (nor are its
             descendants).  The nodes are the last tokens of a sequence of length L, at
             positions c + i, c = L - nodes.  Node i sees itself, its ancestors and the tokens
             j < c; with a window only its `window` nearest of them by depth: of its path the
             nodes at most window - 1 steps up, of the others j > c + depth_i - window.  What is
             no node gives zeros.
  accept     the path starts with node 0 and goes on to the lowest child whose drafted token is
             the one sampled after its parent; `last` is the one sampled after its end.
  move       the row at origin[n] + index[n, i] of sequence n goes to position start[n] + i
             (negative index: none does).
  fork       row i of the new table continues row parents[i] of the old one: it shares the full
             pages of the min(length, want) tokens that stay.  The page that is not full, and
             those after it up to `want` tokens, go to the first such row where nobody else held
             them; otherwise it takes pages that were free before the call, the lowest first, in
             the order of (row, block), and the page that is not full is copied.  A row without
             parent starts with no tokens.  refs counts the entries that name a page.
  grouped    y[r] = x[r] W_e^T for offsets[e] <= r < offsets[e + 1].
  moe        the top_k largest router logits (ties: lower expert), softmax over them,
             y = sum_e w_e * (silu(x Wg_e^T) * (x Wu_e^T)) Wd_e^T.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SPARE_PAGES = 5          # pages of the pool that no sequence of the case holds
TOKENS = 64              # different drafted tokens: siblings are alike now and then


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one short conversation's drafted tree: the smallest call, latency counts
        {"name": "tree_short", "op": "tree", "batch": 1, "nodes": 13, "heads": 32, "kv_heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 509, "window": 0, "dtype": "bf16"},
        # the trees of a batch of conversations of very different lengths
        {"name": "tree_batch", "op": "tree", "batch": 16, "nodes": 32, "heads": 32, "kv_heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 8192, "window": 0, "dtype": "bf16"},
        # a large tree after one long document
        {"name": "tree_long", "op": "tree", "batch": 1, "nodes": 64, "heads": 64, "kv_heads": 8, "dim": 128,
         "group": 128, "page": 256, "length": 131071, "window": 0, "dtype": "fp16"},
        # one conversation's tree has been verified: its path is found and its rows move up
        {"name": "accept_one", "op": "accept", "batch": 1, "nodes": 13, "kv_heads": 8, "dim": 128, "group": 64,
         "page": 64, "length": 509, "dtype": "bf16"},
        # the same for a full batch
        {"name": "accept_batch", "op": "accept", "batch": 64, "nodes": 63, "kv_heads": 8, "dim": 128, "group": 64,
         "page": 16, "length": 1024, "dtype": "bf16"},
        # long sequences keep a quarter of their tokens, in new pages
        {"name": "compact_long", "op": "compact", "batch": 4, "kv_heads": 8, "dim": 128, "group": 32, "page": 64,
         "length": 16384, "keep": 0.25, "dtype": "fp16"},
        # a beam search step: 8 requests of 4 beams each
        {"name": "fork_beams", "op": "fork", "batch": 32, "rows": 32, "kv_heads": 8, "dim": 128, "group": 64,
         "page": 64, "length": 2039, "grow": 1, "dtype": "bf16"},
        # prompts continued by several samples each, pages of many tokens
        {"name": "fork_samples", "op": "fork", "batch": 32, "rows": 128, "kv_heads": 8, "dim": 128, "group": 64,
         "page": 256, "length": 4093, "grow": 300, "dtype": "bf16"},
        # few rows of each of many small experts: the weights' stream counts
        {"name": "grouped_few", "op": "grouped", "rows": 509, "n": 704, "k": 1408, "experts": 128, "bits": 8,
         "group": 32, "dtype": "bf16"},
        # a prompt's rows through one matrix of each of 64 experts
        {"name": "grouped_many", "op": "grouped", "rows": 16384, "n": 1024, "k": 2048, "experts": 64, "bits": 4,
         "group": 64, "dtype": "bf16"},
        # the trees of eight sequences, 32 nodes each, through the repository's expert shape
        {"name": "moe_trees", "op": "moe", "tokens": 256, "hidden": 1408, "inter": 704, "experts": 128, "top_k": 8,
         "bits": 8, "group": 32, "dtype": "bf16"},
        # a prompt through few large experts (the prefill benchmark's matrix)
        {"name": "moe_prompt", "op": "moe", "tokens": 2047, "hidden": 4096, "inter": 14336, "experts": 8, "top_k": 2,
         "bits": 4, "group": 128, "dtype": "fp16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_cache(rng):
    dim = rng.choice([64, 128, 128, 256])
    return {"kv_heads": rng.choice([1, 2, 4, 8]), "dim": dim, "group": rng.choice([g for g in (32, 64, 128) if g <= dim]),
            "page": rng.choice([16, 48, 64, 256]), "dtype": rng.choice(["bf16", "fp16"])}


def _draw_codec(rng):
    return {"bits": rng.choice([4, 4, 4, 8, 8, 3, 6]), "group": rng.choice([32, 64, 128]),
            "dtype": rng.choice(["bf16", "fp16"])}


def draw(rng):
    op = rng.choice(["tree", "tree", "accept", "compact", "fork", "grouped", "moe", "moe"])
    if op == "tree":
        c = {"op": op, **_draw_cache(rng), "batch": _log_int(rng, 1, 32), "nodes": _log_int(rng, 1, 200), "window": 0}
        c["heads"] = c["kv_heads"] * rng.choice([1, 3, 4, 8])
        # no more cached rows than the ragged batch has, no more score work than the long tree's
        length = _log_int(rng, c["nodes"], 131071)
        length = min(length, 2 * 131071 * 8 // (c["kv_heads"] * c["batch"]))
        length = min(length, 64 * 131071 * 64 * 128 // (c["nodes"] * c["heads"] * c["batch"] * c["dim"]))
        c["length"] = max(c["nodes"], length)
        if rng.random() < 0.3:
            c["window"] = _log_int(rng, 1, 8192)
        return c
    if op == "accept":
        c = {"op": op, **_draw_cache(rng), "batch": _log_int(rng, 1, 64), "nodes": _log_int(rng, 1, 63)}
        return {**c, "length": c["nodes"] + _log_int(rng, 1, 1024)}
    if op == "compact":
        c = {"op": op, **_draw_cache(rng), "batch": _log_int(rng, 1, 16), "keep": rng.choice([0.1, 0.25, 0.6, 1.0])}
        return {**c, "length": _log_int(rng, 1, 4 * 16384 // c["batch"])}
    if op == "fork":
        c = {"op": op, **_draw_cache(rng), "batch": _log_int(rng, 1, 64), "rows": _log_int(rng, 1, 128)}
        return {**c, "length": _log_int(rng, 1, 4096), "grow": rng.choice([0, 1, 16, 300])}
    c = _draw_codec(rng)
    group = c["group"]
    if op == "grouped":
        n, k = _log_int(rng, 8, 8192), group * max(1, _log_int(rng, 128, 8192) // group)
        experts = rng.choice([1, 4, 8, 60, 64, 128])
        while experts * n * k > 8 * 4096 * 14336:
            n = max(1, n // 2)
        rows = max(1, min(_log_int(rng, 1, 16384), 2 * 16384 * 1024 * 2048 // (n * k)))
        return {"op": op, "rows": rows, "n": n, "k": k, "experts": experts, **c}
    experts = rng.choice([4, 8, 60, 64, 128])
    top_k = min(rng.choice([1, 2, 4, 8]), experts)
    hidden = group * max(1, _log_int(rng, 256, 4096) // group)
    inter = group * max(1, _log_int(rng, 128, 14336) // group)
    while experts * hidden * inter > 8 * 4096 * 14336:
        inter = group * max(1, inter // 2 // group)
    tokens = min(_log_int(rng, 1, 8192), 4094 * 4096 * 14336 // (top_k * hidden * inter), 65536 // top_k)
    return {"op": op, "tokens": max(1, tokens), "hidden": hidden, "inter": inter, "experts": experts, "top_k": top_k, **c}


def _lengths(case, least=1):
    """Tokens per sequence: evenly spread up to `length`, the last one the longest."""
    n, top = case["batch"], case["length"]
    return [max(least, top * (i + 1) // n) for i in range(n)]


def _row_bytes(case):
    """Bytes of one cached K (or V) row: codes, scales and biases."""
    return case["dim"] // 2 + case["dim"] // case["group"] * 4


def work(case):
    op = case["op"]
    if op == "tree":
        pairs = tokens = 0
        for n in _lengths(case, case["nodes"]):
            ctx = n - case["nodes"]
            seen = min(ctx, case["window"]) if case["window"] else ctx
            pairs, tokens = pairs + case["nodes"] * (seen + 1), tokens + seen + case["nodes"]
        io = 2 * 2 * case["batch"] * case["nodes"] * case["heads"] * case["dim"]
        return {"bytes": tokens * case["kv_heads"] * 2 * _row_bytes(case) + io,
                "flops": 4 * case["dim"] * case["heads"] * pairs}
    if op == "accept":
        rows = case["batch"] * case["nodes"] * case["kv_heads"] * 2
        # new rows read, their cached form written, and read back as the values it stands for
        return {"bytes": rows * (2 * case["dim"] + 2 * _row_bytes(case) + 2 * case["dim"]) + 16 * case["batch"] * case["nodes"],
                "flops": rows * case["dim"] * 6}
    if op == "compact":
        rows = sum(_kept(case, n) for n in _lengths(case)) * case["kv_heads"] * 2
        return {"bytes": rows * (3 * _row_bytes(case) + 2 * case["dim"]), "flops": rows * case["dim"] * 2}
    if op == "fork":
        rows = case["rows"] * case["page"] * case["kv_heads"] * 2 // 2      # about half of the rows copy a page
        blocks = -(-case["length"] // case["page"])
        return {"bytes": rows * (3 * _row_bytes(case) + 2 * case["dim"]) + 12 * (case["rows"] + case["batch"]) * blocks,
                "flops": rows * case["dim"] * 2}
    if op == "grouped":
        e, r, mat = case["experts"], case["rows"], case["n"] * case["k"]
        per = mat * case["bits"] / 8 + mat // case["group"] * 4
        used = e * (1.0 - (1.0 - 1.0 / e) ** r)
        return {"bytes": int(used * per) + 2 * r * (case["n"] + case["k"]), "flops": 2 * r * mat}
    e, k, t = case["experts"], case["top_k"], case["tokens"]
    used = e * (1.0 - (1.0 - k / e) ** t)       # expected experts that any token chooses
    mat = case["hidden"] * case["inter"]
    per = mat * case["bits"] / 8 + mat // case["group"] * 4
    return {"bytes": int(3 * used * per) + 2 * t * (2 * case["hidden"] + e),
            "flops": 2 * 3 * t * k * mat}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _cache_rows(g, rows, case):
    """Keys or values as a model makes them: a few channels much larger than the rest."""
    x = _randn(g, rows, case["kv_heads"], case["dim"])
    loud = 1.0 + 4.0 * (torch.rand(case["kv_heads"], case["dim"], generator=g, device="cuda") < 0.05)
    return (x * loud).to(DTYPES[case["dtype"]])


def _expert_stack(g, experts, n, k, case):
    """Quantized normal weights: codes around the middle of their range, and their s and b."""
    bits, group, dtype = case["bits"], case["group"], DTYPES[case["dtype"]]
    top = 2 ** bits - 1
    words = torch.empty(experts, n, k * bits // 32, dtype=torch.int32, device="cuda")
    at_once = max(1, (1 << 26) // (n * k))
    for e in range(0, experts, at_once):
        m = min(at_once, experts - e)
        codes = torch.clamp(torch.round(_randn(g, m, n, k) * (top / 6.0) + top / 2.0), 0, top).to(torch.int64)
        words[e:e + m] = _pack(codes, bits)
    s = (0.02 * 6.0 / top) * (0.8 + 0.4 * torch.rand(experts, n, k // group, generator=g, device="cuda"))
    return words, s.to(dtype), (s * (-top / 2.0)).to(dtype)


def _tree(case, seed):
    """parents, drafted and sampled tokens int32 [batch, nodes] of random trees, most nodes near
    the last one; every third sequence's tree is smaller than the others."""
    g = torch.Generator().manual_seed(int(seed) * 7 + 3)
    b, n = case["batch"], case["nodes"]
    parents = torch.full((b, n), -1, dtype=torch.int64)
    tokens = torch.randint(0, TOKENS, (b, n), generator=g)
    sampled = torch.randint(0, TOKENS, (b, n), generator=g)
    for i in range(1, n):
        up = torch.clamp((i * torch.rand(b, generator=g) ** 0.5).long(), max=i - 1)
        parents[:, i] = up
        follow = torch.rand(b, generator=g) < 0.6
        r = torch.arange(b)
        sampled[r, up] = torch.where(follow, tokens[:, i], sampled[r, up])
    if case["op"] == "tree":
        parents[2::3, n - n // 4:] = -2
    return parents.to(torch.int32).cuda(), tokens.to(torch.int32).cuda(), sampled.to(torch.int32).cuda()


def _kept(case, n):
    return max(1, int(n * case["keep"]))


def _paged(case, g, lens, spare):
    """pages, block table int32 [batch, blocks], and the slots of every token, sequence by sequence."""
    page = case["page"]
    blocks = [-(-n // page) for n in lens]
    pages = sum(blocks) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device="cuda")
    slots, at = [], 0
    for i, (n, m) in enumerate(zip(lens, blocks)):
        table[i, :m] = perm[at:at + m]
        j = torch.arange(n, device="cuda")
        slots.append(perm[at:at + m][j // page] * page + j % page)
        at += m
    return pages, table, torch.cat(slots).to(torch.int32)


def _inputs(case, seed):
    g = _gen(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    d = {}
    if op == "tree":
        lens = _lengths(case, case["nodes"])
        d["pages"], d["table"], d["slots"] = _paged(case, g, lens, SPARE_PAGES)
        d["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        d["k"], d["v"] = _cache_rows(g, sum(lens), case), _cache_rows(g, sum(lens), case)
        d["q"] = _randn(g, case["batch"], case["nodes"], case["heads"], case["dim"]).to(dtype)
        d["scale"] = case["dim"] ** -0.5
        d["parents"] = _tree(case, seed)[0]
    elif op == "accept":
        n = case["nodes"]
        lens = _lengths(case, n)
        d["pages"], d["table"], slots = _paged(case, g, lens, SPARE_PAGES)
        ends = torch.tensor(lens, device="cuda").cumsum(0)
        d["slots"] = slots[((ends - n)[:, None] + torch.arange(n, device="cuda")).flatten()].contiguous()
        d["start"] = torch.tensor([m - n for m in lens], dtype=torch.int32, device="cuda")
        d["k"], d["v"] = _cache_rows(g, len(lens) * n, case), _cache_rows(g, len(lens) * n, case)
        d["parents"], d["tokens"], d["sampled"] = _tree(case, seed)
    elif op == "compact":
        lens = _lengths(case)
        kept = [_kept(case, n) for n in lens]
        both, table, slots = _paged(case, g, lens + kept, SPARE_PAGES)
        d["pages"], d["table"] = both, table[:len(lens)].contiguous()
        d["to"] = table[len(lens):].contiguous()
        d["slots"], d["to_slots"] = slots[:sum(lens)].contiguous(), slots[sum(lens):].contiguous()
        d["start"] = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        index = torch.full((len(lens), max(kept)), -1, dtype=torch.int32, device="cuda")
        for i, (n, m) in enumerate(zip(lens, kept)):
            index[i, :m] = torch.sort(torch.randperm(n, generator=g, device="cuda")[:m]).values.to(torch.int32)
        d["index"] = index
        d["k"], d["v"] = _cache_rows(g, sum(lens), case), _cache_rows(g, sum(lens), case)
    elif op == "fork":
        lens = _lengths(case)
        rows, page = case["rows"], case["page"]
        most = -(-(case["length"] + case["grow"]) // page)
        d["pages"], table, d["slots"] = _paged(case, g, lens, SPARE_PAGES + rows * (2 + case["grow"] // page))
        d["table"] = table
        d["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        d["refs"] = torch.zeros(d["pages"], dtype=torch.int32, device="cuda")
        d["refs"][table[table >= 0].long()] = 1
        parents = torch.randint(0, len(lens), (rows,), generator=g, device="cuda")
        if rows > 4:
            parents[rows // 2] = -1                # a request that has ended
        d["parents"] = parents.to(torch.int32)
        d["want"] = torch.where(parents >= 0, d["lengths"][parents.clamp(min=0)] + case["grow"], 0).to(torch.int32)
        d["blocks"] = most
        d["k"], d["v"] = _cache_rows(g, sum(lens), case), _cache_rows(g, sum(lens), case)
    elif op == "grouped":
        e, r = case["experts"], case["rows"]
        share = torch.exp(0.7 * _randn(g, e))      # some experts are chosen much more often
        who = torch.sort(torch.multinomial(share, r, replacement=True, generator=g)).values
        counts = torch.bincount(who, minlength=e)
        d["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).to(torch.int32)
        d["host_offsets"] = d["offsets"].tolist()
        d["x"] = _randn(g, r, case["k"]).to(dtype)
        d["w"] = _expert_stack(g, e, case["n"], case["k"], case)
    else:
        e, k, n = case["experts"], case["hidden"], case["inter"]
        d["x"] = _randn(g, case["tokens"], k).to(dtype)
        d["router"] = (1.5 * _randn(g, case["tokens"], e)).to(dtype)
        d["gate"] = _expert_stack(g, e, n, k, case)
        d["up"] = _expert_stack(g, e, n, k, case)
        d["down"] = _expert_stack(g, e, k, n, case)
    return d


# ---------------------------------------------------------------- plain forms

def _pack(codes, bits):
    """int64 codes [..., k] -> int32 words [..., k * bits / 32], one bitstream per row."""
    k = codes.shape[-1]
    if 32 % bits == 0:
        shift = torch.arange(32 // bits, device=codes.device) * bits
        lo = (codes.unflatten(-1, (-1, 32 // bits)) << shift).sum(-1)
        return torch.where(lo >= 2 ** 31, lo - 2 ** 32, lo).to(torch.int32)
    pos = torch.arange(k, device=codes.device) * bits
    lo = torch.zeros(*codes.shape[:-1], k * bits // 32 + 1, dtype=torch.int64, device=codes.device)
    low = (codes << (pos % 32)) & 0xFFFFFFFF
    high = codes >> (32 - pos % 32)
    lo.index_add_(-1, pos // 32, low)
    lo.index_add_(-1, pos // 32 + 1, high)
    lo = lo[..., :-1]
    return torch.where(lo >= 2 ** 31, lo - 2 ** 32, lo).to(torch.int32)


def _unpack(words, bits, k):
    """float32 codes [..., k] of int32 words."""
    pos = torch.arange(k, device=words.device) * bits
    if 32 % bits == 0:
        per = 32 // bits
        shift = torch.arange(per, device=words.device, dtype=torch.int32) * bits
        return ((words[..., None] >> shift) & (2 ** bits - 1)).flatten(-2).float()
    w = words.to(torch.int64) & 0xFFFFFFFF
    nxt = torch.cat([w[..., 1:], torch.zeros_like(w[..., :1])], -1)
    both = w[..., pos // 32] | (nxt[..., pos // 32] << 32)
    return ((both >> (pos % 32)) & (2 ** bits - 1)).float()


def _dequant(words, s, b, bits, group, k):
    q = _unpack(words, bits, k).unflatten(-1, (k // group, group))
    return (q * s.float()[..., None] + b.float()[..., None]).flatten(-2)


def _quantize4(x, group):
    """Rows [..., dim] -> (words, s, b) in float32 steps."""
    g = x.float().unflatten(-1, (x.shape[-1] // group, group))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = (hi - lo) / torch.full_like(lo, 15.0)      # a tensor: torch multiplies by a number's reciprocal
    q = torch.clamp(torch.round((g - lo) / torch.where(s == 0, torch.ones_like(s), s)), 0, 15)
    q = torch.where(s == 0, torch.zeros_like(q), q).to(torch.int64).flatten(-2)
    return _pack(q, 4), s[..., 0].to(x.dtype), lo[..., 0].to(x.dtype)


def _plain_cache(case, d):
    """Flat cache [slot, head, ...] as packed words, scales and biases, empty."""
    n, h, dim = d["pages"] * case["page"], case["kv_heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]
    return [[torch.zeros(n, h, dim // 8, dtype=torch.int32, device="cuda"),
             torch.zeros(n, h, dim // case["group"], dtype=dtype, device="cuda"),
             torch.zeros(n, h, dim // case["group"], dtype=dtype, device="cuda")] for _ in range(2)]


def _plain_append(case, cache, k, v, slots):
    for store, x in zip(cache, (k, v)):
        for dst, src in zip(store, _quantize4(x, case["group"])):
            dst[slots] = src


def _plain_read(case, store, slots):
    """Values of the rows at `slots`; NaN for slots outside the cache."""
    ok = (slots >= 0) & (slots < store[0].shape[0])
    rows = _dequant(*(t[torch.where(ok, slots, 0)] for t in store), 4, case["group"], case["dim"])
    return torch.where(ok[:, None, None], rows, math.nan)


def _plain_move(cache, src, dst, ok):
    """Rows src -> dst where ok, every row read before any is written."""
    src, dst = src[ok], dst[ok]
    for store in cache:
        for t in store:
            t[dst] = t[src]


def _tree_mask(parents, window):
    """(sees bool [batch, nodes, nodes], depth [batch, nodes]) of the trees."""
    b, n = parents.shape
    p = parents.to(torch.int64)
    i = torch.arange(n, device=p.device)
    there = (p >= -1) & (p < i)
    up = torch.full((b, n + 2), n + 1, device=p.device)            # columns n: above a root, n + 1: no node
    up[:, n] = n
    up[:, :n] = torch.where(there, torch.where(p < 0, torch.full_like(p, n), p), up[:, :n])
    sees = torch.zeros(b, n, n + 2, dtype=torch.bool, device=p.device)
    at, depth = i.expand(b, n), torch.zeros_like(p)
    for step in range(n):
        if not window or step < window:
            sees.scatter_(2, at[..., None], True)
        at = torch.gather(up, 1, at)
        depth = depth + (at < n)
    whole = at == n                                                # its path ends above a root
    return sees[..., :n] & whole[..., None], depth * whole, whole


def _run_tree(case, d):
    dtype = DTYPES[case["dtype"]]
    b, lq, hk, dim = case["batch"], case["nodes"], case["kv_heads"], case["dim"]
    rep = case["heads"] // hk
    top = d["table"].shape[1] * case["page"]
    j = torch.arange(top, device="cuda")
    slots = d["table"].clamp(min=0)[:, j // case["page"]] * case["page"] + j % case["page"]    # [b, top]
    k, v = (_plain_read(case, store, slots.flatten()).unflatten(0, (b, top)).transpose(1, 2).contiguous()
            for store in d["cache"])                                       # [b, hk, top, dim]
    q = d["q"].float().unflatten(2, (hk, rep)).permute(0, 2, 3, 1, 4).reshape(b, hk, rep * lq, dim)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * d["scale"]
    sees, depth, there = d["tree"]
    ctx = (d["lengths"].long() - lq)[:, None]                              # [b, 1]
    seen = (j < ctx)[:, None, :] & there[..., None]                        # [b, lq, top]
    if case["window"]:
        seen = seen & (j > (ctx + depth - case["window"])[..., None])
    node = (j - ctx)[:, None, :].expand(b, lq, top)
    inside = (node >= 0) & (node < lq)
    seen = seen | (inside & torch.gather(sees, 2, node.clamp(0, lq - 1)))
    seen = seen[:, None, None]                                             # [b, 1, 1, lq, top]
    s = s.unflatten(2, (rep, lq)).masked_fill(~seen, -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38)).masked_fill(~seen, 0.0)
    e = (e / e.sum(-1, keepdim=True).clamp(min=1e-37)).flatten(2, 3)
    o = torch.matmul(e, v).unflatten(2, (rep, lq))                         # [b, hk, rep, lq, dim]
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(dtype)


def _accept(parents, tokens, sampled):
    b, n = parents.shape
    i = torch.arange(n, device=parents.device)
    at = torch.zeros(b, 1, dtype=torch.int64, device=parents.device)
    live = parents[:, :1] == -1
    path = torch.full((b, n), -1, dtype=torch.int64, device=parents.device)
    count, last = live.long(), torch.full_like(at, -1)
    path[:, :1] = torch.where(live, at, path[:, :1])
    last = torch.where(live, torch.gather(sampled, 1, at).long(), last)
    for step in range(1, n):
        fits = live & (parents == at) & (tokens == last) & (i > at)
        live = fits.any(1, keepdim=True)
        at = torch.where(live, fits.long().argmax(1, keepdim=True), at)
        path[:, step:step + 1] = torch.where(live, at, path[:, step:step + 1])
        last = torch.where(live, torch.gather(sampled, 1, at).long(), last)
        count = count + live.long()
    return path.to(torch.int32), count[:, 0].to(torch.int32), last[:, 0].to(torch.int32)


def _slots_of(table, position, page):
    """Slots of positions [batch, n] of each row's sequence."""
    block = (position // page).clamp(0, table.shape[1] - 1)
    return torch.gather(table.long(), 1, block) * page + position % page


def _run_accept(case, d):
    n = case["nodes"]
    _plain_append(case, d["cache"], d["k"], d["v"], d["slots"])
    path, count, last = _accept(d["parents"], d["tokens"], d["sampled"])
    start = d["start"].long()[:, None]
    ok = path >= 0
    src = _slots_of(d["table"], start + path.clamp(min=0).long(), case["page"])
    dst = _slots_of(d["table"], start + torch.arange(n, device="cuda"), case["page"])
    _plain_move(d["cache"], src.flatten(), dst.flatten(), ok.flatten())
    k, v = (_plain_read(case, store, d["slots"]).to(d["k"].dtype) for store in d["cache"])
    return path, count, last, k, v


def _run_compact(case, d):
    index = d["index"].long()
    m = index.shape[1]
    ok = (index >= 0).flatten()
    src = _slots_of(d["table"], index.clamp(min=0), case["page"]).flatten()
    position = d["start"].long()[:, None] + torch.arange(m, device="cuda")
    dst = _slots_of(d["to"], position, case["page"]).flatten()
    _plain_move(d["cache"], src, dst, ok)
    return tuple(_plain_read(case, store, d["to_slots"]).to(DTYPES[case["dtype"]]) for store in d["cache"])


def _fork(refs, table, lengths, parents, page, want, blocks):
    pages, rows = refs.shape[0], parents.shape[0]
    p = parents.long()
    has = (p >= 0) & (p < table.shape[0])
    q = torch.where(has, p, 0)
    length = torch.where(has, lengths.long()[q], 0)
    want = want.long()
    keep = torch.minimum(length, want)
    full, partial, cover = keep // page, keep % page > 0, -(-want // page)
    r = torch.arange(rows, device=p.device)
    first = has & ~((p[:, None] == p[None, :]) & (r[None, :] < r[:, None])).any(1)
    j = torch.arange(blocks, device=p.device)[None, :]
    wide = torch.full((table.shape[0], max(blocks, table.shape[1])), -1, dtype=torch.int64, device=p.device)
    wide[:, :table.shape[1]] = table.long()
    old = torch.where(has[:, None], wide[q, :blocks], -1)
    valid = (old >= 0) & (old < pages)
    alone = valid & (refs[old.clamp(0, pages - 1)] == 1)
    shared = valid & (j < full[:, None])
    kept = first[:, None] & alone & (j >= full[:, None]) & (j < cover[:, None])
    fresh = (j >= full[:, None]) & (j < cover[:, None]) & ~kept
    number = (fresh.flatten().long().cumsum(0) - 1).view(rows, blocks)
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    open_ = (refs == 0).sum()
    got = torch.where(number < open_, free[number.clamp(0, pages - 1)], -1)
    new = torch.where(shared | kept, old, torch.where(fresh, got, -1))
    at = full.clamp(max=blocks - 1)[:, None]
    copies = partial & (full < blocks) & torch.gather(fresh & valid & (new >= 0), 1, at)[:, 0]
    src = torch.where(copies, torch.gather(old, 1, at)[:, 0], -1)
    dst = torch.where(copies, torch.gather(new, 1, at)[:, 0], -1)
    flat = table.long().flatten()
    some = (flat >= 0) & (flat < pages)
    refs.index_add_(0, torch.where(some, flat, 0), torch.where(some, -1, 0).to(refs.dtype))
    flat = new.flatten()
    refs.index_add_(0, flat.clamp(min=0), (flat >= 0).to(refs.dtype))
    short = (fresh.sum() - open_).clamp(min=0)
    return new.to(torch.int32), src.to(torch.int32), dst.to(torch.int32), short.to(torch.int32).view(1)


def _run_fork(case, d):
    refs = d["refs"].clone()                       # the pool is the program's own, and goes on after the step
    page = case["page"]
    table, src, dst, short = _fork(refs, d["table"], d["lengths"], d["parents"], page, d["want"], d["blocks"])
    inside = torch.arange(page, device="cuda")
    ok = (dst >= 0)[:, None].expand(-1, page).flatten()
    a, b = ((t.clamp(min=0)[:, None] * page + inside).flatten().long() for t in (src, dst))
    _plain_move(d["cache"], a, b, ok)
    slots = torch.where(ok, b, -1)
    k, v = (_plain_read(case, store, slots).to(DTYPES[case["dtype"]]) for store in d["cache"])
    return table, refs, src, dst, short, k, v


def _run_grouped(case, d):
    y = torch.empty(case["rows"], case["n"], device="cuda")
    for e, (a, b) in enumerate(zip(d["host_offsets"], d["host_offsets"][1:])):
        if b > a:
            w = _dequant(*(t[e] for t in d["w"]), case["bits"], case["group"], case["k"])
            y[a:b] = torch.matmul(d["x"][a:b].float(), w.t())
    return y.to(d["x"].dtype)


def _run_moe(case, d):
    bits, group, top_k = case["bits"], case["group"], case["top_k"]
    x = d["x"].float()
    value, index = torch.sort(d["router"].float(), dim=-1, descending=True, stable=True)
    value, index = value[:, :top_k], index[:, :top_k]
    w = torch.exp(value - value[:, :1])
    w = (w / w.sum(-1, keepdim=True)).flatten()
    order = torch.argsort(index.flatten(), stable=True)
    counts = torch.bincount(index.flatten(), minlength=case["experts"]).tolist()
    out = torch.empty(case["tokens"] * top_k, case["hidden"], device="cuda")
    at = 0
    for e, n in enumerate(counts):
        if n:
            pairs = order[at:at + n]
            xe = x[pairs // top_k]
            g, u = (torch.matmul(xe, _dequant(*(t[e] for t in d[m]), bits, group, case["hidden"]).t())
                    for m in ("gate", "up"))
            h = g / (1.0 + torch.exp(-g)) * u
            out[pairs] = torch.matmul(h, _dequant(*(t[e] for t in d["down"]), bits, group, case["inter"]).t())
        at += n
    return (out * w[:, None]).view(case["tokens"], top_k, -1).sum(1).to(d["x"].dtype)


# ---------------------------------------------------------------- preparation and one pass

def prepare(case, seed):
    d = _inputs(case, seed)
    state = {"case": case, "d": d}
    op = case["op"]
    if own:
        import bit_affine_quantized_qmv_amd as qmm
        state["qmm"] = qmm
        if op in ("tree", "accept", "compact", "fork"):
            d["cache"] = qmm.kv_cache(d["pages"], case["page"], case["kv_heads"], case["dim"], case["group"],
                                      case["dtype"], device="cuda")
        if op in ("tree", "compact", "fork"):
            qmm.kv_append(d["cache"], d["k"], d["v"], d["slots"])
        if op == "tree":                           # once per step, for every layer
            state["tree"] = qmm.tree_mask(d["parents"], window=case["window"])
            state["workspace"] = qmm.kv_attend_tree_workspace(d["q"], d["cache"], case["length"])
        if op == "grouped":
            state["w"] = qmm.ExpertWeights(*d["w"], case["n"], case["k"], case["group"], case["bits"])
            state["out"] = torch.empty(case["rows"], case["n"], dtype=DTYPES[case["dtype"]], device="cuda")
            state["workspace"] = qmm.grouped_workspace(d["x"], state["w"])
        if op == "moe":
            for m, n, k in (("gate", case["inter"], case["hidden"]), ("up", case["inter"], case["hidden"]),
                            ("down", case["hidden"], case["inter"])):
                state[m] = qmm.ExpertWeights(*d[m], n, k, case["group"], case["bits"])
            state["workspace"] = qmm.moe_prompt_workspace(d["x"], state["gate"], case["top_k"])
    elif op in ("tree", "accept", "compact", "fork"):
        d["cache"] = _plain_cache(case, d)
        if op != "accept":
            _plain_append(case, d["cache"], d["k"], d["v"], d["slots"])
        if op == "tree":
            d["tree"] = _tree_mask(d["parents"], case["window"])
    if op in ("tree", "compact", "fork"):
        del d["k"], d["v"]
    return state


def run(state):
    case, d = state["case"], state["d"]
    op = case["op"]
    if own:
        qmm = state["qmm"]
        if op == "tree":
            mask, depth = state["tree"]
            return qmm.kv_attend_tree(d["q"], d["cache"], d["table"], d["lengths"], mask, depth, scale=d["scale"],
                                      window=case["window"], max_length=case["length"], workspace=state["workspace"])
        if op == "accept":
            qmm.kv_append(d["cache"], d["k"], d["v"], d["slots"])
            path, count, last = qmm.tree_accept(d["parents"], d["tokens"], d["sampled"])
            qmm.kv_move(d["cache"], d["table"], path, d["start"], origin=d["start"])
            return (path, count, last) + qmm.kv_read(d["cache"], d["slots"])
        if op == "compact":
            qmm.kv_move(d["cache"], d["table"], d["index"], d["start"], to_table=d["to"])
            return qmm.kv_read(d["cache"], d["to_slots"])
        if op == "fork":
            refs = d["refs"].clone()               # the pool is the program's own, and goes on after the step
            table, src, dst, short = qmm.kv_fork(refs, d["table"], d["lengths"], d["parents"], case["page"], d["want"],
                                                 blocks=d["blocks"])
            qmm.kv_copy_pages(d["cache"], src, dst)
            slots = torch.where(dst[:, None] >= 0, dst[:, None] * case["page"]
                                + torch.arange(case["page"], dtype=torch.int32, device="cuda"), -1).flatten()
            return (table, refs, src, dst, short) + qmm.kv_read(d["cache"], slots)
        if op == "grouped":
            return qmm.grouped_qmm(d["x"], state["w"], d["offsets"], out=state["out"], workspace=state["workspace"])
        return qmm.moe_prompt(d["x"], d["router"], state["gate"], state["up"], state["down"], case["top_k"],
                              workspace=state["workspace"])
    return {"tree": _run_tree, "accept": _run_accept, "compact": _run_compact, "fork": _run_fork,
            "grouped": _run_grouped, "moe": _run_moe}[op](case, d)


# ---------------------------------------------------------------- the same in 64 bits

def _fl32(x):
    return x.float().double()


def _exact_codec(rows, group):
    """The values that a 4-bit cache holds for rows [..., dim]: the definition's float32 steps,
    each taken in float64 and rounded."""
    out = torch.empty(rows.shape, dtype=torch.float64, device=rows.device)
    for c in range(0, rows.shape[-1], group):
        x = rows[..., c:c + group].double()
        lo = x.min(-1, keepdim=True).values
        s = _fl32(_fl32(x.max(-1, keepdim=True).values - lo) / 15.0)
        q = torch.where(s > 0, _fl32(_fl32(x - lo) / s.clamp(min=1e-300)), torch.zeros_like(x)).round().clamp(0, 15)
        out[..., c:c + group] = s.to(rows.dtype).double() * q + lo.to(rows.dtype).double()
    return out


def _exact_matrix(stack, e, bits, group, k):
    """float64 [n, k] of expert e, code by code from the bitstream."""
    words, s, b = (t[e] for t in stack)
    w = words.to(torch.int64) % (1 << 32)
    q = torch.empty(w.shape[0], k, dtype=torch.float64, device=w.device)
    run_ = 32                                      # codes per `bits` words
    w = w.view(w.shape[0], k // run_, bits)
    cols = q.view(w.shape[0], k // run_, run_)
    for c in range(run_):
        bit = c * bits
        v = w[:, :, bit // 32] >> (bit % 32)
        if bit % 32 + bits > 32:
            v = v + (w[:, :, bit // 32 + 1] << (32 - bit % 32))
        cols[:, :, c] = (v % (1 << bits)).double()
    return q * s.double().repeat_interleave(group, -1) + b.double().repeat_interleave(group, -1)


def _path_up(parents, i):
    """Node i and its ancestors, nearest first; empty if one of them is no node."""
    path = []
    while i != -1:
        if i < 0 or not parents[i] < i:
            return []
        path.append(i)
        i = parents[i]
    return path


def _exact_tree(case, d):
    rep, n = case["heads"] // case["kv_heads"], case["nodes"]
    out = torch.zeros(case["batch"], n, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    at, parents = 0, d["parents"].tolist()
    for b, length in enumerate(_lengths(case, n)):
        k, v = (_exact_codec(d[m][at:at + length], case["group"]) for m in ("k", "v"))
        at += length
        hidden = torch.ones(n, length, dtype=torch.bool)
        for i in range(n):
            path = _path_up(parents[b], i)
            if path:
                oldest = 0 if not case["window"] else max(0, length - n + len(path) - 1 - case["window"] + 1)
                hidden[i, oldest:length - n] = False
                for up in path[:case["window"] or n]:
                    hidden[i, length - n + up] = False
        hidden = hidden.cuda()
        for h in range(case["heads"]):
            s = d["q"][b, :, h].double() @ k[:, h // rep].T * d["scale"]
            s[hidden] = -math.inf
            out[b, :, h] = torch.softmax(s, -1).nan_to_num(0.0) @ v[:, h // rep]
    return out


def _exact_accept(case, d):
    n = case["nodes"]
    k, v = (_exact_codec(d[m], case["group"]).unflatten(0, (case["batch"], n)) for m in ("k", "v"))
    k2, v2 = k.clone(), v.clone()
    for b, (parents, tokens, sampled) in enumerate(zip(*(d[m].tolist() for m in ("parents", "tokens", "sampled")))):
        at, path = 0, [0]
        while True:
            fits = [i for i in range(at + 1, n) if parents[i] == at and tokens[i] == sampled[at]]
            if not fits:
                break
            at = fits[0]
            path.append(at)
        k2[b, :len(path)], v2[b, :len(path)] = k[b, path], v[b, path]
    return None, None, None, k2.flatten(0, 1), v2.flatten(0, 1)


def _exact_fork(case, d):
    page, lens = case["page"], _lengths(case)
    table, refs = d["table"].tolist(), d["refs"].tolist()
    free = iter([p for p, r in enumerate(refs) if r == 0])
    seen, copied = set(), []
    for p, want in zip(d["parents"].tolist(), d["want"].tolist()):
        length = lens[p] if p >= 0 else 0
        keep, copy = min(length, want), None
        for j in range(keep // page, -(-want // page)):
            has = p >= 0 and j < len(table[p]) and table[p][j] >= 0
            if not (has and p not in seen and refs[table[p][j]] == 1):
                next(free)
                if j == keep // page and keep % page:
                    copy = (p, j)
        seen.add(p)
        copied.append(copy)
    out = []
    starts = [sum(lens[:i]) for i in range(len(lens))]
    for m in ("k", "v"):
        rows = torch.zeros(case["rows"], page, case["kv_heads"], case["dim"], dtype=torch.float64, device="cuda")
        for i, copy in enumerate(copied):
            if copy is None:
                rows[i] = math.nan
            else:
                p, j = copy
                part = d[m][starts[p] + j * page:starts[p] + min(lens[p], (j + 1) * page)]
                rows[i, :part.shape[0]] = _exact_codec(part, case["group"])
        out.append(rows.flatten(0, 1))
    return None, None, None, None, None, out[0], out[1]


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "tree":
        return _exact_tree(case, d)
    if op == "accept":
        return _exact_accept(case, d)
    if op == "compact":
        kept, at, rows = d["index"].tolist(), 0, []
        for n, row in zip(_lengths(case), kept):
            rows += [at + i for i in row if i >= 0]
            at += n
        return tuple(_exact_codec(d[m][rows], case["group"]) for m in ("k", "v"))
    if op == "fork":
        return _exact_fork(case, d)
    if op == "grouped":
        y = torch.empty(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        at = d["offsets"].tolist()
        for e in range(case["experts"]):
            if at[e + 1] > at[e]:
                y[at[e]:at[e + 1]] = d["x"][at[e]:at[e + 1]].double() @ _exact_matrix(
                    d["w"], e, case["bits"], case["group"], case["k"]).T
        return y
    y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    who, share = [[] for _ in range(case["experts"])], [[] for _ in range(case["experts"])]
    for t, row in enumerate(d["router"].double().tolist()):
        chosen = sorted(range(len(row)), key=lambda c: (-row[c], c))[:case["top_k"]]
        total = sum(math.exp(row[c]) for c in chosen)
        for c in chosen:
            who[c].append(t)
            share[c].append(math.exp(row[c]) / total)
    for e in range(case["experts"]):
        if who[e]:
            x = d["x"][who[e]].double()
            g, u = (x @ _exact_matrix(d[m], e, case["bits"], case["group"], case["hidden"]).T for m in ("gate", "up"))
            h = g * torch.sigmoid(g) * u * torch.tensor(share[e], dtype=torch.float64, device="cuda")[:, None]
            y[who[e]] += h @ _exact_matrix(d["down"], e, case["bits"], case["group"], case["inter"]).T
    return y
