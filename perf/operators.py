"""Workloads of the decode-step operators: the 4-bit key/value cache (append, attention), the
quantized mixture-of-experts layer for a few tokens, and sampling from logits.

Each case names one operator call as a serving program makes it.  run() computes it in a plain
form (elementary torch operations in float32, one rounding at the end) or, with `own` set,
through this repository's entry points; exact() computes it in float64, written apart from the
plain form.

Shared definitions
  codec      w = s * q + b per group of `group` consecutive values, q unsigned of `bits` bits;
             a row's codes are one little-endian bitstream of uint32 words; s, b in the
             call's dtype.
  cache      one K and one V row of `dim` values per (token slot, kv head), 4-bit codes; slot =
             page * page_size + offset; quantization in float32 steps: s = (max - min) / 15,
             q = clamp(rint((x - min) / s), 0, 15), q = 0 where s = 0, then s and b = min are
             rounded to the dtype.
  attention  query i of a sequence of length L (L tokens cached, `q_len` queries, the last at
             position L - 1) sits at p = L - q_len + i and sees keys j <= p (causal) with
             j > p - window when window > 0; a query that sees nothing gives zeros.
  moe        the top_k largest router logits (ties: lower expert), softmax over them,
             y = sum_e w_e * (silu(x Wg_e^T) * (x Wu_e^T)) Wd_e^T.
  sample     W_i = floor(2^40 exp((l_i - max l) / T)), l_i NaN or -inf never drawn; the top_k
             largest (ties: lower index); of those the shortest prefix in descending order
             whose sum reaches top_p of the total; of those the ones with exp(..) >= min_p; the
             first index whose running sum (index order) exceeds u times the sum.  T <= 0: the
             first maximum.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SPARE_PAGES = 5          # pages of the pool that no sequence of the case holds
W_ONE = float(2 ** 40)   # sampling weight of the largest logit
U_BITS = 24              # u and top_p are taken in units of 2^-24


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of 32 sequences enters the cache: the call of every decode step
        {"name": "append_step", "op": "append", "tokens": 32, "kv_heads": 8, "dim": 128, "group": 64, "page": 64,
         "dtype": "bf16"},
        # a prompt's keys and values enter the cache at once; an odd token count
        {"name": "append_prompt", "op": "append", "tokens": 8191, "kv_heads": 8, "dim": 128, "group": 32, "page": 16,
         "dtype": "fp16"},
        # one short conversation's next token: the smallest attention call, latency counts
        {"name": "attend_short", "op": "attend", "batch": 1, "q_len": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 509, "window": 0, "dtype": "bf16"},
        # a decode step of a full batch of conversations of very different lengths
        {"name": "attend_batch", "op": "attend", "batch": 32, "q_len": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 8192, "window": 0, "dtype": "bf16"},
        # the next token after one long document
        {"name": "attend_long", "op": "attend", "batch": 1, "q_len": 1, "heads": 64, "kv_heads": 8, "dim": 128,
         "group": 128, "page": 256, "length": 131071, "window": 0, "dtype": "fp16"},
        # a few drafted tokens per sequence checked at once, sliding window, small heads
        {"name": "attend_draft_window", "op": "attend", "batch": 16, "q_len": 5, "heads": 16, "kv_heads": 4, "dim": 64,
         "group": 32, "page": 16, "length": 16384, "window": 4096, "dtype": "bf16"},
        # a chunk of a prompt against what is cached before it
        {"name": "attend_prompt", "op": "attend", "batch": 1, "q_len": 2048, "heads": 32, "kv_heads": 8, "dim": 128,
         "group": 64, "page": 64, "length": 8192, "window": 0, "dtype": "bf16"},
        # one token through a layer of many small experts: latency counts
        {"name": "moe_one", "op": "moe", "tokens": 1, "hidden": 2048, "inter": 1024, "experts": 64, "top_k": 8,
         "bits": 4, "group": 64, "dtype": "bf16"},
        # a decode batch through 8-bit experts of the repository's expert shape
        {"name": "moe_batch", "op": "moe", "tokens": 32, "hidden": 1408, "inter": 704, "experts": 128, "top_k": 8,
         "bits": 8, "group": 32, "dtype": "bf16"},
        # a few tokens through few large experts (the prefill benchmark's matrix)
        {"name": "moe_large", "op": "moe", "tokens": 7, "hidden": 4096, "inter": 14336, "experts": 8, "top_k": 2,
         "bits": 4, "group": 128, "dtype": "fp16"},
        # the next token of one conversation over the lm_head's vocabulary
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 151936, "mode": "filtered", "dtype": "bf16"},
        # the next tokens of a decode batch whose requests ask for different things
        {"name": "sample_batch", "op": "sample", "rows": 32, "vocab": 151936, "mode": "mixed", "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "moe", "moe", "sample"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        return {"op": op, "tokens": _log_int(rng, 1, 8191), "kv_heads": rng.choice([1, 2, 5, 8]),
                "dim": rng.choice([64, 128]), "group": rng.choice([32, 64]), "page": rng.choice([16, 48, 64, 256]),
                "dtype": dtype}
    if op == "attend":
        dim = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        c = {"op": op, "batch": _log_int(rng, 1, 32), "q_len": rng.choice([1, 1, 1, 2, 5, _log_int(rng, 6, 1024)]),
             "heads": kv_heads * rng.choice([1, 3, 4, 8]), "kv_heads": kv_heads, "dim": dim,
             "group": rng.choice([g for g in (32, 64, 128) if g <= dim]), "page": rng.choice([16, 48, 64, 256]),
             "length": _log_int(rng, 1, 131071), "window": 0, "dtype": dtype}
        # no more cached rows than the ragged batch has, no more score work than the prompt's
        c["length"] = max(1, min(c["length"], 2 * 131071 * 8 // (kv_heads * c["batch"])))
        c["length"] = max(1, min(c["length"], 2048 * 8192 * 32 // (c["q_len"] * c["heads"] * c["batch"])))
        if rng.random() < 0.3:
            c["window"] = _log_int(rng, 1, 8192)
        return c
    if op == "moe":
        group = rng.choice([32, 64, 128])
        tokens = _log_int(rng, 1, 32)
        experts = rng.choice([4, 8, 60, 64, 128])
        top_k = min(rng.choice([1, 2, 4, 8]), experts)
        hidden = group * max(1, _log_int(rng, 256, 4096) // group)
        inter = group * max(1, _log_int(rng, 128, 14336) // group)
        while experts * hidden * inter > 8 * 4096 * 14336:
            inter = group * max(1, inter // 2 // group)
        return {"op": op, "tokens": tokens, "hidden": hidden, "inter": inter, "experts": experts, "top_k": top_k,
                "bits": rng.choice([4, 4, 8, 8, 3, 6]), "group": group, "dtype": dtype}
    rows = _log_int(rng, 1, 256)
    vocab = max(2, min(_log_int(rng, 1000, 151936), 32 * 151936 // rows))
    return {"op": op, "rows": rows, "vocab": vocab, "mode": rng.choice(["greedy", "filtered", "free", "mixed"]),
            "dtype": dtype}


def _lengths(case):
    """Cached tokens per sequence: evenly spread up to `length`, the last one the longest."""
    n, top = case["batch"], case["length"]
    return [max(1, top * (i + 1) // n) for i in range(n)]


def _row_bytes(case):
    """Bytes of one cached K (or V) row: codes, scales and biases."""
    return case["dim"] // 2 + case["dim"] // case["group"] * 4


def _seen(length, q_len, window):
    """(query, key) pairs of one sequence, and the cached tokens that any query sees."""
    pairs = 0
    for i in range(q_len):
        p = length - q_len + i
        if p >= 0:
            pairs += min(p + 1, window) if window else p + 1
    first = max(0, length - q_len - window + 1) if window else 0
    return pairs, length - first


def work(case):
    if case["op"] == "append":
        rows = case["tokens"] * case["kv_heads"] * 2
        # new rows read, their cached form written, and read back as the values it stands for
        return {"bytes": rows * (2 * case["dim"] + 2 * _row_bytes(case) + 2 * case["dim"]) + 4 * case["tokens"],
                "flops": rows * case["dim"] * 6}
    if case["op"] == "attend":
        pairs = tokens = 0
        for n in _lengths(case):
            p, t = _seen(n, case["q_len"], case["window"])
            pairs, tokens = pairs + p, tokens + t
        io = 2 * 2 * case["batch"] * case["q_len"] * case["heads"] * case["dim"]
        return {"bytes": tokens * case["kv_heads"] * 2 * _row_bytes(case) + io,
                "flops": 4 * case["dim"] * case["heads"] * pairs}
    if case["op"] == "moe":
        e, k, t = case["experts"], case["top_k"], case["tokens"]
        used = e * (1.0 - (1.0 - k / e) ** t)       # expected experts that any token chooses
        mat = case["hidden"] * case["inter"]
        per = mat * case["bits"] / 8 + mat // case["group"] * 4
        return {"bytes": int(3 * used * per) + 2 * t * (2 * case["hidden"] + e),
                "flops": 2 * 3 * t * k * mat}
    return {"bytes": case["rows"] * (2 * case["vocab"] + 28), "flops": case["rows"] * case["vocab"] * 4}


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
    for e in range(experts):
        codes = torch.clamp(torch.round(_randn(g, n, k) * (top / 6.0) + top / 2.0), 0, top).to(torch.int64)
        words[e] = _pack(codes, bits)
    s = (0.02 * 6.0 / top) * (0.8 + 0.4 * torch.rand(experts, n, k // group, generator=g, device="cuda"))
    return words, s.to(dtype), (s * (-top / 2.0)).to(dtype)


def _inputs(case, seed):
    g = _gen(seed)
    dtype = DTYPES[case["dtype"]]
    d = {}
    if case["op"] == "append":
        t = case["tokens"]
        d["k"], d["v"] = _cache_rows(g, t, case), _cache_rows(g, t, case)
        d["pages"] = -(-t // case["page"]) + SPARE_PAGES
        perm = torch.randperm(d["pages"] * case["page"], generator=g, device="cuda")
        d["slots"] = perm[:t].to(torch.int32)       # any free slot of any page
    elif case["op"] == "attend":
        lens, page = _lengths(case), case["page"]
        blocks = [-(-n // page) for n in lens]
        d["pages"] = sum(blocks) + SPARE_PAGES
        perm = torch.randperm(d["pages"], generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["batch"], max(blocks)), -1, dtype=torch.int32, device="cuda")
        slots, at = [], 0
        for i, (n, m) in enumerate(zip(lens, blocks)):
            table[i, :m] = perm[at:at + m]
            j = torch.arange(n, device="cuda")
            slots.append(perm[at:at + m][j // page] * page + j % page)
            at += m
        d["table"], d["slots"] = table, torch.cat(slots).to(torch.int32)
        d["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        d["k"], d["v"] = _cache_rows(g, sum(lens), case), _cache_rows(g, sum(lens), case)
        d["q"] = _randn(g, case["batch"], case["q_len"], case["heads"], case["dim"]).to(dtype)
        d["scale"] = case["dim"] ** -0.5
    elif case["op"] == "moe":
        e, k, n = case["experts"], case["hidden"], case["inter"]
        d["x"] = _randn(g, case["tokens"], k).to(dtype)
        d["router"] = (1.5 * _randn(g, case["tokens"], e)).to(dtype)
        d["gate"] = _expert_stack(g, e, n, k, case)
        d["up"] = _expert_stack(g, e, n, k, case)
        d["down"] = _expert_stack(g, e, k, n, case)
    else:
        rows, mode = case["rows"], case["mode"]
        d["logits"] = (2.5 * _randn(g, rows, case["vocab"])).to(dtype)
        if mode == "mixed" and rows > 2:            # a request that forbids most of the vocabulary
            d["logits"][rows // 2, torch.rand(case["vocab"], generator=g, device="cuda") < 0.9] = -math.inf
        r = torch.arange(rows, device="cuda")
        kind = {"greedy": torch.zeros_like(r), "filtered": torch.full_like(r, 1), "free": torch.full_like(r, 2),
                "mixed": r % 4}[mode]
        t = 0.6 + 0.6 * torch.rand(rows, generator=g, device="cuda")
        d["temperature"] = torch.where(kind == 0, torch.zeros_like(t), t)
        k = torch.randint(20, 200, (rows,), generator=g, device="cuda")
        d["top_k"] = torch.where((kind == 1) & (r % 8 != 5), k, torch.zeros_like(k)).to(torch.int32)
        p = 0.8 + 0.19 * torch.rand(rows, generator=g, device="cuda")
        d["top_p"] = torch.where((kind == 1) | (kind == 3), p, torch.ones_like(p))
        m = 0.01 + 0.1 * torch.rand(rows, generator=g, device="cuda")
        d["min_p"] = torch.where(kind == 3, m, torch.zeros_like(m))
        d["u"] = torch.rand(rows, generator=g, device="cuda")
    return d


# ---------------------------------------------------------------- plain forms

def _pack(codes, bits):
    """int64 codes [..., k] -> int32 words [..., k * bits / 32], one bitstream per row."""
    k = codes.shape[-1]
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
    return _dequant(*(t[slots] for t in store), 4, case["group"], case["dim"])


def _run_attend(case, d):
    dtype = DTYPES[case["dtype"]]
    b, lq, hk, dim = case["batch"], case["q_len"], case["kv_heads"], case["dim"]
    rep = case["heads"] // hk
    top = d["table"].shape[1] * case["page"]
    j = torch.arange(top, device="cuda")
    slots = d["table"].clamp(min=0)[:, j // case["page"]] * case["page"] + j % case["page"]    # [b, top]
    k, v = (_plain_read(case, store, slots).transpose(1, 2).contiguous() for store in d["cache"])   # [b, hk, top, dim]
    q = d["q"].float().unflatten(2, (hk, rep)).permute(0, 2, 3, 1, 4).reshape(b, hk, rep * lq, dim)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * d["scale"]
    p = d["lengths"][:, None] - lq + torch.arange(lq, device="cuda")       # [b, lq]
    seen = (j <= p[..., None]) & (j < d["lengths"][:, None, None])
    if case["window"]:
        seen = seen & (j > p[..., None] - case["window"])
    seen = seen[:, None, None]                                             # [b, 1, 1, lq, top]
    s = s.unflatten(2, (rep, lq)).masked_fill(~seen, -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38)).masked_fill(~seen, 0.0)
    e = (e / e.sum(-1, keepdim=True).clamp(min=1e-37)).flatten(2, 3)
    o = torch.matmul(e, v).unflatten(2, (rep, lq))                         # [b, hk, rep, lq, dim]
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(dtype)


def _run_moe(case, d):
    bits, group = case["bits"], case["group"]
    x = d["x"].float()
    value, index = torch.sort(d["router"].float(), dim=-1, descending=True, stable=True)
    value, index = value[:, :case["top_k"]], index[:, :case["top_k"]]
    w = torch.exp(value - value[:, :1])
    w = w / w.sum(-1, keepdim=True)
    y = torch.zeros(case["tokens"], case["hidden"], device="cuda")
    for r in range(case["top_k"]):
        e = index[:, r]
        g, u = (torch.bmm(_dequant(*(t[e] for t in d[m]), bits, group, case["hidden"]), x[:, :, None])[..., 0]
                for m in ("gate", "up"))
        h = g / (1.0 + torch.exp(-g)) * u
        down = _dequant(*(t[e] for t in d["down"]), bits, group, case["inter"])
        y += w[:, r:r + 1] * torch.bmm(down, h[:, :, None])[..., 0]
    return y.to(d["x"].dtype)


def _share(total, units):
    """floor(total * units / 2^24) of int64 tensors without overflow."""
    hi, lo = total >> U_BITS, total & (2 ** U_BITS - 1)
    return hi * units + ((lo * units) >> U_BITS)


def _run_sample(case, d):
    l = d["logits"].float()
    open_ = l > -math.inf                                                  # false for NaN too
    l = torch.where(open_, l, torch.full_like(l, -math.inf))
    top = l.amax(-1, keepdim=True)
    t = d["temperature"][:, None]
    greedy = t <= 0
    w = torch.exp((l - top) / torch.where(greedy, torch.ones_like(t), t))
    w = torch.where(l == top, torch.ones_like(w), torch.where(greedy, torch.zeros_like(w), w))
    w = torch.where(open_, w, torch.zeros_like(w))
    _, order = torch.sort(l, dim=-1, descending=True, stable=True)
    ws = torch.gather(w, 1, order)
    big = (ws * W_ONE).to(torch.int64)
    rank = torch.arange(l.shape[1], device="cuda")[None, :]
    k = d["top_k"][:, None].to(torch.int64)
    keep = (rank < torch.where(k > 0, k, torch.full_like(k, l.shape[1]))) & (~greedy | (rank == 0))
    big = torch.where(keep, big, torch.zeros_like(big))
    cum = torch.cumsum(big, -1)
    units = (d["top_p"].clamp(0, 1) * 2.0 ** U_BITS).to(torch.int64)[:, None]
    need = _share(cum[:, -1:], units)
    keep = keep & ((cum - big < need) | (rank == 0)) & ((ws >= d["min_p"][:, None]) | (rank == 0))
    big = torch.where(keep, big, torch.zeros_like(big))
    by_index = torch.zeros_like(big).scatter_(1, order, big)
    cum = torch.cumsum(by_index, -1)
    total = cum[:, -1:]
    target = _share(total, (d["u"].clamp(0, 1) * 2.0 ** U_BITS).to(torch.int64).clamp(max=2 ** U_BITS - 1)[:, None])
    index = (cum <= target).sum(-1)
    some = total[:, 0] > 0
    picked = torch.gather(by_index, 1, index.clamp(max=l.shape[1] - 1)[:, None])[:, 0]
    prob = torch.where(some, picked.double() / total[:, 0].clamp(min=1).double(), torch.zeros_like(picked).double())
    return torch.where(some, index, torch.full_like(index, -1)).to(torch.int32), prob.float()


# ---------------------------------------------------------------- preparation and one pass

def prepare(case, seed):
    d = _inputs(case, seed)
    state = {"case": case, "d": d}
    if own:
        import bit_affine_quantized_qmv_amd as qmm
        state["qmm"] = qmm
        if case["op"] in ("append", "attend"):
            d["cache"] = qmm.kv_cache(d["pages"], case["page"], case["kv_heads"], case["dim"], case["group"],
                                      case["dtype"], device="cuda")
        if case["op"] == "attend":
            qmm.kv_append(d["cache"], d["k"], d["v"], d["slots"])
            state["workspace"] = qmm.kv_attend_workspace(d["q"], d["cache"], case["length"])
        if case["op"] == "moe":
            for m, n, k in (("gate", case["inter"], case["hidden"]), ("up", case["inter"], case["hidden"]),
                            ("down", case["hidden"], case["inter"])):
                state[m] = qmm.ExpertWeights(*d[m], n, k, case["group"], case["bits"])
            state["workspace"] = qmm.moe_workspace(d["x"], state["gate"], case["top_k"])
        if case["op"] == "sample":
            state["workspace"] = qmm.sample_workspace(case["rows"], "cuda")
    elif case["op"] in ("append", "attend"):
        d["cache"] = _plain_cache(case, d)
        if case["op"] == "attend":
            _plain_append(case, d["cache"], d["k"], d["v"], d["slots"])
    if case["op"] == "attend":
        del d["k"], d["v"]
    return state


def run(state):
    case, d = state["case"], state["d"]
    if own:
        qmm = state["qmm"]
        if case["op"] == "append":
            qmm.kv_append(d["cache"], d["k"], d["v"], d["slots"])
            return qmm.kv_read(d["cache"], d["slots"])
        if case["op"] == "attend":
            return qmm.kv_attend(d["q"], d["cache"], d["table"], d["lengths"], scale=d["scale"], causal=True,
                                 window=case["window"], max_length=case["length"], workspace=state["workspace"])
        if case["op"] == "moe":
            return qmm.moe(d["x"], d["router"], state["gate"], state["up"], state["down"], case["top_k"],
                           workspace=state["workspace"])
        return qmm.sample(d["logits"], d["u"], temperature=d["temperature"], top_k=d["top_k"], top_p=d["top_p"],
                          min_p=d["min_p"], workspace=state["workspace"])
    if case["op"] == "append":
        _plain_append(case, d["cache"], d["k"], d["v"], d["slots"])
        return tuple(_plain_read(case, store, d["slots"]).to(d["k"].dtype) for store in d["cache"])
    if case["op"] == "attend":
        return _run_attend(case, d)
    if case["op"] == "moe":
        return _run_moe(case, d)
    return _run_sample(case, d)


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
    run = 32                                       # codes per `bits` words
    w = w.view(w.shape[0], k // run, bits)
    cols = q.view(w.shape[0], k // run, run)
    for c in range(run):
        bit = c * bits
        v = w[:, :, bit // 32] >> (bit % 32)
        if bit % 32 + bits > 32:
            v = v + (w[:, :, bit // 32 + 1] << (32 - bit % 32))
        cols[:, :, c] = (v % (1 << bits)).double()
    return q * s.double().repeat_interleave(group, -1) + b.double().repeat_interleave(group, -1)


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "append":
        return tuple(_exact_codec(d[n], case["group"]) for n in ("k", "v"))
    if case["op"] == "attend":
        rep, lq, out = case["heads"] // case["kv_heads"], case["q_len"], []
        at = 0
        for i, n in enumerate(_lengths(case)):
            o = torch.zeros(lq, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
            k, v = (_exact_codec(d[m][at:at + n], case["group"]) for m in ("k", "v"))
            at += n
            pos = n - lq + torch.arange(lq, device="cuda")[:, None]
            key = torch.arange(n, device="cuda")[None, :]
            hidden = key > pos
            if case["window"]:
                hidden = hidden | (key <= pos - case["window"])
            for h in range(case["heads"]):
                s = d["q"][i, :, h].double() @ k[:, h // rep].T * d["scale"]
                s[hidden] = -math.inf
                o[:, h] = torch.softmax(s, -1).nan_to_num(0.0) @ v[:, h // rep]
            out.append(o)
        return torch.stack(out)
    if case["op"] == "moe":
        y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        router = d["router"].double().tolist()
        for e in range(case["experts"]):
            who, share = [], []
            for t, row in enumerate(router):
                chosen = sorted(range(len(row)), key=lambda c: (-row[c], c))[:case["top_k"]]
                if e in chosen:
                    who.append(t)
                    share.append(math.exp(row[e]) / sum(math.exp(row[c]) for c in chosen))
            if not who:
                continue
            x = d["x"][who].double()
            g, u = (x @ _exact_matrix(d[m], e, case["bits"], case["group"], case["hidden"]).T for m in ("gate", "up"))
            h = g * torch.sigmoid(g) * u * torch.tensor(share, dtype=torch.float64, device="cuda")[:, None]
            y[who] += h @ _exact_matrix(d["down"], e, case["bits"], case["group"], case["inter"]).T
        return y
    prob = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
    for r in range(case["rows"]):
        l = d["logits"][r].double()
        t, k = float(d["temperature"][r]), int(d["top_k"][r])
        if t <= 0:
            prob[r] = 1.0
            continue
        value, index = torch.sort(l, descending=True, stable=True)
        if k > 0:
            value, index = value[:k], index[:k]
        w = torch.exp((value - value[0]) / t)
        before = torch.cumsum(w, 0) - w
        w = torch.where((before < float(d["top_p"][r]) * w.sum()) & (w >= float(d["min_p"][r])), w, torch.zeros_like(w))
        w[0] = 1.0
        line = torch.zeros_like(l)
        line[index] = w
        run_sum = torch.cumsum(line, 0)
        at = int((run_sum <= float(d["u"][r]) * run_sum[-1]).sum().clamp(max=l.shape[0] - 1))
        prob[r] = line[at] / run_sum[-1]
    return None, prob
