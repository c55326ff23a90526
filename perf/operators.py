"""The operators of the paged 8-bit key/value cache, as workloads: sizes, inputs, plain form and definition.

The cache holds keys and values as 8-bit codes (int8 or e4m3) in pages of `page` tokens, with one power-of-two scale for
each page, layer, key/value and head.  Five operators work on it:

  attention  causal attention of each sequence's newest tokens over its cached keys and values
  append     new keys and values rounded into the pages, a page's scale growing with its largest value
  resize     every listed slot to a new length: pages taken from the free ones, given back, and copied where shared
  fork       a slot's sequence shared with empty slots, the unfinished last page copied
  compact    the pages in use moved to the lowest places of the pool, tables rewritten

`own = False` computes them with elementary torch operations, `own = True` through the library's entry points.
"""
import math
import random

import torch

own = False

INT8_MAX, E4M3_MAX = 127.0, 448.0


# ------------------------------------------------------------------------------------------------------------ cases
def listed():
    gpt2 = dict(heads=12, kv_heads=12, head_dim=64, page=16)
    return [
        # one user's sampling loop: one token of one sequence over its prefix; only latency counts
        dict(gpt2, name="attention one sequence", op="attention", fmt="int8", layers=2, n=1, len_lo=777, len_hi=777,
             q_lo=1, q_hi=1, pad=0, mix=1),
        # a sampling batch of GPT-2 sequences of every length up to the block size
        dict(gpt2, name="attention batch 64", op="attention", fmt="e4m3", layers=2, n=64, len_lo=1, len_hi=1024,
             q_lo=1, q_hi=1, pad=3, mix=2),
        # serving long contexts with shared heads, four query heads to a key/value head
        dict(name="attention long shared heads", op="attention", fmt="int8", layers=1, heads=32, kv_heads=8,
             head_dim=128, page=64, n=32, len_lo=4000, len_hi=16384, q_lo=1, q_hi=1, pad=0, mix=3),
        # chunks of prompts: hundreds of new tokens each over what is cached already
        dict(name="attention prompt chunks", op="attention", fmt="e4m3", layers=1, heads=12, kv_heads=12,
             head_dim=64, page=32, n=4, len_lo=1500, len_hi=4096, q_lo=300, q_hi=1024, pad=0, mix=4),
        # one sampled token of each of 256 sequences written to its page
        dict(gpt2, name="append step 256", op="append", fmt="int8", layers=2, n=256, len_lo=1, len_hi=1024,
             q_lo=1, q_hi=1, pad=5, mix=5),
        # a micro-batch of prompts written to fresh pages (B = 16, T up to 1024)
        dict(gpt2, name="append prompts", op="append", fmt="e4m3", layers=1, n=16, len_lo=900, len_hi=1024,
             q_lo=900, q_hi=1024, pad=0, mix=6),
        # before a sampling step: room for one more token in each of 64 slots
        dict(gpt2, name="resize step 64", op="resize", fmt="int8", layers=12, n=64, len_lo=1, len_hi=500, ways=1,
             how="step", mix=7),
        # rejected drafts: 512 slots cut back into a prefix that eight of them share, each copying one page
        dict(gpt2, name="resize rollback shared", op="resize", fmt="e4m3", layers=12, n=512, len_lo=200, len_hi=600,
             ways=8, how="rollback", mix=8),
        # one prompt continued four ways
        dict(gpt2, name="fork one into four", op="fork", fmt="int8", layers=12, n=1, len_lo=333, len_hi=333, ways=4,
             mix=9),
        # a batch of 64 prompts, four samples of each
        dict(gpt2, name="fork 64 into 256", op="fork", fmt="e4m3", layers=12, n=64, len_lo=100, len_hi=1000, ways=4,
             mix=10),
        # a small pool after some of its sequences ended
        dict(gpt2, name="compact small pool", op="compact", fmt="int8", layers=12, n=8, len_lo=50, len_hi=500,
             ways=1, fill=0.6, mix=11),
        # a pool half empty, before half of its memory is given back
        dict(gpt2, name="compact half pool", op="compact", fmt="e4m3", layers=12, n=64, len_lo=100, len_hi=1000,
             ways=2, fill=0.5, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [(c["op"], work(c)) for c in listed()]
    while True:  # until one costs no more than its operator's largest listed case
        c = _any(rng)
        w = work(c)
        if any(op == c["op"] and w["bytes"] <= m["bytes"] and w["flops"] <= max(m["flops"], 4e8) for op, m in most):
            return c


def _any(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "resize", "fork", "compact"])
    kv, d = rng.choice([(12, 64), (1, 64), (4, 64), (8, 128), (2, 128), (16, 64), (3, 64)])
    c = dict(op=op, fmt=rng.choice(["int8", "e4m3"]), kv_heads=kv, head_dim=d, page=rng.choice([16, 16, 32, 64, 128]),
             heads=kv * rng.choice([1, 1, 2, 4, 7, 8]), mix=rng.randrange(1 << 30))
    if op == "attention":
        c["layers"] = rng.choice([1, 2])
        if rng.random() < 0.6:  # single tokens, and a few drafted ones
            c["q_hi"] = rng.choice([1, 1, 1, 2, 5])
            c["n"] = _log(rng, 1, 128)
            c["len_hi"] = _log(rng, 8, max(8, min(100000, 300_000_000 // (c["n"] * kv * d * c["layers"]))))
            c["q_lo"] = rng.choice([0, 1])
        else:
            c["q_hi"] = _log(rng, 6, 900)
            c["n"] = _log(rng, 1, 8)
            most = 150_000_000 // (c["n"] * c["heads"] * c["q_hi"])
            c["len_hi"] = _log(rng, c["q_hi"], max(c["q_hi"], min(8192, most)))
            c["q_lo"] = rng.choice([0, 1, c["q_hi"]])
        c["len_lo"] = rng.choice([c["q_hi"], c["len_hi"]]) if c["len_hi"] > c["q_hi"] else c["q_hi"]
        c["len_hi"] = max(c["len_hi"], c["len_lo"])
        c["pad"] = rng.choice([0, 0, 1, 9])
    elif op == "append":
        c["layers"] = rng.choice([1, 2])
        c["n"] = _log(rng, 1, 300)
        c["q_hi"] = _log(rng, 1, max(1, min(1024, 12_000_000 // (c["n"] * kv * d))))
        c["q_lo"] = rng.choice([0, 1, c["q_hi"]])
        c["len_lo"], c["len_hi"] = c["q_hi"], c["q_hi"] + _log(rng, 1, 400)
        c["pad"] = rng.choice([0, 4])
    else:
        c["layers"] = rng.choice([1, 4, 12])
        c["ways"] = rng.choice([1, 2, 4, 8])
        c["n"] = c["ways"] * _log(rng, 1, 48) if op != "fork" else _log(rng, 1, 64)
        room = 600_000_000 // (c["layers"] * 2 * kv * d * c["n"])
        c["len_hi"] = _log(rng, 8, max(8, min(1000, room)))
        c["len_lo"] = rng.choice([1, c["len_hi"]])
        if op == "resize":
            c["how"] = rng.choice(["step", "rollback", "mixed"])
        if op == "compact":
            c["fill"] = rng.choice([0.3, 0.5, 0.8, 0.95])
    return c


# ------------------------------------------------------------------------------------------------- lengths of a case
def _up(a, b):
    return -(-a // b)


def _lengths(c):
    """(length, new tokens) of every sequence, the same for every seed."""
    r = random.Random(c["mix"])
    lens = [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["n"])]
    if "ways" in c and c["op"] != "fork":  # `ways` slots hold the same sequence
        lens = [lens[i - i % c["ways"]] for i in range(c["n"])]
    news = [min(t, r.randint(c.get("q_lo", 0), c.get("q_hi", 0))) for t in lens]
    if c["op"] in ("attention", "append"):
        news[-1] = max(1, news[-1])
    return lens, news


def _targets(c, lens):
    """The lengths a resize asks for."""
    r = random.Random(c["mix"] + 1)
    if c["how"] == "step":
        return [t + 1 for t in lens]
    if c["how"] == "rollback":
        return [max(0, t - r.randint(1, 2 * c["page"])) for t in lens]
    return [r.choice([0, t, t + 1, t + 3 * c["page"], t // 2]) for t in lens]


def _row_bytes(c):
    return 2 * c["kv_heads"] * c["head_dim"]  # codes of one token in one layer


def _page_bytes(c):
    return c["layers"] * (_row_bytes(c) * c["page"] + 2 * c["kv_heads"] * 4)


def _moves(c):
    """(pages copied, table entries read or written) of a resize, fork or compact."""
    lens, _ = _lengths(c)
    p = c["page"]
    if c["op"] == "fork":
        return c["ways"] * sum(t % p > 0 for t in lens), 2 * c["ways"] * sum(_up(t, p) for t in lens)
    if c["op"] == "resize":
        new = _targets(c, lens)
        shared = c["ways"] > 1
        return (sum(shared and min(a, b) % p > 0 for a, b in zip(lens, new)),
                sum(abs(_up(a, p) - _up(b, p)) + 1 for a, b in zip(lens, new)))
    live = sum(_up(t, p) for t in lens[::c["ways"]])
    pages = _pool_pages(c)
    return live * (pages - live) // pages, 2 * sum(_up(t, p) for t in lens)


def work(case):
    c = case
    lens, news = _lengths(c)
    rows, h, kv, d, p = sum(news), c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    if c["op"] == "attention":
        cached = sum(t for t, q in zip(lens, news) if q)
        pages = sum(_up(t, p) for t, q in zip(lens, news) if q)
        pairs = sum(q * t - q * (q - 1) // 2 for t, q in zip(lens, news))
        return {"bytes": cached * _row_bytes(c) + pages * (2 * kv * 4 + 4) + rows * h * (4 * d + 4) + 12 * len(lens),
                "flops": 4 * pairs * h * d}
    if c["op"] == "append":
        pages = sum(_up(t, p) - (t - q) // p for t, q in zip(lens, news) if q)
        return {"bytes": rows * _row_bytes(c) * 3 + pages * (2 * kv * 8 + 4) + 12 * len(lens), "flops": 4 * rows * 2 * kv * d}
    copies, entries = _moves(c)
    n = c["n"] * (c["ways"] if c["op"] == "fork" else 1)
    return {"bytes": 2 * copies * _page_bytes(c) + 8 * entries + 12 * n + 4 * _pool_pages(c), "flops": 0}


# ------------------------------------------------------------------------------------------------------------ inputs
def _pool_pages(c):
    lens, _ = _lengths(c)
    p, ways = c["page"], c.get("ways", 1)
    if c["op"] == "fork":
        return sum(_up(t, p) for t in lens) + ways * len(lens) + 5
    live = sum(_up(t, p) for t in lens[::ways])
    if c["op"] == "resize":
        grown = sum(max(0, _up(b, p) - _up(a, p)) + 1 for a, b in zip(lens, _targets(c, lens)))
        return live + grown + 5
    if c["op"] == "compact":
        return max(live + 1, int(round(live / c["fill"])))
    return live + max(3, live // 16)


def _two(e):
    """2^e in 32 bits, to the bit, for whole e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens, news = _lengths(c)
    n, p, ways = c["n"], c["page"], c.get("ways", 1)
    kv, h, d, layers = c["kv_heads"], c["heads"], c["head_dim"], c["layers"]
    pages = _pool_pages(c)
    fork = c["op"] == "fork"
    slots_in = torch.randperm(n * (1 + ways if fork else 1) + 3, generator=g, device=dev)
    targets = _targets(c, lens) if c["op"] == "resize" else [0]
    most = max(1, max(_up(t, p) for t in lens + targets))
    shape = (pages, layers, 2, kv, p, d)

    # codes as rounding normal values leaves them, and scales that bring them back to the values' size
    if c["fmt"] == "int8":
        codes = torch.empty(shape, dtype=torch.int8, device=dev)
        for i in range(0, pages, 256):
            m = codes[i:i + 256]
            m.copy_(torch.randn(m.shape, generator=g, device=dev).mul_(36).round_().clamp_(-127, 127))
        low = 5
    else:
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
        for i in range(0, pages, 256):
            m = codes[i:i + 256]
            m.copy_(torch.randn(m.shape, generator=g, device=dev).mul_(90).clamp_(-448, 448))
        low = 6
    scales = _two(-torch.randint(low, low + 2, shape[:4], generator=g, device=dev))

    # reference counts, lengths and page table, one buffer as the program's restore point copies them
    nslots = slots_in.numel()
    cut = (_up(pages, 4) * 4, _up(nslots, 4) * 4)
    meta = torch.zeros(cut[0] + cut[1] + nslots * most, dtype=torch.int32, device=dev)
    refs, slot_lens = meta[:pages], meta[cut[0]:cut[0] + nslots]
    table = meta[cut[0] + cut[1]:].view(nslots, most)
    table.fill_(-1)
    ids = torch.randperm(pages, generator=g, device=dev).int()
    shared = 1 if fork else ways
    counts = torch.tensor([_up(t, p) for t in lens[::shared]], device=dev)
    first = counts.cumsum(0) - counts
    cols = torch.arange(most, device=dev)
    rows = torch.where(cols[None] < counts[:, None], ids[(first[:, None] + cols[None]).clamp_(max=pages - 1)], -1)
    rows = rows.repeat_interleave(shared, 0)
    src = slots_in[:n]
    table[src] = rows
    slot_lens[src] = torch.tensor(lens, dtype=torch.int32, device=dev)
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).int().flatten())

    s = dict(case=c, codes=codes, scales=scales, meta=meta, refs=refs, lens=slot_lens, table=table, layer=layers - 1,
             slots=src.int().contiguous(), work=torch.zeros(64 << 20, dtype=torch.uint8, device=dev))
    if c["op"] in ("attention", "append"):
        cu = [0]
        for q in news:
            cu.append(cu[-1] + q)
        total = cu[-1] + c["pad"]
        qkv = torch.randn(total, (h + 2 * kv) * d, generator=g, device=dev).to(torch.bfloat16)
        if c["op"] == "append":
            # tokens differ in size, so that some pages' scales grow
            qkv.mul_(_two(torch.randint(-1, 3, (total, 1), generator=g, device=dev)).to(torch.bfloat16))
        s["q"] = qkv[:, :h * d].view(total, h, d)
        s["k"] = qkv[:, h * d:(h + kv) * d].view(total, kv, d)
        s["v"] = qkv[:, (h + kv) * d:].view(total, kv, d)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["rows"], s["max_q"], s["max_len"] = cu[-1], max(max(news), 1), max(lens)
        s["out"] = torch.zeros(total, h, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(total, h, dtype=torch.float32, device=dev)
    if c["op"] == "resize":
        s["new"] = torch.tensor(targets, dtype=torch.int32, device=dev)
    if fork:
        s["slots"] = src.int().repeat_interleave(ways).contiguous()
        s["dst"] = slots_in[n:n + n * ways].int().contiguous()
    if c["op"] == "compact":
        s["live"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["op"] in ("resize", "fork", "compact"):
        s["meta0"] = meta.clone()
    return s


# --------------------------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if op in ("resize", "fork", "compact"):
        s["meta"].copy_(s["meta0"])  # back to the restore point: the pass starts from the same pages each time
    if own:
        _run_own(s, op)
    else:
        PLAIN[op](s)
    if op == "attention":
        return {"out": s["out"], "lse": s["lse"]}
    codes = s["codes"] if op == "append" else s["codes"].view(torch.uint8)
    res = {"codes": codes, "scales": s["scales"]}
    if op != "append":
        res["meta"] = s["meta"]
    if op == "compact":
        res["live"] = s["live"]
    return res


def _run_own(s, op):
    cache = s.get("cache")
    if cache is None:  # the handle that a program makes once for its tensors
        from decoder_only_transformer_02_b200 import gpt2 as G
        cache = s["cache"] = G.KV8Cache(s["codes"], s["scales"], s["table"], s["lens"], s["refs"])
    if op == "attention":
        cache.attention(s["layer"], s["q"], s["out"], s["slots"], s["cu"], s["max_q"], s["work"], lse=s["lse"])
    elif op == "append":
        cache.append(s["layer"], s["k"], s["v"], s["slots"], s["cu"])
    elif op == "resize":
        cache.resize(s["slots"], s["new"], s["work"])
    elif op == "fork":
        cache.fork(s["slots"], s["dst"], s["work"])
    else:
        cache.compact(s["work"], live=s["live"])


def _bytes(codes):
    return codes.view(torch.uint8)


def _plain_attention(s):
    c = s["case"]
    p, kv, d, h = c["page"], c["kv_heads"], c["head_dim"], c["heads"]
    n, group, layer = c["n"], h // kv, s["layer"]
    slots, cu = s["slots"].long(), s["cu"].long()
    lens, q_lens = s["lens"][slots].long(), cu[1:] - cu[:-1]
    np_ = _up(s["max_len"], p)
    pages = s["table"][slots, :np_].clamp(min=0).long()
    raw = _bytes(s["codes"])[pages, layer].view(s["codes"].dtype)  # [n, np, 2, kv, page, d]
    vals = raw.float() * s["scales"][pages, layer][..., None, None]
    t = torch.arange(np_ * p, device=vals.device)
    keys, values = vals.permute(2, 0, 3, 1, 4, 5).reshape(2, n, kv, np_ * p, d)
    here = t[None] < lens[:, None]
    values = torch.where(here[:, None, :, None], values, 0.0)
    i = torch.arange(s["max_q"], device=vals.device)
    row = (cu[:-1, None] + i[None]).clamp(max=max(s["q"].shape[0] - 1, 0))
    is_row = i[None] < q_lens[:, None]
    q = s["q"][row].float().view(n, s["max_q"], kv, group, d).permute(0, 2, 1, 3, 4).reshape(n, kv, -1, d)
    score = torch.matmul(q, keys.transpose(2, 3)).view(n, kv, s["max_q"], group, -1) / math.sqrt(d)
    last = lens[:, None] - q_lens[:, None] + i[None]
    seen = (t[None, None] <= last[..., None]) & here[:, None]  # [n, q, T]
    score = torch.where(seen[:, None, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    den = e.sum(-1, keepdim=True)
    out = torch.matmul(e.flatten(2, 3), values).view(n, kv, s["max_q"], group, d) / den
    lse = top + torch.log(den)
    at = row[is_row]
    s["out"][at] = out.permute(0, 2, 1, 3, 4).reshape(n, s["max_q"], h, d)[is_row].to(s["out"].dtype)
    s["lse"][at] = lse.permute(0, 2, 1, 3, 4).reshape(n, s["max_q"], h)[is_row]


def _round_codes(x, dtype):
    """Values over their scale to codes, rounded to nearest even."""
    return x.round().to(torch.int8) if dtype == torch.int8 else x.to(torch.float8_e4m3fn)


def _scale_for(amax, dtype):
    """The smallest power of two, 2^-126 at least, with which amax fits the codes' range."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 127 / 128, x - 7, x - 6) if dtype == torch.int8 else torch.where(m <= 0.875, x - 9, x - 8)
    return _two(torch.where(amax > 0, e, -126).clamp(min=-126))


def _plain_append(s):
    c = s["case"]
    p, layer, dtype = c["page"], s["layer"], s["codes"].dtype
    slots, cu = s["slots"].long(), s["cu"].long()
    lens, q_lens = s["lens"][slots].long(), cu[1:] - cu[:-1]
    r = torch.arange(s["rows"], device=slots.device)
    seq = torch.searchsorted(cu, r, right=True) - 1
    pos = lens[seq] - q_lens[seq] + r - cu[seq]
    page, off = s["table"][slots[seq], pos // p].long(), pos % p
    kv = torch.stack([s["k"][:s["rows"]], s["v"][:s["rows"]]], 1).float()  # [rows, 2, heads, d]
    scales = s["scales"][:, layer]
    need = torch.zeros_like(scales).index_reduce_(0, page, kv.abs().amax(-1), "amax")
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device=r.device).index_fill_(0, page, True)
    fresh = torch.zeros_like(touched).index_fill_(0, page[off == 0], True)
    need = _scale_for(need, dtype)
    new = torch.where(fresh[:, None, None], need, torch.maximum(scales, need))
    new = torch.where(touched[:, None, None], new, scales)
    grown = (touched & ~fresh & (new > scales).flatten(1).any(1)).nonzero().flatten()
    ratio = (scales / new)[grown][..., None, None]
    old = _bytes(s["codes"])[grown, layer].view(dtype).float()
    _bytes(s["codes"])[grown, layer] = _bytes(_round_codes(old * ratio, dtype))
    codes = _round_codes(kv / new[page][..., None], dtype)
    _bytes(s["codes"]).transpose(3, 4)[page, layer, :, off] = _bytes(codes)
    s["scales"][:, layer] = new


def _copy_pages(s, src, dst):
    b = _bytes(s["codes"])
    b[dst] = b[src]
    s["scales"][dst] = s["scales"][src]


def _plain_resize(s):
    p, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    slots, new = s["slots"].long(), s["new"].long()
    old = lens[slots].long()
    have, want, keep = (old + p - 1) // p, (new + p - 1) // p, torch.minimum(old, new)
    col = torch.arange(table.shape[1], device=slots.device)[None]
    rows = table[slots]
    edge = (keep // p).clamp(max=table.shape[1] - 1)
    at_edge = rows.gather(1, edge[:, None])[:, 0].clamp(min=0).long()
    copy = (keep % p > 0) & (refs[at_edge] > 1)
    drop = (col >= want[:, None]) & (col < have[:, None])
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -drop.int().flatten())
    free = (refs == 0).nonzero().flatten().int()
    count = copy.long() + (want - have).clamp(min=0)
    first = count.cumsum(0) - count
    is_copy = copy[:, None] & (col == edge[:, None])
    is_new = (col >= have[:, None]) & (col < want[:, None])
    k = torch.where(is_copy, 0, copy.long()[:, None] + col - have[:, None]) + first[:, None]
    take = is_copy | is_new
    rows = torch.where(drop, -1, rows)
    got = free[k[take]]
    rows[take] = got
    table[slots] = rows
    refs[got.long()] = 1
    refs.index_add_(0, at_edge, -copy.int())
    lens[slots] = new.int()
    _copy_pages(s, at_edge[copy], free[first[copy]].long())


def _plain_fork(s):
    p, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    src, dst = s["slots"].long(), s["dst"].long()
    length = lens[src].long()
    used, part = (length + p - 1) // p, length % p > 0
    col = torch.arange(table.shape[1], device=src.device)[None]
    rows = table[src]
    last = part[:, None] & (col == used[:, None] - 1)
    whole = (col < used[:, None]) & ~last
    old = rows[last].long()
    new = (refs == 0).nonzero().flatten()[:old.numel()]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), whole.int().flatten())
    refs[new] = 1
    rows[last] = new.int()
    table[dst] = torch.where(col < used[:, None], rows, table[dst])
    lens[dst] = length.int()
    _copy_pages(s, old, new)


def _plain_compact(s):
    p, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    ids = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    count = live.sum()
    high, hole = (live & (ids >= count)).nonzero().flatten(), (~live & (ids < count)).nonzero().flatten()
    place = ids.int()
    place[high] = hole.int()
    used = (lens.long() + p - 1) // p
    valid = torch.arange(table.shape[1], device=refs.device)[None] < used[:, None]
    table.copy_(torch.where(valid, place[table.clamp(min=0).long()], table))
    refs[hole] = refs[high]
    refs[high] = 0
    s["live"].copy_(count)
    _copy_pages(s, high, hole)


PLAIN = dict(attention=_plain_attention, append=_plain_append, resize=_plain_resize, fork=_plain_fork,
             compact=_plain_compact)


# ------------------------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    p, op = c["page"], c["op"]
    raw, dtype = s["codes"].view(torch.uint8), s["codes"].dtype
    table, lens, slots = s["table"].tolist(), s["lens"].tolist(), s["slots"].tolist()
    if op == "attention":
        out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.zeros_like(s["lse"], dtype=torch.float64)
        cu = s["cu"].tolist()
        group = c["heads"] // c["kv_heads"]
        for i, slot in enumerate(slots):
            a, b, t = cu[i], cu[i + 1], lens[slot]
            if a == b:
                continue
            ids = torch.tensor(table[slot][:_up(t, p)], device="cuda")
            for j in range(c["kv_heads"]):
                x = raw[ids, s["layer"], :, j].view(dtype).double() * s["scales"][ids, s["layer"], :, j, None, None].double()
                k, v = x.transpose(0, 1).reshape(2, -1, c["head_dim"])[:, :t]
                q = s["q"][a:b, j * group:(j + 1) * group].double()
                z = torch.einsum("qgd,td->qgt", q, k) * c["head_dim"] ** -0.5
                later = torch.arange(t, device="cuda")[None] > torch.arange(t - (b - a), t, device="cuda")[:, None]
                z.masked_fill_(later[:, None], -math.inf)
                lse[a:b, j * group:(j + 1) * group] = torch.logsumexp(z, -1)
                out[a:b, j * group:(j + 1) * group] = torch.einsum("qgt,td->qgd", torch.softmax(z, -1), v)
        return {"out": out, "lse": lse}
    scales = s["scales"].double()
    if op == "append":
        val, lim, y = raw.view(dtype).double(), INT8_MAX if dtype == torch.int8 else E4M3_MAX, s["layer"]
        cu = s["cu"].tolist()
        for i, slot in enumerate(slots):
            pos, end = lens[slot] - (cu[i + 1] - cu[i]), lens[slot]
            row = cu[i]
            while pos < end:
                page, off, m = table[slot][pos // p], pos % p, min(p - pos % p, end - pos)
                x = torch.stack([s["k"][row:row + m], s["v"][row:row + m]]).double().transpose(1, 2)  # [2, kv, m, d]
                top = x.abs().amax((2, 3))
                need = (2.0 ** torch.arange(-126, 128, dtype=torch.float64)).to("cuda")
                need = need[(top[..., None] > lim * need).sum(-1)]
                was = scales[page, y]
                now = need if off == 0 else torch.maximum(was, need)
                if off:
                    val[page, y] = _nearest(val[page, y] * (was / now)[..., None, None], dtype)
                val[page, y, :, :, off:off + m] = _nearest(x / now[..., None, None], dtype)
                scales[page, y] = now
                pos, row = pos + m, row + m
        return {"codes": val.to(torch.int8) if dtype == torch.int8 else val, "scales": scales}
    refs, src, dst = s["refs"].tolist(), [], []
    live = None
    if op == "resize":
        new = s["new"].tolist()
        keep = [min(lens[x], t) for x, t in zip(slots, new)]
        copy = [k % p > 0 and refs[table[x][k // p]] > 1 for x, k in zip(slots, keep)]
        for x, t in zip(slots, new):
            for j in range(_up(t, p), _up(lens[x], p)):
                refs[table[x][j]] -= 1
                table[x][j] = -1
        free = iter([i for i, r in enumerate(refs) if r == 0])
        for x, t, k, y in zip(slots, new, keep, copy):
            for j in ([k // p] if y else []) + list(range(_up(lens[x], p), _up(t, p))):
                if y and j == k // p:
                    src.append(table[x][j])
                    dst.append(next(free))
                    table[x][j] = dst[-1]
                else:
                    table[x][j] = next(free)
                refs[table[x][j]] = 1
            lens[x] = t
        for q in src:
            refs[q] -= 1
    elif op == "fork":
        free = iter([i for i, r in enumerate(refs) if r == 0])
        for x, y in zip(slots, s["dst"].tolist()):
            for j in range(_up(lens[x], p)):
                table[y][j] = table[x][j]
                if (j + 1) * p > lens[x]:
                    table[y][j] = next(free)
                    src.append(table[x][j])
                    dst.append(table[y][j])
                refs[table[y][j]] += 1
            lens[y] = lens[x]
    else:
        live = sum(r > 0 for r in refs)
        src = [i for i, r in enumerate(refs) if r > 0 and i >= live]
        dst = [i for i, r in enumerate(refs) if r == 0 and i < live]
        to = dict(zip(src, dst))
        for x, t in enumerate(lens):
            for j in range(_up(t, p)):
                table[x][j] = to.get(table[x][j], table[x][j])
        for a, b in to.items():
            refs[b], refs[a] = refs[a], 0
    src, dst = torch.tensor(src, device="cuda", dtype=torch.long), torch.tensor(dst, device="cuda", dtype=torch.long)
    raw[dst], scales[dst] = raw[src], scales[src]
    s["refs"].copy_(torch.tensor(refs))
    s["lens"].copy_(torch.tensor(lens))
    s["table"].copy_(torch.tensor(table))
    res = {"codes": raw, "scales": scales, "meta": s["meta"]}
    if live is not None:
        res["live"] = torch.tensor([live], dtype=torch.int32)
    return res


def _nearest(x, dtype):
    """Nearest code's value, ties to even."""
    if dtype == torch.int8:
        return torch.round(x)
    _, e = torch.frexp(x)
    step = _two((e - 4).clamp(min=-9)).double()  # three bits behind the leading one; 2^-9 is the smallest
    return torch.round(x / step) * step
