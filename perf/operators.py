"""Measured cases of the batch operators: attention over packed prompts, the 4-bit page cache, and eviction.

Six kinds of call, each with its plain form in elementary torch operations (32 bits, rounded once at the
end) and the framework's own call:

- ``prompt``: causal attention of packed prompts over their own 16-bit K and V (out, lse)
- ``prompt_weights``: the attention weight that every key of those prompts received, summed over rows and
  the query heads of its kv head (optionally over the last rows of each prompt only)
- ``append``: K and V rows encoded as Q4_0 into pages of the cache, and read back as values
- ``attend``: decode or span attention of a batch of sequences over the 4-bit cache (out, lse)
- ``weights``: the attention weight that every cached token received from those rows, added to a running sum
- ``evict``: per sequence and kv head, the tokens of largest accumulated weight (with the first and the most
  recent ones always) are kept, compacted in order into other pages, and read back as values
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a burst of short chat prompts, ragged down to one token, on the 24 / 4 head, 256-wide layer of the
        # decode benchmark: launch latency and ragged tiles
        dict(name="prompt_short", kind="prompt", lens="1,37,300,211,128", hq=24, hk=4, d=256, dtype="f16"),
        # an ordinary prefill batch of long and short documents, 128-wide heads: tensor-core throughput
        dict(name="prompt_long", kind="prompt", lens="8192,6001,2048,513,1", hq=32, hk=8, d=128, dtype="bf16"),
        # accumulated weight over every row of a prefill batch, as eviction by total weight needs it
        dict(name="prompt_weights_all", kind="prompt_weights", lens="4096,2500,700,33", hq=32, hk=8, d=128,
             dtype="bf16", window=0),
        # the last 64 rows as an observation window over one long prompt
        dict(name="prompt_weights_window", kind="prompt_weights", lens="32768", hq=24, hk=4, d=256, dtype="f16",
             window=64),
        # one decode step of 64 sequences: one new token each, scattered over the pages
        dict(name="append_step", kind="append", lens=",".join(["1"] * 64), hk=8, d=128, page=64, dtype="f16"),
        # the cache filled from prompts: whole pages and ragged ends
        dict(name="append_prompt", kind="append", lens="16384,5000,777", hk=4, d=256, page=256, dtype="bf16"),
        # one sequence, one row, the single-layer geometry of the framework's decode benchmark: latency
        dict(name="attend_one", kind="attend", lens="4096", rows=1, hq=8, hk=2, d=128, page=256, dtype="f32"),
        # a serving batch of mixed lengths with a finished (empty) slot: cache bandwidth
        dict(name="attend_batch", kind="attend",
             lens="32768,30011,28500,25000,21777,20000,18123,16384,15000,12345,11000,9000,8192,7001,6000,5123,"
                  "4096,3500,3001,2500,2048,1500,1024,900,700,513,300,128,64,17,1,0",
             rows=1, hq=32, hk=8, d=128, page=64, dtype="bf16"),
        # one sequence's step that also keeps the running weights
        dict(name="weights_one", kind="weights", lens="4096", rows=1, hq=8, hk=2, d=128, page=256, dtype="f32"),
        # a 4-row verify step of long sequences that also keeps the running weights
        dict(name="weights_batch", kind="weights", lens="65536,40001,20000,4097,33,0", rows=4, hq=24, hk=4, d=256,
             page=256, dtype="f16"),
        # one sequence cut back to a quarter
        dict(name="evict_one", kind="evict", lens="4096", hk=2, d=128, page=64, keep=1024, sinks=4, recent=64),
        # a batch cut back to one budget, the short ones below it
        dict(name="evict_batch", kind="evict", lens="131072,65536,40000,32768,20001,9000,4096,700", hk=8, d=128,
             page=64, keep=4096, sinks=4, recent=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt_weights", "append", "attend", "weights", "evict"])
    d = rng.choice([64, 128, 256])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 6, 8])
    page = rng.choice([32, 64, 128, 256])
    n = _log_int(rng, 1, 24)
    if kind in ("prompt", "prompt_weights"):
        top = 4096 if hq * d <= 4096 else 1024
        case = dict(kind=kind, lens=",".join(str(_log_int(rng, 1, top)) for _ in range(min(n, 8))), hq=hq, hk=hk, d=d,
                    dtype=rng.choice(["f16", "bf16"]))
        if kind == "prompt_weights":
            case["window"] = rng.choice([0, 0, 1, 32, 100])
    elif kind == "append":
        case = dict(kind=kind, lens=",".join(str(_log_int(rng, 1, 600)) for _ in range(n)), hk=hk, d=d, page=page,
                    dtype=rng.choice(["f32", "f16", "bf16"]))
    elif kind in ("attend", "weights"):
        case = dict(kind=kind, lens=",".join(str(_log_int(rng, 1, 8192)) for _ in range(n)), hq=hq, hk=hk, d=d,
                    rows=rng.choice([1, 1, 2, 3, 5, 8]), page=page, dtype=rng.choice(["f32", "f16", "bf16"]))
    else:
        keep = _log_int(rng, 16, 2048)
        sinks = rng.choice([0, 1, 4])
        recent = rng.randint(0, keep // 2 - sinks)
        case = dict(kind=kind, lens=",".join(str(_log_int(rng, 1, 20000)) for _ in range(min(n, 10))), hk=hk, d=d,
                    page=page, keep=keep, sinks=sinks, recent=recent)
    return case


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------------------------------------ 4-bit pages
# A page holds, per kv head, page_tokens / 32 tiles of 36 d bytes: K codes (16 d bytes), K scales (2 d bytes),
# V codes, V scales.  Codes are Q4_0 blocks of 32 dims: byte j holds dims j (low nibble) and j + 16.

def _orders(d, device):
    """Byte offset in its part of a tile of byte j of block b of token t, for K and V codes, and half index of their scales."""
    nb = d // 32
    t = torch.arange(32, device=device).view(32, 1, 1)
    b = torch.arange(nb, device=device).view(1, nb, 1)
    j = torch.arange(16, device=device).view(1, 1, 16)
    u = (t // 8) * nb + b
    kc = ((u // 4) * 32 + (t % 8) * 4 + j // 4) * 16 + (u % 4) * 4 + j % 4
    x = t % 16
    w = ((t // 16) * nb + b) * 2 + x % 4 // 2
    vc = ((w // 4) * 32 + (j % 8) * 4 + x // 4) * 16 + (w % 4) * 4 + (x % 2) * 2 + j // 8
    ks = ((t // 16 * 8 + t % 8) * nb + b) * 2 + t // 8 % 2
    vs = ((t // 4) * nb + b) * 4 + t % 4
    return kc.reshape(-1), vc.reshape(-1), ks.reshape(-1), vs.reshape(-1)


def _quantise(x):
    """Q4_0 of the last axis in 32 bits: codes (uint8) and fp16 scales."""
    blk = x.float().unflatten(-1, (-1, 32))
    mag = blk.abs()
    peak = mag.amax(-1, keepdim=True)
    at = torch.arange(32, device=x.device)
    first = torch.where(mag == peak, at, 32).amin(-1, keepdim=True)
    scale = blk.gather(-1, first) / -8.0
    inv = torch.where(scale != 0, 1.0 / scale, torch.zeros_like(scale))
    codes = torch.trunc(blk * inv + 8.5).clamp(0, 15).to(torch.uint8)
    return codes, scale.squeeze(-1).half()


def _tiles(k, v):
    """Tiles [n, 36 d] (uint8) of K and V rows [n, 32, d]."""
    n, _, d = k.shape
    kc, vc, ks, vs = _orders(d, k.device)
    out = torch.empty((n, 36 * d), dtype=torch.uint8, device=k.device)
    for x, code_at, scale_at, order, sc in ((k, 0, 16 * d, kc, ks), (v, 18 * d, 34 * d, vc, vs)):
        codes, scales = _quantise(x)
        byte = (codes[..., :16] | (codes[..., 16:] << 4)).reshape(n, -1)
        part = torch.empty_like(byte)
        part[:, order] = byte
        out[:, code_at:code_at + 16 * d] = part
        half = torch.empty((n, d), dtype=torch.float16, device=k.device)
        half[:, sc] = scales.reshape(n, -1)
        out[:, scale_at:scale_at + 2 * d] = half.view(torch.uint8)
    return out


def _values(tiles, d):
    """K and V values (fp32) [..., 32, d] of tiles [..., 36 d]."""
    kc, vc, ks, vs = _orders(d, tiles.device)
    got = []
    for code_at, scale_at, order, sc in ((0, 16 * d, kc, ks), (18 * d, 34 * d, vc, vs)):
        byte = tiles[..., code_at:code_at + 16 * d][..., order].unflatten(-1, (32, d // 32, 16))
        codes = torch.cat([byte & 15, byte >> 4], -1).float() - 8.0
        scale = tiles[..., scale_at:scale_at + 2 * d].contiguous().view(torch.float16)[..., sc].float()
        got.append((codes * scale.unflatten(-1, (32, d // 32)).unsqueeze(-1)).flatten(-2))
    return got


def _paged(pages, table, page, hk, d):
    """K and V values [n, hk, width * page, d] of the table's pages."""
    t = pages.view(-1, hk, page // 32, 36 * d)[table.long().clamp(min=0)]  # n, width, hk, tiles, bytes
    return [x.permute(0, 2, 1, 3, 4, 5).flatten(2, 4) for x in _values(t, d)]


def _slots(pages, slots, page, hk, d):
    """K and V values [n, hk, d] at cache slots."""
    t = pages.view(-1, hk, page // 32, 36 * d)
    at = slots.long()
    tile = t[at // page, :, (at % page) // 32]  # n, hk, bytes
    row = (at % 32).view(-1, 1, 1, 1).expand(-1, hk, 1, d)
    return [x.gather(2, row).squeeze(2) for x in _values(tile, d)]


# ------------------------------------------------------------------------------------------------ inputs

def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32).to(dtype)


def _keys(n, hk, d, g):
    """Keys as a model makes them: channels of unequal size around a common offset, a strong first token."""
    size = torch.exp(0.4 * _randn((1, hk, d), g))
    k = _randn((n, hk, d), g) * size + 0.5 * _randn((1, hk, d), g)
    return k


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens, kind, d, hk = _lens(case), case["kind"], case["d"], case["hk"]
    dt = _TYPES[case.get("dtype", "f16")]
    st = dict(case=case, lens=lens)
    if kind in ("prompt", "prompt_weights"):
        n = sum(lens)
        st["q"] = (1.5 * _randn((n, case["hq"], d), g)).to(dt)
        st["k"] = _keys(n, hk, d, g).to(dt)
        st["v"] = _randn((n, hk, d), g, dt)
        st["cu"] = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device=dev)
        if kind == "prompt_weights":  # what the attention of the same prompts returned
            st["lse"] = _prompt_plain(st["q"], st["k"], st["v"], lens)[1]
        return st
    page = case["page"]
    width = max(1, max(-(-x // page) for x in lens))
    pages_used = [max(1, -(-x // page)) for x in lens]
    n_pages = sum(pages_used) + 3
    if kind == "evict":
        keep_w = -(-case["keep"] // page)
        n_pages += keep_w * len(lens)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at, host = 0, perm.cpu()
    for i, u in enumerate(pages_used):
        table[i, :u] = host[at:at + u]
        at += u
    st["table"] = table.to(dev)
    st["lens_t"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    pages = torch.zeros(n_pages * hk * page * d * 9 // 8, dtype=torch.uint8, device=dev)
    st["pages"] = pages
    if kind == "append":
        n = sum(lens)
        st["k"] = _keys(n, hk, d, g).to(dt)
        st["v"] = _randn((n, hk, d), g, dt)
        slots = []
        for i, x in enumerate(lens):  # prompts start at their first page; single tokens inside theirs
            off = torch.arange(x) if x > 1 else torch.tensor([(i * 37) % page])
            slots.append(table[i][off // page].long() * page + off % page)
        st["slots"] = torch.cat(slots).to(dev)
        return st
    tiles = pages.view(n_pages * hk * page // 32, 36 * d)
    step = max(1, (1 << 26) // (32 * d))
    for a in range(0, tiles.shape[0], step):  # every page holds rows, as a pool in use does
        b = min(a + step, tiles.shape[0])
        tiles[a:b] = _tiles(_keys((b - a) * 32, 1, d, g).view(b - a, 32, d), _randn((b - a, 32, d), g))
    if kind in ("attend", "weights"):
        st["q"] = (1.5 * _randn((len(lens), case["rows"], case["hq"], d), g)).to(dt)
        if kind == "weights":
            st["sum"] = torch.rand((len(lens), hk, width * page), generator=g, device=dev)
            st["lse"] = _attend_plain(st)[1]
    else:
        st["dst"] = host[at:at + keep_w * len(lens)].view(len(lens), keep_w).to(dev)
        w = torch.exp(2.0 * _randn((len(lens), hk, width * page), g))
        # tokens no row ever looked at tie at zero
        st["weights"] = torch.where(torch.rand(w.shape, generator=g, device=dev) < 0.1, torch.zeros_like(w), w)
        off = torch.cat([torch.arange(min(x, case["keep"]), device=dev) for x in lens])
        seq = torch.cat([torch.full((min(x, case["keep"]),), i, device=dev) for i, x in enumerate(lens)])
        st["dst_slots"] = st["dst"][seq, off // page].long() * page + off % page
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _prompt_scores(q, k, scale):
    """Masked scores [hk, group, L, L] of one prompt, in 32 bits."""
    n, hq, d = q.shape
    hk = k.shape[1]
    qf = q.float().transpose(0, 1).reshape(hk, -1, d)
    s = torch.matmul(qf, k.float().permute(1, 2, 0)).mul_(scale).view(hk, hq // hk, n, n)
    at = torch.arange(n, device=q.device)
    return s.masked_fill_(at[None, :] > at[:, None], -math.inf)


def _prompt_plain(q, k, v, lens):
    scale = 1.0 / math.sqrt(q.shape[-1])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    a = 0
    for n in lens:  # the packed prompts do not attend to one another
        b = a + n
        s = _prompt_scores(q[a:b], k[a:b], scale)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), v[a:b].float().transpose(0, 1)).view(*p.shape[:3], -1) / total
        out[a:b] = o.flatten(0, 1).transpose(0, 1).to(q.dtype)
        lse[a:b] = (total.log() + top).squeeze(-1).flatten(0, 1).transpose(0, 1)
        a = b
    return out, lse


def _prompt_weights_plain(st):
    q, k, lens, lse = st["q"], st["k"], st["lens"], st["lse"]
    scale, hk = 1.0 / math.sqrt(q.shape[-1]), k.shape[1]
    w = torch.zeros((len(lens), hk, max(lens)), dtype=torch.float32, device=q.device)
    a = 0
    for i, n in enumerate(lens):
        b = a + n
        r = max(0, n - st["case"]["window"]) if st["case"]["window"] else 0
        s = torch.matmul(q[a + r:b].float().transpose(0, 1).reshape(hk, -1, q.shape[-1]), k[a:b].float().permute(1, 2, 0))
        s = s.mul_(scale).view(hk, -1, n - r, n)
        at = torch.arange(n, device=q.device)
        s.masked_fill_(at[None, :] > at[r:, None], -math.inf)
        s -= lse[a + r:b].transpose(0, 1).reshape(hk, -1, n - r, 1)
        w[i, :, :n] = s.exp_().sum((1, 2))
        a = b
    return w


def _cache_scores(st, keys):
    """Masked scores [n, hk, group, rows, tokens]: row r of the last `rows` sees the tokens up to its own."""
    c, q = st["case"], st["q"]
    n, rows, hq, d = q.shape
    hk = c["hk"]
    qf = q.float().permute(0, 2, 1, 3).reshape(n, hk, -1, d)
    s = torch.matmul(qf, keys.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, hk, hq // hk, rows, -1)
    last = st["lens_t"].long()[:, None] - rows + torch.arange(rows, device=q.device)
    hide = torch.arange(s.shape[-1], device=q.device) > last[..., None]
    return s.masked_fill_(hide[:, None, None], -math.inf)


def _attend_plain(st):
    c, q = st["case"], st["q"]
    keys, vals = _paged(st["pages"], st["table"], c["page"], c["hk"], c["d"])
    s = _cache_scores(st, keys)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), vals).view(*p.shape[:4], -1) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (total.log() + top).squeeze(-1)
    n, hk, grp, rows, d = o.shape
    return o.permute(0, 3, 1, 2, 4).reshape(n, rows, hk * grp, d).to(q.dtype), lse.permute(0, 3, 1, 2).reshape(n, rows, -1)


def _weights_plain(st):
    c = st["case"]
    keys, _ = _paged(st["pages"], st["table"], c["page"], c["hk"], c["d"])
    s = _cache_scores(st, keys)
    n, hk, grp, rows, _ = s.shape
    lse = st["lse"].view(n, rows, hk, grp).permute(0, 2, 3, 1).unsqueeze(-1)
    p = torch.where(lse.isinf(), torch.zeros_like(s), (s - lse).exp_())
    return st["sum"] + p.sum((2, 3))


def _append_plain(st):
    c = st["case"]
    hk, d, page = c["hk"], c["d"], c["page"]
    kc, vc, ks, vs = (x.view(32, -1) for x in _orders(d, st["k"].device))
    tiles = st["pages"].view(-1, hk, page // 32, 36 * d)
    at = st["slots"]
    row = (at % 32).view(-1, 1, 1)
    base = (at // page).view(-1, 1, 1), torch.arange(hk, device=at.device).view(1, -1, 1), ((at % page) // 32).view(-1, 1, 1)
    for x, code_at, scale_at, order, sc in ((st["k"], 0, 16 * d, kc, ks), (st["v"], 18 * d, 34 * d, vc, vs)):
        codes, scales = _quantise(x)
        tiles[(*base, code_at + order[row.flatten()].unsqueeze(1))] = (codes[..., :16] | (codes[..., 16:] << 4)).flatten(2)
        where = scale_at + 2 * sc[row.flatten()].unsqueeze(1)
        raw = scales.contiguous().view(torch.uint8).unflatten(-1, (-1, 2))
        tiles[(*base, where)] = raw[..., 0]
        tiles[(*base, where + 1)] = raw[..., 1]
    k, v = _slots(st["pages"], at, page, hk, d)
    return k.half(), v.half()


def _evict_plain(st):
    c, w = st["case"], st["weights"]
    hk, d, page, keep = c["hk"], c["d"], c["page"], c["keep"]
    n, _, width = w.shape
    at = torch.arange(width, device=w.device)
    lens = st["lens_t"].long().view(-1, 1, 1)
    rank = torch.where((at < c["sinks"]) | (at >= lens - c["recent"]), torch.full_like(w, math.inf), w)
    rank = torch.where(at < lens, rank, torch.full_like(w, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]  # ties: the lowest index
    if order.shape[-1] < keep:
        order = torch.cat([order, order.new_full((n, hk, keep - order.shape[-1]), width)], -1)
    kept = torch.sort(torch.where(order < lens, order, width), dim=-1).values
    there = kept < lens
    new_lens = st["lens_t"].clamp(max=keep)
    safe = torch.where(there, kept, 0)
    new_w = torch.where(there, w.gather(2, safe.clamp(max=width - 1)), torch.zeros((), device=w.device))
    # the kept tokens' values, in their new order
    src = st["table"].long().gather(1, (safe // page).flatten(1)).view(n, hk, keep) * page + safe % page
    tiles = st["pages"].view(-1, hk, page // 32, 36 * d)
    head = torch.arange(hk, device=w.device).view(1, hk, 1)
    kc, vc, ks, vs = (x.view(32, -1) for x in _orders(d, w.device))
    dst = (st["dst"].long().gather(1, (torch.arange(keep, device=w.device) // page).expand(n, -1)) * page
           + torch.arange(keep, device=w.device) % page).unsqueeze(1).expand(n, hk, keep)
    src, dst, head = src[there], dst[there], head.expand(n, hk, keep)[there]
    for order, first, count in ((kc, 0, 16 * d), (vc, 18 * d, 16 * d)):
        got = tiles[(src // page).unsqueeze(1), head.unsqueeze(1), (src % page // 32).unsqueeze(1), first + order[src % 32]]
        tiles[(dst // page).unsqueeze(1), head.unsqueeze(1), (dst % page // 32).unsqueeze(1), first + order[dst % 32]] = got
    halves = st["pages"].view(torch.float16).view(-1, hk, page // 32, 18 * d)
    for first, sc in ((8 * d, ks), (17 * d, vs)):
        got = halves[(src // page).unsqueeze(1), head.unsqueeze(1), (src % page // 32).unsqueeze(1), first + sc[src % 32]]
        halves[(dst // page).unsqueeze(1), head.unsqueeze(1), (dst % page // 32).unsqueeze(1), first + sc[dst % 32]] = got
    k, v = _slots(st["pages"], st["dst_slots"], page, hk, d)
    return torch.where(there, kept, -1).int(), new_lens, new_w, k.half(), v.half()


# ------------------------------------------------------------------------------------------------ the framework's calls

def _cache(st):
    """The cache handle that a user's program keeps beside its pages."""
    if "cache" not in st:
        from host_streamed_paged_gb300 import kvs
        c = st["case"]
        st["cache"] = kvs.Q4Cache(pages=st["pages"], page_tokens=c["page"], n_kv_head=c["hk"], head_dim=c["d"])
    return st["cache"]


def _run_own(st):
    from host_streamed_paged_gb300 import kvs
    c = st["case"]
    kind = c["kind"]
    if kind == "prompt":
        return kvs.prompt_attend(st["q"], st["k"], st["v"], st["cu"])
    if kind == "prompt_weights":
        return kvs.prompt_weights(st["q"], st["k"], st["lse"], st["cu"], max(st["lens"]), window=c["window"])
    cache = _cache(st)
    if kind == "append":
        cache.append(st["slots"], st["k"], st["v"])
        return cache.read(st["slots"], torch.float16)
    if kind == "attend":
        return cache.attend(st["table"], st["lens_t"], st["q"])
    if kind == "weights":
        return cache.weights(st["table"], st["lens_t"], st["q"], st["lse"].contiguous(), prev=st["sum"])
    kept, lens, w = cache.evict(st["table"], st["dst"], st["lens_t"], st["weights"], c["keep"], sinks=c["sinks"],
                                recent=c["recent"])
    k, v = cache.read(st["dst_slots"], torch.float16)
    return kept, lens, w, k, v


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind == "prompt":
        return _prompt_plain(state["q"], state["k"], state["v"], state["lens"])
    if kind == "prompt_weights":
        return _prompt_weights_plain(state)
    return {"append": _append_plain, "attend": _attend_plain, "weights": _weights_plain, "evict": _evict_plain}[kind](state)


# ------------------------------------------------------------------------------------------------ work and exact values

def work(case):
    lens, kind, d, hk = _lens(case), case["kind"], case["d"], case["hk"]
    e = _BYTES[case.get("dtype", "f16")]
    n = sum(lens)
    tok = hk * d * 9 // 8  # bytes of one cached token, K and V
    if kind == "prompt":
        pairs = sum(x * (x + 1) // 2 for x in lens)
        return dict(bytes=n * (2 * case["hq"] + 2 * hk) * d * e + 4 * n * case["hq"], flops=4 * pairs * d * case["hq"])
    if kind == "prompt_weights":
        win = case["window"]
        rows = [min(x, win) if win else x for x in lens]
        pairs = sum(r * x - r * (r - 1) // 2 for r, x in zip(rows, lens))
        return dict(bytes=sum(rows) * case["hq"] * (d * e + 4) + n * hk * d * e + 4 * hk * max(lens) * len(lens),
                    flops=2 * pairs * d * case["hq"])
    if kind == "append":  # rows in, codes and scales out and in, values out
        return dict(bytes=n * hk * d * 2 * e + 2 * n * tok + n * hk * d * 2 * 2 + 16 * n, flops=12 * n * hk * d)
    if kind in ("attend", "weights"):
        rows, hq = case["rows"], case["hq"]
        pairs = sum(max(0, x - rows + r + 1) for x in lens for r in range(rows))
        q = len(lens) * rows * hq
        if kind == "attend":
            return dict(bytes=n * tok + q * (2 * d * e + 4), flops=4 * pairs * hq * d)
        width = -(-max(1, max(lens)) // case["page"]) * case["page"]
        return dict(bytes=n * tok // 2 + q * (d * e + 4) + 8 * len(lens) * hk * width, flops=2 * pairs * hq * d)
    kept = sum(min(x, case["keep"]) for x in lens)
    # every weight in; the kept tokens in, out, and out as values; their indices and weights
    return dict(bytes=4 * n * hk + 3 * kept * tok + 4 * kept * hk * d + 12 * len(lens) * hk * case["keep"], flops=8 * n * hk)


def _exact_values(tiles, d):
    """K and V values (float64) [n, 32, d] of whole tiles, read nibble by nibble."""
    nb = d // 32
    out = []
    for kind in (0, 1):
        base = 18 * d * kind
        scales = tiles[:, base + 16 * d:base + 18 * d].contiguous().view(torch.float16).double()
        val = torch.empty((tiles.shape[0], 32, d), dtype=torch.float64, device=tiles.device)
        for t in range(32):
            for b in range(nb):
                half = ((t // 16 * 8 + t % 8) * nb + b) * 2 + t // 8 % 2 if kind == 0 else ((t // 4) * nb + b) * 4 + t % 4
                s = scales[:, half, None]
                offs = []
                for j in range(16):
                    if kind == 0:
                        u = (t // 8) * nb + b
                        offs.append(((u // 4) * 32 + (t % 8) * 4 + j // 4) * 16 + (u % 4) * 4 + j % 4)
                    else:
                        u = ((t // 16) * nb + b) * 2 + t % 4 // 2
                        offs.append(((u // 4) * 32 + (j % 8) * 4 + t % 16 // 4) * 16 + (u % 4) * 4 + (t % 2) * 2 + j // 8)
                raw = tiles[:, torch.tensor(offs, device=tiles.device) + base].to(torch.int32)
                val[:, t, b * 32:b * 32 + 16] = (raw % 16 - 8) * s
                val[:, t, b * 32 + 16:b * 32 + 32] = (raw // 16 - 8) * s
        out.append(val)
    return out


def _exact_prompt(q, k, v, lens, window, lse_in=None):
    """One query head at a time, in 64 bits: (out, lse), or the weights under the given lse."""
    n, hq, d = q.shape
    hk = k.shape[1]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((n, hq), dtype=torch.float64, device=q.device)
    w = torch.zeros((len(lens), hk, max(lens)), dtype=torch.float64, device=q.device)
    first = 0
    for i, x in enumerate(lens):
        for h in range(hq):
            kk, vv = k[first:first + x, h // (hq // hk)].double(), v[first:first + x, h // (hq // hk)].double()
            for r0 in range(0, x, 2048):
                r1 = min(x, r0 + 2048)
                s = q[first + r0:first + r1, h].double() @ kk[:r1].T / math.sqrt(d)
                s = s + torch.triu(torch.full((r1 - r0, r1), -math.inf, dtype=torch.float64, device=q.device), r0 + 1)
                if lse_in is None:
                    z = torch.logsumexp(s, 1)
                    lse[first + r0:first + r1, h] = z
                    out[first + r0:first + r1, h] = torch.exp(s - z[:, None]) @ vv[:r1]
                else:
                    p = torch.exp(s - lse_in[first + r0:first + r1, h, None].double())
                    if window:
                        p = p[max(0, x - window - r0):]
                    w[i, h // (hq // hk), :r1] += p.sum(0)
        first += x
    return (out, lse) if lse_in is None else w


def exact(case, seed):
    kind, d, hk = case["kind"], case["d"], case["hk"]
    if kind in ("prompt", "prompt_weights") and work(case)["flops"] > 2e12:
        return None
    st = prepare(case, seed)
    lens = st["lens"]
    if kind == "prompt":
        return _exact_prompt(st["q"], st["k"], st["v"], lens, 0)
    if kind == "prompt_weights":
        return _exact_prompt(st["q"], st["k"], st["v"], lens, case["window"], st["lse"])
    if kind == "append":  # the format is defined by its 32-bit steps; the values that it holds are exact
        import numpy as np
        got = []
        for name in ("k", "v"):
            x = st[name].float().cpu().numpy().reshape(-1, 32)
            pos = np.abs(x).argmax(1)  # the first of equal ones
            dd = x[np.arange(len(x)), pos] / np.float32(-8)
            with np.errstate(divide="ignore", invalid="ignore"):
                inv = np.where(dd != 0, np.float32(1) / dd, np.float32(0)).astype(np.float32)
            code = np.minimum(15, np.floor((x * inv[:, None]).astype(np.float32) + np.float32(8.5)))
            val = (code.astype(np.float64) - 8) * dd.astype(np.float16).astype(np.float64)[:, None]
            got.append(torch.from_numpy(val.reshape(st[name].shape)))
        return tuple(got)
    page = case["page"]
    tiles = st["pages"].view(-1, hk, page // 32, 36 * d)
    if kind in ("attend", "weights"):
        q, rows, hq = st["q"].double(), case["rows"], case["hq"]
        grp = hq // hk
        out, lse = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
        w = st["sum"].double() if kind == "weights" else None
        for i, x in enumerate(lens):
            used = st["table"][i, :max(1, -(-x // page))].long()
            for h in range(hk):
                kk, vv = _exact_values(tiles[used, h].flatten(0, 1), d)
                kk, vv = kk.flatten(0, 1)[:x], vv.flatten(0, 1)[:x]
                for r in range(rows):
                    see = max(0, x - rows + r + 1)
                    s = q[i, r, h * grp:(h + 1) * grp] @ kk[:see].T / math.sqrt(d)
                    if kind == "weights":
                        if see:
                            w[i, h, :see] += torch.exp(s - st["lse"][i, r, h * grp:(h + 1) * grp, None].double()).sum(0)
                        continue
                    z = torch.logsumexp(s, 1) if see else torch.full((grp,), -math.inf, dtype=torch.float64, device=q.device)
                    lse[i, r, h * grp:(h + 1) * grp] = z
                    if see:
                        out[i, r, h * grp:(h + 1) * grp] = torch.exp(s - z[:, None]) @ vv[:see]
        return w if kind == "weights" else (out, lse)
    keep, sinks, recent = case["keep"], case["sinks"], case["recent"]
    kept = torch.full((len(lens), hk, keep), -1, dtype=torch.int32)
    new_w = torch.zeros((len(lens), hk, keep), dtype=torch.float64)
    ks, vs = [], []
    for i, x in enumerate(lens):
        m = min(x, keep)
        seq_k, seq_v = torch.empty((m, hk, d), dtype=torch.float64), torch.empty((m, hk, d), dtype=torch.float64)
        for h in range(hk):
            vals = st["weights"][i, h, :x].double().cpu().numpy()
            forced = [t for t in range(x) if t < sinks or t >= x - recent] if x > keep else list(range(x))
            chosen = set(forced[:keep])
            if len(chosen) < m:
                import numpy as np
                for t in np.lexsort((np.arange(x), -vals)):
                    if len(chosen) == m:
                        break
                    chosen.add(int(t))
            idx = torch.tensor(sorted(chosen), dtype=torch.long)
            kept[i, h, :m] = idx.int()
            new_w[i, h, :m] = torch.from_numpy(vals)[idx]
            dev = idx.to(tiles.device)
            used = st["table"][i, :max(1, -(-x // page))].long()
            kk, vv = _exact_values(tiles[used, h].flatten(0, 1), d)
            seq_k[:, h], seq_v[:, h] = kk.flatten(0, 1)[dev].cpu(), vv.flatten(0, 1)[dev].cpu()
        ks.append(seq_k)
        vs.append(seq_v)
    return kept, torch.tensor([min(x, keep) for x in lens], dtype=torch.int32), new_w, torch.cat(ks), torch.cat(vs)


def _self_check():
    """Small cases of every kind on this machine: the plain forms against the exact values."""
    rng = random.Random(1)
    for _ in range(40):
        c = draw(rng)
        c["lens"] = ",".join(str(1 + int(x) % 90) for x in c["lens"].split(",")[:3])
        if c["kind"] == "evict":
            c.update(keep=24, sinks=min(2, c["sinks"]), recent=5)
        got, want = run(prepare(c, 3)), exact(c, 3)
        got, want = (x if isinstance(x, tuple) else (x,) for x in (got, want))
        for a, b in zip(got, want):
            a, b = a.double().cpu(), b.double().cpu()
            fin = torch.isfinite(b)
            assert torch.equal(fin, torch.isfinite(a)), c
            assert (a[fin] - b[fin]).norm() <= 4e-3 * b[fin].norm() + 1e-30, c


if __name__ == "__main__":
    _self_check()
    print("plain forms agree with the exact values")
