"""Measured cases of the operators around the caches: query and key preparation, chunks over the 4-bit cache, windows.

Six kinds of call, each with its plain form in elementary torch operations (32 bits, angles in 64, rounded once at
the end) and the framework's own call:

- ``rotate``: rotary positions of query and key rows: pairs of neighbours or of halves, the whole head or its first
  part, frequencies as they are or scaled for long contexts
- ``norm_rotate``: the norm of every head's query and key first (root mean square, a weight per dim), the same rotation
  after it
- ``chunk``: attention of a packed batch of chunks (new rows of each sequence, one to thousands) over the 4-bit cache
- ``window_chunk``: the same where a row sees the last ``window`` tokens up to its own and the first ``sinks``
- ``window_prompt``: packed prompts over themselves under such a window (out, lse)
- ``window_step``: decode or span rows of a batch over the 4-bit cache under such a window (out, lse)
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_BASE = 500000.0  # of the rotary frequencies
_CONTEXT = 8192   # that scaled frequencies were trained for


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences at scattered positions: launch latency
        dict(name="rotate_step", kind="rotate", rows=64, hq=32, hk=8, d=128, rot=128, pairs="halves", scaling="none",
             top=131072, dtype="bf16"),
        # a long prefill batch of the wide-headed layer, a quarter of the head rotated, frequencies scaled for a long
        # context and positions to match: bandwidth
        dict(name="rotate_prompt", kind="rotate", rows=16755, hq=24, hk=4, d=256, rot=64, pairs="neighbours", scaling="yarn",
             top=1048576, dtype="f16"),
        # one token of the single-layer geometry of the framework's decode benchmark: latency
        dict(name="norm_rotate_one", kind="norm_rotate", rows=1, hq=8, hk=2, d=128, rot=128, pairs="halves", scaling="none",
             top=4096, dtype="f32"),
        # a prefill batch of a layer with normed queries and keys: bandwidth
        dict(name="norm_rotate_prompt", kind="norm_rotate", rows=12001, hq=32, hk=8, d=128, rot=128, pairs="halves",
             scaling="bands", top=131072, dtype="bf16"),
        # one short turn of a chat on top of a cached history: latency
        dict(name="chunk_one", kind="chunk", rows="37", past="4059", hq=8, hk=2, d=128, page=256, dtype="f16"),
        # a serving batch that mixes prefill chunks with decode rows, a new prompt, a row of nobody and an idle sequence
        dict(name="chunk_batch", kind="chunk", rows="512,1,256,1,64,33,777,1,1,0,1,5",
             past="32256,30011,16384,20000,7001,500,0,8191,65,4096,-1,12345", hq=32, hk=8, d=128, page=64, dtype="bf16"),
        # a large prefill chunk deep in one long context: tensor-core throughput
        dict(name="chunk_long", kind="chunk", rows="2048", past="63488", hq=32, hk=8, d=128, page=64, dtype="bf16"),
        # ragged chunks of the wide-headed layer
        dict(name="chunk_wide", kind="chunk", rows="1000,129,300", past="24000,40001,0", hq=24, hk=4, d=256, page=256, dtype="f16"),
        # packed prompts under a window of 1024 with 4 sinks, longer and shorter than it
        dict(name="window_prompt", kind="window_prompt", rows="8192,6001,2048,513,1", hq=32, hk=8, d=128, window=1024, sinks=4,
             dtype="bf16"),
        # prefill chunks of sequences far longer than the window
        dict(name="window_chunk", kind="window_chunk", rows="1024,511,64,1", past="98304,20000,131000,5000", hq=32, hk=8, d=128,
             page=64, window=4096, sinks=4, dtype="bf16"),
        # one sequence's step: latency
        dict(name="window_step_one", kind="window_step", lens="8192", rows=1, hq=24, hk=4, d=256, page=256, window=1000, sinks=1,
             dtype="f16"),
        # a decode batch, most of it past the window, one sequence finished: bandwidth
        dict(name="window_step", kind="window_step",
             lens="60000,50011,48000,40001,32768,30000,28123,25000,20000,17777,16384,12345,10000,9000,8192,7000,"
                  "6001,5000,4500,4097,4096,4000,2500,1500,1024,900,513,300,128,33,1,0",
             rows=1, hq=32, hk=8, d=128, page=64, window=4096, sinks=4, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "norm_rotate", "chunk", "window_chunk", "window_prompt", "window_step"])
    d = rng.choice([64, 128, 256])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 6, 8])
    case = dict(kind=kind, hq=hq, hk=hk, d=d, dtype=rng.choice(["f16", "bf16"]))
    if kind in ("rotate", "norm_rotate"):
        case.update(rows=_log_int(rng, 1, 12000), rot=rng.choice([d, d, d // 2, d // 4, 16 * rng.randint(1, d // 16)]),
                    pairs=rng.choice(["halves", "neighbours"]), scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    top=_log_int(rng, 64, 1 << 20), dtype=rng.choice(["f32", "f16", "bf16"]))
        return case
    n = _log_int(rng, 1, 16)
    if kind != "chunk":
        case.update(window=_log_int(rng, 1, 3000), sinks=rng.choice([0, 1, 4, 40]))
    if kind == "window_prompt":
        top = 4096 if hq * d <= 4096 else 1024
        case.update(rows=",".join(str(_log_int(rng, 1, top)) for _ in range(min(n, 8))))
        return case
    case.update(page=rng.choice([32, 64, 128, 256]))
    if kind == "window_step":
        case.update(lens=",".join(str(_log_int(rng, 1, 16384)) for _ in range(n)), rows=rng.choice([1, 1, 2, 3, 5, 8]),
                    dtype=rng.choice(["f32", "f16", "bf16"]))
        return case
    top = 600 if hq * d <= 4096 else 200
    case.update(rows=",".join(str(_log_int(rng, 1, top)) for _ in range(n)),
                past=",".join(str(_log_int(rng, 1, 8192) - 1) for _ in range(n)))
    return case


def _ints(text):
    return [int(x) for x in text.split(",")]


def _chunk_lens(case):
    """Rows of each sequence and its cached tokens, the rows' own among them (past -1: a row of nobody, nothing cached)."""
    rows, past = _ints(case["rows"]), _ints(case["past"])
    return rows, [0 if p < 0 else p + r for r, p in zip(rows, past)]


# ------------------------------------------------------------------------------------------------ rotary frequencies

_SCALED = dict(none=1.0, linear=4.0, ntk=8.0, yarn=16.0, bands=8.0)


def _frequencies(case):
    """Radians per position of each pair (float64, on the host), and the factor on the rotated values."""
    rot, scaling = case["rot"], case["scaling"]
    factor, base = _SCALED[scaling], _BASE
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def at(turns):
            return rot * math.log(_CONTEXT / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    if scaling == "bands":
        turns = _CONTEXT * f / (2 * math.pi)
        smooth = ((turns - 1) / (4 - 1)).clamp(0, 1)
        return f / factor * (1 - smooth) + f * smooth, 1.0
    return f, 1.0


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


def _tiles(k, v):
    """Tiles [n, 36 d] (uint8) of K and V rows [n, 32, d], encoded as the cache does."""
    n, _, d = k.shape
    kc, vc, ks, vs = _orders(d, k.device)
    out = torch.empty((n, 36 * d), dtype=torch.uint8, device=k.device)
    for x, code_at, scale_at, order, sc in ((k, 0, 16 * d, kc, ks), (v, 18 * d, 34 * d, vc, vs)):
        blk = x.unflatten(-1, (-1, 32))
        scale = blk.gather(-1, blk.abs().argmax(-1, keepdim=True)) / -8.0
        inv = torch.where(scale != 0, 1.0 / scale, torch.zeros_like(scale))
        codes = torch.trunc(blk * inv + 8.5).clamp(0, 15).to(torch.uint8)
        part = torch.empty((n, 16 * d), dtype=torch.uint8, device=k.device)
        part[:, order] = (codes[..., :16] | (codes[..., 16:] << 4)).reshape(n, -1)
        out[:, code_at:code_at + 16 * d] = part
        half = torch.empty((n, d), dtype=torch.float16, device=k.device)
        half[:, sc] = scale.squeeze(-1).half().reshape(n, -1)
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


def _cached(st, table, tiles):
    """K and V values [n, hk, m * 32, d] of the tiles [n, m] of sequences whose page tables are `table` [n, width]."""
    c = st["case"]
    per = c["page"] // 32
    page = table.long().gather(1, (tiles // per).clamp(max=table.shape[1] - 1)).clamp(min=0)
    t = st["pages"].view(-1, c["hk"], per, 36 * c["d"])[page, :, tiles % per]  # n, m, hk, bytes
    return [x.permute(0, 2, 1, 3, 4).flatten(2, 3) for x in _values(t, c["d"])]


# ------------------------------------------------------------------------------------------------ inputs

def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32).to(dtype)


def _keys(n, hk, d, g):
    """Keys as a model makes them: channels of unequal size around a common offset."""
    size = torch.exp(0.4 * _randn((1, hk, d), g))
    return _randn((n, hk, d), g) * size + 0.5 * _randn((1, hk, d), g)


def _offsets(rows, dev):
    return torch.tensor([0] + [sum(rows[:i + 1]) for i in range(len(rows))], dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind, d, hk, hq = case["kind"], case["d"], case["hk"], case["hq"]
    dt = _TYPES[case["dtype"]]
    st = dict(case=case)
    if kind in ("rotate", "norm_rotate"):
        n = case["rows"]
        st["pos"] = torch.randint(0, case["top"], (n,), generator=g, device=dev)
        # queries and keys side by side, as one projection gives them
        both = _randn((n, hq + hk, d), g) * torch.exp(0.4 * _randn((1, hq + hk, d), g))
        both = both.to(dt)
        st["q"], st["k"] = both[:, :hq], both[:, hq:]
        freq, st["magnitude"] = _frequencies(case)
        st["freq"] = freq.to(dev)
        if kind == "norm_rotate":
            st["wq"], st["wk"] = (1 + 0.2 * _randn((d,), g)).to(dt), (1 + 0.2 * _randn((d,), g)).to(dt)
        return st
    if kind == "window_prompt":
        rows = _ints(case["rows"])
        n = sum(rows)
        st["rows"], st["cu"] = rows, _offsets(rows, dev)
        st["q"], st["k"], st["v"] = (1.5 * _randn((n, hq, d), g)).to(dt), _keys(n, hk, d, g).to(dt), _randn((n, hk, d), g, dt)
        return st
    page = case["page"]
    if kind == "window_step":
        lens, rows = _ints(case["lens"]), [case["rows"]] * len(_ints(case["lens"]))
        st["q"] = (1.5 * _randn((len(lens), case["rows"], hq, d), g)).to(dt)
    else:
        rows, lens = _chunk_lens(case)
        st["cu"] = _offsets(rows, dev)
        st["q"] = (1.5 * _randn((sum(rows), hq, d), g)).to(dt)
    st["rows"], st["lens"] = rows, lens
    width = max(1, max(-(-x // page) for x in lens))
    used = [-(-x // page) for x in lens]
    n_pages = sum(used) + 3
    host = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).cpu()
    table, at = torch.full((len(lens), width), -1, dtype=torch.int32), 0
    for i, u in enumerate(used):
        table[i, :u] = host[at:at + u]
        at += u
    st["table"] = table.to(dev)
    st["lens_t"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["pages"] = torch.zeros(n_pages * hk * page * d * 9 // 8, dtype=torch.uint8, device=dev)
    tiles = st["pages"].view(n_pages * hk * page // 32, 36 * d)
    step = max(1, (1 << 26) // (32 * d))
    for a in range(0, tiles.shape[0], step):  # every page holds rows, as a pool in use does
        b = min(a + step, tiles.shape[0])
        tiles[a:b] = _tiles(_keys((b - a) * 32, 1, d, g).view(b - a, 32, d), _randn((b - a, 32, d), g))
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _rotated(x, st):
    """Rows [n, h, d] (32 bits) with their first `rot` dims rotated; angles and their cosines in 64 bits."""
    c = st["case"]
    rot = c["rot"]
    angle = st["pos"].double()[:, None] * st["freq"]
    cos, sin = (st["magnitude"] * torch.cos(angle)).float()[:, None], (st["magnitude"] * torch.sin(angle)).float()[:, None]
    if c["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., :rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _rotate_plain(st):
    return tuple(_rotated(st[x].float(), st).to(st[x].dtype) for x in ("q", "k"))


def _norm_rotate_plain(st):
    out = []
    for name, w in (("q", "wq"), ("k", "wk")):
        x = st[name].float()
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * st[w].float()
        out.append(_rotated(x, st).to(st[name].dtype))
    return tuple(out)


def _attention(q, k, v, see):
    """Queries [n, hk, group * r, d], keys and values [n, hk, t, d], what sees what [n, r, t]: (out, lse), 32 bits."""
    n, hk, gr, d = q.shape
    s = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, hk, gr // see.shape[1], see.shape[1], -1)
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).view(*p.shape[:4], d) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (total.log() + top).squeeze(-1)


def _sees(row_pos, token, window, sinks):
    """Whether the row at position row_pos [..., r, 1] sees token [..., 1, t]."""
    see = token <= row_pos
    return see & ((token > row_pos - window) | (token < sinks)) if window else see


def _packed_queries(q, hk):
    r, hq, d = q.shape
    return q.float().transpose(0, 1).reshape(1, hk, hq // hk * r, d)


def _chunk_plain(st):
    c, q, out = st["case"], st["q"], torch.zeros_like(st["q"])
    window, sinks, dev = c.get("window", 0), c.get("sinks", 0), st["q"].device
    at = 0
    for i, (r, t) in enumerate(zip(st["rows"], st["lens"])):  # the sequences share nothing
        if r and t:
            first = max(0, t - r - window + 1) // 32 if window else 0
            keep = min(first, -(-sinks // 32))  # tiles of the first tokens, then those of the window
            tiles = torch.cat([torch.arange(keep, device=dev), torch.arange(first, -(-t // 32), device=dev)])
            k, v = _cached(st, st["table"][i:i + 1], tiles[None])
            token = (tiles[:, None] * 32 + torch.arange(32, device=dev)).view(1, 1, -1)
            see = _sees(torch.arange(t - r, t, device=dev).view(1, r, 1), token, window, sinks)
            o, _ = _attention(_packed_queries(q[at:at + r], c["hk"]), k, v, see)
            out[at:at + r] = o.flatten(0, 2).transpose(0, 1).to(q.dtype)
        at += r
    return out


def _window_prompt_plain(st):
    c, q, k, v = st["case"], st["q"], st["k"], st["v"]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    window, sinks, at = c["window"], c["sinks"], 0
    for n in st["rows"]:  # the packed prompts do not attend to one another
        for r0 in range(0, n, 2048):  # rows in pieces, each with the keys that a window can reach
            r1, k0 = min(n, r0 + 2048), max(0, r0 - window + 1)
            token = torch.cat([torch.arange(min(sinks, k0), device=q.device), torch.arange(k0, r1, device=q.device)])
            kk, vv = (x[at + token].float().transpose(0, 1)[None] for x in (k, v))
            see = _sees(torch.arange(r0, r1, device=q.device).view(1, -1, 1), token.view(1, 1, -1), window, sinks)
            o, z = _attention(_packed_queries(q[at + r0:at + r1], c["hk"]), kk, vv, see)
            out[at + r0:at + r1] = o.flatten(0, 2).transpose(0, 1).to(q.dtype)
            lse[at + r0:at + r1] = z.flatten(0, 2).transpose(0, 1)
        at += n
    return out, lse


def _window_step_plain(st):
    c, q, dev = st["case"], st["q"], st["q"].device
    n, rows, hq, d = q.shape
    window, sinks = c["window"], c["sinks"]
    lens = st["lens_t"].long()
    first = (lens - rows - window + 1).clamp(min=0)[:, None] // 32  # the tile where the window of the first row begins
    front = torch.arange(-(-sinks // 32), device=dev).expand(n, -1)
    span = first + torch.arange(-(-(window + rows) // 32) + 1, device=dev)
    tiles = torch.cat([front, span], 1)
    # a tile is counted once, and none past the length
    there = torch.cat([front < first, span * 32 < lens[:, None]], 1)
    k, v = _cached(st, st["table"], torch.where(there, tiles, 0))
    token = (tiles[..., None] * 32 + torch.arange(32, device=dev)).flatten(1)[:, None]
    pos = (lens[:, None] - rows + torch.arange(rows, device=dev))[..., None]
    see = _sees(pos, token, window, sinks) & there.repeat_interleave(32, 1)[:, None]
    o, lse = _attention(q.float().permute(0, 2, 1, 3).reshape(n, c["hk"], -1, d), k, v, see)
    return o.permute(0, 3, 1, 2, 4).reshape(n, rows, hq, d).to(q.dtype), lse.permute(0, 3, 1, 2).reshape(n, rows, hq)


# ------------------------------------------------------------------------------------------------ the framework's calls

def _handle(st):
    """What a user's program keeps: the cache beside its pages, the rotary plan beside its frequencies."""
    if "handle" not in st:
        from host_streamed_paged_gb300 import kvs
        c = st["case"]
        if "pages" in st:
            st["handle"] = kvs.Q4Cache(pages=st["pages"], page_tokens=c["page"], n_kv_head=c["hk"], head_dim=c["d"])
        else:
            st["handle"] = kvs.Rotary(c["d"], rot_dim=c["rot"], base=_BASE, interleaved=c["pairs"] == "neighbours",
                                      scaling=None if c["scaling"] == "none" else c["scaling"], factor=_SCALED[c["scaling"]],
                                      context=_CONTEXT, device=st["q"].device)
    return st["handle"]


def _run_own(st):
    from host_streamed_paged_gb300 import kvs
    c = st["case"]
    kind = c["kind"]
    if kind == "rotate":
        return _handle(st).rotate(st["pos"], st["q"], st["k"])
    if kind == "norm_rotate":
        return _handle(st).norm_rotate(st["pos"], st["q"], st["k"], st["wq"], st["wk"], eps=1e-6)
    if kind == "window_prompt":
        return kvs.prompt_attend(st["q"], st["k"], st["v"], st["cu"], window=c["window"], sinks=c["sinks"])
    if kind == "window_step":
        return _handle(st).attend(st["table"], st["lens_t"], st["q"], window=c["window"], sinks=c["sinks"])
    return _handle(st).attend_chunk(st["table"], st["lens_t"], st["cu"], st["q"], window=c.get("window", 0), sinks=c.get("sinks", 0))


def run(state):
    if own:
        return _run_own(state)
    return {"rotate": _rotate_plain, "norm_rotate": _norm_rotate_plain, "chunk": _chunk_plain, "window_chunk": _chunk_plain,
            "window_prompt": _window_prompt_plain, "window_step": _window_step_plain}[state["case"]["kind"]](state)


# ------------------------------------------------------------------------------------------------ work and exact values

def _reach(pos0, rows, window, sinks):
    """Of rows at pos0 .. pos0 + rows - 1 (those below 0 see nothing): (row, token) pairs seen, and tokens seen by any."""
    pairs, lo, hi = 0, None, 0
    for p in range(max(0, pos0), pos0 + rows):
        first = max(0, p - window + 1) if window else 0
        pairs += p - first + 1 + min(first, sinks)
        lo = first if lo is None else lo
        hi = p + 1
    return pairs, (hi - lo + min(lo, sinks)) if hi else 0


def work(case):
    kind, d, hk, hq = case["kind"], case["d"], case["hk"], case["hq"]
    e = _BYTES[case["dtype"]]
    if kind in ("rotate", "norm_rotate"):
        n = case["rows"] * (hq + hk)
        norm = kind == "norm_rotate"
        return dict(bytes=2 * n * d * e + 8 * case["rows"] + (2 * d * e if norm else 0), flops=n * (3 * case["rot"] + (4 * d if norm else 0)))
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    if kind == "window_prompt":
        rows = _ints(case["rows"])
        pairs = sum(_reach(0, r, window, sinks)[0] for r in rows)
        return dict(bytes=sum(rows) * ((2 * hq + 2 * hk) * d * e + 4 * hq), flops=4 * pairs * hq * d)
    if kind == "window_step":
        lens, rows = _ints(case["lens"]), [case["rows"]] * len(_ints(case["lens"]))
    else:
        rows, lens = _chunk_lens(case)
    got = [_reach(t - r, r, window, sinks) for r, t in zip(rows, lens)]
    n = sum(rows)
    return dict(bytes=sum(t for _, t in got) * hk * d * 9 // 8 + n * hq * (2 * d * e + (4 if kind == "window_step" else 0)),
                flops=4 * sum(p for p, _ in got) * hq * d)


def _exact_rotate(st):
    """Each pair as a complex number times magnitude * exp(i angle); the norms as they are defined."""
    c, out = st["case"], []
    rot, f, m = c["rot"], [], 1.0
    for i in range(rot // 2):
        base, s = _BASE, c["scaling"]
        if s == "ntk" and rot > 2:
            base *= 8.0 ** (rot / (rot - 2.0))
        w = math.exp(-math.log(base) * (2.0 * i / rot))
        if s == "linear":
            w /= 4.0
        elif s == "yarn":
            m = 1.0 + 0.1 * math.log(16.0)
            lo = max(0, math.floor(rot * math.log(_CONTEXT / (64.0 * math.pi)) / math.log(base) / 2))
            hi = min(rot - 1, math.ceil(rot * math.log(_CONTEXT / (2.0 * math.pi)) / math.log(base) / 2))
            a = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = w * (1.0 - a) + w * a / 16.0
        elif s == "bands":
            turns = _CONTEXT * w / (2.0 * math.pi)
            w = w / 8.0 if turns <= 1 else w if turns >= 4 else w * (turns - 1) / 3.0 + w / 8.0 * (4 - turns) / 3.0
        f.append(w)
    angle = st["pos"].double().unsqueeze(1) * torch.tensor(f, dtype=torch.float64, device=st["pos"].device)
    turn = torch.polar(torch.full_like(angle, m), angle).unsqueeze(1)
    for name, weight in (("q", "wq"), ("k", "wk")):
        x = st[name].double()
        if c["kind"] == "norm_rotate":
            x = x * st[weight].double() * (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).rsqrt()
        y = x.clone()
        a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if c["pairs"] == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
        z = torch.complex(x[..., a], x[..., b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_cache(st, i, h, t):
    """K and V (float64) [t, d] of one sequence and kv head, each element looked up by its place in the page."""
    c = st["case"]
    d, page, dev = c["d"], c["page"], st["pages"].device
    nb = d // 32
    tok, dim = torch.arange(t, device=dev).view(-1, 1), torch.arange(d, device=dev).view(1, -1)
    x, b, j = tok % 32, dim // 32, dim % 16
    base = (st["table"][i].long()[tok // page] * c["hk"] + h) * (page // 32 * 36 * d) + tok % page // 32 * (36 * d)
    u, w = x // 8 * nb + b, (x // 16 * nb + b) * 2 + x % 4 // 2
    at_k = (u // 4 * 32 + x % 8 * 4 + j // 4) * 16 + u % 4 * 4 + j % 4
    at_v = 18 * d + (w // 4 * 32 + j % 8 * 4 + x % 16 // 4) * 16 + w % 4 * 4 + x % 2 * 2 + j // 8
    sc_k = 8 * d + ((x // 16 * 8 + x % 8) * nb + b) * 2 + x // 8 % 2
    sc_v = 17 * d + (x // 4 * nb + b) * 4 + x % 4
    halves = st["pages"].view(torch.float16)
    high = (dim % 32) // 16
    return [(torch.where(high == 1, st["pages"][base + at] // 16, st["pages"][base + at] % 16).double() - 8)
            * halves[base // 2 + sc].double() for at, sc in ((at_k, sc_k), (at_v, sc_v))]


def _exact_rows(q, kk, vv, first, window, sinks):
    """One query head: rows [r, d] at positions first .. over keys [t, d], all in 64 bits."""
    r, d = q.shape
    out, lse = torch.zeros_like(q), torch.full((r,), -math.inf, dtype=torch.float64, device=q.device)
    for r0 in range(0, r, 1024):
        r1 = min(r, r0 + 1024)
        end = min(kk.shape[0], max(0, first + r1))
        if end == 0:
            continue
        pos = first + torch.arange(r0, r1, device=q.device)[:, None]
        tok = torch.arange(end, device=q.device)[None]
        s = q[r0:r1] @ kk[:end].T / math.sqrt(d)
        hidden = tok > pos
        if window:
            hidden = hidden | ((tok <= pos - window) & (tok >= sinks))
        s[hidden] = -math.inf
        z = torch.logsumexp(s, 1)
        lse[r0:r1] = z
        w = torch.exp(s - torch.where(z.isinf(), torch.zeros_like(z), z)[:, None])
        out[r0:r1] = w @ vv[:end]
    return out, lse


def exact(case, seed):
    kind, hk, hq = case["kind"], case["hk"], case["hq"]
    st = prepare(case, seed)
    if kind in ("rotate", "norm_rotate"):
        return _exact_rotate(st)
    window, sinks = case.get("window", 0), case.get("sinks", 0)
    rows = st["rows"]
    lens = rows if kind == "window_prompt" else st["lens"]
    if sum(r * t for r, t in zip(rows, lens)) * hq * case["d"] > 8e11:
        return None
    q = st["q"].double().view(-1, hq, case["d"])
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    at = 0
    for i, (r, t) in enumerate(zip(rows, lens)):
        for g in range(hk):
            if r and t:
                if kind == "window_prompt":
                    kk, vv = st["k"][at:at + r, g].double(), st["v"][at:at + r, g].double()
                else:
                    kk, vv = _exact_cache(st, i, g, t)
                for h in range(g * hq // hk, (g + 1) * hq // hk):
                    out[at:at + r, h], lse[at:at + r, h] = _exact_rows(q[at:at + r, h], kk, vv, t - r, window, sinks)
        at += r
    if kind in ("chunk", "window_chunk"):
        return out
    return out.view(st["q"].shape), lse.view(st["q"].shape[:-1])


def _self_check():
    """Small cases of every kind on this machine: the plain forms against the exact values."""
    rng = random.Random(2)
    for _ in range(60):
        c = draw(rng)
        for key, top in (("rows", 70), ("past", 200), ("lens", 300)):
            if isinstance(c.get(key), str):
                c[key] = ",".join(str((int(x) - 1) % top + (key == "rows")) for x in c[key].split(",")[:3])
        if c["kind"].endswith("rotate"):
            c["rows"] = 1 + c["rows"] % 50
        if "window" in c:
            c["window"] = 1 + c["window"] % 90
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
