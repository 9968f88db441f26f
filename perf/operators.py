"""Cases for the operators of the 4-bit key/value cache: writing it, reading it
back, and attention over it.

The cache holds keys and values of one layer in pages.  A page holds
``page_tokens`` tokens of every kv head as tiles of 16 tokens of one head,

    K codes [16][D/2] | V codes [16][D/2] | K words [D/32][16] | V words [D/32][16]

two codes a byte (the even dimension in the low half) and one 16-bit word for
each group of 32 dimensions of a token: an fp16 scale of seven significant
bits, with the group's integral zero point in the four bits that leaves free.
A code q stands for scale * (q - zero).

``run`` computes the operators with elementary torch operations in 32 bits
(64 for the scales, where a quotient may lie next to a border), or, where
``own`` is true, by the library's calls.
"""
import math

import torch

own = False

GROUP = 32       # values that share a scale and a zero point
TILE = 16        # tokens of a tile
CLAMP = 57344.0  # larger magnitudes are taken as this
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of each of 33 sequences, K and V slices of a fused projection
        dict(name="write_step", kind="write", tokens=33, kv_heads=8, dim=128, page=16, dtype="fp16", fused=True),
        # a 52-head layer (6656 wide) filling its cache from a mid-sized prompt, padding rows among the tokens
        dict(name="write_wide", kind="write", tokens=2011, kv_heads=52, dim=128, page=64, dtype="fp16", fused=False),
        # a long prompt of a grouped-query layer
        dict(name="write_prompt", kind="write", tokens=16384, kv_heads=8, dim=128, page=64, dtype="bf16", fused=True),
        # part of one sequence fetched for inspection: few tokens, small heads, 32-bit values
        dict(name="read_part", kind="read", tokens=777, kv_heads=3, dim=64, page=32, dtype="fp32"),
        # a whole 64k-token context restored to 16 bits
        dict(name="read_context", kind="read", tokens=65536, kv_heads=8, dim=128, page=64, dtype="fp16"),
        # one token of one short sequence, the 32 heads of a 4096-wide layer: latency counts
        dict(name="token_short", kind="attend", batch=1, new=1, ragged=False, longest=333, shortest=333, q_heads=32,
             kv_heads=32, dim=128, page=64, dtype="fp16", causal=True, window=0),
        # a serving batch of uneven contexts, grouped-query heads
        dict(name="token_batch", kind="attend", batch=48, new=1, ragged=False, longest=4096, shortest=17, q_heads=32,
             kv_heads=8, dim=128, page=64, dtype="fp16", causal=True, window=0),
        # long contexts, where the bytes of the cache are everything
        dict(name="token_long", kind="attend", batch=4, new=1, ragged=False, longest=131072, shortest=100000, q_heads=64,
             kv_heads=8, dim=128, page=64, dtype="bf16", causal=True, window=0),
        # 1 to 5 draft tokens checked at once, 52 query heads on 4 kv heads
        dict(name="verify", kind="attend", batch=16, new=5, ragged=True, longest=8190, shortest=500, q_heads=52,
             kv_heads=4, dim=128, page=32, dtype="fp16", causal=True, window=0),
        # wide heads that share one kv head, each token seeing the last 1024
        dict(name="token_window", kind="attend", batch=24, new=1, ragged=False, longest=32768, shortest=900, q_heads=16,
             kv_heads=1, dim=256, page=128, dtype="bf16", causal=True, window=1024),
        # uneven prompts with small heads, the first of them behind a context that is there already
        dict(name="prompt_uneven", kind="attend", batch=6, new=1531, ragged=True, longest=2600, shortest=1, q_heads=12,
             kv_heads=12, dim=64, page=16, dtype="fp16", causal=True, window=0),
        # one long prompt of a grouped-query layer
        dict(name="prompt_long", kind="attend", batch=1, new=6000, ragged=False, longest=6000, shortest=6000, q_heads=32,
             kv_heads=8, dim=128, page=64, dtype="bf16", causal=True, window=0),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 12, 32])
    if kind != "attend":
        most = max(1, (1 << 24) // (kv_heads * dim))
        c = dict(kind=kind, tokens=_between(rng, 1, min(65536, most)), kv_heads=kv_heads, dim=dim, page=page,
                 dtype=rng.choice(["fp16", "bf16"] if kind == "write" else ["fp16", "bf16", "fp32"]))
        if kind == "write":
            c["fused"] = rng.random() < 0.5
        return c
    share = rng.choice([1, 1, 4, 7, 8, 16])
    q_heads = kv_heads * share
    prompt = rng.random() < 0.4
    if prompt:  # rows x keys of all heads stay under those of the largest listed case
        batch = _between(rng, 1, 8)
        longest = _between(rng, 24, max(25, min(4096, int(math.sqrt(6.0e8 * 64 / (dim * q_heads * batch))))))
        new = _between(rng, max(1, longest // 4), longest)
    else:
        batch = _between(rng, 1, 64)
        new = rng.choice([1, 1, 1, 2, 5, 8])
        longest = _between(rng, 16, max(17, min(131072, (1 << 28) // (kv_heads * dim * batch))))
        longest = min(longest, max(16, (1 << 29) // (q_heads * batch * new)))
    return dict(kind="attend", batch=batch, new=new, ragged=rng.random() < 0.5, longest=longest,
                shortest=_between(rng, 1, longest), q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page,
                dtype=rng.choice(["fp16", "bf16"]), causal=rng.random() < 0.9,
                window=0) | ({"causal": True, "window": _between(rng, 8, 2048)} if rng.random() < 0.2 else {})


def _spread(lo, hi, n):
    """n lengths from lo to hi, the first of them hi, the same for every seed."""
    return [hi] + [lo + int((hi - lo + 1) * ((0.6180339887 * k) % 1.0)) for k in range(1, n)]


def _lengths(case):
    """Cached tokens and new tokens (the last of the cached ones) of each sequence."""
    kv = _spread(case["shortest"], case["longest"], case["batch"])
    new = _spread(1, case["new"], case["batch"]) if case["ragged"] else [case["new"]] * case["batch"]
    if case["ragged"]:
        new = [min(n, k) for n, k in zip(new, kv)]
    return kv, new


def _visible(case, kv, n):
    """Pairs of a query and a key it sees, and keys that any query sees, of one sequence."""
    pairs, first = 0, kv
    for i in range(n):
        pos = kv - n + i
        hi = min(kv, pos + 1) if case["causal"] else kv
        lo = max(0, pos - case["window"] + 1) if case["window"] else 0
        pairs += max(0, hi - lo)
        first = min(first, lo)
    return pairs, kv - first


def work(case):
    h, d = case["kv_heads"], case["dim"]
    held = 2 * h * d * 9 / 16  # bytes of a token in the cache: 4 bits a value and a word for 32
    if case["kind"] == "write":  # the rows are read and written; the values come back
        t = case["tokens"]
        return {"bytes": t * (2 * h * d * 2 + held + 2 * h * d * 2 + 8), "flops": 0}
    if case["kind"] == "read":
        t = case["tokens"]
        return {"bytes": t * (held + 2 * h * d * (4 if case["dtype"] == "fp32" else 2) + 8), "flops": 0}
    pairs = keys = rows = 0
    for kv, n in zip(*_lengths(case)):
        p, k = _visible(case, kv, n)
        pairs, keys, rows = pairs + p, keys + k, rows + n
    return {"bytes": keys * held + rows * case["q_heads"] * (2 * d * 2 + 4), "flops": 4 * d * case["q_heads"] * pairs}


# ---------------------------------------------------------------- the inputs

def _tile_bytes(d):
    return TILE * (d + d // 8)


def _encode(x):
    """Codes (uint8, one a byte) and group words (int16) of x [..., D]."""
    n = x.shape[-1] // GROUP
    x = x.float().unflatten(-1, (n, GROUP))
    bad = torch.isnan(x).any(-1)
    x = torch.where(bad[..., None], 0.0, x.clamp(-CLAMP, CLAMP))
    lo, hi = x.amin(-1).clamp(max=0).double(), x.amax(-1).clamp(min=0).double()
    d = (hi - lo) / 15
    power = (d.view(torch.int64) >> 52).clamp(min=1023 - 14) - 6  # of the scale's last bit, biased: no power function, whose values may be off by a bit
    unit = (power << 52).view(torch.float64)
    s = (torch.ceil(d / unit) * unit).clamp(min=2.0 ** -20)
    z = torch.round(-lo / s)
    q = (torch.round(x / s.float()[..., None]) + z.float()[..., None]).clamp(0, 15)
    q = torch.where(bad[..., None], 0.0, q)
    word = s.half().view(torch.int16).int() | z.int()
    word = torch.where(bad, 0x7E00, word).short()
    return q.flatten(-2).to(torch.uint8), word


def _sections(cache, case):
    """The four sections of every tile, as views: codes [pages, H, tiles, 16, D/2] and words [pages, H, tiles, D/32, 16]."""
    d, h = case["dim"], case["kv_heads"]
    t = cache.view(-1, h, case["page"] // TILE, _tile_bytes(d))
    c, w = TILE * d // 2, TILE * d // 16
    codes = [t[..., i * c:(i + 1) * c].unflatten(-1, (TILE, d // 2)) for i in (0, 1)]
    words = [t[..., 2 * c + i * w:2 * c + (i + 1) * w].view(torch.int16).unflatten(-1, (d // GROUP, TILE)) for i in (0, 1)]
    return codes[0], codes[1], words[0], words[1]


def _store(cache, case, k, v, slots):
    """Writes rows k, v [tokens, H, D] at their slots; rows of negative slots go to the last slot, which holds no token."""
    at = torch.where(slots < 0, cache.numel() // _tile_bytes(case["dim"]) // case["kv_heads"] * TILE - 1, slots)
    page, tile, row = at // case["page"], at % case["page"] // TILE, at % TILE
    kc, vc, kw, vw = _sections(cache, case)
    for x, codes, words in ((k, kc, kw), (v, vc, vw)):
        q, w = _encode(x)
        codes[page, :, tile, row] = q[..., 0::2] | (q[..., 1::2] << 4)
        words[page, :, tile, :, row] = w


def _values(codes, words):
    """fp32 values of codes [..., D/2] and words [..., D/32]."""
    w = words.int() & 0xFFFF
    s = (w & 0xFFF0).short().view(torch.float16).float()
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    q = q.unflatten(-1, (-1, GROUP)).float() - (w & 15).float()[..., None]
    return (q * s[..., None]).flatten(-2)


def _load(cache, case, slots):
    page, tile, row = slots // case["page"], slots % case["page"] // TILE, slots % TILE
    kc, vc, kw, vw = _sections(cache, case)
    return tuple(_values(c[page, :, tile, row], w[page, :, tile, :, row]) for c, w in ((kc, kw), (vc, vw)))


def _rows(gen, n, h, d, dtype):
    """Key or value rows: some dimensions several times as large as others, as trained heads have them."""
    x = torch.randn(n, h, d, generator=gen, device="cuda")
    return (x * torch.exp(0.6 * torch.randn(h, d, generator=gen, device="cuda"))).to(dtype)


def _fill(gen, pages, case):
    """A cache of written rows."""
    p, h, d = case["page"], case["kv_heads"], case["dim"]
    cache = torch.empty(pages * h * (p // TILE) * _tile_bytes(d), dtype=torch.uint8, device="cuda")
    kc, vc, kw, vw = _sections(cache, case)
    for codes, words in ((kc, kw), (vc, vw)):
        q, w = _encode(_rows(gen, pages * p, h, d, torch.float16))
        b = q[..., 0::2] | (q[..., 1::2] << 4)
        codes.copy_(b.view(pages, p // TILE, TILE, h, d // 2).permute(0, 3, 1, 2, 4))
        words.copy_(w.view(pages, p // TILE, TILE, h, d // GROUP).permute(0, 3, 1, 4, 2))
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    h, d, p, dtype = case["kv_heads"], case["dim"], case["page"], DTYPES[case["dtype"]]
    s = {"case": case}
    if case["kind"] != "attend":
        t = case["tokens"]
        pages = -(-t // p) + 3
        if case["kind"] == "write":
            s["cache"] = torch.zeros(pages * h * (p // TILE) * _tile_bytes(d), dtype=torch.uint8, device="cuda")
            if case["fused"]:
                x = torch.cat([_rows(gen, t, h, d, dtype) for _ in range(2)], 1).view(t, 2, h, d)
                s["k"], s["v"] = x[:, 0], x[:, 1]
            else:
                s["k"], s["v"] = (_rows(gen, t, h, d, dtype) for _ in range(2))
            s["slots"] = torch.randperm((pages - 1) * p, generator=gen, device="cuda")[:t] if t < 4096 else torch.arange(t, device="cuda") + p
            if t > 1000:  # padding rows
                s["slots"][torch.randperm(t, generator=gen, device="cuda")[:t // 50]] = -1
        else:
            s["cache"] = _fill(gen, pages, case)
            order = torch.randperm(pages, generator=gen, device="cuda")
            s["slots"] = (order[:, None] * p + torch.arange(p, device="cuda")).flatten()[:t].contiguous()
        s["out"] = [torch.zeros(t, h, d, dtype=dtype, device="cuda") for _ in range(2)]
    else:
        kv, new = _lengths(case)
        need = [-(-n // p) for n in kv]
        cols, pages = max(need), sum(need) + 1
        s["cache"] = _fill(gen, pages, case)
        order = torch.randperm(pages, generator=gen, device="cuda").int().split(need + [1])
        table = torch.zeros(case["batch"], cols, dtype=torch.int32, device="cuda")
        for b, ids in enumerate(order[:-1]):
            table[b, :len(ids)] = ids
        s["table"] = table
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        rows = sum(new) + (7 if case["ragged"] else 0)  # rows behind the last sequence
        s["q_start"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["q"] = torch.randn(rows, case["q_heads"], d, generator=gen, device="cuda").to(dtype)
        s["out"] = torch.zeros(rows, case["q_heads"], d, dtype=dtype, device="cuda")
        s["lse"] = torch.zeros(rows, case["q_heads"], dtype=torch.float32, device="cuda")
    if own:
        import dense_sparse_quantized_b200 as dsq
        s["kv"] = dsq.KVCache(h, d, pages, p, data=s["cache"])
        if case["kind"] == "attend":
            s["work"] = s["kv"].attend_workspace(s["q"].shape[0], case["q_heads"], case["batch"])
    return s


# ------------------------------------------------------------------- the runs

def _attend(s):
    """Attention of every query row over its sequence's cached tokens."""
    case, q, lens = s["case"], s["q"], s["kv_lens"].long()
    b, h, d, p = case["batch"], case["kv_heads"], case["dim"], case["page"]
    share = case["q_heads"] // h
    start = s["q_start"].long() if s["q_start"] is not None else torch.arange(b + 1, device=q.device) * (q.shape[0] // b)
    n = start[1:] - start[:-1]
    i = torch.arange(case["new"], device=q.device)
    at = start[:-1, None] + i                                            # [b, new]
    x = q[at.clamp(max=q.shape[0] - 1)].float()                          # [b, new, Hq, D]
    x = x.unflatten(2, (h, share)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [b, h, share*new, D]
    cols = s["table"].shape[1]
    kc, vc, kw, vw = _sections(s["cache"], case)
    pick = s["table"].long()

    def gathered(codes, words):
        c = codes[pick].permute(0, 2, 1, 3, 4, 5).reshape(b, h, cols * p, d // 2)
        w = words[pick].permute(0, 2, 1, 3, 5, 4).reshape(b, h, cols * p, d // GROUP)
        return _values(c, w)

    score = x @ gathered(kc, kw).transpose(-1, -2) * (1.0 / math.sqrt(d))
    pos = (lens - n)[:, None] + i                                        # [b, new]
    key = torch.arange(cols * p, device=q.device)
    seen = (key < lens[:, None])[:, None].expand(b, case["new"], -1)
    if case["causal"]:
        seen = seen & (key <= pos[..., None])
    if case["window"]:
        seen = seen & (key > pos[..., None] - case["window"])
    score = score.unflatten(2, (share, case["new"])).masked_fill_(~seen[:, None, None], -torch.inf).flatten(2, 3)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    y = e @ gathered(vc, vw) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    y = y.unflatten(2, (share, case["new"])).permute(0, 3, 1, 2, 4).flatten(2, 3)      # [b, new, Hq, D]
    lse = lse.unflatten(2, (share, case["new"])).permute(0, 3, 1, 2).flatten(2, 3)
    row = torch.arange(q.shape[0], device=q.device)
    seq = (torch.searchsorted(start, row, right=True) - 1).clamp(max=b - 1)
    i = row - start[seq]
    valid, i = i < n[seq], i.clamp(max=case["new"] - 1)
    s["out"].copy_(torch.where(valid[:, None, None], y[seq, i].to(q.dtype), s["out"]))
    s["lse"].copy_(torch.where(valid[:, None], lse[seq, i], s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    case = s["case"]
    if own:
        kv = s["kv"]
        if case["kind"] == "attend":
            kv.attend(s["q"], s["table"], s["kv_lens"], q_start=s["q_start"], causal=case["causal"], window=case["window"],
                      out=s["out"], lse=s["lse"], workspace=s["work"])
            return {"out": s["out"], "lse": s["lse"]}
        if case["kind"] == "write":
            kv.append(s["k"], s["v"], s["slots"])
        k, v = kv.read(s["slots"], k=s["out"][0], v=s["out"][1])
        return {"k": k, "v": v}
    if case["kind"] == "attend":
        return _attend(s)
    if case["kind"] == "write":
        _store(s["cache"], case, s["k"], s["v"], s["slots"])
    there = (s["slots"] >= 0)[:, None, None]
    for x, y in zip(s["out"], _load(s["cache"], case, s["slots"].clamp(min=0))):
        x.copy_(torch.where(there, y.to(x.dtype), x))
    return {"k": s["out"][0], "v": s["out"][1]}


# ------------------------------------------------------------- the definition

def _exact_round(x):
    """What a row of 64-bit numbers [..., D] stands for once it is held in 4 bits."""
    out = torch.empty_like(x)
    powers = torch.tensor([2.0 ** k for k in range(-20, 8)], dtype=torch.float64, device=x.device)
    for g in range(x.shape[-1] // GROUP):
        part = torch.clamp(x[..., g * GROUP:(g + 1) * GROUP], -CLAMP, CLAMP)
        lo = torch.minimum(part.min(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=x.device))
        hi = torch.maximum(part.max(-1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=x.device))
        step = (hi - lo) / 15.0
        power = torch.frexp(step).exponent.long() - 1                    # step in [2^power, 2^(power+1))
        unit = powers[torch.where(step > 0, power - 6, -20).clamp(min=-20) + 20]
        scale = torch.ceil(step / unit) * unit
        scale = torch.where(scale < 2.0 ** -20, torch.full_like(scale, 2.0 ** -20), scale)
        zero = torch.round(-lo / scale)
        code = torch.minimum(torch.maximum(torch.round(part / scale) + zero, torch.zeros_like(part)), torch.full_like(part, 15.0))
        out[..., g * GROUP:(g + 1) * GROUP] = scale * (code - zero)
    return out


def _exact_rows(cache, case, slots):
    """64-bit K and V rows [tokens, H, D] at the slots, byte by byte."""
    d, h, p = case["dim"], case["kv_heads"], case["page"]
    size, tiles = _tile_bytes(d), case["page"] // TILE
    tile = ((slots // p)[:, None] * h + torch.arange(h, device=slots.device)) * tiles + (slots % p // TILE)[:, None]
    base, row = tile * size, (slots % TILE)[:, None, None]
    dims = torch.arange(d, device=slots.device)
    found = []
    for which in (0, 1):
        codes = cache[base[..., None] + which * TILE * d // 2 + row * (d // 2) + dims // 2]
        codes = torch.where(dims % 2 == 0, codes % 16, codes // 16).double()
        at = base[..., None] + TILE * d + which * TILE * d // 16 + (dims // GROUP) * 2 * TILE + 2 * row
        word = cache[at].long() + 256 * cache[at + 1].long()
        zero, e, m = word % 16, word // 1024 % 32, word // 16 % 64 * 16
        powers = torch.tensor([2.0 ** (k - 25) for k in range(32)], dtype=torch.float64, device=cache.device)
        scale = torch.where(e == 0, m.double() * 2.0 ** -24, (1024.0 + m) * powers[e])
        found.append((codes - zero) * scale)
    return found


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "write":
        there = (s["slots"] >= 0)[:, None, None]
        return {n: torch.where(there, _exact_round(s[n].double()), 0.0) for n in ("k", "v")}
    if case["kind"] == "read":
        k, v = _exact_rows(s["cache"], case, s["slots"])
        return {"k": k, "v": v}
    rows, share, p = s["q"].shape[0], case["q_heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(rows, case["q_heads"], case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, case["q_heads"], dtype=torch.float64, device="cuda")
    first = 0
    for b, (kv, n) in enumerate(zip(*_lengths(case))):
        t = torch.arange(kv, device="cuda")
        k, v = _exact_rows(s["cache"], case, s["table"][b].long()[t // p] * p + t % p)
        for i in range(0, n, 512):
            m = min(512, n - i)
            pos = kv - n + i + torch.arange(m, device="cuda")[:, None]
            seen = torch.ones(m, kv, dtype=torch.bool, device="cuda")
            if case["causal"]:
                seen &= t <= pos
            if case["window"]:
                seen &= t > pos - case["window"]
            for head in range(case["q_heads"]):
                y = s["q"][first + i:first + i + m, head].double() @ k[:, head // share].T / math.sqrt(case["dim"])
                y = y.masked_fill(~seen, -torch.inf)
                total = torch.logsumexp(y, -1)
                lse[first + i:first + i + m, head] = total
                out[first + i:first + i + m, head] = torch.where(seen, torch.exp(y - total[:, None]), 0.0) @ v[:, head // share]
        first += n
    return {"out": out, "lse": lse}
