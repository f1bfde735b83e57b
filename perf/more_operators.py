"""Operators that carry an agent's tokens into its paged cache by way of the
position rotation, and that hold the cache in 4 bits: the cases that are measured.

The sequences are those of the paged private caches: token j of sequence s is
slot j % page_tokens of page table[s, j // page_tokens]. The operators:

"rotary"  writes a layer's new K, rotated by position, and V into bf16 pages,
          and rotates the new tokens' Q on the way.
"store"   the same into pages that hold 4 bits per value, then reads the tokens
          back as the values that the codes stand for.
"read"    whole sequences of the 4-bit cache as bf16 (a cache handed on).
"attend"  attention of single tokens, drafts, chunks and prompts over the 4-bit
          cache, with a cap, a bias by distance or a window where a layer has them.

Rotation: channel pairs (i, i + R/2), or (2i, 2i + 1) where interleaved, of the
first R channels turn by the angle whose cosine and sine stand in row offset + p
of two float32 tables, for a token at position p.

4 bits: a head-vector x of d channels becomes y = H x (H the Walsh-Hadamard
matrix in Sylvester's order), whose coordinates come near N(0, n^2), n = |x|.
With the step 0.3352 n (the best uniform 16-level quantiser of a normal
variable: J. Max, 1960) channel i has the code u_i = clamp(floor(y_i / step) + 8,
0, 15); the vector has one float32 scale t = step / d and stands for
t H (u - 7.5). Eight channels share a 32-bit word, channel 2k in bits 4k ...
4k + 3 and channel 2k + 1 sixteen bits above.
"""

import math

import torch

own = False

#: (kv_heads, q_heads, head_dim): the shapes of this repository's workloads, and one whose group of query heads is odd
HEADS = {"tiny": (2, 4, 64), "smollm2": (32, 32, 64), "llama3": (8, 32, 128), "qwen3": (8, 64, 128), "group7": (4, 28, 128)}
STEP = 0.3352


def listed():
    return [
        # one decode step of three agents right after they started: launch latency
        dict(name="decode_tiny", kind="attend", heads="tiny", page=16, seqs=3, q_min=1, q_max=1, kv_min=40, kv_max=129),
        # one decode step of 32 agents, 32K tokens each: bandwidth
        dict(name="decode_qwen3_32k", kind="attend", heads="qwen3", page=128, seqs=32, q_min=1, q_max=1, kv_min=30001, kv_max=32768),
        # a few draft tokens of one agent verified over a long history: little parallelism but the context's
        dict(name="verify_group7", kind="attend", heads="group7", page=32, seqs=1, q_min=5, q_max=5, kv_min=20011, kv_max=20011),
        # one decode step of 15 agents in a layer whose scores are capped, fall with the distance and end at a window
        dict(name="scored_decode", kind="attend", heads="llama3", page=64, seqs=15, q_min=1, q_max=1, kv_min=600, kv_max=7194,
             cap=30.0, slopes=True, window=4096),
        # a prompt read in chunks: 2,048 new tokens at the end of 16K
        dict(name="chunk_llama3_16k", kind="attend", heads="llama3", page=64, seqs=1, q_min=2048, q_max=2048, kv_min=16384, kv_max=16384),
        # a mixed batch: tool answers of up to 777 tokens next to decoding agents
        dict(name="mixed_llama3", kind="attend", heads="llama3", page=16, seqs=12, q_min=1, q_max=777, kv_min=900, kv_max=4099),
        # one layer's new token of 15 agents behind a shared context of 4,096 tokens: launch latency
        dict(name="rotary_decode", kind="rotary", heads="llama3", page=64, seqs=15, q_min=1, q_max=1, kv_min=600, kv_max=7194,
             offset=4096, rot=128, interleaved=False),
        # one layer's new tokens of a batch of long chunks, half of the channels rotated, in adjacent pairs
        dict(name="rotary_chunks", kind="rotary", heads="llama3", page=16, seqs=9, q_min=500, q_max=4096, kv_min=4096, kv_max=8192,
             offset=0, rot=64, interleaved=True),
        # the decode step's token of 15 agents into 4 bits: launch latency
        dict(name="store_decode", kind="store", heads="llama3", page=64, seqs=15, q_min=1, q_max=1, kv_min=600, kv_max=7194,
             offset=4096, rot=128, interleaved=False),
        # a batch of long chunks into 4 bits
        dict(name="store_chunks", kind="store", heads="qwen3", page=64, seqs=7, q_min=501, q_max=4096, kv_min=4096, kv_max=8191,
             offset=0, rot=128, interleaved=False),
        # one short agent's cache handed on
        dict(name="read_short", kind="read", heads="smollm2", page=32, seqs=1, q_min=333, q_max=333, kv_min=333, kv_max=333),
        # the caches of 15 agents with up to the repository's long context handed on
        dict(name="read_long", kind="read", heads="llama3", page=64, seqs=15, q_min=600, q_max=7194, kv_min=600, kv_max=7194),
    ]


def _spread(lo, hi, n, turn):
    """n whole numbers from lo to hi, spread over the range, the largest among them."""
    return [hi if i == 0 else lo + int((hi - lo) * math.modf(i * turn)[0] + 0.5) for i in range(n)]


def _lengths(c):
    """New tokens and held tokens (the new ones among them) of each sequence."""
    q = _spread(c["q_min"], c["q_max"], c["seqs"], 0.6180339887498949)
    t = _spread(c["kv_min"], c["kv_max"], c["seqs"], 0.4142135623730951)
    if c["q_min"] == c["kv_min"] and c["q_max"] == c["kv_max"]:  # whole sequences
        return q, q
    return q, [max(a, b) for a, b in zip(q, t)]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["decode", "decode", "chunk", "chunk", "prompts", "rotary", "store", "read"])
    heads = rng.choice(list(HEADS))
    hk, hq, d = HEADS[heads]
    page = rng.choice([16, 32, 64, 128])
    if kind in ("rotary", "store"):
        q = log(1, 4096)
        return dict(kind=kind, heads=heads, page=page, seqs=log(1, max(1, min(16, 20000 // q))), q_min=max(1, q // 8), q_max=q,
                    kv_min=q, kv_max=q + log(1, 4096), offset=rng.choice([0, 0, 4096, 7194]), rot=rng.choice([d, d, d // 2]),
                    interleaved=rng.random() < 0.3)
    if kind == "read":
        t = log(1, 7194)
        low = max(1, t // rng.randrange(1, 9))
        return dict(kind="read", heads=heads, page=page, seqs=log(1, max(1, min(16, 60000 // t))), q_min=low, q_max=t, kv_min=low, kv_max=t)
    if kind == "decode":
        kv = log(1, 32768)
        seqs = log(1, max(1, min(32, (1 << 28) // (kv * hk * d))))
        c = dict(kind="attend", heads=heads, page=page, seqs=seqs, q_min=1, q_max=rng.choice([1, 1, 1, 2, 4]),
                 kv_min=max(1, kv // rng.randrange(1, 9)), kv_max=kv)
    else:
        q = log(2, 2048)
        kv = q if kind == "prompts" else q + log(1, 16384 - q)
        seqs = log(1, max(1, min(16, (1 << 30) // (q * hq * kv))))
        low = max(1, q // rng.randrange(1, 9))
        c = dict(kind="attend", heads=heads, page=page, seqs=seqs, q_min=low, q_max=q, kv_min=low if kind == "prompts" else max(1, kv // 2), kv_max=kv)
    if rng.random() < 0.3:
        c["cap"] = rng.choice([0.0, 20.0, 50.0])
        c["slopes"] = rng.random() < 0.5
        if rng.random() < 0.5:
            c["window"] = log(1, 4096)
    return c


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _channels(shape, g):
    """Standard deviations of channels as KV caches show them: log-normal, one in a hundred ten times larger."""
    std = torch.exp(0.5 * torch.randn(shape, generator=g, device="cuda"))
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.01, 10 * std, std).to(torch.bfloat16)


def prepare(case, seed):
    hk, hq, d = HEADS[case["heads"]]
    P = case["page"]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    q, t = _lengths(case)
    need = [(x + P - 1) // P for x in t]
    pages = sum(need) + 3
    s = {"kind": case["kind"], "d": d, "P": P}
    if case["kind"] == "rotary":
        s["K"], s["V"] = (normal(1, pages, hk, P, d) for _ in range(2))
    else:
        # a cache as appends leave it: coordinates near normal, norms about sqrt(d) times the heads' own sizes
        for name in ("K", "V"):
            codes = torch.empty(pages, hk, P, d // 2, dtype=torch.uint8, device="cuda")
            for a in range(0, pages, 512):
                z = torch.randn((min(512, pages - a), hk, P, d), generator=g, device="cuda")
                u = torch.floor(z / STEP).add_(8).clamp_(0, 15).to(torch.uint8)
                codes[a: a + 512] = u[..., 0::2] | u[..., 1::2] << 4
            s[name] = codes[None]
            size = torch.exp(0.3 * torch.randn((hk, 1), generator=g, device="cuda"))
            norm = math.sqrt(d) * size * (1 + 0.1 * torch.randn((1, pages, hk, P), generator=g, device="cuda")).clamp_(0.5, 1.5)
            s[name + "_scale"] = (STEP / d * norm).contiguous()
    # each sequence's pages lie scattered over the cache; entries behind its last page are not used
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(q), max(need), dtype=torch.int32, device="cuda")
    used = torch.arange(max(need), device="cuda")[None, :] < _ints(need)[:, None]
    table[used] = order[: sum(need)]
    start = [0]
    for n in q:
        start.append(start[-1] + n)
    s |= {"table": table, "kv_len": _ints(t), "q_start": _ints(start), "max_q": max(q), "max_kv": max(t), "tokens": start[-1]}
    if case["kind"] in ("rotary", "store"):
        # what a projection gives: Q, K and V next to each other in one row per token
        qkv = normal(start[-1], hq + 2 * hk, d)
        qkv[:, hq:] *= torch.cat([_channels((hk, d), g), _channels((hk, d), g)])
        s["Q"], s["new_k"], s["new_v"] = qkv[:, :hq], qkv[:, hq: hq + hk], qkv[:, hq + hk:]
        # cosines and sines of every position that a program expects, from angles in 64 bits
        R = case["rot"]
        at = torch.arange(case["offset"] + max(t), dtype=torch.float64, device="cuda")
        angle = at[:, None] * 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        s |= {"cos": angle.cos().float(), "sin": angle.sin().float(), "interleaved": case["interleaved"], "offset": case["offset"]}
    elif case["kind"] == "attend":
        s["Q"] = normal(start[-1], hq, d)
        s["score"] = {}
        if case.get("cap"):
            s["score"]["cap"] = case["cap"]
        if case.get("slopes"):
            s["score"]["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq)
        if case.get("window"):
            s["score"]["window"] = case["window"]
    return s


def _slots(s):
    """Position, page and slot of every new token."""
    row = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    at = s["kv_len"].long()[seq] - s["q_start"].long()[seq + 1] + row
    return at, s["table"].long()[seq, at // s["P"]], at % s["P"]


def _turned(s, x, at):
    """Rows [tokens, heads, d] in 32 bits, rotated by the positions."""
    x = x.float()
    c, n = (s[k][s["offset"] + at][:, None] for k in ("cos", "sin"))
    R = 2 * c.shape[-1]
    out = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if s["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    out[..., a] = x[..., a] * c - x[..., b] * n
    out[..., b] = x[..., b] * c + x[..., a] * n
    return out


def _power_of_two(e):
    return (e + 127 << 23).to(torch.int32).view(torch.float32)


def _coded(x):
    """Codes and scales of vectors [..., d], step by step in 32 bits: the largest value brought into [1/2, 1), so that squares
    stay in range; the butterflies of the transform; the squares summed in neighbouring pairs."""
    d = x.shape[-1]
    e = torch.frexp(x.abs().amax(-1, keepdim=True))[1].clamp_(-126, 126)
    y = x * _power_of_two(-e)
    sq = y * y
    while sq.shape[-1] > 1:
        sq = sq[..., 0::2] + sq[..., 1::2]
    step = torch.tensor(STEP, dtype=torch.float32, device=x.device) * sq.sqrt()
    h = 1
    while h < d:
        y = y.view(*x.shape[:-1], d // (2 * h), 2, h)
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2)
        h *= 2
    y = y.reshape(x.shape) * (1.0 / step)
    u = torch.where(step > 0, torch.floor(y) + 8, 8).clamp_(0, 15).to(torch.uint8)
    # channels 0, 2, 4, 6, 1, 3, 5, 7 of every eight, two to a byte
    u = u.view(*x.shape[:-1], d // 8, 4, 2).transpose(-1, -2).reshape(*x.shape[:-1], d // 2, 2)
    return u[..., 0] | u[..., 1] << 4, (step * _power_of_two(e))[..., 0] / d


def _levels(codes):
    """u - 7.5 of packed codes [..., d / 2] in 32 bits, channels in order."""
    u = torch.stack([codes & 15, codes >> 4], -1).view(*codes.shape[:-1], -1, 2, 4).transpose(-1, -2)
    return u.reshape(*codes.shape[:-1], -1).float() - 7.5


def _hadamard(d, dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _values(codes, scale):
    """What codes stand for, in 32 bits."""
    return torch.matmul(_levels(codes), _hadamard(2 * codes.shape[-1], torch.float32)) * scale[..., None]


def _plain_append(s):
    at, page, slot = _slots(s)
    k, v = _turned(s, s["new_k"], at), s["new_v"]
    q = _turned(s, s["Q"], at).to(torch.bfloat16)
    if s["kind"] == "rotary":
        s["K"][0][page, :, slot] = k.to(torch.bfloat16)
        s["V"][0][page, :, slot] = v
        return s["K"], s["V"], q
    for name, x in (("K", k), ("V", v.float())):
        s[name][0][page, :, slot], s[name + "_scale"][0][page, :, slot] = _coded(x)
    return *_plain_read(s), q


def _plain_read(s):
    at, page, slot = _slots(s)
    return tuple(_values(s[x][0][page, :, slot], s[x + "_scale"][0][page, :, slot]).to(torch.bfloat16) for x in ("K", "V"))


def _plain_attend(s, cap=0.0, slopes=None, window=0):
    P, d = s["P"], s["d"]
    hk = s["K"].shape[2]
    tokens, hq = s["Q"].shape[:2]
    S, n, T = s["table"].shape[0], s["max_q"], s["table"].shape[1] * P
    count, held = s["q_start"].diff().long(), s["kv_len"].long()
    i, j = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    # rows of the batch, one sequence each, as [S, n]; places behind a sequence's last row go to a row that is dropped
    row = torch.where(i < count[:, None], s["q_start"][:-1].long()[:, None] + i, tokens)
    q = torch.cat([s["Q"], s["Q"].new_zeros(1, hq, d)])[row].float().view(S, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    page = s["table"].long()

    def rows(name):
        return _values(s[name][0][page], s[name + "_scale"][0][page]).transpose(1, 2).reshape(S, hk, T, d)

    x = torch.matmul(q.reshape(S, hk, -1, d), rows("K").transpose(2, 3)).mul_(d ** -0.5).view(S, hk, hq // hk, n, T)
    at = (held - count)[:, None] + i
    if cap:
        x = x.div_(cap).tanh_().mul_(cap)
    if slopes is not None:
        x = x.sub_(slopes.view(1, hk, hq // hk, 1, 1) * (at[:, :, None] - j).abs()[:, None, None])
    seen = j <= at[:, :, None]
    if window:
        seen = seen & (j > at[:, :, None] - window)
    x = x.masked_fill_(~(seen & (j < held[:, None, None]))[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S, hk, -1, T), rows("V")).view(S, hk, hq // hk, n, d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out = s["Q"].new_zeros(tokens + 1, hq, d)
    out[row] = o.permute(0, 3, 1, 2, 4).reshape(S, n, hq, d).to(torch.bfloat16)
    at_row = torch.zeros(tokens + 1, hq, device="cuda")
    at_row[row] = lse.permute(0, 3, 1, 2).reshape(S, n, hq)
    return out[:tokens], at_row[:tokens]


def _own(s):
    from shared_quantized_kv_gb300 import kvpool

    batch = s["table"], s["kv_len"], s["q_start"]
    if s["kind"] in ("rotary", "store"):
        turn = kvpool.Rotary(s["cos"], s["sin"], s["interleaved"], s["offset"])
    if s["kind"] == "rotary":
        q = kvpool.pages_append_rotary(s["K"], s["V"], 0, s["new_k"], s["new_v"], *batch, turn, Q=s["Q"])
        return s["K"], s["V"], q
    pages = kvpool.Pages4(s["K"], s["V"], s["K_scale"], s["V_scale"])
    if s["kind"] == "store":
        q = kvpool.pages4_append(pages, 0, s["new_k"], s["new_v"], *batch, rotary=turn, Q=s["Q"])
        return *kvpool.pages4_read(pages, 0, *batch, s["tokens"]), q
    if s["kind"] == "read":
        return kvpool.pages4_read(pages, 0, *batch, s["tokens"])
    return kvpool.pages4_attend(pages, 0, s["Q"], *batch, max_q=s["max_q"], max_kv=s["max_kv"], return_lse=True, **s["score"])


def run(state):
    if own:
        return _own(state)
    if state["kind"] in ("rotary", "store"):
        return _plain_append(state)
    if state["kind"] == "read":
        return _plain_read(state)
    return _plain_attend(state, **state["score"])


def work(case):
    hk, hq, d = HEADS[case["heads"]]
    q, t = _lengths(case)
    new, held4 = sum(q), d // 2 + 4  # bytes of a vector in 4 bits, with its scale
    where = 4 * (2 * len(q) + 1 + sum((x + case["page"] - 1) // case["page"] for x in t))
    if case["kind"] in ("rotary", "store"):
        spans, rows, end = sorted((x - n, x) for n, x in zip(q, t)), 0, 0
        for a, b in spans:  # the tables' rows that any token turns by
            rows += max(0, b - max(a, end))
            end = max(end, b)
        moved = new * (2 * hq + 2 * hk) * d * 2 + rows * case["rot"] * 4 + where
        # the new K and V rows: two bytes per value, or codes and scales, and what is read back
        return {"bytes": moved + 2 * new * hk * (2 * d if case["kind"] == "rotary" else held4 + 2 * d),
                "flops": new * hk * d * (3 if case["kind"] == "rotary" else 3 + 3 * 2 * (d.bit_length() - 1)) + 3 * new * hq * d}
    if case["kind"] == "read":
        return {"bytes": 2 * new * hk * (held4 + 2 * d) + where, "flops": 2 * new * hk * d * d.bit_length()}
    window = case.get("window") or 1 << 40
    pairs = sum(sum(min(p + 1, window) for p in range(x - n, x)) for n, x in zip(q, t))
    held = sum(min(x, window + n - 1) for n, x in zip(q, t))
    rows = new * hq
    return {"bytes": rows * d * 2 * 2 + rows * 4 + 2 * held * hk * held4 + where, "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    hk, hq, d = HEADS[case["heads"]]
    q, t = _lengths(case)
    table, P = s["table"].tolist(), case["page"]
    # H by its definition: (-1)^(ones that the binary numbers i and j share)
    i = torch.arange(d, device="cuda")
    both = i[:, None] & i[None, :]
    H = torch.ones(d, d, dtype=torch.float64, device="cuda")
    for k in range(d.bit_length() - 1):
        H = torch.where((both >> k & 1).bool(), -H, H)

    def held(name, pages, x):
        """The first x tokens of a sequence as [heads, x, d]."""
        which = torch.tensor(pages[: (x + P - 1) // P], device="cuda")
        words = s[name][0, which].transpose(0, 1).reshape(hk, -1, d // 2)[:, :x].contiguous().view(torch.int32).long()
        scale = s[name + "_scale"][0, which].transpose(0, 1).reshape(hk, -1)[:, :x].double()
        u = torch.empty(hk, x, d, dtype=torch.float64, device="cuda")
        for c in range(8):
            u[..., c::8] = (words >> (4 * (c // 2) + 16 * (c % 2)) & 15).double()
        return ((u - 7.5) @ H) * scale[..., None]

    if case["kind"] == "read":
        return tuple(torch.cat([held(name, pages, x).transpose(0, 1) for x, pages in zip(t, table)]) for name in ("K", "V"))
    if case["kind"] in ("rotary", "store"):
        R = case["rot"]
        first = torch.arange(0, R, 2, device="cuda") if case["interleaved"] else torch.arange(R // 2, device="cuda")
        second = first + (1 if case["interleaved"] else R // 2)
        at = torch.tensor([case["offset"] + p for n, x in zip(q, t) for p in range(x - n, x)], device="cuda")
        # a pair is a complex number, the rotation a product with one of size 1
        turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]

        def turned(x):
            x = x.double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        k, v, rows = turned(s["new_k"]), s["new_v"].double(), turned(s["Q"])
        if case["kind"] == "store":
            def kept(x):
                step = STEP * x.norm(dim=-1, keepdim=True)
                u = torch.floor((x @ H) / step).clamp(-8, 7) + 0.5
                return (u @ H) * step / d

            return kept(k), kept(v), rows
        K, V = s["K"].double(), s["V"].double()
        r = 0
        for n, x, pages in zip(q, t, table):
            p = x - n
            while p < x:  # the part of the new tokens that falls into one page
                m = min(P - p % P, x - p)
                for X, new in ((K, k), (V, v)):
                    X[0, pages[p // P], :, p % P: p % P + m] = new[r: r + m].transpose(0, 1)
                p, r = p + m, r + m
        return K, V, rows
    group = hq // hk
    out = torch.zeros(sum(q), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(q), hq, dtype=torch.float64, device="cuda")
    slopes, window = s["score"].get("slopes"), case.get("window") or 1 << 40
    r = 0
    for n, x, pages in zip(q, t, table):
        k, v = held("K", pages, x), held("V", pages, x)
        key = torch.arange(x, device="cuda")[None, :]
        for b in range(0, n, 1024):  # rows in blocks, to keep the scores small
            m = min(1024, n - b)
            p = (x - n + b + torch.arange(m, device="cuda"))[:, None]
            hidden = (key > p) | (key <= p - window)
            for head in range(hq):
                y = (s["Q"][r + b: r + b + m, head].double() @ k[head // group].T) / math.sqrt(d)
                if case.get("cap"):
                    y = case["cap"] * torch.tanh(y / case["cap"])
                if slopes is not None:
                    y = y - float(slopes[head]) * (p - key).abs().double()
                y[hidden] = -math.inf
                z = torch.logsumexp(y, 1)
                lse[r + b: r + b + m, head] = z
                out[r + b: r + b + m, head] = torch.exp(y - z[:, None]) @ v[head // group]
        r += n
    return out, lse
