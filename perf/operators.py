"""Operators over paged private KV caches: the cases that are measured.

An agent that reads the shared pool keeps its own tokens in pages of a bf16
cache, K and V [layers, pages, kv_heads, page_tokens, head_dim]. Token j of
sequence s is slot j % page_tokens of page table[s, j // page_tokens]. The
operators write a layer's new tokens into their slots ("append"), copy whole
pages of every layer when a sequence forks or the cache is compacted ("copy"),
and attend chunks of new tokens over the pages ("attend"), with optional
modifiers of the scores ("scored": a tanh cap, a bias by distance, a window, a
document mask, a prefix mask).
"""

import math

import torch

own = False

#: (kv_heads, q_heads, head_dim): the shapes of this repository's workloads, and one whose group of query heads is odd
HEADS = {"tiny": (2, 4, 64), "smollm2": (32, 32, 64), "llama3": (8, 32, 128), "qwen3": (8, 64, 128), "group7": (4, 28, 128)}


def listed():
    return [
        # one decode step of three agents right after they started: launch latency
        dict(name="decode_tiny", kind="attend", heads="tiny", page=16, seqs=3, q_min=1, q_max=1, kv_min=40, kv_max=129),
        # one decode step of 32 agents, 32K tokens each: bandwidth
        dict(name="decode_qwen3_32k", kind="attend", heads="qwen3", page=128, seqs=32, q_min=1, q_max=1, kv_min=30001, kv_max=32768),
        # a few draft tokens of one agent verified over a long history: little parallelism but the context's
        dict(name="verify_group7", kind="attend", heads="group7", page=32, seqs=1, q_min=5, q_max=5, kv_min=20011, kv_max=20011),
        # a mixed batch: tool answers of up to 777 tokens next to decoding agents
        dict(name="mixed_llama3", kind="attend", heads="llama3", page=16, seqs=12, q_min=1, q_max=777, kv_min=900, kv_max=4099),
        # a prompt read in chunks: 2,048 new tokens at the end of 16K
        dict(name="chunk_llama3_16k", kind="attend", heads="llama3", page=64, seqs=1, q_min=2048, q_max=2048, kv_min=16384, kv_max=16384),
        # whole short prompts of ragged lengths, one query head per KV head
        dict(name="prompts_smollm2", kind="attend", heads="smollm2", page=32, seqs=6, q_min=100, q_max=1851, kv_min=100, kv_max=1851),
        # one decode step of 15 agents with private histories of 600 to 7,194 tokens (the repository's long context), in a layer
        # whose scores are capped, fall with the distance and end at a window
        dict(name="scored_decode", kind="attend", heads="llama3", page=64, seqs=15, q_min=1, q_max=1, kv_min=600, kv_max=7194,
             cap=30.0, slopes=True, window=4096),
        # packed documents behind a common prefix, capped scores
        dict(name="scored_chunk", kind="attend", heads="llama3", page=64, seqs=2, q_min=1000, q_max=1500, kv_min=3500, kv_max=4000,
             cap=50.0, slopes=True, document=300, prefix=257),
        # one layer's new token of 15 agents into their pages: launch latency
        dict(name="append_decode", kind="append", heads="llama3", page=64, seqs=15, q_min=1, q_max=1, kv_min=600, kv_max=7194, layers=2),
        # one layer's new tokens of a batch of long chunks
        dict(name="append_chunks", kind="append", heads="llama3", page=16, seqs=9, q_min=500, q_max=4096, kv_min=4096, kv_max=8192, layers=1),
        # 15 forks: the last, partly filled page of each, in 32 layers
        dict(name="copy_forks", kind="copy", heads="llama3", page=16, pairs=15, pages=256, layers=32),
        # a cache compacted: every second page moves
        dict(name="copy_compact", kind="copy", heads="qwen3", page=64, pairs=500, pages=1000, layers=8),
    ]


def _spread(lo, hi, n, turn):
    """n whole numbers from lo to hi, spread over the range, the largest among them."""
    return [hi if i == 0 else lo + int((hi - lo) * math.modf(i * turn)[0] + 0.5) for i in range(n)]


def _lengths(c):
    """New tokens and held tokens (the new ones among them) of each sequence."""
    q = _spread(c["q_min"], c["q_max"], c["seqs"], 0.6180339887498949)
    t = _spread(c["kv_min"], c["kv_max"], c["seqs"], 0.4142135623730951)
    if c["q_min"] == c["kv_min"] and c["q_max"] == c["kv_max"]:  # whole prompts
        return q, q
    return q, [max(a, b) for a, b in zip(q, t)]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["decode", "decode", "chunk", "chunk", "chunk", "prompts", "append", "copy"])
    heads = rng.choice(list(HEADS))
    hk, hq, d = HEADS[heads]
    page = rng.choice([16, 32, 64, 128])
    if kind == "copy":
        layers = log(1, 32)
        most = max(1, min(1000, (500 << 20) // (layers * hk * page * d * 2)))
        pairs = log(1, most)
        return dict(kind="copy", heads=heads, page=page, pairs=pairs, pages=2 * pairs + rng.randrange(9), layers=layers)
    if kind == "decode":
        kv = log(1, 32768)
        seqs = log(1, max(1, min(32, (1 << 28) // (kv * hk * d))))
        c = dict(kind="attend", heads=heads, page=page, seqs=seqs, q_min=1, q_max=rng.choice([1, 1, 1, 2, 4]),
                 kv_min=max(1, kv // rng.randrange(1, 9)), kv_max=kv)
    elif kind == "append":
        q = log(1, 4096)
        c = dict(kind="append", heads=heads, page=page, seqs=log(1, max(1, min(16, 20000 // q))), q_min=max(1, q // 8), q_max=q,
                 kv_min=q, kv_max=q + log(1, 4096), layers=rng.randrange(1, 3))
    else:
        q = log(2, 2048)
        kv = q if kind == "prompts" else q + log(1, 16384 - q)
        seqs = log(1, max(1, min(16, (1 << 30) // (q * hq * kv))))
        low = max(1, q // rng.randrange(1, 9))
        c = dict(kind="attend", heads=heads, page=page, seqs=seqs, q_min=low, q_max=q, kv_min=low if kind == "prompts" else max(1, kv // 2), kv_max=kv)
    if c["kind"] == "attend" and rng.random() < 0.4:
        c["cap"] = rng.choice([0.0, 20.0, 50.0])
        c["slopes"] = rng.random() < 0.5
        pick = rng.randrange(4)
        if pick == 1:
            c["window"] = log(1, 4096)
        elif pick == 2:
            c["document"] = log(16, 1024)
        elif pick == 3:
            c["prefix"] = log(1, 2 * c["q_max"])
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

    s = {"kind": case["kind"], "layer": case.get("layers", 1) - 1}
    if case["kind"] == "copy":
        s["K"], s["V"] = (normal(case["layers"], case["pages"], hk, P, d) for _ in range(2))
        order = torch.randperm(case["pages"], generator=g, device="cuda").cpu()
        s["src"], s["dst"] = order[: case["pairs"]].tolist(), order[case["pairs"]: 2 * case["pairs"]].tolist()
        return s
    q, t = _lengths(case)
    need = [(x + P - 1) // P for x in t]
    pages = sum(need) + 3
    s["K"], s["V"] = (normal(case.get("layers", 1), pages, hk, P, d) * _channels((hk, 1, d), g) for _ in range(2))
    # each sequence's pages lie scattered over the cache; entries behind its last page are not used
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(q), max(need), dtype=torch.int32, device="cuda")
    used = torch.arange(max(need), device="cuda")[None, :] < _ints(need)[:, None]
    table[used] = order[: sum(need)]
    start = [0]
    for n in q:
        start.append(start[-1] + n)
    s |= {"table": table, "kv_len": _ints(t), "q_start": _ints(start), "max_q": max(q), "max_kv": max(t)}
    if case["kind"] == "append":
        # what a projection gives: K and V next to each other in one row per token
        kv = normal(start[-1], 2, hk, d)
        s["new_k"], s["new_v"] = kv[:, 0], kv[:, 1]
        return s
    s["Q"] = normal(start[-1], hq, d)
    s["score"] = {}
    if case.get("cap"):
        s["score"]["cap"] = case["cap"]
    if case.get("slopes"):
        s["score"]["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda", dtype=torch.float32) / hq)
    if case.get("window"):
        s["score"]["window"] = case["window"]
    if case.get("document"):
        at = [(x - n + i) // case["document"] * case["document"] for n, x in zip(q, t) for i in range(n)]
        s["score"]["first"] = _ints(at)
    if case.get("prefix"):
        s["score"]["prefix"] = _ints([case["prefix"]] * len(q))
    return s


def _plain_append(s):
    P = s["K"].shape[3]
    row = torch.arange(s["new_k"].shape[0], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    at = s["kv_len"].long()[seq] - s["q_start"].long()[seq + 1] + row
    page = s["table"].long()[seq, at // P]
    s["K"][s["layer"]][page, :, at % P] = s["new_k"]
    s["V"][s["layer"]][page, :, at % P] = s["new_v"]
    return s["K"], s["V"]


def _plain_attend(s, cap=0.0, slopes=None, window=0, first=None, prefix=None):
    hk, P, d = s["K"].shape[2:]
    tokens, hq = s["Q"].shape[:2]
    S, n, T = s["table"].shape[0], s["max_q"], s["table"].shape[1] * P
    count, held = s["q_start"].diff().long(), s["kv_len"].long()
    i, j = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    # rows of the batch, one sequence each, as [S, n]; places behind a sequence's last row go to a row that is dropped
    real = i < count[:, None]
    row = torch.where(real, s["q_start"][:-1].long()[:, None] + i, tokens)
    q = torch.cat([s["Q"], s["Q"].new_zeros(1, hq, d)])[row].float().view(S, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    k, v = (x[s["layer"]][s["table"].long()].transpose(1, 2).reshape(S, hk, T, d).float() for x in (s["K"], s["V"]))
    x = torch.matmul(q.reshape(S, hk, -1, d), k.transpose(2, 3)).mul_(d ** -0.5).view(S, hk, hq // hk, n, T)
    at = (held - count)[:, None] + i
    if cap:
        x = x.div_(cap).tanh_().mul_(cap)
    if slopes is not None:
        x = x.sub_(slopes.view(1, hk, hq // hk, 1, 1) * (at[:, :, None] - j).abs()[:, None, None])
    seen = j <= at[:, :, None]
    if window:
        seen = seen & (j > at[:, :, None] - window)
    if prefix is not None:
        seen = seen | (j < prefix[:, None, None])
    if first is not None:
        seen = seen & (j >= torch.cat([first, first.new_zeros(1)])[row][:, :, None])
    seen = (seen & (j < held[:, None, None]))[:, None, None]
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S, hk, -1, T), v).view(S, hk, hq // hk, n, d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    out = s["Q"].new_zeros(tokens + 1, hq, d)
    out[row] = o.permute(0, 3, 1, 2, 4).reshape(S, n, hq, d).to(torch.bfloat16)
    at_row = torch.zeros(tokens + 1, hq, device="cuda")
    at_row[row] = lse.permute(0, 3, 1, 2).reshape(S, n, hq)
    return out[:tokens], at_row[:tokens]


def run(state):
    s = state
    if own:
        from shared_quantized_kv_gb300 import kvpool

        if s["kind"] == "copy":
            kvpool.pages_copy(s["K"], s["V"], s["src"], s["dst"])
            return s["K"], s["V"]
        if s["kind"] == "append":
            kvpool.pages_append(s["K"], s["V"], s["layer"], s["new_k"], s["new_v"], s["table"], s["kv_len"], s["q_start"])
            return s["K"], s["V"]
        return kvpool.pages_attend(s["K"], s["V"], s["layer"], s["Q"], s["table"], s["kv_len"], s["q_start"], max_q=s["max_q"],
                                   max_kv=s["max_kv"], return_lse=True, **s["score"])
    if s["kind"] == "copy":
        s["K"][:, s["dst"]] = s["K"][:, s["src"]]
        s["V"][:, s["dst"]] = s["V"][:, s["src"]]
        return s["K"], s["V"]
    if s["kind"] == "append":
        return _plain_append(s)
    return _plain_attend(s, **s["score"])


def _seen_from(case, p):
    """The keys up to its own that a row at position p sees, as (first, end); and the end of the prefix that it sees besides."""
    lo = p - case["window"] + 1 if case.get("window") else 0
    doc = p // case["document"] * case["document"] if case.get("document") else 0
    return max(lo, doc, 0), p + 1, max(doc, 0), case.get("prefix") or 0


def work(case):
    hk, hq, d = HEADS[case["heads"]]
    if case["kind"] == "copy":
        return {"bytes": 2 * 2 * case["pairs"] * case["layers"] * hk * case["page"] * d * 2, "flops": 0}
    q, t = _lengths(case)
    if case["kind"] == "append":
        return {"bytes": 2 * 2 * sum(q) * hk * d * 2 + 4 * (3 * len(q) + 1), "flops": 0}
    pairs = held = 0
    for n, x in zip(q, t):
        used_from, used_to, pre = x, 0, 0
        for p in range(x - n, x):
            lo, end, doc, prefix = _seen_from(case, p)
            more = min(prefix, x)
            # the union of [lo, end) and [doc, more)
            pairs += end - lo + max(0, min(more, lo) - doc) + max(0, more - max(end, doc))
            used_from, used_to, pre = min(used_from, lo), max(used_to, end), max(pre, more if more > doc else 0)
        held += used_to - used_from + max(0, min(pre, used_from))
    rows = sum(q) * hq
    return {"bytes": rows * d * 2 * 2 + rows * 4 + 2 * held * hk * d * 2, "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    P = case["page"]
    if case["kind"] == "copy":
        for a, b in zip(s["src"], s["dst"]):
            for X in (s["K"], s["V"]):
                X[:, b].copy_(X[:, a])
        return s["K"], s["V"]
    q, t = _lengths(case)
    table = s["table"].tolist()
    if case["kind"] == "append":
        r = 0
        for n, x, pages in zip(q, t, table):
            at = x - n
            while at < x:  # the part of the new tokens that falls into one page
                m = min(P - at % P, x - at)
                for X, new in ((s["K"], s["new_k"]), (s["V"], s["new_v"])):
                    X[s["layer"], pages[at // P], :, at % P: at % P + m] = new[r: r + m].transpose(0, 1)
                at, r = at + m, r + m
        return s["K"], s["V"]
    hk, hq, d = HEADS[case["heads"]]
    group = hq // hk
    out = torch.zeros(sum(q), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(q), hq, dtype=torch.float64, device="cuda")
    slopes = s["score"].get("slopes")
    r = 0
    for n, x, pages in zip(q, t, table):
        which = torch.tensor(pages[: (x + P - 1) // P], device="cuda")
        for h in range(hk):
            k, v = (X[0, which, h].reshape(-1, d)[:x].double() for X in (s["K"], s["V"]))
            for b in range(0, n, 1024):  # rows in blocks, to keep the scores small
                m = min(1024, n - b)
                rows = [_seen_from(case, x - n + b + i) for i in range(m)]
                lo, end, doc, more = (torch.tensor(z, device="cuda")[:, None] for z in zip(*rows))
                key = torch.arange(x, device="cuda")[None, :]
                hidden = ~(((key >= lo) & (key < end)) | ((key >= doc) & (key < more)))
                for e in range(group):
                    head = h * group + e
                    y = (s["Q"][r + b: r + b + m, head].double() @ k.T) / math.sqrt(d)
                    if case.get("cap"):
                        y = case["cap"] * torch.tanh(y / case["cap"])
                    if slopes is not None:
                        y = y - float(slopes[head]) * (end - 1 - key).abs().double()
                    y[hidden] = -math.inf
                    z = torch.logsumexp(y, 1)
                    lse[r + b: r + b + m, head] = z
                    out[r + b: r + b + m, head] = torch.exp(y - torch.where(z == -math.inf, 0.0, z)[:, None]) @ v
        r += n
    return out, lse
