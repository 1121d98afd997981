"""Cases of the operators that serve attention from a paged K/V cache.

Five calls of ``token_indexed_sparse_b200.qsa``: rotary positions and their
gradient (``rope``, ``rope_backward``), writing a step's new K/V into the pages
with the rotation on the way (``cache_append``), and attention of new tokens
over the pages, by route IDs (``paged_forward``) or by position with an
optional window and first tokens that stay visible (``paged_causal``).

Cache layout: pools ``[n_pages, page_size, G, 256]``, a block table ``[B,
max_pages]`` of page IDs, ``kv_len [B]`` tokens held per sequence (the new ones
included) and ``cu_q [B + 1]`` offsets of each sequence's new tokens in the
packed rows; the i-th of a sequence's n new tokens sits at position
``kv_len - n + i``.  Heads are 12 per K/V head, 256 dims, BF16.
"""

import math

import torch

own = False

D = 256     # head dimension
R12 = 12    # query heads per K/V head
SCALE = 1.0 / 16.0
ROPE_BASE = 1.0e6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # training: q and k of a 32768-token sequence, 24 heads on 2, whole head, half layout
        {"name": "rope_train", "op": "rope", "T": 32768, "G": 2, "rot": 256, "inter": False, "factor": 1.0, "docs": 1},
        # the gradient at 16384 packed tokens of 8 documents: a quarter of the head, interleaved, scaled 8 times
        {"name": "rope_grad", "op": "rope_backward", "T": 16384, "G": 1, "rot": 64, "inter": True, "factor": 8.0,
         "docs": 8},
        # a handful of tokens of a decode step, scaled positions far out: latency counts
        {"name": "rope_step", "op": "rope", "T": 7, "G": 2, "rot": 128, "inter": False, "factor": 4.0, "docs": 7},
        # a decode step of 61 sequences: one token each is rotated and written to 16-token pages
        {"name": "append_step", "op": "append", "B": 61, "new": 1, "past": 8192, "G": 2, "page": 16, "rot": 256,
         "inter": False, "factor": 1.0},
        # prefill chunks of 9 sequences, about 16384 tokens in all, onto 64-token pages, half of the head, interleaved
        {"name": "append_chunk", "op": "append", "B": 9, "new": 3640, "past": 4096, "G": 2, "page": 64, "rot": 128,
         "inter": True, "factor": 4.0},
        # one token of one long sequence, 2048 routes over 131072 cached tokens: latency counts
        {"name": "routed_one", "op": "routed", "B": 1, "new": 1, "past": 131071, "G": 1, "page": 64, "W": 2048,
         "blocks": 512, "dup": 0.0, "pad": 0.0},
        # a decode step of 53 sequences of mixed lengths, 564 routes with a tenth repeated
        {"name": "routed_step", "op": "routed", "B": 53, "new": 1, "past": 32768, "G": 2, "page": 16, "W": 564,
         "blocks": 128, "dup": 0.10, "pad": 0.0},
        # a chunk of 2048 tokens at the end of 131072, 2048 routes each, some rows all padding
        {"name": "routed_chunk", "op": "routed", "B": 1, "new": 2048, "past": 129024, "G": 1, "page": 128, "W": 2048,
         "blocks": 512, "dup": 0.0, "pad": 0.05},
        # one token over a whole cache of 131072: the cache read once, latency counts
        {"name": "causal_one", "op": "causal", "B": 1, "new": 1, "past": 131071, "G": 1, "page": 64, "window": 0,
         "sinks": 0},
        # a decode step of 48 sequences of mixed lengths up to 32768 on small pages
        {"name": "causal_step", "op": "causal", "B": 48, "new": 1, "past": 32767, "G": 2, "page": 16, "window": 0,
         "sinks": 0},
        # a prefill chunk of 2048 tokens behind 30000 cached ones
        {"name": "causal_chunk", "op": "causal", "B": 1, "new": 2048, "past": 30000, "G": 2, "page": 64, "window": 0,
         "sinks": 0},
        # ragged chunks of 7 sequences that see a window of 1021 tokens and the first 4
        {"name": "causal_window", "op": "causal", "B": 7, "new": 1150, "past": 8192, "G": 1, "page": 32,
         "window": 1021, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_backward", "append", "routed", "routed", "causal", "causal", "causal"])
    G = rng.choice([1, 2])
    if op in ("rope", "rope_backward"):
        return {"op": op, "T": _log(rng, 1, 32768), "G": G, "rot": rng.choice([32, 64, 96, 128, 256]),
                "inter": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 8.0]), "docs": rng.randint(1, 9)}
    page = rng.choice([16, 32, 64, 128, 256])
    decode = rng.random() < 0.5
    B = _log(rng, 1, 61) if decode else rng.randint(1, 9)
    if op == "append":
        return {"op": op, "B": B, "new": 1 if decode else _log(rng, 2, 3640), "past": _log(rng, 1, 8192), "G": G,
                "page": page, "rot": rng.choice([64, 128, 256]), "inter": rng.random() < 0.5,
                "factor": rng.choice([1.0, 4.0])}
    past = _log(rng, 1, 131071 // B if decode else 30000 // B)
    if op == "routed":
        blocks = _log(rng, 4, 512)
        new = 1 if decode else _log(rng, 2, max(2, 2048 * 512 // (blocks * B)) if blocks > 128 else 2048 // B + 2)
        dup = rng.choice([0.0, 0.10])
        return {"op": op, "B": B, "new": min(new, 2048), "past": past, "G": G, "page": page,
                "W": 4 * blocks + (math.ceil(0.4 * blocks) if dup else 0) + rng.randint(0, 3), "blocks": blocks,
                "dup": dup, "pad": rng.choice([0.0, 0.05])}
    window = rng.choice([0, 0, _log(rng, 1, 4096)])
    return {"op": op, "B": B, "new": 1 if decode else _log(rng, 2, 2048 // B), "past": past, "G": G, "page": page,
            "window": window, "sinks": rng.choice([0, 1, 4, 130]) if window else 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """New and past tokens per sequence, on the host: one sequence takes the
    stated sizes, the others spread below them (so batches are ragged)."""
    B, new, past = case["B"], case["new"], case["past"]
    news = [new if (b == 0 or new == 1) else max(1, new * (1 + (b * 7919) % 97) // 98) for b in range(B)]
    pasts = [past if b == 0 else past * (1 + (b * 6007) % 101) // 102 for b in range(B)]
    return news, pasts


def _frequencies(rot, factor, device):
    """Rotary angles per token step of each pair, in 64 bits.  A factor above 1
    stretches the slow pairs (fewer than one turn over the original 4096
    positions) by it, leaves the fast ones (over 32 turns) as they are and goes
    from one to the other linearly between, with the magnitude that goes with it."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    inv = ROPE_BASE ** (-2.0 * i / rot)
    if factor == 1.0:
        return inv.to(device), 1.0
    turns = 4096.0 * inv / (2.0 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (inv * keep + inv / factor * (1.0 - keep)).to(device), 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16)

    G, op = case["G"], case["op"]
    H = R12 * G
    s = dict(case)
    if op in ("rope", "rope_backward"):
        T = case["T"]
        s["q"], s["k"] = randn(T, H, D), randn(T, G, D)
        # packed documents start over at their own positions; a decode step's tokens are far out
        if case["docs"] >= T:
            s["positions"] = torch.randint(0, 131072, (T,), generator=g, device=dev, dtype=torch.int32)
        else:
            n = -(-T // case["docs"])
            s["positions"] = (torch.arange(T, device=dev) % n).to(torch.int32)
        s["inv_freq"], s["mscale"] = _frequencies(case["rot"], case["factor"], dev)
        return s
    B, page = case["B"], case["page"]
    news, pasts = _lengths(case)
    lens = [a + b for a, b in zip(news, pasts)]
    T, L = sum(news), max(lens)
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + sum(held) // 10 + 1
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(held)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    s["k_pages"], s["v_pages"] = randn(n_pages, page, G, D), randn(n_pages, page, G, D)
    s["block_table"] = table
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["cu_q"] = torch.tensor([0] + news, device=dev).cumsum(0).to(torch.int32)
    s["T"], s["L"], s["n_max"] = T, L, max(news)
    s["q"] = randn(T, H, D)
    if op == "append":
        s["k_new"], s["v_new"] = randn(T, G, D), randn(T, G, D)
        s["inv_freq"], s["mscale"] = _frequencies(case["rot"], case["factor"], dev)
    if op == "routed":
        # four-token blocks: the token's own block and others drawn from those before it, some IDs twice, -1 behind them
        seq = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(news, device=dev))
        pos = s["kv_len"][seq] - s["cu_q"][seq + 1] + torch.arange(T, device=dev)
        own_block = pos // 4
        W, nb = case["W"], case["blocks"]
        routes = torch.full((T, W), -1, dtype=torch.int32, device=dev)
        step = 1 + (1 << 27) // (L // 4 + 1)
        for t0 in range(0, T, step):
            ob = own_block[t0:t0 + step, None]
            w = torch.rand(ob.shape[0], L // 4 + 1, generator=g, device=dev)
            at = torch.arange(L // 4 + 1, device=dev)
            w = torch.where(at == ob, 2.0, torch.where(at < ob, w, -1.0))
            best, pick = w.topk(min(nb, L // 4 + 1), dim=1)
            tok = pick[:, :, None] * 4 + torch.arange(4, device=dev)
            tok = torch.where((best[:, :, None] >= 0) & (tok <= pos[t0:t0 + step, None, None]), tok, -1)
            tok = tok.reshape(ob.shape[0], -1)
            routes[t0:t0 + step, :tok.shape[1]] = tok.to(torch.int32)
        if case["dup"]:
            n = min(W - 4 * nb, math.ceil(4 * nb * case["dup"]))
            routes[:, 4 * nb:4 * nb + n] = routes[:, :n]
            routes = routes[:, torch.randperm(W, generator=g, device=dev)].contiguous()
        if case["pad"]:
            routes[torch.rand(T, generator=g, device=dev) < case["pad"]] = -1
        s["routes"] = routes
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope, "rope_backward": _rope, "append": _append, "routed": _routed, "causal": _causal}[s["op"]](s)


def _run_own(s):
    from token_indexed_sparse_b200 import qsa

    op = s["op"]
    if op == "rope":
        return qsa.rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=s["inter"], mscale=s["mscale"])
    if op == "rope_backward":
        return qsa.rope_backward(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=s["inter"],
                                 mscale=s["mscale"])
    cache = (s["k_pages"], s["v_pages"])
    where = (s["block_table"], s["kv_len"], s["cu_q"])
    if op == "append":
        q = qsa.cache_append(s["k_new"], s["v_new"], *cache, *where, q=s["q"], inv_freq=s["inv_freq"],
                             interleaved=s["inter"], mscale=s["mscale"])
        return q, s["k_pages"], s["v_pages"]
    if op == "routed":
        return qsa.paged_forward(s["q"], *cache, s["routes"], *where, scale=SCALE)
    return qsa.paged_causal(s["q"], *cache, *where, scale=SCALE, window=s["window"], sinks=s["sinks"])


def _rotate(x, positions, inv_freq, mscale, inter, sign):
    angle = positions.double()[:, None] * inv_freq
    cos, sin = (angle.cos() * mscale).float()[:, None], (angle.sin() * (sign * mscale)).float()[:, None]
    n = inv_freq.numel()
    x = x.float()
    head, rest = x[..., :2 * n], x[..., 2 * n:]
    a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., :n], head[..., n:])
    a, b = a * cos - b * sin, a * sin + b * cos
    head = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((head, rest), -1).to(torch.bfloat16)


def _rope(s):
    sign = 1.0 if s["op"] == "rope" else -1.0
    args = (s["positions"], s["inv_freq"], s["mscale"], s["inter"], sign)
    return _rotate(s["q"], *args), _rotate(s["k"], *args)


def _rows(s):
    """Sequence and position of every packed row."""
    row = torch.arange(s["T"], device=s["q"].device)
    seq = torch.searchsorted(s["cu_q"], row.to(torch.int32), right=True) - 1
    return seq, s["kv_len"][seq] - s["cu_q"][seq + 1] + row


def _slots(s, seq, pos):
    """Rows of the pools, seen as [n_pages * page_size, G, D], of positions of sequences."""
    page = s["page"]
    return s["block_table"][seq, pos // page].long() * page + pos % page


def _append(s):
    seq, pos = _rows(s)
    args = (pos, s["inv_freq"], s["mscale"], s["inter"], 1.0)
    at = _slots(s, seq, pos)
    s["k_pages"].view(-1, s["G"], D)[at] = _rotate(s["k_new"], *args)
    s["v_pages"].view(-1, s["G"], D)[at] = s["v_new"]
    return _rotate(s["q"], *args), s["k_pages"], s["v_pages"]


def _softmax(scores, visible):
    """Probabilities and the natural-log sum over the last axis; rows that see nothing get zeros and -inf."""
    scores = scores.masked_fill_(~visible, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (scores - top).exp()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    return p / torch.where(total == 0, 1.0, total), lse


def _routed(s):
    T, G = s["T"], s["G"]
    seq, pos = _rows(s)
    r = s["routes"].sort(1).values
    seen = (r >= 0) & (r < s["kv_len"][seq][:, None])
    seen[:, 1:] &= r[:, 1:] != r[:, :-1]
    at = torch.where(seen, _slots(s, seq[:, None], r.clamp(min=0).where(seen, 0)), 0)
    k = s["k_pages"].view(-1, G, D)[at].float().transpose(1, 2)      # [T, G, W, D]
    v = s["v_pages"].view(-1, G, D)[at].float().transpose(1, 2)
    q = s["q"].float().view(T, G, R12, D)
    p, lse = _softmax(q @ k.mT * SCALE, seen[:, None, None])
    return (p @ v).reshape(T, G * R12, D).to(torch.bfloat16), lse.reshape(T, G * R12)


def _causal(s):
    T, G, L, N = s["T"], s["G"], s["L"], s["n_max"]
    B = s["B"]
    dev = s["q"].device
    seq, pos = _rows(s)
    row = torch.arange(T, device=dev) - s["cu_q"][seq]
    # every sequence's cache, and its new tokens, side by side
    j = torch.arange(L, device=dev).expand(B, L)
    inside = j < s["kv_len"][:, None]
    at = torch.where(inside, _slots(s, torch.arange(B, device=dev)[:, None], j), 0)
    k = s["k_pages"].view(-1, G, D)[at].float().permute(0, 2, 3, 1)  # [B, G, D, L]
    v = s["v_pages"].view(-1, G, D)[at].float().transpose(1, 2)      # [B, G, L, D]
    q = torch.zeros(B, N, G, R12, D, device=dev)
    q[seq, row] = s["q"].float().view(T, G, R12, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, G, N * R12, D)
    p_of = torch.full((B, N), -1, dtype=pos.dtype, device=dev)
    p_of[seq, row] = pos
    sees = j[:, None] <= p_of[:, :, None]
    if s["window"]:
        sees &= (j[:, None] > p_of[:, :, None] - s["window"]) | (j[:, None] < s["sinks"])
    sees = sees[:, None, :, None].expand(B, 1, N, R12, L).reshape(B, 1, N * R12, L)
    p, lse = _softmax((q @ k).mul_(SCALE), sees)
    out = (p @ v).view(B, G, N, R12, D)[seq, :, row].reshape(T, G * R12, D)
    return out.to(torch.bfloat16), lse.view(B, G, N, R12)[seq, :, row].reshape(T, G * R12)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _visible(pos, window, sinks):
    """Keys that a token at `pos` sees."""
    if not window or window > pos:
        return pos + 1
    return window + min(sinks, pos + 1 - window)


def work(case):
    G = case["G"]
    H = R12 * G
    row = D * 2
    if case["op"] in ("rope", "rope_backward"):
        # q and k in and out, positions and frequencies in; a rotation is 6 operations a pair
        T = case["T"]
        return {"bytes": 2 * T * (H + G) * row + 4 * T + 4 * case["rot"], "flops": 3 * T * (H + G) * case["rot"]}
    news, pasts = _lengths(case)
    T = sum(news)
    tables = 4 * sum(-(-(a + b) // case["page"]) for a, b in zip(news, pasts)) + 8 * case["B"] + 4
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * G) * row + 4 * 2 * case["B"] + 4 * T + 4 * case["rot"],
                "flops": 3 * T * (H + G) * case["rot"]}
    outputs = 2 * T * H * row + 4 * T * H
    if case["op"] == "routed":
        # the pages' rows that some route names, each once (at most all that is held)
        pairs = named = 0
        for n, past in zip(news, pasts):
            seq_pairs = sum(min(4 * case["blocks"], past + i + 1) for i in range(n))
            pairs += seq_pairs
            named += min(seq_pairs, past + n)
        pairs, named = pairs * (1 - case["pad"]), named if T > 1000 else named * (1 - case["pad"])
        return {"bytes": outputs + 4 * T * case["W"] + 2 * named * G * row + tables, "flops": 4 * pairs * H * D}
    pairs = keys = 0
    for n, past in zip(news, pasts):
        pairs += sum(_visible(past + i, case["window"], case["sinks"]) for i in range(n))
        first = max(0, past + 1 - case["window"]) if case["window"] else 0
        keys += past + n - first + min(case["sinks"] if case["window"] else 0, first)
    return {"bytes": outputs + 2 * keys * G * row + tables, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _turned(x, positions, inv_freq, mscale, inter, sign):
    """Each pair as a complex number times mscale * exp(i * sign * angle)."""
    x = x.to(torch.float64).clone()
    n = inv_freq.numel()
    turn = torch.polar(torch.full((positions.numel(), n), mscale, dtype=torch.float64, device=x.device),
                       sign * positions.to(torch.float64)[:, None] * inv_freq)[:, None, :]
    first = slice(0, 2 * n, 2) if inter else slice(0, n)
    second = slice(1, 2 * n, 2) if inter else slice(n, 2 * n)
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op, G = s["op"], s["G"]
    if op in ("rope", "rope_backward"):
        sign = 1.0 if op == "rope" else -1.0
        args = (s["positions"], s["inv_freq"], s["mscale"], s["inter"], sign)
        return _turned(s["q"], *args), _turned(s["k"], *args)
    news, pasts = _lengths(case)
    page, dev = s["page"], s["q"].device
    starts = s["cu_q"].tolist()
    table = s["block_table"].long()
    if op == "append":
        kp, vp = (s[n].to(torch.float64).reshape(-1, G, D) for n in ("k_pages", "v_pages"))
        q = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        for b, (n, past) in enumerate(zip(news, pasts)):
            a, z = starts[b], starts[b] + n
            pos = torch.arange(past, past + n, device=dev)
            at = table[b][pos // page] * page + pos % page
            args = (pos, s["inv_freq"], s["mscale"], s["inter"], 1.0)
            q[a:z] = _turned(s["q"][a:z], *args)
            kp[at] = _turned(s["k_new"][a:z], *args)
            vp[at] = s["v_new"][a:z].to(torch.float64)
        return q, kp.view(s["k_pages"].shape), vp.view(s["v_pages"].shape)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=dev)
    for b, (n, past) in enumerate(zip(news, pasts)):
        length = past + n
        j = torch.arange(length, device=dev)
        at = table[b][j // page] * page + j % page
        step = max(1, (1 << 28) // (length * R12))  # query rows at a time
        for g in range(G):
            k = s["k_pages"].view(-1, G, D)[at, g].to(torch.float64)
            v = s["v_pages"].view(-1, G, D)[at, g].to(torch.float64)
            heads = slice(g * R12, (g + 1) * R12)
            for a in range(starts[b], starts[b] + n, step):
                z = min(a + step, starts[b] + n)
                if op == "routed":
                    # membership of every cached token in the row's set, one column more for what is padding
                    r = s["routes"][a:z].long()
                    r = torch.where((r < 0) | (r >= length), length, r)
                    sees = torch.zeros(z - a, length + 1, dtype=torch.bool, device=dev).scatter_(1, r, True)[:, :-1]
                else:
                    p = past + torch.arange(a - starts[b], z - starts[b], device=dev)[:, None]
                    sees = j <= p
                    if s["window"]:
                        sees &= (p - j < s["window"]) | (j < s["sinks"])
                dots = torch.einsum("thd,jd->thj", s["q"][a:z, heads].to(torch.float64), k) * SCALE
                dots = torch.where(sees[:, None], dots, -math.inf)
                lse[a:z, heads] = torch.logsumexp(dots, -1)
                weight = torch.where(sees[:, None], (dots - lse[a:z, heads, None]).exp(), 0.0)
                out[a:z, heads] = weight @ v
    return out, lse
