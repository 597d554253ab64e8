"""Operators on the 4-bit paged cache around drafted tokens and bounded memory: what is measured, and their plain forms.

Four operators; a step of a server that verifies drafted trees under a bound on the cache runs them in
this order (behind the append of the drafted tokens):

* ``tree``     attention of a tree of drafted tokens over the cache: a row sees the keys in front of the
               tree and those drafted keys that its mask names (its ancestors and itself)
* ``accept``   the accepted path's keys and values move together behind the committed ones
* ``weights``  each key's accumulated attention weight: the sum over rows and heads of its probability
* ``evict``    sequences longer than a budget keep their first and newest keys and those of the largest
               weights; the places of the others are filled from behind

The cache is uint8 [pages][kv heads][page_size / 16][18 * head_dim]: 16 tokens at a time, the codes of K
(16 x head_dim / 2 bytes, even dimension in the low nibble), those of V, K's scales (16 x head_dim / 16
bytes) and V's.  A value is e2m1(code) * e4m3(scale of its 16 dimensions) * the cache's own factor.
"""
import math
import random

import torch

own = False

K_SCALE, V_SCALE = 1.0 / 32, 1.0 / 64
WORKSPACE = 96 << 20
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    tree = dict(op="tree", head_dim=128, window=0)
    acc = dict(op="accept", head_dim=128)
    wei = dict(op="weights", head_dim=128, window=0, path=False)
    evi = dict(op="evict", head_dim=128)
    return [
        # one request's small tree: the latency of the call
        dict(tree, name="tree 1 x 15", seqs=1, q_min=15, q_max=15, kv_min=700, kv_max=700, q_heads=32, kv_heads=8,
             page_size=16, dtype="bf16"),
        # a batch of requests with trees of all sizes up to 64 nodes
        dict(tree, name="tree 32 x 64", seqs=32, q_min=9, q_max=64, kv_min=500, kv_max=4000, q_heads=32, kv_heads=8,
             page_size=16, dtype="bf16"),
        # trees in a window, narrow heads, the other type, more than one word of mask
        dict(tree, name="tree 20 x 37 window f16", seqs=20, q_min=33, q_max=37, kv_min=200, kv_max=5000, q_heads=24,
             kv_heads=4, page_size=32, dtype="f16", head_dim=64, window=2048),
        # two very long requests, every head with keys of its own
        dict(tree, name="tree 2 x 60 x 100000", seqs=2, q_min=50, q_max=60, kv_min=60000, kv_max=100000, q_heads=32,
             kv_heads=32, page_size=64, dtype="bf16"),
        # one request's accepted path: the latency of the call
        dict(acc, name="accept 1", seqs=1, q_min=15, q_max=15, kv_min=700, kv_max=700, kv_heads=8, page_size=16),
        # a full batch, every head with keys of its own
        dict(acc, name="accept 256 x 64", seqs=256, q_min=9, q_max=64, kv_min=64, kv_max=500, kv_heads=32,
             page_size=32),
        # one request's next token: the latency of the call
        dict(wei, name="weights 1 x 700", seqs=1, q_min=1, q_max=1, kv_min=700, kv_max=700, q_heads=32, kv_heads=8,
             page_size=16, dtype="bf16"),
        # a full decode batch with histories of all lengths
        dict(wei, name="weights 256 x 4096", seqs=256, q_min=1, q_max=1, kv_min=1, kv_max=4096, q_heads=32, kv_heads=8,
             page_size=16, dtype="bf16"),
        # prompts: chunks of several requests, some with a history
        dict(wei, name="weights prefill 6 x 2000", seqs=6, q_min=700, q_max=2000, kv_min=2000, kv_max=5000, q_heads=32,
             kv_heads=8, page_size=64, dtype="bf16"),
        # one request, one token past its budget: the latency of the call
        dict(evi, name="evict 1 x 1025", seqs=1, kv_min=1025, kv_max=1025, kv_heads=8, page_size=16, budget=1024,
             sink=4, recent=128, prompt=False),
        # a batch that evicts after every few tokens; some sequences are still within the budget
        dict(evi, name="evict 256 x 2100", seqs=256, kv_min=2000, kv_max=2100, kv_heads=8, page_size=16, budget=2048,
             sink=4, recent=256, prompt=False),
        # prompts that shrink to their budget at once
        dict(evi, name="evict prompts 6 x 30000", seqs=6, kv_min=10000, kv_max=30000, kv_heads=8, page_size=64,
             budget=2000, sink=16, recent=64, prompt=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "weights", "accept", "evict", "evict"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 48, 64])
    kvh = rng.choice([1, 2, 3, 4, 8, 8, 32])
    qh = kvh * rng.choice([1, 2, 4, 5, 6, 8] if kvh <= 8 else [1, 2])
    case = dict(op=op, kv_heads=kvh, head_dim=d, page_size=page)
    if op == "evict":
        prompt = rng.random() < 0.4
        budget = _log(rng, 20, 4000)
        kv_max = budget + (_log(rng, 1, 30000 - budget) if prompt else _log(rng, 1, 100))
        seqs = _log(rng, 1, max(1, min(256, 256 * 2100 * 8 // (kv_max * kvh))))
        sink = rng.choice([0, 4, budget // 10])
        return dict(case, seqs=seqs, kv_min=rng.randint(1, kv_max), kv_max=kv_max, budget=budget, sink=sink,
                    recent=rng.choice([0, 1, budget // 4, budget - sink]), prompt=prompt)
    if op == "accept":
        q_max = _log(rng, 1, 128)
        return dict(case, seqs=_log(rng, 1, max(1, min(256, 256 * 32 // kvh))), q_min=rng.randint(1, q_max), q_max=q_max,
                    kv_min=q_max, kv_max=q_max + _log(rng, 1, 500))
    case = dict(case, q_heads=qh, dtype=rng.choice(["bf16", "bf16", "f16"]), window=rng.choice([0, 0, 0, 200, 1000]))
    kind = "tree" if op == "tree" else rng.choice(["decode", "decode", "path", "prefill"])
    if kind == "prefill":
        q_max = _log(rng, 40, 2000)
        kv_max = q_max + _log(rng, 1, 3000)
        seqs = _log(rng, 1, max(1, min(8, int(1.2e4 * 32 / (q_max * qh)))))
        return dict(case, path=False, seqs=seqs, q_min=rng.randint(1, q_max), q_max=q_max, kv_min=rng.randint(1, q_max),
                    kv_max=kv_max)
    q_max = 1 if kind == "decode" else _log(rng, 2, 128)
    kv_max = q_max + _log(rng, 1, 100000 if kind == "tree" else 30000)
    most = min(256 * 4096 * 8 / (kv_max * kvh), 2 * 60 * 80000 * 32 / (kv_max * q_max * qh))
    case = dict(case, seqs=_log(rng, 1, max(1, min(256, int(most)))), q_min=rng.randint(1, q_max), q_max=q_max,
                kv_min=q_max, kv_max=kv_max)
    return case if kind == "tree" else dict(case, path=kind == "path")


def _rng(case):
    return random.Random(1000003 * case["seqs"] + 1009 * case["kv_max"] + case.get("q_max", 0))


def _lengths(case):
    """The sequences' (rows, keys): part of the case, not of the inputs' seed."""
    r = _rng(case)
    got = []
    for _ in range(case["seqs"]):
        kv = r.randint(case["kv_min"], case["kv_max"])
        got.append((r.randint(case["q_min"], case["q_max"]) if "q_min" in case else 1, kv))
    return got


def _trees(case):
    """Each sequence's tree (a row's ancestors and itself as bits) and an accepted path (rows, maybe none)."""
    r = _rng(case)
    r.random()
    masks, paths = [], []
    for m, _ in _lengths(case):
        mask = []
        for i in range(m):  # drafters go deep along their best guesses
            parent = i - 1 if r.random() < 0.5 else r.randint(-1, i - 1)
            mask.append((mask[parent] if parent >= 0 else 0) | 1 << i)
        last = r.randint(-1, m - 1)
        masks.append(mask)
        paths.append([i for i in range(m) if last >= 0 and mask[last] >> i & 1])
    return masks, paths


def _step(case):
    """By how much the positions of an eviction's sequences go on from pass to pass."""
    return case["kv_max"] - (0 if case["prompt"] else case["budget"])


def _pairs(q, kv, window):
    """(query row, key) pairs that the causal mask of one sequence leaves, and the keys that any row sees."""
    first = kv - q  # position of the first row
    pairs = sum(max(0, min(p, kv - 1) - max(0, p - window + 1 if window else 0) + 1)
                for p in range(max(0, first), kv))
    lo = max(0, first - window + 1) if window else 0
    return pairs, max(0, kv - lo) if pairs else 0


def work(case):
    d, kvh, op = case["head_dim"], case["kv_heads"], case["op"]
    entry = d * 9 // 8  # bytes of a token's K and V in one head
    lengths = _lengths(case)
    if op == "evict":
        # a weight and a position a key, and what has to move; new positions are written
        n = sum(kv for _, kv in lengths)
        over = [kv - case["budget"] for _, kv in lengths if kv > case["budget"]]
        moved = sum(min(x, case["budget"]) if not case["prompt"] else
                    round(case["budget"] * x / (x + case["budget"])) for x in over)
        return {"bytes": kvh * (8 * n + moved * (2 * entry + 16) + 4 * sum(over)), "flops": kvh * n}
    if op == "accept":
        _, paths = _trees(case)
        moved = sum(i != c for p in paths for i, c in enumerate(p))
        return {"bytes": kvh * moved * 2 * entry + 12 * case["seqs"] + 4 * sum(len(p) for p in paths), "flops": 0}
    qh, w = case["q_heads"], case["window"]
    if op == "tree":
        masks, _ = _trees(case)
        rows = pairs = keys = 0
        for (m, kv), mask in zip(lengths, masks):
            seen = [min(kv - m, max(0, w - bin(x).count("1")) if w else kv - m) for x in mask]
            rows, keys = rows + m, keys + m + max(seen)
            pairs += sum(seen) + sum(bin(x).count("1") for x in mask)
        return {"bytes": rows * (qh * (4 * d + 4) + 4 * -(-case["q_max"] // 32)) + keys * kvh * entry +
                4 * keys // case["page_size"], "flops": 4 * d * qh * pairs}
    if case["path"]:
        _, paths = _trees(case)
        lengths = [(len(p), kv - m + len(p)) for (m, kv), p in zip(lengths, paths)]
    got = [(q,) + _pairs(q, kv, w) for q, kv in lengths]
    rows, pairs, keys = (sum(x[i] for x in got) for i in range(3))
    return {"bytes": rows * qh * (2 * d + 4) + keys * kvh * (entry // 2 + 8) + 4 * keys // case["page_size"],
            "flops": 2 * d * qh * pairs}


# ------------------------------------------------------------------ inputs

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, d, kvh, page = case["op"], case["head_dim"], case["kv_heads"], case["page_size"]
    lengths = _lengths(case)
    # the pages: in any order, NaN until filled, and behind a sequence's last key
    per = [-(-kv // page) for _, kv in lengths]
    wide, pages = max(per), sum(per) + 2
    cache = torch.full((pages, kvh, page // 16, 18 * d), 255, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (kvh * page * d))
    for a in range(0, pages, step):
        m = min(step, pages - a)
        k, v = (torch.randn(m, kvh, page, d, generator=g, device="cuda") for _ in range(2))
        part = _sections(cache[a:a + m], d)
        for x, factor, codes, scales in ((k, K_SCALE, part[0], part[2]), (v, V_SCALE, part[1], part[3])):
            c, sc = _quantise(x, factor)
            codes.copy_(c.view(codes.shape))
            scales.copy_(sc.view(torch.uint8).view(scales.shape))
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((len(per), wide), pages - 1, dtype=torch.int64)
    at = 0
    for b, m in enumerate(per):
        table[b, :m] = torch.arange(at, at + m)
        at += m
    table = order[table.cuda()]
    for b, (_, kv) in enumerate(lengths):
        if kv % page:
            behind = (torch.arange(page, device="cuda") >= kv % page).view(page // 16, 16, 1)
            for scales in _sections(cache[table[b, per[b] - 1]], d)[2:]:
                scales.masked_fill_(behind, 255)
    s = dict(case=case, cache=cache, table=table.int(), kv_len=_i32([kv for _, kv in lengths]),
             max_kv=max(kv for _, kv in lengths))
    if op in ("accept", "evict"):
        s["kv_len_out"] = torch.zeros(len(per), dtype=torch.int32, device="cuda")
        codes_k, codes_v, scales_k, scales_v = _sections(cache, d)
        s["held"] = [codes_k, codes_v] + [x.view(torch.float8_e4m3fn) for x in (scales_k, scales_v)]
    if op == "evict":
        cap, n = s["max_kv"], s["kv_len"].long()[:, None]
        shape = (len(per), kvh, cap)
        # few keys draw most of the weight; some have drawn none at all
        w = torch.exp(2.0 * torch.randn(shape, generator=g, device="cuda"))
        s["weights"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.05, 0.0, w)
        s["prompt_weights"] = s["weights"].clone() if case["prompt"] else None
        j = torch.arange(cap, device="cuda")
        # what earlier evictions have kept stands anywhere in a longer history; new keys have no position yet
        kept = torch.zeros_like(n) if case["prompt"] else n.clamp(max=case["budget"])
        gaps = torch.randint(1, 4, shape, generator=g, device="cuda").cumsum(-1)
        shuffled = gaps.gather(-1, torch.where(j < kept[..., None], torch.rand(
            shape, generator=g, device="cuda"), 2.0 + j).argsort(-1))
        s["key_pos"] = torch.where(j < kept[..., None], shuffled, -1).int()
        s["last_pos"] = (s["key_pos"].amax((1, 2)) + (n - kept)[:, 0]).int()
        return s
    starts = [0]
    for q, _ in lengths:
        starts.append(starts[-1] + q)
    s |= dict(q_start=_i32(starts), max_q=max(q for q, _ in lengths))
    if op == "accept" or op == "tree" or case["path"]:
        masks, paths = _trees(case)
        s["path"] = _i32([(p + [-1] * s["max_q"])[:s["max_q"]] for p in paths])
        s["path_len"] = _i32([len(p) for p in paths])
    if op == "accept":
        return s
    rows, qh, dt = starts[-1], case["q_heads"], DTYPES[case["dtype"]]
    s["q"] = torch.randn(rows, qh, d, generator=g, device="cuda").to(dt)
    if op == "tree":
        words = -(-s["max_q"] // 32)
        bits = [[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for mask in masks for x in mask]
        s |= dict(mask=torch.tensor([[x - (x >> 31 << 32) for x in row] for row in bits], dtype=torch.int32, device="cuda"),
                  out=torch.zeros(rows, qh, d, dtype=dt, device="cuda"), lse=torch.zeros(rows, qh, device="cuda"),
                  workspace=torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda"))
        return s
    if case["path"]:  # the accepted path's keys have moved together
        s["kv_len"] = (s["kv_len"] - s["q_start"].diff() + s["path_len"]).int()
    else:
        s["path"] = s["path_len"] = None
    score, row, live = _causal_scores(s)  # what the attention has left
    total = torch.logsumexp(score, -1).permute(0, 3, 1, 2).flatten(2, 3)
    s["lse"] = torch.zeros(rows, qh, device="cuda")
    s["lse"][row[live]] = total[live]
    s["weights"] = torch.rand(len(per), kvh, s["max_kv"], generator=g, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _sections(cache, d):
    """K's codes, V's codes, K's scales and V's of a cache, as views [page][head][page_size / 16][16][...]."""
    k, v, ks, vs = cache.split([8 * d, 8 * d, d, d], -1)
    return k.unflatten(-1, (16, d // 2)), v.unflatten(-1, (16, d // 2)), ks.unflatten(-1, (16, d // 16)), \
        vs.unflatten(-1, (16, d // 16))


def _quantise(x, factor):
    """Codes (two a byte) and e4m3 scales of fp32 x[..., d], in blocks of 16."""
    x = (x * (1.0 / factor)).unflatten(-1, (-1, 16))
    sc = (x.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = sc.float()
    y = torch.where(sf > 0, x / torch.where(sf > 0, sf, 1.0), 0.0)
    a = y.abs()
    c = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    c = (c + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), sc.squeeze(-1)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(codes, scales, factor):
    """fp32 values of codes [..., d / 2] and scales [..., d / 16] (bytes)."""
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = lut[c.int()].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.flatten(-2) * factor


def _side(s, which, factor):
    """K (0) or V (1) of the sequences side by side, fp32 [b][j][kv head][d], zero behind their last keys."""
    page, d = s["case"]["page_size"], s["case"]["head_dim"]
    j = torch.arange(s["max_kv"], device="cuda")
    pages = s["table"].long()[:, j // page]
    inside = (j % page).expand_as(pages)
    sections = _sections(s["cache"], d)
    codes, scales = (sections[which + i][pages, :, inside // 16, inside % 16] for i in (0, 2))
    return torch.where((j < s["kv_len"][:, None])[:, :, None, None], _values(codes, scales, factor), 0.0)


def _scores(s, row, seen):
    """Scaled scores [b][kv head][head of it][i][j] of the rows row [b][i], -inf where not seen [b][i][j]."""
    qh, kvh, d = s["case"]["q_heads"], s["case"]["kv_heads"], s["case"]["head_dim"]
    k = _side(s, 0, K_SCALE).permute(0, 2, 3, 1)
    q = s["q"].float()[row].unflatten(2, (kvh, qh // kvh)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (q @ k).mul_(1.0 / math.sqrt(d)).unflatten(2, (qh // kvh, -1))
    return score.masked_fill_(~seen[:, None, None], -math.inf)


def _causal_scores(s):
    """The scores of the rows whose weights are wanted, those rows [b][i], and which of them there are."""
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    first, n = s["q_start"][:-1].long()[:, None], s["kv_len"].long()[:, None]
    if s["path"] is None:
        row, m = first + i, s["q_start"].diff().long()[:, None]
    else:
        row, m = first + s["path"].long(), s["path_len"].long()[:, None]
    live = i < m
    row = torch.where(live, row, first)
    at = (n - m + i)[..., None]
    seen = live[..., None] & (j <= at) & (j < n[..., None])
    if s["case"]["window"]:
        seen = seen & (j > at - s["case"]["window"])
    return _scores(s, row, seen), row, live


def _tree_plain(s):
    c, m, n = s["case"], s["q_start"].diff().long()[:, None], s["kv_len"].long()[:, None]
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_kv"], device="cuda")
    live = i < m
    row = torch.where(live, s["q_start"][:-1].long()[:, None] + i, 0)
    mask = s["mask"].long()[row]  # [b][i][words]
    bits = (mask[..., None] >> torch.arange(32, device="cuda") & 1).flatten(2).bool()
    drafted = j - (n - m)  # [b][j]
    named = bits.gather(2, drafted.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, bits.shape[1], -1))
    seen = torch.where((drafted < 0)[:, None], True, named)
    if c["window"]:
        at = n - m + (bits.sum(-1) - 1).clamp(min=0)  # the row's position
        seen = seen & ((drafted >= 0)[:, None] | (j > at[..., None] - c["window"]))
    score = _scores(s, row, seen & live[..., None] & (j < n)[:, None])
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = _side(s, 1, V_SCALE).permute(0, 2, 1, 3)
    o = (p.flatten(2, 3) @ v).unflatten(2, (c["q_heads"] // c["kv_heads"], -1)) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    o, lse = o.permute(0, 3, 1, 2, 4).flatten(2, 3), lse.permute(0, 3, 1, 2).flatten(2, 3)
    s["out"][:] = o[live].to(s["out"].dtype)
    s["lse"][:] = lse[live]
    return [s["out"], s["lse"]]


def _accept_plain(s):
    page, d = s["case"]["page_size"], s["case"]["head_dim"]
    base = (s["kv_len"] - s["q_start"].diff()).long()[:, None]
    i = torch.arange(s["path"].shape[1], device="cuda")
    taken = i < s["path_len"][:, None]
    to = base + i
    # rows that are not taken copy a place of their own onto itself
    wide = s["table"].shape[1] * page - 1
    of, to = torch.where(taken, base + s["path"].long(), to).clamp(max=wide), to.clamp(max=wide)
    of = torch.where(taken, of, to)
    pages, pages_of = s["table"].long().gather(1, to // page), s["table"].long().gather(1, of // page)
    for x in _sections(s["cache"], d):
        new = x[pages_of, :, of % page // 16, of % 16]
        old = x[pages, :, to % page // 16, to % 16]
        # places behind a table's end were clamped to one: only the taken are written for certain
        x[pages, :, to % page // 16, to % 16] = torch.where(taken[..., None, None], new, old)
    s["kv_len_out"][:] = base[:, 0] + s["path_len"]
    return [s["kv_len_out"], *s["held"]]


def _weights_plain(s):
    score, row, live = _causal_scores(s)
    lse = s["lse"][row].unflatten(2, score.shape[1:3]).permute(0, 2, 3, 1)[..., None]
    p = torch.exp(score - torch.where(lse == -math.inf, 0.0, lse))
    j = torch.arange(s["max_kv"], device="cuda")
    m = live.sum(-1)[:, None]
    old = (j < s["kv_len"].long()[:, None] - m)[:, None]
    there = (j < s["kv_len"][:, None])[:, None]
    s["weights"][:] = torch.where(there, torch.where(old, s["weights"], 0.0) + p.sum((2, 3)), s["weights"])
    return [s["weights"]]


def _evict_plain(s):
    c, w, pos = s["case"], s["weights"], s["key_pos"]
    budget, page, d = c["budget"], c["page_size"], c["head_dim"]
    n, last = s["kv_len"].long()[:, None, None], s["last_pos"].long()[:, None, None]
    j = torch.arange(w.shape[2], device="cuda")
    there = j < n
    p = torch.where(there & (pos < 0), last - (n - 1 - j), pos.long())
    # 32-bit numbers as whole ones that order alike; protected keys above them, what is not there below
    bits = (w + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    order = torch.where(torch.isnan(w), -(1 << 40), order)
    order = torch.where((p < c["sink"]) | (p > last - c["recent"]), 1 << 40, order)
    order = torch.where(there, order, -(1 << 41))
    ranked = order.sort(stable=True, dim=-1, descending=True).indices[..., :budget]
    keep = torch.zeros_like(there.expand_as(order)).scatter(-1, ranked, True) & there
    keep = keep | (there & (n <= budget))
    if w.shape[2] > budget:
        most = min(budget, w.shape[2] - budget)
        hole, mover = there & ~keep & (j < budget), keep & (j >= budget)
        to = (~hole).int().sort(stable=True, dim=-1).indices[..., :most]
        of = (~mover).int().sort(stable=True, dim=-1).indices[..., :most]
        real = mover.gather(-1, of)
        of = torch.where(real, of, to)  # (the others onto themselves)
        b, h = torch.arange(w.shape[0], device="cuda")[:, None, None], torch.arange(w.shape[1], device="cuda")[:, None]
        pages, pages_of = (s["table"].long()[b, x // page] for x in (to, of))
        for x in _sections(s["cache"], d):
            new, old = x[pages_of, h, of % page // 16, of % 16], x[pages, h, to % page // 16, to % 16]
            x[pages, h, to % page // 16, to % 16] = torch.where(real[..., None], new, old)
        w.scatter_(-1, to, w.gather(-1, of))
        p = p.scatter(-1, to, p.gather(-1, of))
    left = n.clamp(max=budget)
    pos[:] = torch.where(j < left, p, torch.where(there, -1, pos)).int()
    s["kv_len_out"][:] = left[:, 0, 0]
    return [s["kv_len_out"], pos, w, *s["held"]]


def run(s):
    c = s["case"]
    if c["op"] == "evict":  # the next step: positions go on, and a prompt's weights are another prompt's
        s["last_pos"] += _step(c)
        if c["prompt"]:
            s["weights"].copy_(s["prompt_weights"])
    if not own:
        return {"tree": _tree_plain, "accept": _accept_plain, "weights": _weights_plain, "evict": _evict_plain}[c["op"]](s)
    from gathered_rank_gemm_gb300 import binding as B
    if c["op"] == "tree":
        B.lora_kv4_tree_attention(s["cache"], s["q"], s["out"], s["q_start"], s["kv_len"], s["table"], s["max_q"],
                                  s["mask"], 1.0 / math.sqrt(c["head_dim"]), s["workspace"], window=c["window"],
                                  k_scale=K_SCALE, v_scale=V_SCALE, lse=s["lse"])
        return [s["out"], s["lse"]]
    if c["op"] == "accept":
        B.lora_kv4_accept(s["cache"], s["q_start"], s["kv_len"], s["table"], s["path"], s["path_len"], s["kv_len_out"])
        return [s["kv_len_out"], *s["held"]]
    if c["op"] == "weights":
        B.lora_kv4_key_weights(s["weights"], s["cache"], s["q"], s["lse"], s["q_start"], s["kv_len"], s["table"],
                               s["max_q"], 1.0 / math.sqrt(c["head_dim"]), window=c["window"], k_scale=K_SCALE,
                               path=s["path"], path_len=s["path_len"])
        return [s["weights"]]
    B.lora_kv4_evict(s["cache"], s["weights"], s["key_pos"], s["kv_len"], s["last_pos"], s["table"], c["budget"],
                     s["kv_len_out"], sink=c["sink"], recent=c["recent"])
    return [s["kv_len_out"], s["key_pos"], s["weights"], *s["held"]]


# ------------------------------------------------------------------ the definition in 64 bits

def _keys_64(s, b, h, n, v):
    """K (or V) of n keys of one sequence and head, in 64 bits."""
    d = s["case"]["head_dim"]
    raw = s["cache"][s["table"][b].long(), h].reshape(-1, 18 * d)
    magnitude = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    codes = raw[:, 8 * d * v:8 * d * (v + 1)].reshape(-1, d // 2)[:n].long()
    scales = raw[:, (16 + v) * d:(17 + v) * d].contiguous().view(torch.float8_e4m3fn).double().reshape(-1, d // 16)[:n]
    x = torch.empty(n, d, dtype=torch.float64, device="cuda")
    for half in range(2):
        nib = (codes >> (4 * half)) % 16
        x[:, half::2] = magnitude[nib % 8] * (1 - 2 * (nib // 8))
    return x * scales.repeat_interleave(16, 1) * (V_SCALE if v else K_SCALE)


def exact(case, seed):
    s = prepare(case, seed)
    op, d, kvh = case["op"], case["head_dim"], case["kv_heads"]
    lengths = _lengths(case)
    if op in ("accept", "evict"):
        blocks = s["cache"].cpu()
        table, page = s["table"].tolist(), case["page_size"]

        def move(b, heads, of, to):
            """Places `of` of a sequence to the places `to`, read before any is written."""
            of, to = ([torch.tensor(x) for x in zip(*[(table[b][x // page], x % page // 16, x % 16) for x in xs])]
                      for xs in (of, to))
            for x in _sections(blocks, d) if of else ():
                x[to[0], heads, to[1], to[2]] = x[of[0], heads, of[1], of[2]].clone()

        def held():
            parts = [x.cuda() for x in _sections(blocks, d)]
            return parts[:2] + [x.contiguous().view(torch.float8_e4m3fn).double() for x in parts[2:]]

        if op == "accept":
            _, paths = _trees(case)
            for b, ((m, n), path) in enumerate(zip(lengths, paths)):
                move(b, slice(None), [n - m + x for x in path], [n - m + i for i in range(len(path))])
            return [_i32([n - m + len(p) for (m, n), p in zip(lengths, paths)]), *held()]
        if sum(n for _, n in lengths) * kvh > 3e6 or case["seqs"] * kvh * case["budget"] > 1.5e5:
            return None
        w, pos = s["weights"].cpu().double().numpy(), s["key_pos"].cpu().numpy().copy()
        last = [x + _step(case) for x in s["last_pos"].tolist()]
        for b, (_, n) in enumerate(lengths):
            for h in range(kvh):
                for j in range(n):
                    if pos[b, h, j] < 0:
                        pos[b, h, j] = last[b] - (n - 1 - j)
                if n <= case["budget"]:
                    continue
                shield = [(x < case["sink"]) or (x > last[b] - case["recent"]) for x in pos[b, h, :n].tolist()]
                ranked = sorted(range(n), key=lambda j: (not shield[j], -w[b, h, j], j))
                gone = sorted(j for j in ranked[case["budget"]:] if j < case["budget"])
                stay = sorted(j for j in ranked[:case["budget"]] if j >= case["budget"])
                move(b, h, stay, gone)
                w[b, h, gone], pos[b, h, gone] = w[b, h, stay], pos[b, h, stay]
                pos[b, h, case["budget"]:n] = -1
        return [_i32([min(n, case["budget"]) for _, n in lengths]), torch.from_numpy(pos).cuda(),
                torch.from_numpy(w).cuda(), *held()]
    qh = case["q_heads"]
    if sum(q * kv for q, kv in lengths) * qh * d > 1.5e12:
        return None
    group, window, row = qh // kvh, case["window"], 0
    masks, paths = _trees(case)
    q = s["q"].double()
    if op == "tree":
        out, lse = torch.zeros_like(q), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    else:
        weights, lse = s["weights"].double(), s["lse"].double()
    for b, (m, n) in enumerate(lengths):
        rows = torch.arange(row, row + m, device="cuda")
        row += m
        if op == "tree":
            base = n - m
            hidden = torch.ones(m, n, dtype=torch.bool)
            for i, x in enumerate(masks[b]):
                depth = bin(x).count("1") - 1
                hidden[i, max(0, base + depth - window + 1) if window else 0:base] = False
                hidden[i, [base + c for c in range(m) if x >> c & 1]] = False
            hidden = hidden.cuda()
        else:
            if case["path"]:
                n, m = n - m + len(paths[b]), len(paths[b])
                rows = rows[paths[b]]
            at, key = torch.arange(n - m, n, device="cuda")[:, None], torch.arange(n, device="cuda")
            hidden = (key > at) | ((key <= at - window) if window else False)
        for h in range(kvh):
            x = torch.einsum("rgd,kd->grk", q[rows, h * group:(h + 1) * group], _keys_64(s, b, h, n, 0)) / d ** 0.5
            x = x.masked_fill(hidden, -math.inf)
            if op == "tree":
                total = torch.logsumexp(x, -1)
                p = torch.exp(x - total[..., None])
                out[rows, h * group:(h + 1) * group] = torch.einsum("grk,kd->rgd", p, _keys_64(s, b, h, n, 1))
                lse[rows, h * group:(h + 1) * group] = total.T
            else:
                weights[b, h, max(0, n - m):n] = 0
                of = lse[rows, h * group:(h + 1) * group].T[..., None]
                p = torch.exp(x - torch.where(of == -math.inf, 0.0, of))
                weights[b, h, :n] += p.sum((0, 1))
    return [out, lse] if op == "tree" else [weights]
