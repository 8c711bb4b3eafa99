"""Serving with drafted tokens and with caches that are kept short, as they are timed: appending tokens
whose positions are not their places in the cache, attention for trees of drafted tokens over the bf16
paged cache, keeping the accepted ones, adding up the attention that each cached token draws, and
evicting the tokens that draw the least.

Where ``own`` is false ``run`` computes each operator's plain form with elementary torch operations in
32 bits, rounded once at the end; where it is true it makes the package's calls.

Pages.  Logical token p of sequence b is row p % block_size of page block_table[b, p / block_size] of the
cache [pages, block_size, H_kv, d].  Tokens of a step are packed, sequence b's at [cu[b], cu[b+1]);
seqlens[b] counts the sequence's tokens with these, which are its last n = cu[b+1] - cu[b].

Append.  Token t's query and keys are rotated by positions[t] and written to the cache as they would be
without; the 4-bit cache is the one of append_paged_q4 (16 elements: scale = e4m3(max |x| / (6 descale)),
codes to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6).

Tree.  Query token i of a sequence sees all tokens in front of the step's, and of these those whose bits
are set in tree[cu[b] + i], bit j % 32 of word j / 32 for the step's token j; without a tree, j <= i.

Accept.  Of the step's tokens those at accepted[b, :n_accepted[b]], ascending, move to the front of the
step's places; the sequence is then as long as its tokens in front of the step and these.

Weights [pages, H_kv, block_size] follow the pages.  A step with queries q and their lse makes of them

    w[p] = decay * w[p] + sum over its query tokens that see p, and the query heads that share the
                          key head, of exp(scale * q . k[p] - lse)

with 0 for the w[p] of tokens from weighed[b] on.

Evict.  Of each sequence with more than budgets[b] tokens every key head keeps so many: the first
``keep_first``, the last ``keep_last`` and between them those of the largest weights, the lower position
where they are equal.  What is kept goes in order to the pages of a new block table.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DESCALE_K, DESCALE_V = (float(torch.tensor(x / 2688, dtype=torch.float32)) for x in (5.8137, 5.7219))
MOST_BYTES = 2.0e9      # of a drawn case: below the largest listed ones
MOST_FLOPS = 5.0e11
MOST_SCORES = 1.0e9     # of a drawn attention case: padded (query, key, head) triples


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _case(name, op, seqs, new, old, H, H_kv, d, block, **more):
    """``new`` and ``old``: each sequence's tokens of the step and in front of it, as "lo-hi" from which its
    own count is taken (by ``lens``, not by the inputs' seed, so that the work is the case's)."""
    c = {"op": op, "seqs": seqs, "new": new, "old": old, "H": H, "H_kv": H_kv, "d": d, "block": block,
         "tree": False, "rotary": 0, "interleaved": False, "evicted": 0, "decay": 1.0, "weighed": True,
         "budget": "0-0", "first": 0, "last": 0, "lens": 1}
    c.update(more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # drafted trees of four sequences into the bf16 cache: every node at its depth's position
        _case("append_tree_4x26", "append", 4, "26-26", "100-2000", 32, 8, 128, 64, tree=True, rotary=128),
        # steps of mixed length into 4-bit caches that were cut short before: positions are far ahead of places
        _case("append_q4_24xmixed", "append_q4", 24, "1-1024", "0-2000", 32, 8, 128, 32, rotary=64, interleaved=True, evicted=20000),
        # one sequence's small tree over a thousand tokens: the smallest call, all latency
        _case("tree_1x8", "tree", 1, "8-8", "1000-1000", 32, 8, 128, 64, tree=True),
        # trees of mixed size for a batch of mixed lengths
        _case("tree_16xmixed", "tree", 16, "1-60", "500-8188", 32, 8, 128, 64, tree=True),
        # single tokens over long caches, eight query heads a key head
        _case("tree_16x1_32768", "tree", 16, "1-1", "32767-32767", 32, 4, 128, 128),
        # the last 512 tokens of four 16384-token prompts, computed against all before them
        _case("tree_4x512_chain", "tree", 4, "512-512", "15872-15872", 32, 8, 128, 128),
        # the accepted paths of a few sequences' trees
        _case("accept_4x26", "accept", 4, "26-26", "100-2000", 8, 8, 128, 64, tree=True),
        # those of a large batch with large trees
        _case("accept_128x64", "accept", 128, "64-64", "100-1000", 8, 8, 128, 64, tree=True),
        # a decoding step of a batch of mixed lengths
        _case("weigh_32x1", "weigh", 32, "1-1", "100-8191", 32, 8, 128, 64, decay=0.98),
        # two whole prompts
        _case("weigh_2x4096", "weigh", 2, "4096-4096", "0-0", 32, 8, 128, 128),
        # one sequence that has grown over its budget by a page
        _case("evict_1x4160", "evict", 1, "0-0", "4160-4160", 8, 8, 128, 64, budget="4096-4096", first=4, last=512),
        # prompts cut to a quarter and less
        _case("evict_16x16384", "evict", 16, "0-0", "10000-16384", 8, 8, 128, 64, budget="1024-4096", first=4, last=256),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _span(rng, lo, hi):
    """A range of counts: all one number half the time, else from anywhere below it."""
    top = _log(rng, max(1, lo), hi)
    return "%d-%d" % ((top, top) if rng.random() < 0.5 else (rng.randint(lo, top), top))


def draw(rng):
    while True:
        op = rng.choice(["append", "append_q4", "tree", "tree", "tree", "accept", "weigh", "weigh", "evict"])
        d = rng.choice([64, 128, 128])
        H_kv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
        H = H_kv * rng.choice([1, 1, 2, 4, 4, 5, 8, 16])
        block = rng.choice([16, 32, 48, 64, 128, 256])
        seqs, more = _log(rng, 1, 64), {"tree": rng.random() < 0.6}
        if op in ("append", "append_q4"):
            new = _span(rng, 1, 200 if more["tree"] else 2048)
            old = "0-%d" % _log(rng, 1, 8192)
            more.update(rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.4,
                        evicted=0 if more["tree"] else _log(rng, 1, 30000))
        elif op == "tree":
            new = "1-1" if rng.random() < 0.3 else _span(rng, 1, 200 if more["tree"] else 1024)
            old = "0-%d" % _log(rng, 1, 32768) if rng.random() < 0.5 else _span(rng, 1, 32768)
        elif op == "accept":
            seqs, more["tree"] = _log(rng, 1, 128), True
            new, old, H = _span(rng, 1, 200), "0-%d" % _log(rng, 1, 2000), H_kv
        elif op == "weigh":
            more = {"decay": rng.choice([1.0, 0.98, 0.5]), "weighed": rng.random() < 0.6}
            if rng.random() < 0.4:                  # a prompt's tokens, or its last ones behind those in front
                new, old = _span(rng, 1, 4096), rng.choice(["0-0", "0-%d" % _log(rng, 1, 8192)])
            else:                                   # a decoding step, or the accepted tokens of one
                new, old = "1-%d" % _log(rng, 1, 16), _span(rng, 0, 32767)
        else:
            top = _log(rng, 16, 32768)
            keep = _log(rng, 1, top)
            new, old, H = "0-0", "%d-%d" % (rng.randint(1, top), top), H_kv
            more = {"budget": "%d-%d" % (rng.randint(1, keep), keep)}
            least = int(more["budget"].split("-")[0])
            more["first"] = rng.choice([0, min(4, least)])
            more["last"] = rng.randint(0, least - more["first"])
        c = _case(None, op, seqs, new, old, H, H_kv, d, block, lens=rng.randint(1, 1 << 20), **more)
        w = work(c)
        n, k = _counts(c)
        pool = seqs * H_kv * max(k) * d
        padded = seqs * H * max(n) * max(k) if op in ("tree", "weigh") else 0
        if H <= 64 and max(k) and w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS and max(padded, pool) <= MOST_SCORES:
            return c


def _counts(case):
    """(the step's tokens of each sequence, its tokens with these)."""
    r = random.Random(case["lens"])
    ends = [[int(x) for x in case[k].split("-")] for k in ("new", "old")]
    n = [r.randint(*ends[0]) for _ in range(case["seqs"])]
    return n, [a + r.randint(*ends[1]) for a in n]


def _budgets(case):
    r = random.Random(case["lens"] + 1)
    lo, hi = (int(x) for x in case["budget"].split("-"))
    return [r.randint(lo, hi) for _ in range(case["seqs"])]


def _trees(case):
    """Each sequence's parents: -1, or an earlier node, mostly one of the last few (trees are laid out by depth)."""
    r = random.Random(case["lens"] + 2)
    return [[-1 if i == 0 or r.random() < 0.1 else max(0, i - r.randint(1, min(i, 12))) for i in range(n)] for n in _counts(case)[0]]


def _path(parents, i):
    """The nodes from the root down to node i."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path[::-1]


def _accepted(case):
    """A node's path for each sequence, or nothing."""
    r = random.Random(case["lens"] + 3)
    return [_path(p, r.randrange(len(p))) if r.random() < 0.9 else [] for p in _trees(case)]


def work(case):
    n, k = _counts(case)
    H, H_kv, d, op = case["H"], case["H_kv"], case["d"], case["op"]
    total, row, row4, ints = sum(n), 2 * d, d // 2 + d // 16, 4 * (2 * case["seqs"] + 1 + sum(-(-x // case["block"]) for x in k))
    if op in ("append", "append_q4"):   # q read and written, keys and values read and written (in 4 bits: and read back)
        new_kv = 2 * total * H_kv
        rot = {"flops": 3 * total * (H + H_kv) * case["rotary"] + (0 if op == "append" else 4 * new_kv * d)}
        there = row if op == "append" else 2 * row4 + row
        return dict(rot, bytes=2 * total * H * row + new_kv * (row + there) + 4 * total * (case["rotary"] + 1) + ints)
    if op == "accept":
        moved = sum(sum(i != j for i, j in enumerate(a)) for a in _accepted(case))
        return {"bytes": 4 * moved * H_kv * row + 4 * sum(len(a) for a in _accepted(case)) + ints + 8 * case["seqs"], "flops": 0}
    if op == "evict":
        kept = sum(min(x, y) for x, y in zip(k, _budgets(case)))
        return {"bytes": H_kv * (4 * sum(k) + kept * (4 * row + 8)) + 2 * ints, "flops": 0}
    if op == "tree":
        if case["tree"]:
            pairs = sum(x * (y - x) for x, y in zip(n, k)) + sum(len(_path(p, i)) for p in _trees(case) for i in range(len(p)))
        else:
            pairs = sum(x * y - x * (x - 1) // 2 for x, y in zip(n, k))
        return {"bytes": 2 * sum(k) * H_kv * row + total * H * (2 * row + 4) + ints, "flops": 4 * d * H * pairs}
    pairs = sum(x * y - x * (x - 1) // 2 for x, y in zip(n, k))
    old = sum(y - x for x, y in zip(n, k)) if case["weighed"] else 0
    return {"bytes": sum(k) * H_kv * (row + 4) + 4 * old * H_kv + total * H * (row + 4) + ints, "flops": 2 * d * H * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tables(lens, block, spare, order, at):
    """Block tables for sequences of these lengths, of the pages order[at:]; unused entries are -1."""
    table = torch.full((len(lens), max(-(-x // block) for x in lens) + spare), -1, dtype=torch.int32)
    for b, x in enumerate(lens):
        need = -(-x // block)
        table[b, :need] = order[at:at + need]
        at += need
    return table.to(DEV), at


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, k = _counts(case)
    B, H, H_kv, d, bs, op = case["seqs"], case["H"], case["H_kv"], case["d"], case["block"], case["op"]
    total = sum(n)
    budgets = _budgets(case) if op == "evict" else []
    lens = [min(x, y) for x, y in zip(k, budgets)]
    pages = sum(-(-x // bs) for x in k + lens) + 3                # a pool with a few pages to spare, in any order
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table, at = _tables(k, bs, 1, order, 0)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s = {"op": op, "table": table, "cu": _ints(cu), "seqlens": _ints(k), "max_q": max(n), "max_k": max(k), "total": total,
         "scale": d ** -0.5, "interleaved": case["interleaved"], "tree": None}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    trees = _trees(case) if case["tree"] else None
    if op == "tree" and trees:
        words = -(-max(n) // 32)
        bits = []
        for p in trees:
            rows = []
            for i, up in enumerate(p):
                rows.append((rows[up] if up >= 0 else 0) | 1 << i)
            bits += [[(x >> 32 * w & 0xffffffff) - (x >> 32 * w + 31 & 1) * (1 << 32) for w in range(words)] for x in rows]
        s["tree"] = _ints(bits)
    if op in ("append", "append_q4"):
        # keys, values and queries as one fused projection leaves them: rows of one wide matrix
        qkv = normal(total, (H + 2 * H_kv) * d)
        s["q"] = qkv[:, :H * d].unflatten(1, (H, d))
        s["k"] = qkv[:, H * d:(H + H_kv) * d].unflatten(1, (H_kv, d))
        s["v"] = qkv[:, (H + H_kv) * d:].unflatten(1, (H_kv, d))
        at = []
        for b, (x, y) in enumerate(zip(n, k)):
            if trees:
                depth = []
                for up in trees[b]:
                    depth.append(depth[up] + 1 if up >= 0 else 0)
                at += [y - x + i for i in depth]
            else:
                at += range(y - x + case["evicted"], y + case["evicted"])
        s["positions"] = _ints(at)
        p = torch.arange(max(at) + 1, dtype=torch.float64, device=DEV)
        angle = p[:, None] * 10000.0 ** (-torch.arange(0, case["rotary"], 2, dtype=torch.float64, device=DEV) / case["rotary"])
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["descale_k"], s["descale_v"] = DESCALE_K, DESCALE_V
        if op == "append_q4":
            for x in ("k", "v"):
                s[x + "_codes"] = torch.zeros((pages, H_kv, bs, d // 2), dtype=torch.uint8, device=DEV)
                s[x + "_scales"] = torch.zeros((pages, H_kv, bs, d // 16), dtype=torch.uint8, device=DEV)
            return s
    for x in ("k", "v") if op != "weigh" else ("k",):
        s[x + "_cache"] = cache = torch.zeros((pages, bs, H_kv, d), dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 27) // (H_kv * bs * d))
        for i in range(0, pages if op != "append" else 0, step):
            cache[i:i + step] = torch.randn(cache[i:i + step].shape, generator=g, device=DEV)
    if op in ("tree", "weigh"):
        s["q"] = normal(total, H, d)
    if op == "accept":
        paths = _accepted(case)
        deep = max(1, max(len(p) for p in paths))
        s["accepted"], s["n_accepted"] = _ints([p + [-1] * (deep - len(p)) for p in paths]), _ints([len(p) for p in paths])
    if op == "weigh":
        # what the attention left of each row
        s["lse"] = torch.empty((H, total), device=DEV)
        for b, (x, y) in enumerate(zip(n, k)):
            K = s["k_cache"][table[b, :-(-y // bs)].long()].flatten(0, 1)[:y]
            hidden = torch.arange(y, device=DEV) > torch.arange(y - x, y, device=DEV)[:, None]
            for h in range(H_kv):
                G = H // H_kv
                z = torch.einsum("ngd,kd->gnk", s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].float(), K[:, h].float()).mul_(s["scale"])
                s["lse"][h * G:(h + 1) * G, cu[b]:cu[b + 1]] = z.masked_fill_(hidden, -math.inf).logsumexp(-1)
        s["decay"] = case["decay"]
        s["weighed"] = None if case["weighed"] else torch.zeros(B, dtype=torch.int32, device=DEV)
    if op in ("weigh", "evict"):
        # a few tokens draw most of the attention, and many none that 32 bits show
        w = torch.randn((pages, H_kv, bs), generator=g, device=DEV).mul_(2).exp_()
        s["weights"] = torch.where(w < 0.1, torch.zeros_like(w), w)
    if op == "evict":
        s["new_table"], _ = _tables(lens, bs, 0, order, at)
        s["budgets"], s["max_kept"], s["first"], s["last"] = _ints(budgets), max(lens), case["first"], case["last"]
    return s


# ---------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------

def _places(s):
    """(page, row) of each packed token."""
    t = torch.arange(s["total"], device=DEV)
    cu = s["cu"].long()
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = s["seqlens"].long()[b] - (cu[b + 1] - cu[b]) + t - cu[b]
    block = (s["k_cache"] if "k_cache" in s else s["k_codes"].transpose(1, 2)).shape[1]
    return s["table"].long()[b, pos // block], pos % block


def _rotate(x, s):
    """fp32 rotation of x [total, heads, d]."""
    x = x.float()
    at = s["positions"].long()
    c, n = s["cos"][at][:, None], s["sin"][at][:, None]
    r = 2 * c.shape[-1]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((y, x[..., r:]), -1)


def _quantise(x, descale):
    """Codes, one a byte, and e4m3 scales of fp32 x [..., d]."""
    b = x.unflatten(-1, (-1, 16))
    # a tensor as the divisor: by a plain number torch multiplies with the reciprocal, one rounding more
    s = (b.abs().amax(-1) / torch.full((), 6.0 * descale, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float().unsqueeze(-1) * descale
    y = torch.where(f > 0, b.abs() / f, torch.zeros_like(b))
    code = ((y > .25).to(torch.uint8) + (y >= .75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = code.to(torch.uint8) + 8 * torch.signbit(b).to(torch.uint8)
    return code.flatten(-2), s.view(torch.uint8)


def _dequantise(codes, scales, descale):
    """fp32 values of packed codes [..., d/2] and scales [..., d/16]."""
    v = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1., -1.5, -2., -3., -4., -6.], device=codes.device)
    x = torch.stack((v[(codes & 15).int()], v[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2) * descale


def _append(s):
    page, row = _places(s)
    s["k_cache"][page, row] = _rotate(s["k"], s).to(torch.bfloat16)
    s["v_cache"][page, row] = s["v"]
    return _rotate(s["q"], s).to(torch.bfloat16)


def _append_q4(s):
    page, row = _places(s)
    back = []
    for x, y in (("k", _rotate(s["k"], s)), ("v", s["v"].float())):
        c, e = _quantise(y, s["descale_" + x])
        s[x + "_codes"][page, :, row] = c[..., 0::2] | (c[..., 1::2] << 4)
        s[x + "_scales"][page, :, row] = e
        back.append(_dequantise(s[x + "_codes"][page, :, row], s[x + "_scales"][page, :, row], s["descale_" + x]).to(torch.bfloat16))
    return [_rotate(s["q"], s).to(torch.bfloat16)] + back


def _scores(s):
    """Padded scores [B, H_kv, G, n, keys], -inf where a query does not see a key."""
    bs, H_kv, d = s["k_cache"].shape[1:]
    B = s["table"].shape[0]
    K = s["k_cache"][s["table"].long()].flatten(1, 2)[:, :s["max_k"]].permute(0, 2, 3, 1).float()   # [B, H_kv, d, keys]
    cu, lens = s["cu"].long(), s["seqlens"].long()
    n = cu[1:] - cu[:-1]
    i, j = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    at = (cu[:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][at].float().unflatten(2, (H_kv, -1)).permute(0, 2, 3, 1, 4)                          # [B, H_kv, G, n, d]
    G, m = q.shape[2], q.shape[3]
    of = j[None] - (lens - n)[:, None]                                                              # [B, keys]: the step's token
    if s["tree"] is None:
        seen = of[:, None] <= i[None, :, None]
    else:
        word = s["tree"][at].gather(2, (of.clamp(0, 32 * s["tree"].shape[1] - 1) // 32)[:, None].expand(B, m, -1))
        seen = (word >> (of.clamp(min=0) % 32)[:, None] & 1).bool() | (of < 0)[:, None]
    seen &= (j[None] < lens[:, None])[:, None] & (i[None] < n[:, None])[:, :, None]
    x = torch.matmul(q.reshape(B, H_kv, G * m, d), K).mul_(s["scale"]).unflatten(2, (G, m))
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _tree(s):
    x = _scores(s)
    B, H_kv, G, m = x.shape[:4]
    V = s["v_cache"][s["table"].long()].flatten(1, 2)[:, :s["max_k"]].transpose(1, 2).float()
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H_kv, G * m, -1), V).unflatten(2, (G, m))
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).flatten(2, 3)         # [B, n, H, d]
    lse = (top + l.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)                             # [B, n, H]
    cu, t = s["cu"].long(), torch.arange(s["total"], device=DEV)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return o[b, t - cu[b]].to(torch.bfloat16), lse[b, t - cu[b]].t().contiguous()


def _accept(s):
    bs = s["k_cache"].shape[1]
    old = s["seqlens"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["accepted"].shape[1], device=DEV)
    b, i = torch.nonzero(i[None] < s["n_accepted"][:, None], as_tuple=True)
    src, dst = old[b] + s["accepted"][b, i].long(), old[b] + i
    page = s["table"].long()
    for x in ("k_cache", "v_cache"):
        s[x][page[b, dst // bs], dst % bs] = s[x][page[b, src // bs], src % bs]
    return (old + s["n_accepted"]).to(torch.int32)


def _weigh(s):
    x = _scores(s)                                                                                  # [B, H_kv, G, n, keys]
    B, H_kv, G, m = x.shape[:4]
    cu, lens = s["cu"].long(), s["seqlens"].long()
    at = (cu[:-1, None] + torch.arange(m, device=DEV)).clamp(max=s["total"] - 1)
    lse = s["lse"][:, at].unflatten(0, (H_kv, G)).permute(2, 0, 1, 3)                               # [B, H_kv, G, n]
    drawn = x.sub_(lse[..., None]).exp_().sum((2, 3))                                               # [B, H_kv, keys]
    j = torch.arange(s["max_k"], device=DEV)
    b, j = torch.nonzero((j[None] < lens[:, None]) & (cu[1:] > cu[:-1])[:, None], as_tuple=True)
    bs = s["k_cache"].shape[1]
    page, row = s["table"].long()[b, j // bs], j % bs
    weighed = lens - (cu[1:] - cu[:-1]) if s["weighed"] is None else s["weighed"].long()
    before = torch.where((j < weighed[b])[:, None], s["weights"][page, :, row] * s["decay"], torch.zeros((), device=DEV))
    s["weights"][page, :, row] = before + drawn[b, :, j]


def _evict(s):
    bs, H_kv = s["k_cache"].shape[1:3]
    page, new = s["table"].long(), s["new_table"].long()
    lens, B = s["seqlens"].long(), page.shape[0]
    left = torch.minimum(lens, s["budgets"].long())
    j = torch.arange(s["max_k"], device=DEV)
    w = s["weights"][page].transpose(1, 2).flatten(2)[..., :s["max_k"]]                             # [B, H_kv, tokens]
    w = torch.where(w.isnan(), torch.full_like(w, -math.inf), w)
    kind = torch.where((j < s["first"]) | (j >= (lens - s["last"])[:, None]), 0, 1)                 # kept in any case, perhaps, none
    kind = torch.where(j >= lens[:, None], 2, kind)[:, None].expand(B, H_kv, -1)
    order = w.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, kind.gather(-1, order).sort(dim=-1, stable=True).indices)                  # by kind, then by weight
    i = torch.arange(s["max_kept"], device=DEV)
    some = (i < left[:, None])[:, None].expand(B, H_kv, -1)
    kept = torch.where(some, order[..., :s["max_kept"]], s["max_k"]).sort(-1).values
    b, h, i = torch.nonzero(some, as_tuple=True)
    src = kept[b, h, i]
    p0, r0, p1, r1 = page[b, src // bs], src % bs, new[b, i // bs], i % bs
    for x in ("k_cache", "v_cache"):
        s[x][p1, r1, h] = s[x][p0, r0, h]
    s["weights"][p1, h, r1] = s["weights"][p0, h, r0]
    return torch.where(some, kept, -1).to(torch.int32), left.to(torch.int32)


def run(s):
    op = s["op"]
    if own:
        import exact_io_aware_08_gb300 as fa
    if op == "append":
        if own:
            q = fa.append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"], q=s["q"],
                                cos=s["cos"], sin=s["sin"], interleaved=s["interleaved"], positions=s["positions"])
        else:
            q = _append(s)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "append_q4":
        # what was appended is read back as the values it stands for
        if own:
            cache = [s[x] for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
            scales = {"descale_k": s["descale_k"], "descale_v": s["descale_v"]}
            q = fa.append_paged_q4(s["k"], s["v"], *cache, s["table"], s["cu"], s["seqlens"], q=s["q"], cos=s["cos"], sin=s["sin"],
                                   interleaved=s["interleaved"], positions=s["positions"], **scales)
            k, v = fa.gather_paged_q4(*cache, s["table"], s["cu"], s["seqlens"], s["total"], **scales)
        else:
            q, k, v = _append_q4(s)
        return {"q": q, "k": k, "v": v}
    if op == "tree":
        if own:
            o, lse = fa.forward_paged_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"], s["max_q"],
                                           s["max_k"], tree=s["tree"], scale=s["scale"])
        else:
            o, lse = _tree(s)
        return {"o": o, "lse": lse}
    if op == "accept":
        if own:
            lens = fa.accept_paged(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"], s["accepted"], s["n_accepted"])
        else:
            lens = _accept(s)
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "seqlens": lens}
    if op == "weigh":
        if own:
            fa.weigh_paged(s["q"], s["lse"], s["k_cache"], s["weights"], s["table"], s["cu"], s["seqlens"], s["max_q"], s["max_k"],
                           weighed=s["weighed"], decay=s["decay"], scale=s["scale"])
        else:
            _weigh(s)
        return {"weights": s["weights"]}
    if own:
        kept, lens = fa.evict_paged(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["new_table"], s["seqlens"], s["budgets"],
                                    s["max_k"], s["max_kept"], keep_first=s["first"], keep_last=s["last"])
    else:
        kept, lens = _evict(s)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"], "kept": kept, "seqlens": lens}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, one sequence after another
# ---------------------------------------------------------------------------------------------

def _exact_rotate(x, at, case):
    """x [n, heads, d] at the positions ``at``, as complex numbers; the tables hold 32 bits."""
    r = case["rotary"]
    w = 10000.0 ** (-2 * torch.arange(r // 2, dtype=torch.float64, device=DEV) / r)
    angle = at.double()[:, None] * w
    turn = torch.complex(angle.cos().float().double(), angle.sin().float().double())[:, None]
    x, rest = x[..., :r], x[..., r:]
    z = x.unflatten(-1, (r // 2, 2)) if case["interleaved"] else x.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(z[..., 0].contiguous(), z[..., 1].contiguous()) * turn)
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, rest), -1)


def _exact_round(x, descale):
    """x [..., d] in 64 bits as the 4-bit cache holds it."""
    b = x.unflatten(-1, (-1, 16))
    a = (b.abs().amax(-1, keepdim=True) / (6 * descale)).clamp(max=448.0)
    u = torch.exp2(a.clamp(min=2.0 ** -6).log2().floor() - 3)                # spacing of e4m3 numbers there
    s = (a / u).round() * u * descale
    y = torch.where(s > 0, b.abs() / s, torch.zeros_like(b)).clamp(max=6.0)
    u = torch.exp2(y.clamp(min=1.0).log2().floor() - 1)
    return (torch.sign(b) * (y / u).round() * u * s).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    n, k = _counts(case)
    H_kv, bs, op = case["H_kv"], case["block"], case["op"]
    G = case["H"] // H_kv
    if op == "append_q4":
        at = s["positions"]
        return {"q": _exact_rotate(s["q"].double(), at, case), "k": _exact_round(_exact_rotate(s["k"].double(), at, case), DESCALE_K),
                "v": _exact_round(s["v"].double(), DESCALE_V)}
    caches = {x: s[x].double() if op == "append" else s[x] for x in ("k_cache", "v_cache") if x in s}
    o, lse, moved = [], [], {x: y.clone() for x, y in s.items() if op in ("accept", "evict") and x in ("k_cache", "v_cache", "weights")}
    weights = s["weights"].double() if op == "weigh" else None
    kept = torch.full((case["seqs"], H_kv, s["max_kept"]), -1, dtype=torch.int32) if op == "evict" else None
    left, first = [], 0
    for b, (new, length) in enumerate(zip(n, k)):
        mine = slice(first, first + new)
        first += new
        at = torch.arange(length, device=DEV)
        page, row, step = s["table"][b].long()[at // bs], at % bs, at[length - new:]
        if op == "append":
            caches["k_cache"][page[step], row[step]] = _exact_rotate(s["k"][mine].double(), s["positions"][mine], case)
            caches["v_cache"][page[step], row[step]] = s["v"][mine].double()
        elif op == "accept":
            path = _accepted(case)[b]
            for i, j in enumerate(path):
                for x in moved:
                    moved[x][page[length - new + i], row[length - new + i]] = s[x][page[length - new + j], row[length - new + j]]
            left.append(length - new + len(path))
        elif op == "evict":
            count = min(length, _budgets(case)[b])
            left.append(count)
            to = torch.arange(count, device=DEV)
            to_page, to_row = s["new_table"][b].long()[to // bs], to % bs
            for h in range(H_kv):
                w = s["weights"][page, h, row].tolist()
                sure = [j for j in range(length) if j < case["first"] or j >= length - case["last"]] if count < length else list(range(length))
                rest = sorted((j for j in range(case["first"], length - case["last"])), key=lambda j: (-w[j], j)) if count < length else []
                these = torch.tensor(sorted(sure + rest[:count - len(sure)]), dtype=torch.long)
                kept[b, h, :count] = these.int()
                these = these.to(DEV)
                for x in ("k_cache", "v_cache"):
                    moved[x][to_page, to_row, h] = s[x][page[these], row[these], h]
                moved["weights"][to_page, h, to_row] = s["weights"][page[these], h, row[these]]
        else:
            seen = at[None] < length - new + torch.zeros(new, dtype=torch.long, device=DEV)[:, None]
            if case["tree"] and op == "tree":
                for i, up in enumerate(_trees(case)[b]):
                    if up >= 0:
                        seen[i, length - new:] = seen[up, length - new:]
                    seen[i, length - new + i] = True
            else:
                seen = at[None] <= step[:, None]
            K = caches["k_cache"][page, row].double()
            q = s["q"][mine].double()
            outs, sums = [], []
            for h in range(H_kv):
                z = torch.einsum("ngd,kd->ngk", q[:, h * G:(h + 1) * G], K[:, h]) * s["scale"]
                z = z.masked_fill(~seen[:, None], -math.inf)
                if op == "weigh":
                    drawn = torch.exp(z - s["lse"][h * G:(h + 1) * G, mine].double().t()[..., None]).sum((0, 1))
                    had = weights[page, h, row] * s["decay"]
                    had[(length - new if case["weighed"] else 0):] = 0
                    weights[page, h, row] = had + drawn
                    continue
                e = torch.logsumexp(z, -1)
                outs.append(torch.einsum("ngk,kd->ngd", torch.exp(z - e[..., None]), caches["v_cache"][page, row, h].double()))
                sums.append(e)
            if op == "tree":
                o.append(torch.cat(outs, 1))
                lse.append(torch.cat(sums, 1))
    if op == "append":
        return {"q": _exact_rotate(s["q"].double(), s["positions"], case), "k_cache": caches["k_cache"], "v_cache": caches["v_cache"]}
    if op == "weigh":
        return {"weights": weights}
    if op == "tree":
        return {"o": torch.cat(o), "lse": torch.cat(lse).t().contiguous()}
    out = {"k_cache": moved["k_cache"], "v_cache": moved["v_cache"], "seqlens": _ints(left)}
    return out if op == "accept" else dict(out, weights=moved["weights"], kept=kept.to(DEV))
