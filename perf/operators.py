"""Serving operators over a paged key/value cache, as they are timed: appending rotated keys and
values (to a bf16 cache, and to one held in 4 bits), reading a 4-bit cache back, and attention
over it, for one new token a sequence and for several.

Where ``own`` is false ``run`` computes each operator's plain form with elementary torch
operations in 32 bits, rounded once at the end; where it is true it makes the package's calls.

The 4-bit cache.  A token's row of one head (d values) is held as d/2 bytes of codes, element 2i
in the low and 2i+1 in the high four bits of byte i, and d/16 scales of 8 bits, one for each 16
consecutive elements.  A code is sign, two exponent bits and one mantissa bit: 0, 0.5, 1, 1.5, 2,
3, 4, 6 and their negatives; a scale is an e4m3 number.  The value is code * scale * descale, with
one ``descale`` for all keys and one for all values.  Of 16 elements x:

    scale = e4m3(max |x| / (6 descale)), at most 448;  code = nearest(x / (scale descale)), at most 6

both to nearest, ties to the even code; a scale of 0 gives codes of 0.

Pages.  Logical token p of sequence b is row p % block_size of page block_table[b, p / block_size].
The bf16 cache is [pages, block_size, H_kv, d]; codes are [pages, H_kv, block_size, d/2] and scales
[pages, H_kv, block_size, d/16].  Tokens of a step are packed, sequence b's at [cu[b], cu[b+1]);
seqlens[b] counts the sequence's tokens with these, so that token cu[b] + i has the position
seqlens[b] - (cu[b+1] - cu[b]) + i.

Rotation of a pair (x1, x2) at position p: (x1 cos - x2 sin, x2 cos + x1 sin), with the tables' row
p.  Pairs are (i, i + rotary/2), or (2i, 2i+1) where ``interleaved``; elements from ``rotary`` on stay.
"""
import math
import random

import torch

own = False

DEV = "cuda"
# a calibration's largest key and value over 6 * 448, in 32 bits: the values here stay below 5.8
DESCALE_K, DESCALE_V = (float(torch.tensor(x / 2688, dtype=torch.float32)) for x in (5.8137, 5.7219))
MOST_BYTES = 2.4e9      # of a drawn case: below the largest listed ones
MOST_FLOPS = 1.0e12
MOST_SCORES = 2.2e9     # of a drawn attention case: padded (query, key, head) triples


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _case(name, op, seqs, new, old, H, H_kv, d, block, **more):
    """``new`` and ``old``: each sequence's new and already cached tokens, as "lo-hi" from which a
    sequence's own count is taken (by ``lens``, not by the inputs' seed, so that the work is the case's)."""
    c = {"op": op, "seqs": seqs, "new": new, "old": old, "H": H, "H_kv": H_kv, "d": d, "block": block,
         "rotary": 0, "interleaved": False, "lens": 1}
    c.update(more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token for each of eight running sequences, a bf16 cache with as many heads as the
        # queries: the smallest call, all latency
        _case("append_8x1", "append", 8, "1-1", "100-1000", 32, 32, 128, 128, rotary=128),
        # four whole prompts of the benchmark's length and heads
        _case("append_4x4096", "append", 4, "4096-4096", "0-0", 32, 32, 128, 128, rotary=128),
        # one token for each sequence of a large batch into the 4-bit cache, and those read back
        _case("append_q4_64x1", "append_q4", 64, "1-1", "1-8192", 32, 8, 128, 64, rotary=128),
        # prompts of mixed length behind shared prefixes, half of each head rotated, pairs side by side
        _case("append_q4_24xmixed", "append_q4", 24, "1-4096", "0-2000", 32, 8, 128, 32, rotary=64, interleaved=True),
        # a few short sequences handed to a path that takes bf16
        _case("gather_q4_6xshort_d64", "gather_q4", 6, "1-700", "0-0", 4, 4, 64, 16),
        # long prefixes handed back whole
        _case("gather_q4_8x16384", "gather_q4", 8, "16384-16384", "0-0", 8, 8, 128, 128),
        # decode: one sequence of about a thousand tokens, the smallest step
        _case("decode_q4_1x1000", "decode_q4", 1, "1-1", "999-999", 32, 8, 128, 64),
        # decode: a batch of mixed lengths up to 8192 tokens over 256-token pages, one query head a key head
        _case("decode_q4_32xmixed", "decode_q4", 32, "1-1", "0-8191", 8, 8, 128, 256),
        # decode: 64 sequences of 32768 tokens, four query heads a key head
        _case("decode_q4_64x32768", "decode_q4", 64, "1-1", "32767-32767", 32, 8, 128, 128),
        # a few tokens a sequence at once (drafted tokens being checked) over long caches
        _case("forward_q4_16x4", "forward_q4", 16, "4-4", "500-8188", 32, 8, 128, 64),
        # short prompts of mixed length behind short prefixes, 64-wide heads
        _case("forward_q4_8xmixed_d64", "forward_q4", 8, "1-1024", "0-300", 16, 16, 64, 128),
        # the last 1024 tokens of four 16384-token prompts, computed against all before them
        _case("forward_q4_4x1024", "forward_q4", 4, "1024-1024", "15360-15360", 32, 8, 128, 128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _span(rng, lo, hi):
    """A range of counts: all one number half the time, else from anywhere below it."""
    top = _log(rng, max(1, lo), hi)
    return "%d-%d" % ((top, top) if rng.random() < 0.5 else (rng.randint(lo, top), top))


def draw(rng):
    while True:
        op = rng.choice(["append", "append_q4", "gather_q4", "decode_q4", "decode_q4", "forward_q4", "forward_q4"])
        d = rng.choice([64, 128, 128])
        H_kv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
        H = H_kv * rng.choice([1, 1, 2, 4, 4, 5, 8, 16])
        block = rng.choice([64, 128, 256] if op == "append" else [16, 32, 48, 64, 128, 256])
        seqs, old, more = _log(rng, 1, 64), "0-0", {}
        if op in ("append", "append_q4"):
            new = "1-1" if rng.random() < 0.4 else _span(rng, 1, 4096)
            old = "0-0" if rng.random() < 0.3 else "0-%d" % _log(rng, 1, 8192)
            more = {"rotary": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.4}
        elif op == "gather_q4":
            new = _span(rng, 1, 16384)
            H = H_kv
        elif op == "decode_q4":
            new, old = "1-1", _span(rng, 0, 32767)
        else:
            new, old = _span(rng, 1, 1024), "0-%d" % _log(rng, 1, 16384)
        c = _case(None, op, seqs, new, old, H, H_kv, d, block, lens=rng.randint(1, 1 << 20), **more)
        w = work(c)
        n, k = _counts(c)
        padded = seqs * H * max(n) * max(k) if op in ("decode_q4", "forward_q4") else 0
        if H <= 64 and w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS and max(padded, seqs * H_kv * max(k) * d) <= MOST_SCORES:
            return c


def _counts(case):
    """(new tokens of each sequence, its tokens with these)."""
    r = random.Random(case["lens"])
    ends = [[int(x) for x in case[k].split("-")] for k in ("new", "old")]
    n = [r.randint(*ends[0]) for _ in range(case["seqs"])]
    return n, [a + r.randint(*ends[1]) for a in n]


def work(case):
    n, k = _counts(case)
    H, H_kv, d, op = case["H"], case["H_kv"], case["d"], case["op"]
    total, row, row4, ints = sum(n), 2 * d, d // 2 + d // 16, 4 * (2 * case["seqs"] + 1 + sum(-(-x // case["block"]) for x in k))
    new_kv, table = 2 * total * H_kv, 4 * case["rotary"] * max(k)
    if op == "append":          # q, keys and values read and written
        return {"bytes": 2 * (total * H + new_kv) * row + table + ints, "flops": 3 * total * (H + H_kv) * case["rotary"]}
    if op == "append_q4":       # and, in 4 bits, written, read back and written out
        return {"bytes": 2 * total * H * row + new_kv * (2 * row + 2 * row4) + table + ints,
                "flops": 3 * total * (H + H_kv) * case["rotary"] + 4 * new_kv * d}
    if op == "gather_q4":
        return {"bytes": new_kv * (row4 + row) + ints, "flops": 2 * new_kv * d}
    pairs = sum(x * y - x * (x - 1) // 2 for x, y in zip(n, k))     # query i of x sees y - x + i + 1 keys
    return {"bytes": 2 * sum(k) * H_kv * row4 + total * H * (2 * row + 4) + ints, "flops": 4 * d * H * pairs}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _values(dev):
    return torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1., -1.5, -2., -3., -4., -6.], device=dev)


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


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _dequantise(codes, scales, descale):
    """fp32 values of packed codes [..., d/2] and scales [..., d/16]."""
    v = _values(codes.device)
    x = torch.stack((v[(codes & 15).int()], v[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2) * descale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, k = _counts(case)
    B, H, H_kv, d, bs, op = case["seqs"], case["H"], case["H_kv"], case["d"], case["block"], case["op"]
    total = sum(n)
    need = [-(-x // bs) for x in k]
    pages = sum(need) + 3                                         # a pool with a few pages to spare, in any order
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)
    at = [sum(need[:b]) for b in range(B)]
    order_h = order.cpu()
    for b in range(B):
        table[b, :need[b]] = order_h[at[b]:at[b] + need[b]]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s = {"op": op, "table": table.to(DEV), "cu": torch.tensor(cu, dtype=torch.int32, device=DEV),
         "seqlens": torch.tensor(k, dtype=torch.int32, device=DEV), "max_q": max(n), "max_k": max(k), "total": total,
         "scale": d ** -0.5, "descale_k": DESCALE_K, "descale_v": DESCALE_V, "interleaved": case["interleaved"]}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    if op in ("append", "append_q4"):
        # keys, values and queries as one fused projection leaves them: rows of one wide matrix
        qkv = normal(total, (H + 2 * H_kv) * d)
        s["q"] = qkv[:, :H * d].unflatten(1, (H, d))
        s["k"] = qkv[:, H * d:(H + H_kv) * d].unflatten(1, (H_kv, d))
        s["v"] = qkv[:, (H + H_kv) * d:].unflatten(1, (H_kv, d))
        p = torch.arange(max(k), dtype=torch.float64, device=DEV)
        angle = p[:, None] * 10000.0 ** (-torch.arange(0, case["rotary"], 2, dtype=torch.float64, device=DEV) / case["rotary"])
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if op == "append":
        s["k_cache"] = torch.zeros((pages, bs, H_kv, d), dtype=torch.bfloat16, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        return s
    for x in ("k", "v"):
        codes = torch.zeros((pages, H_kv, bs, d // 2), dtype=torch.uint8, device=DEV)
        scales = torch.zeros((pages, H_kv, bs, d // 16), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 27) // (H_kv * bs * d))
        for i in range(0, pages if op != "append_q4" else 0, step):
            c, e = _quantise(torch.randn(codes[i:i + step].shape[:3] + (d,), generator=g, device=DEV), s["descale_" + x])
            codes[i:i + step], scales[i:i + step] = _pack(c), e
        s[x + "_codes"], s[x + "_scales"] = codes, scales
    if op == "decode_q4":
        s["q"] = normal(B, H, 1, d)
    elif op == "forward_q4":
        s["q"] = normal(total, H, d)
    return s


# ---------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------

def _places(s):
    """(sequence, position, page, row) of each packed token."""
    t = torch.arange(s["total"], device=DEV)
    cu = s["cu"].long()
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = s["seqlens"].long()[b] - (cu[b + 1] - cu[b]) + t - cu[b]
    block = (s["k_cache"] if "k_cache" in s else s["k_codes"].transpose(1, 2)).shape[1]
    return b, pos, s["table"].long()[b, pos // block], pos % block


def _rotate(x, s, pos):
    """fp32 rotation of x [total, heads, d]."""
    x = x.float()
    c, n = s["cos"][pos][:, None], s["sin"][pos][:, None]
    r = 2 * c.shape[-1]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((y, x[..., r:]), -1)


def _append(s):
    _, pos, page, row = _places(s)
    s["k_cache"][page, row] = _rotate(s["k"], s, pos).to(torch.bfloat16)
    s["v_cache"][page, row] = s["v"]
    return _rotate(s["q"], s, pos).to(torch.bfloat16)


def _append_q4(s):
    _, pos, page, row = _places(s)
    for x, y in (("k", _rotate(s["k"], s, pos)), ("v", s["v"].float())):
        c, e = _quantise(y, s["descale_" + x])
        s[x + "_codes"][page, :, row] = _pack(c)
        s[x + "_scales"][page, :, row] = e
    return _rotate(s["q"], s, pos).to(torch.bfloat16)


def _gather_q4(s):
    _, _, page, row = _places(s)
    return [_dequantise(s[x + "_codes"][page, :, row], s[x + "_scales"][page, :, row], s["descale_" + x]).to(torch.bfloat16)
            for x in ("k", "v")]


def _attend_q4(s):
    """Attention of padded queries [B, n, H, d] over the padded cache."""
    page = s["table"].long()
    H_kv, block, d = s["k_codes"].shape[1], s["k_codes"].shape[2], 2 * s["k_codes"].shape[3]
    B = page.shape[0]

    def cached(x):
        y = _dequantise(s[x + "_codes"][page], s[x + "_scales"][page], s["descale_" + x])    # [B, pages, H_kv, block, d]
        return y.transpose(1, 2).reshape(B, H_kv, -1, d)[:, :, :s["max_k"]]

    lens = s["seqlens"].long()
    if s["op"] == "decode_q4":
        q = s["q"].transpose(1, 2)
        n = torch.ones_like(lens)
    else:
        cu = s["cu"].long()
        n = cu[1:] - cu[:-1]
        q = s["q"][(cu[:-1, None] + torch.arange(s["max_q"], device=DEV)).clamp(max=s["total"] - 1)]
    q = q.float().unflatten(2, (H_kv, -1)).permute(0, 2, 3, 1, 4)                            # [B, H_kv, G, n, d]
    G, m = q.shape[2], q.shape[3]
    i, j = torch.arange(m, device=DEV), torch.arange(s["max_k"], device=DEV)
    seen = j[None, None] <= (lens - n)[:, None, None] + i[None, :, None]                     # [B, n, keys]
    x = torch.matmul(q.reshape(B, H_kv, G * m, d), cached("k").transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (G, m))
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, H_kv, G * m, -1), cached("v")).unflatten(2, (G, m))
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, n, H, d]
    lse = (top + l.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2, 3)                      # [B, n, H]
    if s["op"] == "decode_q4":
        return o.transpose(1, 2).to(torch.bfloat16), lse.transpose(1, 2)
    t = torch.arange(s["total"], device=DEV)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return o[b, t - cu[b]].to(torch.bfloat16), lse[b, t - cu[b]].t().contiguous()


def run(s):
    op = s["op"]
    if own:
        import exact_io_aware_08_gb300 as fa
    if op == "append":
        if own:
            q = fa.append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"], q=s["q"],
                                cos=s["cos"], sin=s["sin"], interleaved=s["interleaved"])
        else:
            q = _append(s)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    cache = [s[x] for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
    if own:
        scales = {"descale_k": s["descale_k"], "descale_v": s["descale_v"]}
    if op == "append_q4":
        # what was appended is read back as the values it stands for; the whole pool's bytes beside
        # them show that nothing else was touched
        if own:
            q = fa.append_paged_q4(s["k"], s["v"], *cache, s["table"], s["cu"], s["seqlens"], q=s["q"], cos=s["cos"], sin=s["sin"],
                                   interleaved=s["interleaved"], **scales)
            k, v = fa.gather_paged_q4(*cache, s["table"], s["cu"], s["seqlens"], s["total"], **scales)
        else:
            q = _append_q4(s)
            k, v = _gather_q4(s)
        return {"q": q, "k": k, "v": v, "k_codes": cache[0], "k_scales": cache[1].view(torch.float8_e4m3fn),
                "v_codes": cache[2], "v_scales": cache[3].view(torch.float8_e4m3fn)}
    if op == "gather_q4":
        k, v = fa.gather_paged_q4(*cache, s["table"], s["cu"], s["seqlens"], s["total"], **scales) if own else _gather_q4(s)
        return {"k": k, "v": v}
    if op == "decode_q4" and own:
        o, lse = fa.decode_paged_q4(s["q"], *cache, s["table"], s["seqlens"], s["max_k"], scale=s["scale"], **scales)
    elif own:
        o, lse = fa.forward_paged_q4(s["q"], *cache, s["table"], s["cu"], s["seqlens"], s["max_q"], s["max_k"], causal=True,
                                     scale=s["scale"], **scales)
    else:
        o, lse = _attend_q4(s)
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, one sequence after another
# ---------------------------------------------------------------------------------------------

def _exact_values(codes, scales, descale):
    """Values in 64 bits from the numbers' own bits."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).double()
    m = c % 8
    a = torch.where(m < 2, m / 2, torch.exp2((m / 2).floor() - 1) * (1 + (m % 2) / 2))
    a = torch.where(c >= 8, -a, a)
    e, f = (scales // 8 % 16).double(), (scales % 8).double()
    s = torch.where(e == 0, f / 512, torch.exp2(e - 7) * (1 + f / 8))
    return a * s.repeat_interleave(16, -1) * descale


def _exact_round(x, descale):
    """x [..., d] in 64 bits as the 4-bit cache holds it."""
    b = x.unflatten(-1, (-1, 16))
    a = (b.abs().amax(-1, keepdim=True) / (6 * descale)).clamp(max=448.0)
    u = torch.exp2(a.clamp(min=2.0 ** -6).log2().floor() - 3)                # spacing of e4m3 numbers there
    s = (a / u).round() * u * descale
    y = torch.where(s > 0, b.abs() / s, torch.zeros_like(b)).clamp(max=6.0)
    u = torch.exp2(y.clamp(min=1.0).log2().floor() - 1)
    return (torch.sign(b) * (y / u).round() * u * s).flatten(-2)


def _exact_rotate(x, at, case):
    """One sequence's x [n, heads, d] at the positions ``at``, as complex numbers."""
    r = case["rotary"]
    w = 10000.0 ** (-2 * torch.arange(r // 2, dtype=torch.float64, device=DEV) / r)
    angle = at.double()[:, None] * w
    turn = torch.complex(angle.cos().float().double(), angle.sin().float().double())[:, None]
    x, rest = x[..., :r], x[..., r:]
    z = x.unflatten(-1, (r // 2, 2)) if case["interleaved"] else x.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.complex(z[..., 0], z[..., 1]) * turn)
    z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat((z, rest), -1)


def exact(case, seed):
    s = prepare(case, seed)
    n, k = _counts(case)
    H_kv, d, block, op = case["H_kv"], case["d"], case["block"], case["op"]
    out, first = {}, 0
    if op == "append":
        caches = {x: s[x + "_cache"].double() for x in ("k", "v")}
    parts = {x: [] for x in ("q", "k", "v", "o", "lse")}
    for b, (new, length) in enumerate(zip(n, k)):
        at = torch.arange(length - new, length, device=DEV)
        mine = slice(first, first + new)
        first += new
        page = s["table"][b].long()
        if op in ("append", "append_q4"):
            rot = {"q": _exact_rotate(s["q"][mine].double(), at, case), "k": _exact_rotate(s["k"][mine].double(), at, case),
                   "v": s["v"][mine].double()}
            parts["q"].append(rot["q"])
            for x in ("k", "v"):
                if op == "append":
                    caches[x][page[at // block], at % block] = rot[x]
                else:
                    parts[x].append(_exact_round(rot[x], s["descale_" + x]))
            continue
        if op == "gather_q4":
            for x in ("k", "v"):
                parts[x].append(_exact_values(s[x + "_codes"][page[at // block], :, at % block],
                                              s[x + "_scales"][page[at // block], :, at % block], s["descale_" + x]))
            continue
        page = page[:-(-length // block)]
        K, V = (_exact_values(s[x + "_codes"][page], s[x + "_scales"][page], s["descale_" + x]).transpose(0, 1).flatten(1, 2)[:, :length]
                for x in ("k", "v"))
        q = (s["q"][b].transpose(0, 1) if op == "decode_q4" else s["q"][mine]).double()      # [new, H, d]
        o, lse = [], []
        for h in range(H_kv):
            G = case["H"] // H_kv
            z = torch.einsum("ngd,kd->ngk", q[:, h * G:(h + 1) * G], K[h]) * s["scale"]
            z = z.masked_fill(torch.arange(length, device=DEV) > at[:, None, None], -math.inf)
            e = torch.logsumexp(z, -1)
            o.append(torch.einsum("ngk,kd->ngd", torch.exp(z - e[..., None]), V[h]))
            lse.append(e)
            del z
        parts["o"].append(torch.cat(o, 1))
        parts["lse"].append(torch.cat(lse, 1))
    if op in ("append", "append_q4"):
        out["q"] = torch.cat(parts["q"])
        if op == "append":
            return dict(out, k_cache=caches["k"], v_cache=caches["v"])
    if op in ("append_q4", "gather_q4"):
        out["k"], out["v"] = torch.cat(parts["k"]), torch.cat(parts["v"])
        return out if op == "gather_q4" else dict(out, k_codes=None, k_scales=None, v_codes=None, v_scales=None)
    o, lse = torch.cat(parts["o"]), torch.cat(parts["lse"])
    return {"o": o[:, :, None], "lse": lse[:, :, None]} if op == "decode_q4" else {"o": o, "lse": lse.t().contiguous()}
