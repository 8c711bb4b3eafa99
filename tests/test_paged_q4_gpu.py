"""The paged-cache operators on the GPU against the plain oracle (oracle/paged.py): appended bytes
exactly, attention within bounds that follow from its roundings.

Caches start with a sentinel in every byte, pages are scattered over a pool in a seeded order,
unused table entries are -1, and what lies behind a sequence's end holds scales that are no number,
so that a stray read or write shows."""
import numpy as np
import pytest
import torch

import exact_io_aware_08_gb300 as fa
from oracle import paged as P
from tests.gpu_common import cuda, poisoned, require_gpu
from tests.test_canaries_gpu import Guarded

pytestmark = pytest.mark.gpu

DK, DV = 0.0021627, 0.0021286        # descales of no special form


def make_pages(lens, block_size, spare, seed):
    """(num_blocks, table [n, max_blocks + 1] int32 with -1 where unused)."""
    need = [-(-n // block_size) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return max(1, sum(need) + spare), table


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(shape, seed, outliers=False):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    if outliers:                                     # a few large elements: running maxima jump
        x.view(-1)[::997] *= 8
    return x


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# (new tokens, tokens with these, H, H_kv, d, block, rotary, interleaved, padding rows, wide rows)
APPENDS = [
    ([1], [1], 1, 1, 64, 64, 64, False, 0, False),
    ([1, 1, 1], [130, 1, 64], 8, 2, 128, 64, 128, False, 2, True),
    ([5, 0, 70, 1], [5, 0, 100, 33], 6, 3, 128, 32, 64, True, 3, True),
    ([3, 2], [50, 2], 5, 5, 64, 16, 32, False, 0, True),
    ([0, 0, 33, 0], [7, 0, 33, 0], 4, 4, 128, 48, 0, False, 1, False),
    ([1] * 70, list(range(1, 71)), 16, 1, 64, 16, 64, True, 5, True),
    ([300, 1, 17], [900, 1025, 17], 7, 1, 128, 128, 96, False, 0, True),
    ([1500, 700, 3], [1500, 800, 30], 32, 8, 128, 64, 128, False, 2, True),
    # enough tokens for several heads a warp: 1, 2, 3 and 8 rounds of them a token
    ([9000, 801], [9000, 900], 2, 2, 64, 64, 64, True, 1, True), ([5000, 7], [5001, 7], 4, 2, 128, 32, 128, False, 0, False),
    ([3300], [3300], 6, 3, 128, 64, 64, True, 1, True), ([1300], [1310], 16, 8, 128, 128, 128, True, 0, False),
]
APPEND_IDS = [f"{len(c[0])}seqs_{sum(c[0])}tok_d{c[4]}_b{c[5]}_r{c[6]}{'i' if c[7] else ''}" for c in APPENDS]


def append_case(case, with_q=True):
    new, lens, H, H_kv, d, block, rotary, inter, pad, wide = case
    total = sum(new) + pad
    seed = sum(lens) + d + H
    cu = np.concatenate(([0], np.cumsum(new)))
    nb, table = make_pages(lens, block, 2, seed)
    if wide:                                        # slices of one projection
        qkv = normal((total, (H + 2 * H_kv) * d), seed)
        q, k, v = (x.unflatten(1, (-1, d)) for x in cuda(qkv).split((H * d, H_kv * d, H_kv * d), 1))
    else:
        q, k, v = (cuda(normal((total, h, d), seed + h)) for h in (H, H_kv, H_kv))
    cos, sin = fa.rotary_tables(max(lens) + 1, rotary, device="cuda") if rotary else (None, None)
    return dict(q=q, k=k, v=v, cu=cu, lens=lens, table=table, nb=nb, cos=cos, sin=sin, H=H, H_kv=H_kv, d=d, block=block,
                inter=inter, total=total, owned=int(cu[-1]))


class Rotation:
    """Host copies of a case's inputs and tables."""

    def __init__(self, c):
        self.c = c
        self.x = {n: f64(c[n]) for n in "qkv"}
        self.cos, self.sin = (None, None) if c["cos"] is None else (f64(c["cos"]), f64(c["sin"]))

    def __call__(self, name, tok, pos, f32=False):
        x = self.x[name][tok]
        if self.cos is None:
            return x
        return (P.rotate_f32 if f32 else P.rotate)(x, self.cos[pos], self.sin[pos], self.c["inter"])

    def check(self, got, name, tok, pos):
        """bf16 of the fp32 rotation: half a bf16 step, and three fp32 roundings of terms no larger
        than |x1| + |x2|."""
        want = self(name, tok, pos)
        big = np.abs(self.x[name][tok]).max(-1, keepdims=True) * 2
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * big).all()


def bf16_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def sample(places):
    """All places of a small case, some of a large one (the first and last among them)."""
    return places if len(places) < 400 else places[:20] + places[20:-20:37] + places[-20:]


@pytest.mark.parametrize("case", APPENDS, ids=APPEND_IDS)
def test_append_bf16(case):
    require_gpu()
    c = append_case(case)
    shape = (c["nb"], c["block"], c["H_kv"], c["d"])
    kc, vc = (torch.full(shape, -7.25, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_out = torch.full((c["total"], c["H"], c["d"]), -7.25, dtype=torch.bfloat16, device="cuda")
    got = fa.append_paged(c["k"], c["v"], kc, vc, i32(c["table"]), i32(c["cu"]), i32(c["lens"]), q=c["q"], cos=c["cos"],
                          sin=c["sin"], interleaved=c["inter"], q_out=q_out)
    fa.fa_sync_status()
    assert got is q_out
    k, v, qo = f64(kc), f64(vc), f64(q_out)
    vbits, vcbits = bf16_bits(c["v"]), bf16_bits(vc)
    touched = np.zeros(shape[:2], bool)
    rot, places = Rotation(c), P.places(c["cu"], c["lens"], c["table"], c["block"])
    for tok, b, pos, page, row in places:
        np.testing.assert_array_equal(vcbits[page, row], vbits[tok])
        touched[page, row] = True
    for tok, b, pos, page, row in sample(places):
        rot.check(k[page, row], "k", tok, pos)
        rot.check(qo[tok], "q", tok, pos)
    for x in (k, v):
        assert (x[~touched] == -7.25).all() and (x[touched] != -7.25).any(-1).all()
    assert (qo[c["owned"]:] == -7.25).all() and (qo[:c["owned"]] != -7.25).any(-1).all()


@pytest.mark.parametrize("case", APPENDS, ids=APPEND_IDS)
def test_append_q4_and_gather(case):
    require_gpu()
    c = append_case(case)
    d, rows = c["d"], (c["nb"], c["H_kv"], c["block"])
    cache = [torch.full((*rows, n), 0xA5, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 16, d // 2, d // 16)]
    table, cu, lens = i32(c["table"]), i32(c["cu"]), i32(c["lens"])
    q_out = fa.append_paged_q4(c["k"], c["v"], *cache, table, cu, lens, q=c["q"], cos=c["cos"], sin=c["sin"], descale_k=DK,
                               descale_v=DV, interleaved=c["inter"], q_out=torch.full_like(c["q"].contiguous(), -7.25))
    ko, vo = (torch.full((c["total"], c["H_kv"], d), -7.25, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_gather_paged_q4(*cache, ko, vo, cu, lens, table, DK, DV)
    fa.fa_sync_status()
    kc, ks, vc, vs = (x.cpu().numpy() for x in cache)
    qo, kf, vf = f64(q_out), f64(ko), f64(vo)
    touched = np.zeros((c["nb"], c["block"]), bool)
    rot, places = Rotation(c), P.places(c["cu"], c["lens"], c["table"], c["block"])
    for tok, b, pos, page, row in places:
        for codes, scales, dscale, back in ((kc, ks, DK, kf), (vc, vs, DV, vf)):
            want = P.values(codes[page, :, row], scales[page, :, row], dscale)
            assert (np.abs(back[tok] - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -15)).all()
        touched[page, row] = True
    for tok, b, pos, page, row in sample(places):
        rot.check(qo[tok], "q", tok, pos)
        for src, codes, scales, dscale in ((rot("k", tok, pos, f32=True), kc, ks, DK), (rot.x["v"][tok], vc, vs, DV)):
            code, s = P.quantise_f32(src.astype(np.float32), dscale)
            np.testing.assert_array_equal(scales[page, :, row], s)
            np.testing.assert_array_equal(codes[page, :, row], P.pack(code))
    for x in (kc, ks, vc, vs):
        assert (x.swapaxes(1, 2)[~touched] == 0xA5).all()
    for x in (qo, kf, vf):
        assert (x[c["owned"]:] == -7.25).all()


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,d,rotary", [(4000, 128, 128), (3, 128, 128), (2500, 64, 32)])
def test_rotation_rounds_every_operation(n, d, rotary, inter, q4):
    """The rotated queries (and bf16 keys) are those of separately rounded fp32 products and sums, bit for
    bit: one product too few rounded would change one in some 2^16 of them."""
    require_gpu()
    H, H_kv, block = 16, 4, 64
    nb, table = make_pages([n], block, 0, 5)
    q, k, v = (cuda(normal((n, h, d), 90 + h)) for h in (H, H_kv, H_kv))
    cos, sin = fa.rotary_tables(n, rotary, device="cuda")

    def rotated(x):
        y = x.float()
        a, e = (slice(0, rotary, 2), slice(1, rotary, 2)) if inter else (slice(rotary // 2), slice(rotary // 2, rotary))
        c, s = cos[:, None], sin[:, None]
        x1, x2 = y[..., a].clone(), y[..., e].clone()
        p, r = x1 * c, x2 * s
        y[..., a] = p - r
        p, r = x2 * c, x1 * s
        y[..., e] = p + r
        return y.to(torch.bfloat16)

    args = (i32(table), i32([0, n]), i32([n]))
    if q4:
        cache = [torch.zeros(nb, H_kv, block, m, dtype=torch.uint8, device="cuda") for m in (d // 2, d // 16, d // 2, d // 16)]
        qo = fa.append_paged_q4(k, v, *cache, *args, q=q, cos=cos, sin=sin, descale_k=DK, descale_v=DV, interleaved=inter)
    else:
        kc, vc = (torch.zeros(nb, block, H_kv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        qo = fa.append_paged(k, v, kc, vc, *args, q=q, cos=cos, sin=sin, interleaved=inter)
        pages = i32(table[0, :-(-n // block)]).long()
        assert torch.equal(kc[pages].view(-1, H_kv, d)[:n], rotated(k))
        assert torch.equal(vc[pages].view(-1, H_kv, d)[:n], v)
    fa.fa_sync_status()
    assert torch.equal(qo, rotated(q))


def test_append_in_place_and_without_queries():
    """q_out may be q; without queries only keys and values move."""
    require_gpu()
    c = append_case(([4, 9], [20, 9], 4, 2, 128, 16, 128, False, 0, False))
    rows = (c["nb"], c["block"], c["H_kv"], c["d"])
    kc, vc, kc2, vc2 = (torch.zeros(rows, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    idx = i32(c["table"]), i32(c["cu"]), i32(c["lens"])
    rot = dict(cos=c["cos"], sin=c["sin"])
    want = fa.append_paged(c["k"], c["v"], kc, vc, *idx, q=c["q"], **rot)
    q = c["q"].clone()
    assert fa.append_paged(c["k"], c["v"], kc2, vc2, *idx, q=q, q_out=q, **rot) is q
    assert torch.equal(q, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    kc2.zero_()
    assert fa.append_paged(c["k"], c["v"], kc2, vc2, *idx, **rot) is None
    assert torch.equal(kc, kc2)
    fa.fa_sync_status()


def test_quantiser_borders():
    """Zeros, ties, tiny and huge blocks, infinities and NaN: the bytes of the fp32 definition, and
    something finite for what is not finite."""
    require_gpu()
    d, H = 64, 1
    rows = torch.zeros(8, H, d)
    rows[1] = -0.0
    rows[2, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5.])
    rows[3] = 2.0 ** -30
    rows[4] = 3e38
    rows[5, 0, ::2] = -2688.0
    rows[5, 0, 1::2] = 2.0 ** -9
    rows[6, 0] = torch.linspace(-448 * 6, 448 * 6, d)
    rows[7, 0, 5] = 2.0 ** -133
    v = rows.to(torch.bfloat16).cuda()
    bad = v.clone()
    bad[0, 0, 3], bad[1, 0, 20], bad[2, 0, 40] = float("inf"), float("-inf"), float("nan")
    for x, exact in ((v, True), (bad, False)):
        cache = [torch.zeros((1, H, 16, n), dtype=torch.uint8, device="cuda") for n in (32, 4, 32, 4)]
        idx = i32([[0]]), i32([0, 8]), i32([8])
        fa.append_paged_q4(x, x, *cache, *idx)
        k, w = fa.gather_paged_q4(*cache, *idx, 8)
        fa.fa_sync_status()
        assert torch.isfinite(k.float()).all() and torch.equal(k, w)
        if exact:
            code, s = P.quantise_f32(f64(x).astype(np.float32), 1.0)
            np.testing.assert_array_equal(cache[0][0, 0, :8].cpu().numpy(), P.pack(code)[:, 0])
            np.testing.assert_array_equal(cache[1][0, 0, :8].cpu().numpy(), s[:, 0])


# ------------------------------------------------------------------------------------------- attention

def fill_cache(lens, H_kv, d, block, seed, outliers=False):
    """A 4-bit cache with every sequence's tokens (drawn, quantised by the oracle), garbage elsewhere
    (scales that are no number among it); the fp64 values per sequence."""
    nb, table = make_pages(lens, block, 3, seed)
    rng = np.random.default_rng(seed)
    cache = {x: (rng.integers(0, 256, (nb, H_kv, block, d // 2), dtype=np.uint8), np.full((nb, H_kv, block, d // 16), 0x7F, np.uint8))
             for x in "kv"}
    val = {"k": [], "v": []}
    for x, dscale in (("k", DK), ("v", DV)):
        codes, scales = cache[x]
        for b, n in enumerate(lens):
            y = f64(normal((n, H_kv, d), seed + 7 * b + ord(x), outliers)).astype(np.float32)
            code, s = P.quantise_f32(y, dscale)
            packed = P.pack(code)
            p = np.arange(n)
            codes[table[b, p // block], :, p % block] = packed
            scales[table[b, p // block], :, p % block] = s
            val[x].append(P.values(packed, s, dscale))
    return [cuda(torch.from_numpy(a)) for x in "kv" for a in cache[x]], table, val


def check_attention(o, lse, want):
    ro, rl, bo, bl = want
    assert np.isfinite(o).all()
    none = np.isneginf(rl)
    assert (np.isneginf(lse) == none).all() and (o[none] == 0).all()
    assert (np.abs(o - ro) <= bo).all(), float((np.abs(o - ro) / bo)[~none].max())
    off = np.abs(lse[~none] - rl[~none]) / bl[~none]
    assert (off <= 1).all(), float(off.max())


# (lens, H, H_kv, d, block, n_splits)
DECODES = [
    ([1], 1, 1, 64, 16, 1), ([1], 4, 1, 128, 64, 0), ([63, 64, 65], 2, 2, 128, 64, 1), ([0, 5, 0, 300], 8, 2, 64, 32, 3),
    ([1000, 37, 513], 32, 8, 128, 16, 7), ([700], 5, 1, 128, 48, 0), ([257, 31], 12, 4, 64, 48, 2), ([640, 200], 9, 1, 128, 128, 0),
    ([500, 100], 16, 1, 64, 64, 4), ([333], 40, 2, 128, 32, 2), ([90, 1], 64, 1, 128, 16, 1), ([2000, 3], 8, 8, 128, 256, 64),
    ([4096, 4000], 3, 3, 64, 256, 0), ([0, 0], 4, 2, 128, 64, 2), ([1100], 200, 1, 128, 64, 0),
    # rows of many states: few of them, and more than a thousand
    ([9000], 8, 8, 128, 64, 0), ([6000, 0, 10], 4, 1, 64, 32, 0), ([5000] + [70, 0, 300, 1] * 9, 32, 2, 128, 16, 0),
    ([700, 90] * 18, 32, 4, 64, 64, 20), ([3000, 17], 8, 2, 128, 64, 24),
    # short row blocks that are not divided, and just too long for it
    ([640, 0, 1, 129, 500] * 10, 8, 4, 128, 64, 0), ([300, 0, 77] * 11, 40, 4, 64, 32, 0), ([641, 0, 1, 129, 500] * 10, 8, 4, 128, 64, 0),
    ([0, 0, 0, 128] + [0] * 200, 2, 1, 128, 64, 0), ([600] + [0] * 200, 2, 1, 64, 64, 0),
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"{len(c[0])}x{max(c[0])}_{c[1]}of{c[2]}_d{c[3]}_b{c[4]}_s{c[5]}")
def test_decode_q4(case):
    require_gpu()
    lens, H, H_kv, d, block, n_splits = case
    B, N, G = len(lens), max(max(lens), 1), H // H_kv
    cache, table, val = fill_cache(lens, H_kv, d, block, sum(lens) + d, outliers=True)
    q = normal((B, H, 1, d), 5 + N)
    need = fa.fa_decode_paged_q4_workspace_size(B, H, H_kv, N, d, n_splits)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    o, lse = poisoned((B, H, 1, d), torch.bfloat16), poisoned((B, H, 1), torch.float32)
    fa.fa_decode_paged_q4(cuda(q), *cache, o, lse, i32(table), i32(lens), N, d ** -0.5, DK, DV, n_splits, ws)
    fa.fa_sync_status()
    for b in range(B):
        for h in range(H_kv):
            s = slice(h * G, (h + 1) * G)
            want = P.attend(f64(q[b, s, 0]), val["k"][b][:, h], val["v"][b][:, h], d ** -0.5, [lens[b]] * G)
            check_attention(f64(o[b, s, 0]), f64(lse[b, s, 0]), want)


# (query tokens, lens, H, H_kv, d, block, causal, n_splits, padding rows)
FORWARDS = [
    ([1], [1], 1, 1, 128, 16, True, 1, 0), ([4, 4], [100, 70], 8, 2, 128, 64, True, 0, 2), ([1, 0, 9], [65, 30, 9], 4, 4, 64, 32, True, 2, 3),
    ([33, 2], [33, 400], 6, 2, 128, 48, True, 3, 0), ([40], [10], 2, 1, 64, 16, True, 1, 0), ([40], [10], 2, 1, 128, 16, True, 4, 1),
    ([50, 7], [200, 0], 4, 2, 128, 64, True, 1, 0), ([17, 64], [129, 300], 16, 2, 64, 128, False, 0, 4),
    ([200, 1, 77], [700, 513, 77], 8, 2, 128, 64, True, 0, 0), ([130], [130], 3, 3, 64, 16, True, 1, 0),
    ([129, 260], [129, 1000], 5, 1, 128, 32, True, 2, 5), ([150], [450], 12, 12, 128, 256, False, 1, 0),
    ([256], [256], 4, 4, 128, 128, True, 1, 0), ([300, 20], [900, 20], 10, 2, 64, 64, True, 1, 0),
    ([1, 600], [3, 600], 4, 1, 128, 16, True, 0, 1), ([520], [1500], 8, 1, 64, 48, True, 5, 0),
    # on either side of the rows from which on tiles are used
    ([8, 3], [300, 900], 8, 2, 128, 64, True, 0, 1), ([9, 2], [300, 900], 8, 2, 128, 64, True, 0, 1), ([12, 1], [700, 90], 8, 2, 64, 32, True, 0, 0),
    ([13, 0], [700, 90], 8, 2, 64, 32, True, 3, 0),
    ([3, 1, 0, 4] * 20, [500, 1, 70, 4] * 20, 8, 2, 128, 64, True, 0, 3), ([1, 2] * 40, [600, 40] * 40, 4, 2, 64, 32, True, 0, 0),
    # row blocks that are split because they do not fill the SMs
    ([70], [5000], 4, 4, 128, 64, True, 0, 0), ([64], [9000], 4, 1, 64, 64, True, 0, 2), ([300], [2500], 4, 1, 128, 64, True, 0, 1), ([200, 90], [2200, 1100], 4, 2, 64, 32, True, 0, 2), ([70, 0, 3], [3100, 40, 1030], 4, 2, 128, 48, False, 0, 0),
]


@pytest.mark.parametrize("case", FORWARDS, ids=lambda c: f"{len(c[0])}x{max(c[0])}of{max(c[1])}_{c[2]}of{c[3]}_d{c[4]}_b{c[5]}{'_c' if c[6] else ''}_s{c[7]}")
def test_forward_q4(case):
    require_gpu()
    new, lens, H, H_kv, d, block, causal, n_splits, pad = case
    cu = np.concatenate(([0], np.cumsum(new)))
    total, N, G = int(cu[-1]) + pad, max(lens), H // H_kv
    cache, table, val = fill_cache(lens, H_kv, d, block, sum(lens) + d + H, outliers=True)
    q = normal((total, H, d), 9 + N)
    need = fa.fa_fwd_paged_q4_workspace_size(len(lens), H, H_kv, total, max(new), N, d, n_splits)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    o = torch.full((total, H, d), -7.25, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, total), -7.25, dtype=torch.float32, device="cuda")
    fa.fa_fwd_paged_q4(cuda(q), *cache, o, lse, i32(cu), i32(lens), i32(table), max(new), N, d ** -0.5, DK, DV, causal, n_splits, ws)
    fa.fa_sync_status()
    for b, n in enumerate(new):
        rows = slice(cu[b], cu[b + 1])
        seen = [lens[b] - n + i + 1 if causal else lens[b] for i in range(n)]
        for h in range(H):
            want = P.attend(f64(q[rows, h]), val["k"][b][:, h // G], val["v"][b][:, h // G], d ** -0.5, seen)
            check_attention(f64(o[rows, h]), f64(lse[h, rows]), want)
    assert (o[cu[-1]:] == -7.25).all() and (lse[:, cu[-1]:] == -7.25).all()


@pytest.mark.parametrize("n,keys,d", [(1, 200, 128), (40, 200, 128), (1, 1500, 128), (4, 1500, 128), (40, 900, 128), (300, 900, 128),
                                      (1, 1500, 64), (4, 1500, 64), (40, 900, 64)])
def test_q4_attention_with_queries_of_any_size(n, keys, d):
    """Rows of tiny, huge and zero queries beside ordinary ones: each keeps its own factor."""
    require_gpu()
    lens, H, block = [keys], 8, 64
    cache, table, val = fill_cache(lens, 1, d, block, 3)
    q = normal((n, H, d), 4)
    for h, f in enumerate((1.0, 2.0 ** -40, 2.0 ** -120, 0.0, 2.0 ** 6, 2.0 ** 40, 2.0 ** -20, 1.0)):
        q[:, h] *= f
    q[0, 7, 3] = 300.0
    o, lse = fa.forward_paged_q4(cuda(q), *cache, i32(table), i32([0, n]), i32(lens), n, keys, causal=False, descale_k=DK,
                                 descale_v=DV)
    fa.fa_sync_status()
    rows = [0, 1, 2, 3, 4, 6, 7]
    for t in range(n):
        want = P.attend(f64(q[t]), val["k"][0][:, 0], val["v"][0][:, 0], d ** -0.5, [keys] * H)
        check_attention(f64(o[t, rows]), f64(lse[rows, t]), [x[rows] for x in want])
        # scores of 2^40 leave one key: its value exactly, and the score itself for lse
        best = int(np.argmax(val["k"][0][:, 0] @ f64(q[t, 5])))
        np.testing.assert_allclose(f64(o[t, 5]), val["v"][0][best, 0], rtol=2.0 ** -8)
        np.testing.assert_allclose(f64(lse[5, t]), want[1][5], rtol=2.0 ** -16)


def test_q4_attention_is_the_same_twice_and_captured():
    """No atomics: the same bits on a second call, on another stream, and replayed from a graph."""
    require_gpu()
    new, lens, H, H_kv, d = [3, 90, 1], [500, 90, 1000], 8, 2, 128
    cu = np.concatenate(([0], np.cumsum(new)))
    cache, table, _ = fill_cache(lens, H_kv, d, 64, 21)
    q = cuda(normal((94, H, d), 6))
    args = (*cache, i32(table), i32(cu), i32(lens), 90, 1000)
    more = dict(descale_k=DK, descale_v=DV)
    o, lse = fa.forward_paged_q4(q, *args, **more)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, lse2 = fa.forward_paged_q4(q, *args, **more)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = fa.forward_paged_q4(q, *args, **more)
    for _ in range(2):
        o3.fill_(0)
        graph.replay()
    fa.fa_sync_status()
    for a, b in ((o2, lse2), (o3, lse3)):
        assert torch.equal(o, a) and torch.equal(lse, b)


@pytest.mark.parametrize("n", [1, 4, 40, 300])
def test_q4_attention_with_a_vanishing_score_factor(n):
    """Scores below fp32's range: every key weighs the same."""
    require_gpu()
    lens, H, d = [200], 4, 128
    cache, table, val = fill_cache(lens, 2, d, 64, 3)
    q = normal((n, H, d), 4) * 2.0 ** -100
    o, lse = fa.forward_paged_q4(cuda(q), *cache, i32(table), i32([0, n]), i32(lens), n, 200, causal=False, descale_k=1e-20,
                                 descale_v=DV)
    fa.fa_sync_status()
    for h in range(H):
        want = P.attend(f64(q[:, h]), val["k"][0][:, h // 2] * (1e-20 / DK), val["v"][0][:, h // 2], d ** -0.5, [200] * n)
        check_attention(f64(o[:, h]), f64(lse[h]), want)


@pytest.mark.parametrize("n_splits", [0, 1, 3])
@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_numbers_that_are_none_stay_none(n, n_splits):
    """A query row that holds no number, and rows that see a key or value whose scale is none, give NaN;
    the other rows, rows without keys and the other sequences keep their results."""
    require_gpu()
    H, H_kv, d, lens = 4, 2, 128, [700, 700, 0, 300]
    cu = np.arange(5) * n
    cache, table, _ = fill_cache(lens, H_kv, d, 64, 11)
    q = cuda(normal((4 * n, H, d), 3))
    args = (i32(table), i32(cu), i32(lens), n, 700)
    more = dict(causal=False, n_splits=n_splits, descale_k=DK, descale_v=DV)
    o, lse = fa.forward_paged_q4(q, *cache, *args, **more)
    bad = q.clone()
    bad[0, 1, 5] = float("nan")
    bad[2 * n + n - 1, 0, 0] = float("nan")                  # a sequence without keys: nothing to be seen
    ks, vs = cache[1].clone(), cache[3].clone()
    ks[int(table[1, 2]), 0, 9, 3] = 0x7F                     # sequence 1, key 137, key head 0
    vs[int(table[3, 4]), 1, 2, 7] = 0xFF                     # sequence 3, value 258, key head 1, the last 16 elements
    o2, lse2 = fa.forward_paged_q4(bad, cache[0], ks, cache[2], vs, *args, **more)
    fa.fa_sync_status()
    o, lse, o2, lse2 = (x.cpu() for x in (o, lse, o2, lse2))
    lost = torch.zeros(4 * n, H, d, dtype=torch.bool)
    lost[0, 1] = True
    lost[n:2 * n, :2] = True
    lost[3 * n:, 2:, 112:] = True
    assert (o2.isnan() == lost).all()
    assert torch.equal(o2[~lost], o[~lost])
    gone = torch.zeros(H, 4 * n, dtype=torch.bool)
    gone[1, 0] = True
    gone[:2, n:2 * n] = True
    assert (lse2.isnan() == gone).all()
    assert torch.equal(lse2[~gone], lse[~gone])


def test_outputs_belong_to_the_stream_that_is_given():
    """What a call allocates for another stream than the current one is that stream's memory."""
    require_gpu()
    lens = [500, 90]
    cache, table, _ = fill_cache(lens, 2, 128, 64, 21)
    q = cuda(normal((2, 8, 1, 128), 6))
    args = (*cache, i32(table), i32(lens), 500)
    o, lse = fa.decode_paged_q4(q, *args, descale_k=DK, descale_v=DV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        o2, lse2 = fa.decode_paged_q4(q, *args, descale_k=DK, descale_v=DV, stream=stream)
        side.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for t in (o2, lse2):
            segment = [x for x in torch.cuda.memory_snapshot() if x["address"] <= t.data_ptr() < x["address"] + x["total_size"]]
            assert [x["stream"] for x in segment] == [side.cuda_stream]
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    fa.fa_sync_status()


def test_append_of_one_token_with_any_token_stride():
    require_gpu()
    nb, table = make_pages([70], 64, 0, 1)
    x = cuda(normal((3, 2, 128), 4))
    caches = []
    for k in (x[:1], x.view(-1)[:256].as_strided((1, 2, 128), (3, 128, 1))):
        kc, vc = (torch.zeros(nb, 64, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        fa.append_paged(k, k, kc, vc, i32(table), i32([0, 1]), i32([70]))
        caches.append((kc, vc))
    fa.fa_sync_status()
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    assert torch.equal(caches[1][0][int(table[0, 1]), 5], x[0])


def test_decode_equals_forward_of_one_token():
    require_gpu()
    lens, H, H_kv, d = [700, 64, 0, 333], 8, 4, 128
    cache, table, _ = fill_cache(lens, H_kv, d, 32, 8)
    q = cuda(normal((4, H, 1, d), 2))
    more = dict(descale_k=DK, descale_v=DV, n_splits=3)
    o, lse = fa.decode_paged_q4(q, *cache, i32(table), i32(lens), 700, **more)
    o2, lse2 = fa.forward_paged_q4(q[:, :, 0].contiguous(), *cache, i32(table), i32([0, 1, 2, 3, 4]), i32(lens), 1, 700, **more)
    fa.fa_sync_status()
    assert torch.equal(o[:, :, 0], o2) and torch.equal(lse[:, :, 0].t(), lse2)


def test_serving_run_bf16():
    """Prompts appended, then tokens one by one, each step attended by fa_decode_paged."""
    require_gpu()
    H, d, block, lens = 2, 64, 64, [70, 3]
    steps = 3
    nb, table = make_pages([n + steps for n in lens], block, 1, 0)
    kc, vc = (torch.full((nb, block, H, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cos, sin = fa.rotary_tables(128, d, device="cuda")
    t = i32(table)
    ks, vs = [[], []], [[], []]
    now = list(lens)
    for step in range(steps + 1):
        new = lens if step == 0 else [1, 1]
        now = [a if step == 0 else a + 1 for a in now]
        cu = np.concatenate(([0], np.cumsum(new)))
        q, k, v = (normal((int(cu[-1]), H, d), 100 * step + i) for i in range(3))
        q_rot = fa.append_paged(cuda(k), cuda(v), kc, vc, t, i32(cu), i32(now), q=cuda(q), cos=cos, sin=sin)
        for b in range(2):
            for i in range(new[b]):
                p = now[b] - new[b] + i
                ks[b].append(P.rotate(f64(k[cu[b] + i]), f64(cos[p]), f64(sin[p]), False))
                vs[b].append(f64(v[cu[b] + i]))
        last = torch.stack([q_rot[cu[b + 1] - 1] for b in range(2)])[:, :, None].contiguous()
        o, lse = fa.decode_paged(last, kc, vc, t, i32(now), max(now))
        fa.fa_sync_status()
        for b in range(2):
            K, V = np.stack(ks[b]), np.stack(vs[b])
            for h in range(H):
                p = now[b] - 1
                qr = P.rotate(f64(q[cu[b + 1] - 1]), f64(cos[p]), f64(sin[p]), False)[h]
                ro, rl, bo, bl = P.attend(qr[None], K[:, h], V[:, h], d ** -0.5, [len(K)])
                # q and K were rounded to bf16: scores move by 2^-7 of their terms
                move = 2.0 ** -7 * d ** -0.5 * (np.abs(K[:, h]) @ np.abs(qr)).max()
                assert np.abs(f64(lse[b, h, 0]) - rl[0]) <= bl[0] + 1.01 * move
                assert (np.abs(f64(o[b, h, 0]) - ro[0]) <= bo[0] + 2.2 * move * np.abs(V[:, h]).max()).all()


def test_serving_run_q4():
    """Prompts in two parts, then single tokens, then a few drafted ones, over one 4-bit cache: each
    step's attention against the values the cache then holds, read back by gather."""
    require_gpu()
    H, H_kv, d, block = 6, 2, 128, 16
    parts = [[40, 3], [25, 0], [1, 1], [1, 1], [4, 4]]
    ends = np.cumsum(parts, 0)
    nb, table = make_pages(ends[-1].tolist(), block, 1, 1)
    rows = (nb, H_kv, block)
    cache = [torch.full((*rows, n), 0x7F, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 16, d // 2, d // 16)]
    cos, sin = fa.rotary_tables(256, d, device="cuda")
    t, scales = i32(table), dict(descale_k=DK, descale_v=DV)
    for step, (new, now) in enumerate(zip(parts, ends)):
        cu = np.concatenate(([0], np.cumsum(new)))
        q, k, v = (cuda(normal((int(cu[-1]), h, d), 50 * step + i)) for i, h in enumerate((H, H_kv, H_kv)))
        q_rot = fa.append_paged_q4(k, v, *cache, t, i32(cu), i32(now), q=q, cos=cos, sin=sin, **scales)
        if max(new) == 1:
            o, lse = fa.decode_paged_q4(q_rot[:, :, None].contiguous(), *cache, t, i32(now), int(max(now)), **scales)
            o, lse = o[:, :, 0], lse[:, :, 0].t()
        else:
            o, lse = fa.forward_paged_q4(q_rot, *cache, t, i32(cu), i32(now), int(max(new)), int(max(now)), **scales)
        whole = np.concatenate(([0], np.cumsum(now)))
        K, V = fa.gather_paged_q4(*cache, t, i32(whole), i32(now), int(whole[-1]), **scales)
        fa.fa_sync_status()
        kc, ksc, vc, vsc = (x.cpu().numpy() for x in cache)
        for b in range(2):
            at = np.arange(now[b])
            kv = P.values(kc[table[b, at // block], :, at % block], ksc[table[b, at // block], :, at % block], DK)
            vv = P.values(vc[table[b, at // block], :, at % block], vsc[table[b, at // block], :, at % block], DV)
            np.testing.assert_allclose(f64(K[whole[b]:whole[b + 1]]), kv, rtol=2.0 ** -8 * (1 + 2.0 ** -15))
            np.testing.assert_allclose(f64(V[whole[b]:whole[b + 1]]), vv, rtol=2.0 ** -8 * (1 + 2.0 ** -15))
            if new[b] == 0:
                continue
            mine = slice(cu[b], cu[b + 1])
            seen = [now[b] - new[b] + i + 1 for i in range(new[b])]
            for h in range(H):
                g = h // (H // H_kv)
                check_attention(f64(o[mine, h]), f64(lse[h, mine]), P.attend(f64(q_rot[mine, h]), kv[:, g], vv[:, g], d ** -0.5, seen))


def test_gathered_prefix_feeds_the_varlen_forward():
    """A 4-bit prefix handed to fa_fwd_varlen as bf16 gives what the 4-bit attention gives, up to the
    roundings of the keys and values to bf16."""
    require_gpu()
    lens, H, d = [130, 64], 2, 128
    cache, table, val = fill_cache(lens, H, d, 64, 77)
    cu = i32([0, 130, 194])
    K, V = fa.gather_paged_q4(*cache, i32(table), cu, i32(lens), 194, descale_k=DK, descale_v=DV)
    q = normal((194, H, d), 1)
    o, lse = fa.forward_varlen(cuda(q), K, V, cu, cu, 130, 130, causal=False)
    o2, lse2 = fa.forward_paged_q4(cuda(q), *cache, i32(table), cu, i32(lens), 130, 130, causal=False, descale_k=DK, descale_v=DV)
    fa.fa_sync_status()
    for b, (lo, hi) in enumerate(((0, 130), (130, 194))):
        for h in range(H):
            k, v = val["k"][b][:, h], val["v"][b][:, h]
            move = 2.0 ** -8 * d ** -0.5 * (np.abs(f64(q[lo:hi, h])) @ np.abs(k).T).max(1)
            assert (np.abs(f64(lse[h, lo:hi]) - f64(lse2[h, lo:hi])) <= 1.05 * move + 2.0 ** -9).all()
            # each result's weights and output roundings, and the move of scores and values
            top = np.abs(v).max()
            assert (np.abs(f64(o[lo:hi, h]) - f64(o2[lo:hi, h])) <= (2.2 * move[:, None] + 5 * 2.0 ** -8) * top).all()


# ------------------------------------------------------------------------------------------- bad contents

@pytest.mark.parametrize("n_splits", [0, 1, 3, 12])
@pytest.mark.parametrize("n,d", [(1, 128), (3, 64), (4, 128), (8, 128), (37, 64), (37, 128), (150, 128), (150, 64)])
def test_everything_stays_in_bounds(n, d, n_splits):
    """Pools, outputs and workspaces between guard bands, at sizes that fill no tile."""
    require_gpu()
    H, H_kv, block, lens = 10, 2, 48, [n + 700, n, n + 3001]
    cu = np.arange(4) * n
    total, N = 3 * n, max(lens)
    nb, table = make_pages(lens, block, 0, 3)
    pool = [Guarded((nb, H_kv, block, m), torch.uint8) for m in (d // 2, d // 16, d // 2, d // 16)]
    for x in pool:
        x.t.random_(0, 0x70)                                  # codes of any kind, scales that are numbers
    q, k, v = (cuda(normal((total, h, d), h)) for h in (H, H_kv, H_kv))
    cos, sin = fa.rotary_tables(N, d, device="cuda")
    caches = [x.t for x in pool]
    qo = Guarded((total, H, d), torch.bfloat16)
    fa.fa_append_paged_q4(q, k, v, qo.t, *caches, cos, sin, i32(cu), i32(lens), i32(table), DK, DV)
    ko, vo = (Guarded((total, H_kv, d), torch.bfloat16) for _ in "kv")
    fa.fa_gather_paged_q4(*caches, ko.t, vo.t, i32(cu), i32(lens), i32(table), DK, DV)
    o, lse = Guarded((total, H, d), torch.bfloat16), Guarded((H, total), torch.float32)
    ws = Guarded((fa.fa_fwd_paged_q4_workspace_size(3, H, H_kv, total, n, N, d, n_splits),), torch.uint8)
    fa.fa_fwd_paged_q4(qo.t, *caches, o.t, lse.t, i32(cu), i32(lens), i32(table), n, N, d ** -0.5, DK, DV, True, n_splits, ws.t)
    fa.fa_sync_status()
    for x, name in ((qo, "q"), (ko, "k"), (vo, "v"), (o, "o"), (lse, "lse")):
        x.check(name)
    for x in (*pool, ws):
        x.check("pool or workspace", fully_written=False)
    kc, vc = (Guarded((nb, block, H_kv, d), torch.bfloat16) for _ in "kv")
    q2 = Guarded((total, H, d), torch.bfloat16)
    fa.fa_append_paged(q, k, v, q2.t, kc.t, vc.t, cos, sin, i32(cu), i32(lens), i32(table))
    fa.fa_sync_status()
    q2.check("q")
    for x in (kc, vc):
        x.check("pool", fully_written=False)
    if n == 1:
        o, lse = Guarded((3, H, 1, d), torch.bfloat16), Guarded((3, H, 1), torch.float32)
        ws = Guarded((fa.fa_decode_paged_q4_workspace_size(3, H, H_kv, N, d, n_splits),), torch.uint8)
        fa.fa_decode_paged_q4(qo.t[:, :, None], *caches, o.t, lse.t, i32(table), i32(lens), N, d ** -0.5, DK, DV, n_splits, ws.t)
        fa.fa_sync_status()
        for x, name in ((o, "o"), (lse, "lse")):
            x.check(name)
        ws.check("workspace", fully_written=False)


def test_captured_step_follows_the_lengths():
    """A step (append, then attention) captured once and replayed as the sequences grow, beside the same
    steps called one by one: the lengths are read on the device."""
    require_gpu()
    lens, H, H_kv, d, block, steps = [300, 0, 127, 900], 8, 2, 128, 64, 4
    B, N = len(lens), 1024
    cache, table, _ = fill_cache(lens, H_kv, d, block, 13)
    pages = np.arange(B * 16, dtype=np.int32).reshape(B, 16)             # a pool of its own, sequence by sequence
    pool = [torch.zeros(B * 16, H_kv, block, x.shape[3], dtype=torch.uint8, device="cuda") for x in cache]
    for b, n in enumerate(lens):
        for i in range(-(-n // block)):
            for x, y in zip(pool, cache):
                x[int(pages[b, i])] = y[int(table[b, i])]
    other = [x.clone() for x in pool]
    cos, sin = fa.rotary_tables(N, d, device="cuda")
    cu, tab = i32(np.arange(B + 1)), i32(pages)
    qkv = [cuda(normal((B, (H + 2 * H_kv) * d), 40 + i)) for i in range(steps)]

    def step(x, pool, n):
        q, k, v = (y.unflatten(1, (-1, d)) for y in x.split((H * d, H_kv * d, H_kv * d), 1))
        q = fa.append_paged_q4(k, v, *pool, tab, cu, n, q=q, cos=cos, sin=sin, descale_k=DK, descale_v=DV)
        return fa.decode_paged_q4(q[:, :, None], *pool, tab, n, N, descale_k=DK, descale_v=DV)

    want, n = [], i32(lens)
    for x in qkv:
        n += 1
        want.append(step(x, pool, n))
    x, n = qkv[0].clone(), i32(lens)
    step(x, [y.clone() for y in other], n + 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n += 1
        o, lse = step(x, other, n)
    for i in range(steps):
        x.copy_(qkv[i])
        graph.replay()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    fa.fa_sync_status()
    for y, z in zip(pool, other):
        assert torch.equal(y, z)


@pytest.mark.parametrize("n", [1, 4, 70])
def test_calls_side_by_side(n):
    """Calls on two streams at once, each with outputs and workspace of its own."""
    require_gpu()
    H, H_kv, d = 8, 2, 128
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls, want = [], []
    for i in range(2):
        lens = [3000 + 200 * i, 64, 900]
        cache, table, _ = fill_cache(lens, H_kv, d, 64, 50 + i)
        q = cuda(normal((3 * n, H, d), 60 + i))
        calls.append((q, *cache, i32(table), i32(np.arange(4) * n), i32(lens), n, max(lens)))
        want.append(fa.forward_paged_q4(*calls[i], descale_k=DK, descale_v=DV))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append((i, fa.forward_paged_q4(*calls[i], descale_k=DK, descale_v=DV)))
    torch.cuda.synchronize()
    fa.fa_sync_status()
    for i, (o, lse) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_pages_past_32_bits():
    """The last pages of pools whose bytes and elements pass 2^32: the same as in a small pool."""
    require_gpu()
    H, H_kv, d, block, n, old = 16, 8, 128, 64, 70, 330
    need = -(-(old + n) // block)
    small, big = need, (2 ** 32 // (H_kv * block * d)) + need + 5              # bf16 elements past 2^32
    cos, sin = fa.rotary_tables(old + n, d, device="cuda")
    q, k, v = (cuda(normal((old + n, h, d), 70 + h)) for h in (H, H_kv, H_kv))
    first, new = i32([0, old]), i32([0, n])
    got = []
    for pages in (small, big):
        table = i32(np.arange(pages - need, pages)[None])
        at = slice(pages - need, pages)
        kc, vc = (torch.empty(pages, block, H_kv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        for x, lens, part in ((first, [old], slice(0, old)), (new, [old + n], slice(old, None))):
            fa.append_paged(k[part], v[part], kc, vc, table, x, i32(lens), q=q[part], cos=cos, sin=sin)
        got.append([torch.cat([c[at].view(-1, H_kv, d)[:old + n] for c in (kc, vc)])])
        del kc, vc
    for pages in (small, 2 * big):                                             # code bytes past 2^32
        table = i32(np.arange(pages - need, pages)[None])
        cache = [torch.empty(pages, H_kv, block, m, dtype=torch.uint8, device="cuda") for m in (d // 2, d // 16, d // 2, d // 16)]
        for x, lens, part in ((first, [old], slice(0, old)), (new, [old + n], slice(old, None))):
            qo = fa.append_paged_q4(k[part], v[part], *cache, table, x, i32(lens), q=q[part], cos=cos, sin=sin, descale_k=DK, descale_v=DV)
        more = dict(descale_k=DK, descale_v=DV)
        out = list(fa.gather_paged_q4(*cache, table, i32([0, old + n]), i32([old + n]), old + n, **more))
        out += fa.forward_paged_q4(qo, *cache, table, new, i32([old + n]), n, old + n, **more)
        out += fa.forward_paged_q4(qo[:5].contiguous(), *cache, table, i32([0, 5]), i32([old + n]), 5, old + n, causal=False, **more)
        out += fa.decode_paged_q4(qo[-1:, :, None], *cache, table, i32([old + n]), old + n, **more)
        got.append(out)
        del cache
    fa.fa_sync_status()
    for a, b in ((got[0], got[1]), (got[2], got[3])):
        for x, y in zip(a, b):
            assert x.isfinite().all() and torch.equal(x, y)


@pytest.mark.parametrize("what", ["page", "minus", "short", "beyond", "position", "order", "end"])
@pytest.mark.parametrize("q4", [False, True])
def test_append_reports_bad_places(what, q4):
    """Out of range pages, positions, lengths and boundaries are reported, and only the tokens they
    concern are left out."""
    require_gpu()
    H_kv, d, block = 2, 64, 16
    new, lens, table = [4, 4], [20, 4], np.array([[1, 2], [3, 0]], np.int32)
    cu, n_pos = [0, 4, 8], 64
    if what == "page":
        table[0, 1] = 4
    elif what == "minus":
        table[0, 1] = -1
    elif what == "short":
        lens[0] = 3
    elif what == "beyond":
        lens[0] = 33 + 4
    elif what == "position":
        n_pos = 18
    elif what == "order":
        cu = [0, 9, 8]
    else:
        cu = [0, 4, 9]
    k = cuda(normal((8, H_kv, d), 1))
    cos, sin = fa.rotary_tables(n_pos, d, device="cuda")
    idx = i32(table), i32(cu), i32(lens)
    rot = dict(q=k, cos=cos, sin=sin, q_out=torch.full_like(k, -7.25))
    if q4:
        cache = [torch.full((4, H_kv, block, n), 0xA5, dtype=torch.uint8, device="cuda") for n in (32, 4, 32, 4)]
        q = fa.append_paged_q4(k, k, *cache, *idx, **rot)
        touched = (cache[0] != 0xA5).any(-1).any(1)
    else:
        cache = [torch.full((4, block, H_kv, d), -7.25, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        q = fa.append_paged(k, k, *cache, *idx, **rot)
        touched = (cache[0] != -7.25).any(-1).any(-1)
    with pytest.raises(fa.FaError) as e:
        fa.fa_sync_status()
    assert e.value.status == 1
    fa.fa_sync_status()
    if what in ("page", "minus", "short", "beyond"):          # the second sequence went through
        assert touched[3, :4].all() and not touched[:3].any()
        assert (q[:4] == -7.25).all() and (q[4:] != -7.25).any()


@pytest.mark.parametrize("what", ["page", "long", "negative", "boundary", "many"])
@pytest.mark.parametrize("tokens", [3, 70])
def test_attention_reports_bad_contents(what, tokens):
    require_gpu()
    lens, H, d = [100, 200], 4, 64
    cache, table, _ = fill_cache(lens, 2, d, 64, 5)
    cu, new, max_q = [0, tokens, tokens + 2], tokens + 2, tokens
    if what == "page":
        table[1, 2] = cache[0].shape[0]
    elif what == "long":
        lens = [100, 201]
    elif what == "negative":
        lens = [-1, 200]
    elif what == "boundary":
        cu = [0, tokens, tokens + 3]
    else:
        max_q = tokens - 1
    q = cuda(normal((new, H, d), 1))
    calls = [lambda: fa.forward_paged_q4(q, *cache, i32(table), i32(cu), i32(lens), max_q, 200)]
    if what in ("page", "long", "negative"):
        calls.append(lambda: fa.decode_paged_q4(q[:2, :, None].contiguous(), *cache, i32(table), i32(lens), 200))
    for call in calls:
        call()
        with pytest.raises(fa.FaError) as e:
            fa.fa_sync_status()
        assert e.value.status == 1
        fa.fa_sync_status()


def test_gather_reports_bad_places():
    require_gpu()
    cache, table, _ = fill_cache([40], 2, 64, 16, 5)
    table[0, 1] = 100
    k, v = (torch.full((40, 2, 64), -7.25, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_gather_paged_q4(*cache, k, v, i32([0, 40]), i32([40]), i32(table), DK, DV)
    with pytest.raises(fa.FaError):
        fa.fa_sync_status()
    assert (k[16:32] == -7.25).all() and not (k[:16] == -7.25).all() and not (v[32:] == -7.25).all()


def test_package_refuses_wrong_tensors():
    """Types, shapes and layouts that the pointers alone would not show."""
    require_gpu()
    cache, table, _ = fill_cache([40], 2, 64, 16, 5)
    t, n = i32(table), i32([40])
    q = cuda(normal((1, 4, 1, 64), 1))
    for bad in (lambda: fa.decode_paged_q4(q.half(), *cache, t, n, 40), lambda: fa.decode_paged_q4(q, *cache, t.long(), n, 40),
                lambda: fa.decode_paged_q4(q, *cache, t, i32([40, 40]), 40), lambda: fa.decode_paged_q4(q.repeat(1, 1, 2, 1), *cache, t, n, 40),
                lambda: fa.decode_paged_q4(q, cache[0], cache[1][:, :1], *cache[2:], t, n, 40),
                lambda: fa.decode_paged_q4(q[:, :3], *cache, t, n, 40),
                lambda: fa.decode_paged_q4(q, *cache, t, n, 40, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                lambda: fa.gather_paged_q4(*cache, t, i32([0, 40]).float(), n, 40),
                lambda: fa.append_paged_q4(q[0].transpose(0, 2), q[0], *cache, t, i32([0, 1]), n),
                lambda: fa.append_paged_q4(q[:, :2, 0], q[:, :2, 0], *cache, t, i32([0, 1]), n, cos=torch.ones(3, 32, device="cuda"))):
        with pytest.raises(fa.FaError) as e:
            bad()
        assert e.value.status == 1
    fa.fa_sync_status()
