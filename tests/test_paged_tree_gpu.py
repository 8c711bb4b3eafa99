"""Drafted trees, attention weights and eviction over the bf16 paged cache on the GPU, against the plain oracle
(oracle/paged.py) within bounds that follow from the roundings.

Pages are scattered over a pool in a seeded order, unused table entries are -1, and every cache row that no
sequence holds is NaN, so that a stray read shows; outputs start as NaN or as a sentinel, so that a row which is
not written, or one that should not be, does."""
import numpy as np
import pytest
import torch

import exact_io_aware_08_gb300 as fa
from oracle import paged as P
from tests.gpu_common import cuda, poisoned, require_gpu
from tests.test_paged_q4_gpu import f64, i32, make_pages, normal

pytestmark = pytest.mark.gpu
NAN = float("nan")


def random_tree(r, n):
    return [-1 if i == 0 or r.random() < 0.15 else int(r.integers(max(0, i - 9), i)) for i in range(n)]


class Step:
    """A step of packed queries over a cache of random keys and values."""

    def __init__(self, new, lens, H, H_kv, d, block, kind, pad=0, scale=None, outliers=False, seed=0):
        self.new, self.lens, self.H, self.H_kv, self.d, self.block = new, lens, H, H_kv, d, block
        r = np.random.default_rng(seed + sum(lens) + H)
        self.cu = np.concatenate(([0], np.cumsum(new)))
        self.total, self.max_q, self.max_k = sum(new) + pad, max(new), max(lens)
        self.scale = d ** -0.5 if scale is None else scale
        self.nb, self.table = make_pages(lens, block, 2, seed + 1)
        shape = (self.nb, block, H_kv, d)
        self.k, self.v = (normal(shape, seed + i, outliers) for i in (2, 3))
        held = torch.zeros(shape[:2], dtype=torch.bool)
        for b, n in enumerate(lens):
            p = np.arange(n)
            held[self.table[b][p // block], p % block] = True
        self.k[~held] = NAN
        self.v[~held] = NAN
        self.q = normal((self.total, H, d), seed + 4, outliers)
        if kind is None:
            self.seen = [np.tril(np.ones((n, n), bool)) for n in new]
        elif kind == "tree":
            self.seen = [P.tree_mask(random_tree(r, n)) for n in new]
        else:                                        # any bits, some rows without one
            self.seen = [(r.random((n, n)) < 0.4) & (r.random((n, 1)) < 0.8) for n in new]
        self.tree = None
        if kind is not None:
            words = -(-self.max_q // 32) + (1 if kind == "bits" else 0)
            bits = [P.pack_bits(s, words) for s in self.seen] + [np.full((pad, words), -1, np.int32)]
            self.tree = np.concatenate(bits)
            if kind == "bits":                       # bits behind the step's tokens are not looked at
                for b, n in enumerate(new):
                    wide = np.zeros((n, 32 * words), bool)
                    wide[:, n:] = r.random((n, 32 * words - n)) < 0.5
                    self.tree[self.cu[b]:self.cu[b + 1]] |= P.pack_bits(wide, words)

    def gpu(self):
        return [cuda(self.q), cuda(self.k), cuda(self.v), i32(self.table), i32(self.cu), i32(self.lens)]

    def attend(self, **kw):
        q, k, v, table, cu, lens = self.gpu()
        tree = None if self.tree is None else i32(self.tree)
        ws = torch.full((fa.fa_fwd_paged_tree_workspace_size(self.H, self.H_kv, self.max_q, self.d) // 4,), NAN, device="cuda")
        o, lse = poisoned((self.total, self.H, self.d), torch.bfloat16), poisoned((self.H, self.total), torch.float32)
        fa.fa_fwd_paged_tree(q, k, v, o, lse, tree, cu, lens, table, self.max_q, self.max_k, self.scale, ws, **kw)
        fa.fa_sync_status()
        return o, lse

    def keys(self, b, h):
        p = np.arange(self.lens[b])
        page, row = self.table[b][p // self.block], p % self.block
        return f64(self.k[page, row, h]), f64(self.v[page, row, h])

    def rows(self, b, h, tokens):
        """(k, v, query rows, seen) of some tokens and all query heads of key head h."""
        n, m, G = self.new[b], self.lens[b], self.H // self.H_kv
        k, v = self.keys(b, h)
        q = f64(self.q[self.cu[b]:self.cu[b + 1]][tokens][:, h * G:(h + 1) * G]).reshape(-1, self.d)
        seen = np.ones((n, m), bool)
        seen[:, m - n:] = self.seen[b]
        return k, v, q, np.repeat(seen[tokens], G, 0)

    def check(self, o, lse, sequences=None, most=24):
        G = self.H // self.H_kv
        og, lg = f64(o), f64(lse)
        if sequences is None:
            sequences = sorted({*range(min(12, len(self.new))), *range(0, len(self.new), 5), len(self.new) - 1})
        for b in sequences:
            n = self.new[b]
            if n == 0:
                continue
            tokens = sorted({0, n - 1, *np.linspace(0, n - 1, most).astype(int)})
            for h in sorted({0, self.H_kv - 1, self.H_kv // 2}):
                k, v, q, seen = self.rows(b, h, tokens)
                want, l, bo, bl = P.attend_seen(q, k, v, self.scale, seen)
                at = self.cu[b] + np.array(tokens)
                got = og[at][:, h * G:(h + 1) * G].reshape(-1, self.d)
                gl = lg[h * G:(h + 1) * G][:, at].T.reshape(-1)
                assert (np.abs(got - want) <= bo).all(), (b, h, np.abs(got - want).max(), (np.abs(got - want) / bo).max())
                none = l == -np.inf
                assert (gl[none] == -np.inf).all() and (got[none] == 0).all()
                assert (np.abs(gl[~none] - l[~none]) <= bl[~none]).all()
        assert np.isnan(og[self.cu[-1]:]).all() and np.isnan(lg[:, self.cu[-1]:]).all()
        assert not np.isnan(og[:self.cu[-1]]).any() and not np.isnan(lg[:, :self.cu[-1]]).any()


# (new tokens, tokens with these, H, H_kv, d, block, kind, padding rows)
STEPS = [
    ([1], [1], 1, 1, 64, 16, None, 0),
    ([1], [1], 1, 1, 128, 16, "bits", 0),
    ([1, 1, 1], [129, 1, 128], 8, 2, 128, 64, None, 2),
    ([8], [1008], 32, 8, 128, 64, "tree", 0),
    ([3, 0, 5, 1], [3, 40, 100, 257], 6, 2, 64, 48, "bits", 3),
    ([1, 1], [5000, 3], 16, 1, 128, 128, None, 0),
    ([7, 26, 1, 33], [700, 26, 4000, 129], 5, 1, 128, 16, "tree", 1),
    ([128], [128], 1, 1, 128, 32, "bits", 0),
    ([127, 128, 1], [255, 256, 2049], 2, 2, 64, 256, "tree", 0),
    ([129, 2], [129, 3000], 1, 1, 128, 64, "tree", 0),                     # two row tiles, shares
    ([60, 50, 0, 64], [1000, 50, 7, 1500], 8, 2, 128, 64, "tree", 5),
    ([40, 33], [140, 3333], 8, 1, 64, 16, "bits", 0),                      # row blocks, split keys
    ([300, 1, 77], [300, 900, 1077], 4, 4, 128, 64, None, 0),
    ([300], [4300], 7, 1, 128, 48, None, 2),
    ([513, 200], [513, 2000], 2, 1, 64, 128, "tree", 0),
    ([3], [2000], 160, 1, 64, 64, "tree", 0),                              # more query heads than a tile has rows
    ([1] * 70, list(range(1, 1401, 20)), 8, 4, 128, 32, None, 0),
    ([4] * 40, [4] * 40, 4, 2, 64, 16, "bits", 0),
    ([0, 0, 1], [9, 0, 1], 3, 3, 64, 16, None, 4),
    ([8] * 64, [1000] * 64, 32, 8, 128, 64, "tree", 0),
    # one and two tiles of rows by turns, several sequences a CTA
    ([60, 1, 1, 33, 2, 40, 1, 64, 31, 32] * 7, [20 * i + 70 for i in range(70)], 16, 4, 128, 64, "tree", 0),
    ([1, 1, 250, 3, 129, 1, 128] * 9, [17 * i + 260 for i in range(63)], 8, 8, 64, 16, None, 0),
]
STEP_IDS = [f"{len(c[0])}seqs_{sum(c[0])}tok_H{c[2]}x{c[3]}_d{c[4]}_b{c[5]}_{c[6]}" for c in STEPS]


@pytest.mark.parametrize("case", STEPS, ids=STEP_IDS)
def test_tree_attention(case):
    require_gpu()
    new, lens, H, H_kv, d, block, kind, pad = case
    s = Step(new, lens, H, H_kv, d, block, kind, pad)
    o, lse = s.attend()
    s.check(o, lse)
    again = s.attend()
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), again[1].view(torch.int32))


@pytest.mark.parametrize("case", [STEPS[3], STEPS[10], STEPS[11]], ids=lambda c: f"{sum(c[0])}tok")
@pytest.mark.parametrize("scale", [1e-30, 1.0, 40.0])
def test_tree_attention_of_large_scores(case, scale):
    """Outliers: running maxima jump, one key has nearly all of a row, references are far from 0."""
    require_gpu()
    s = Step(*case, scale=scale, outliers=True)
    s.check(*s.attend())


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("case", [STEPS[3], STEPS[7], STEPS[10], STEPS[12], STEPS[13]], ids=lambda c: f"{sum(c[0])}tok")
def test_what_is_not_seen_does_not_count(case, where, value):
    """Drafted tokens whose keys or values are no finite numbers reach the rows that see them, and no others."""
    require_gpu()
    s = Step(*case)
    n, m = s.new[0], s.lens[0]
    j = n // 2
    page, row = s.table[0][(m - n + j) // s.block], (m - n + j) % s.block
    getattr(s, where)[page, row, :, 3] = value
    o, lse = (f64(x) for x in s.attend())
    sees = s.seen[0][:, j]
    assert sees.any() and not sees.all()
    if where == "v":
        got = o[:n][sees][..., 3]
        assert (np.isnan(got) if np.isnan(value) else got == value).all()
        assert np.isfinite(np.delete(o[:n][sees], 3, -1)).all() and not np.isnan(lse[:, :n]).any()
    elif np.isnan(value):
        assert np.isnan(o[:n][sees]).all() and np.isnan(lse[:, :n][:, sees]).all()
    tokens = [int(t) for t in np.flatnonzero(~sees)][:40]
    G = s.H // s.H_kv
    for h in range(s.H_kv):
        k, v, q, seen = s.rows(0, h, tokens)
        k, v = np.where(np.isfinite(k), k, 0), np.where(np.isfinite(v), v, 0)
        want, l, bo, bl = P.attend_seen(q, k, v, s.scale, seen)
        got, gl = o[tokens][:, h * G:(h + 1) * G].reshape(-1, s.d), lse[h * G:(h + 1) * G][:, tokens].T.reshape(-1)
        none = l == -np.inf
        assert (np.abs(got - want) <= bo).all() and (gl[none] == -np.inf).all() and (np.abs(gl[~none] - l[~none]) <= bl[~none]).all()


@pytest.mark.parametrize("case", [
    ([7, 9, 1], [700, 9, 257], 5, 1, 128, 16, "tree", 0),                  # 35, 45 and 5 rows: warps that rows fill in part
    ([9, 30], [1009, 4000], 4, 1, 64, 64, "bits", 2),
    ([21, 33, 5], [300, 2033, 5], 8, 1, 128, 64, "tree", 0),               # 168, 264 (shares) and 40 rows
    ([77, 130, 3], [177, 1130, 259], 7, 1, 128, 48, None, 1),              # row blocks
], ids=lambda c: f"{sum(c[0])}tok_{c[6]}")
def test_values_that_are_no_numbers_beside_lanes_without_a_row(case):
    """Warps in which some lanes have no row, some see a value that is no finite number and some do not, in every
    block of columns: each row has what it sees, and every other result stays bit for bit."""
    require_gpu()
    s = Step(*case)
    clean = [x.clone() for x in s.attend()]
    G, d = s.H // s.H_kv, s.d
    planted = []
    for b, n in enumerate(s.new):
        for i, c in enumerate(range(1, d, 15)):
            j, value = (i * 5) % n, (NAN, float("inf"), -float("inf"))[i % 3]
            p = s.lens[b] - n + j
            s.v[s.table[b][p // s.block], p % s.block, :, c] = value
            planted.append((b, j, c, value))
    j = s.new[1] // 2                                                      # and two that meet in one column
    for k, value in ((0, float("inf")), (j, -float("inf"))):
        p = s.lens[1] - s.new[1] + k
        s.v[s.table[1][p // s.block], p % s.block, :, d - 2] = value
        planted.append((1, k, d - 2, value))
    want = f64(clean[0])
    for b, n in enumerate(s.new):
        for c in {x[2] for x in planted}:
            sums = np.zeros(n)
            with np.errstate(invalid="ignore"):
                for _, j, _, value in (x for x in planted if x[0] == b and x[2] == c):
                    sums += np.where(s.seen[b][:, j], value, 0.0)
            hit = ~np.isfinite(sums)
            want[s.cu[b]:s.cu[b + 1], :, c][hit] = sums[hit, None]
    for _ in range(2):
        o, lse = s.attend()
        np.testing.assert_array_equal(f64(o), want)
        assert torch.equal(lse.view(torch.int32), clean[1].view(torch.int32))


def test_values_that_are_no_numbers_in_many_sequences():
    """Every second sequence has one, with one and two tiles of rows by turns and several sequences a CTA."""
    require_gpu()
    s = Step([60, 1, 3, 33, 2, 40, 64] * 10, [9 * i + 70 for i in range(70)], 16, 4, 128, 64, "tree")
    clean = f64(s.attend()[0])
    for b in range(0, 70, 2):
        p = s.lens[b] - s.new[b]
        s.v[s.table[b][p // 64], p % 64, :, 100] = NAN          # the first drafted token's
    o = f64(s.attend()[0])
    for b in range(70):
        sees = s.seen[b][:, 0] & (b % 2 == 0)
        at = slice(s.cu[b], s.cu[b + 1])
        assert np.isnan(o[at][sees][..., 100]).all()
        np.testing.assert_array_equal(o[at][~sees], clean[at][~sees])
        np.testing.assert_array_equal(np.delete(o[at][sees], 100, -1), np.delete(clean[at][sees], 100, -1))


@pytest.mark.parametrize("case,more", [(STEPS[2], 40), (STEPS[7], 300), (STEPS[12], 500), (STEPS[16], 1000)], ids=lambda x: str(x)[:8])
def test_loose_maxima_and_guards(case, more):
    """Maxima above the lengths (other tile counts, empty row blocks), and bytes around the outputs and the workspaces."""
    require_gpu()
    new, lens, H, H_kv, d, block, kind, _ = case
    s = Step(new, lens, H, H_kv, d, block, kind, more)
    s.max_q, s.max_k = min(s.total, s.max_q + more), min(s.max_k + more, s.table.shape[1] * block)
    if s.tree is not None:
        s.tree = np.pad(s.tree, ((0, 0), (0, -(-s.max_q // 32) - s.tree.shape[1])))
    o, lse = s.attend()
    s.check(o, lse)
    q, k, v, table, cu, ln = s.gpu()
    size = fa.fa_fwd_paged_tree_workspace_size(H, H_kv, s.max_q, d)
    room, pad = [size, o.numel() * 2, lse.numel() * 4], 256
    held = [torch.full((pad + -(-n // 16) * 16 + pad,), 0xA5, dtype=torch.uint8, device="cuda") for n in room]
    ws, og, lg = (x[pad:pad + n] for x, n in zip(held, room))
    fa.fa_fwd_paged_tree(q, k, v, og.view(torch.bfloat16).view(o.shape), lg.view(torch.float32).view(lse.shape), None if s.tree is None else i32(s.tree),
                         cu, ln, table, s.max_q, s.max_k, s.scale, ws)
    size = fa.fa_weigh_paged_workspace_size(H, H_kv, s.max_q)
    held.append(torch.full((pad + size + pad,), 0xA5, dtype=torch.uint8, device="cuda"))
    room.append(size)
    rows = lse.clone()
    rows[:, s.cu[-1]:] = 0
    w = torch.zeros((s.nb, H_kv, block), device="cuda")
    fa.fa_weigh_paged(q, rows, k, w, None, cu, ln, table, s.max_q, s.max_k, s.scale, 1.0, held[3][pad:pad + size])
    fa.fa_sync_status()
    n = s.cu[-1]
    assert torch.equal(og.view(torch.int16).view(o.shape)[:n], o.view(torch.int16)[:n])
    assert torch.equal(lg.view(torch.int32).view(lse.shape)[:, :n], lse.view(torch.int32)[:, :n])
    for x, y in zip(held, room):
        assert (x[:pad] == 0xA5).all() and (x[pad + y:] == 0xA5).all()
    assert (og.view(o.shape[0], -1)[n:] == 0xA5).all()
    if kind is None:                                              # (a row's weights sum to 1: each is off by some 2^-18 of itself at most)
        assert abs(f64(w).sum() - n * H) <= n * H * 1e-4


def test_long_caches_and_many_shares():
    require_gpu()
    s = Step([1, 3, 2], [70001, 5, 40000], 8, 2, 128, 64, "tree")
    s.check(*s.attend())
    s = Step([90], [30000], 4, 1, 64, 256, "tree")
    s.check(*s.attend(), most=6)
    s = Step([100, 7, 300], [30000, 9, 2300], 8, 2, 128, 64, None)          # whole row blocks and a rest
    s.check(*s.attend(), most=6)
    s = Step([700, 1, 50, 650], [700, 5, 3000, 9000], 16, 4, 64, 64, None)
    s.check(*s.attend(), most=6)
    s = Step([600] * 10, [600 + 10 * i for i in range(10)], 8, 8, 128, 64, "tree")
    s.check(*s.attend(), most=6)


def test_pages_past_32_bits():
    """The last pages of caches of more than 2^32 bytes (and elements' bytes past 2^31 rows of them)."""
    require_gpu()
    H_kv, d, block = 8, 128, 64
    nb = (5 << 30) // (block * H_kv * d * 2)
    k, v = (torch.zeros((nb, block, H_kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = Step([9], [200], 16, 8, d, block, "tree")
    need = 4
    table = np.array([[nb - 1, nb - 7, nb - 3, nb - 2]], np.int32)
    for i in range(need):
        k[int(table[0, i])], v[int(table[0, i])] = cuda(s.k[s.table[0, i]]), cuda(s.v[s.table[0, i]])
    q, cu, lens, tree = cuda(s.q), i32(s.cu), i32(s.lens), i32(s.tree)
    o, lse = fa.forward_paged_tree(q, k, v, i32(table), cu, lens, 9, 200, tree=tree)
    s.check(o, lse)
    w = torch.full((nb, H_kv, block), NAN, device="cuda")
    chain = fa.forward_paged_tree(q, k, v, i32(table), cu, lens, 9, 200)[1]
    fa.weigh_paged(q, chain, k, w, i32(table), cu, lens, 9, 200, weighed=i32([0]))
    kept, left = fa.evict_paged(k, v, w, i32(table), i32([[nb - 10, nb - 12]]), lens, i32([100]), 200, 100, keep_last=10)
    fa.fa_sync_status()
    got = kept[0].cpu().numpy()
    wc = f64(w)
    for h in range(H_kv):
        at = [wc[table[0, p // block], h, p % block] for p in range(200)]
        assert list(got[h]) == P.evict(np.array(at), 100, 0, 10)
        for i in (0, 63, 64, 99):
            p = int(got[h, i])
            assert torch.equal(k[(nb - 10, nb - 12)[i // block], i % block, h], k[int(table[0, p // block]), p % block, h])
    path = i32([[1, 4, 8]])
    before = [k[int(table[0, p // block]), p % block].clone() for p in (192, 195, 199)]
    assert fa.accept_paged(k, v, i32(table), cu, lens, path, i32([3])).tolist() == [194]
    for i, x in enumerate(before):
        assert torch.equal(k[int(table[0, (191 + i) // block]), (191 + i) % block], x)


@pytest.mark.parametrize("what", ["boundaries", "too many tokens", "length", "short length", "page"])
def test_bad_sequences_are_reported_and_left(what):
    """A sequence that is not sound is reported and its rows stay; the others are computed."""
    require_gpu()
    s = Step([4, 4, 4], [300, 200, 150], 8, 2, 128, 64, "tree")
    good = [0, 2]
    q, k, v, table, cu, lens = s.gpu()
    max_q, max_k = 4, 300
    if what == "boundaries":
        cu = i32([0, 4, 13, 12])
        good = [0]
    elif what == "too many tokens":
        s = Step([2, 6, 2], [300, 200, 150], 8, 2, 128, 64, "tree")
        q, k, v, table, cu, lens = s.gpu()
        max_q = 5
    elif what == "length":
        lens = i32([300, 301, 150])
    elif what == "short length":
        lens = i32([300, 3, 150])
    else:
        table[1, 1] = s.nb
    tree = i32(s.tree)
    ws = torch.empty(fa.fa_fwd_paged_tree_workspace_size(8, 2, max_q, 128), dtype=torch.uint8, device="cuda")
    o, lse = poisoned(q.shape, torch.bfloat16), poisoned((8, s.total), torch.float32)
    fa.fa_fwd_paged_tree(q, k, v, o, lse, tree, cu, lens, table, max_q, max_k, s.scale, ws)
    with pytest.raises(fa.FaError, match="invalid sequence boundaries"):
        fa.fa_sync_status()
    og, lg = f64(o), f64(lse)
    keep = np.concatenate([np.arange(s.cu[b], s.cu[b + 1]) for b in good])
    for b in good:
        for h in range(2):
            kk, vv, qq, seen = s.rows(b, h, list(range(s.new[b])))
            want, l, bo, bl = P.attend_seen(qq, kk, vv, s.scale, seen)
            got = og[s.cu[b]:s.cu[b + 1], 4 * h:4 * h + 4].reshape(-1, 128)
            assert (np.abs(got - want) <= bo).all()
    if what != "page":
        rest = np.setdiff1d(np.arange(s.total), keep)
        assert np.isnan(og[rest]).all() and np.isnan(lg[:, rest]).all()
    # and the weights of a chain
    w = torch.full((s.nb, 2, 64), 7.0, device="cuda")
    fa.weigh_paged(q, torch.zeros((8, s.total), device="cuda"), k, w, table, cu, lens, max_q, max_k)
    with pytest.raises(fa.FaError, match="invalid sequence boundaries"):
        fa.fa_sync_status()
    if what != "page":
        for b in sorted({0, 1, 2} - set(good)):
            pages = s.table[b][s.table[b] >= 0]
            assert (f64(w)[pages] == 7).all()


@pytest.mark.parametrize("what", ["tree", "weigh"])
def test_a_step_over_caches_of_no_tokens(what):
    """max_seqlen_k of 0: nothing is written where all sequences are empty, and one that is not is reported."""
    require_gpu()
    q, c = cuda(normal((3, 8, 64), 1)), torch.full((2, 16, 2, 64), NAN, dtype=torch.bfloat16, device="cuda")
    o, lse = poisoned((3, 8, 64), torch.bfloat16), poisoned((8, 3), torch.float32)
    w = torch.full((2, 2, 16), 7.0, device="cuda")
    ws = torch.empty(max(fa.fa_fwd_paged_tree_workspace_size(8, 2, 3, 64), fa.fa_weigh_paged_workspace_size(8, 2, 3)), dtype=torch.uint8, device="cuda")

    def call(cu, lens, max_k, max_q=2):
        if what == "tree":
            fa.fa_fwd_paged_tree(q, c, c, o, lse, None, i32(cu), i32(lens), i32([[0], [1]]), max_q, max_k, 0.125, ws)
        else:
            fa.fa_weigh_paged(q, lse, c, w, None, i32(cu), i32(lens), i32([[0], [1]]), max_q, max_k, 0.125, 1.0, ws)
        fa.fa_sync_status()

    call([0, 0, 0], [0, 0], 0)                                   # padding rows alone
    for cu, lens in (([0, 2, 2], [2, 0]), ([0, 0, 0], [0, 1]), ([0, 1, 1], [0, 0])):
        with pytest.raises(fa.FaError, match="invalid sequence boundaries"):
            call(cu, lens, 0)
    call([0, 0, 0], [0, 0], 0, 3)
    assert torch.isnan(o).all() and torch.isnan(lse).all() and (w == 7).all()


# --------------------------------------------------------------------------------------------
# weights
# --------------------------------------------------------------------------------------------

# (new tokens, tokens with these, H, H_kv, d, block, weighed, decay)
WEIGHS = [
    ([1], [1], 1, 1, 64, 16, None, 1.0),
    ([1, 1, 1], [700, 1, 257], 8, 2, 128, 64, None, 0.98),
    ([3, 0, 5], [300, 40, 5], 6, 2, 64, 48, [10, 0, 0], 0.5),
    ([1], [4000], 160 // 2, 1, 128, 128, None, 1.0),
    ([128], [128], 1, 1, 128, 16, None, 1.0),
    ([9, 12], [2000, 12], 12, 4, 64, 32, [0, 5], 0.0),
    ([129], [400], 1, 1, 64, 64, None, 0.9),                              # more than one tile of rows
    ([300, 1, 40], [300, 900, 1040], 4, 2, 128, 64, None, 1.0),
    ([64, 64], [1000, 700], 20, 4, 128, 256, [0, 0], 1.0),
    ([700], [700], 5, 1, 128, 16, None, 1.0),
    ([1] * 70, list(range(1, 1401, 20)), 8, 8, 64, 32, None, 0.7),
    ([520, 2, 511], [1040, 5, 511], 3, 3, 128, 32, None, 0.25),
    ([1000, 3, 0, 600], [1000, 9, 50, 4000], 8, 2, 128, 64, [0, 9, 5, 100], 0.5),      # ranges of rows
    ([1100], [1300], 2, 2, 64, 64, None, 1.0),
    ([700, 650], [1400, 650], 100, 1, 64, 16, None, 1.0),                             # a token a tile
    ([96, 1, 33, 0, 64, 32] * 12, [31 * i + 96 for i in range(72)], 16, 4, 128, 64, None, 0.98),   # up to three tiles of rows
    ([90, 7], [9000, 4000], 8, 2, 64, 32, [0, 1000], 0.5),
    ([97, 1], [3000, 1], 8, 2, 128, 64, None, 1.0),                                   # one more
]


@pytest.mark.parametrize("case", WEIGHS, ids=[f"{len(c[0])}seqs_{sum(c[0])}tok_H{c[2]}x{c[3]}_d{c[4]}_b{c[5]}" for c in WEIGHS])
def test_weights(case):
    require_gpu()
    new, lens, H, H_kv, d, block, weighed, decay = case
    s = Step(new, lens, H, H_kv, d, block, None)
    G = H // H_kv
    q, k, v, table, cu, ln = s.gpu()
    at0 = [m - n for n, m in zip(new, lens)] if weighed is None else weighed
    w0 = torch.rand((s.nb, H_kv, block), generator=torch.Generator().manual_seed(1))
    held = np.zeros((s.nb, block), bool)
    for b, m in enumerate(lens):
        if new[b] == 0:
            continue
        p = np.arange(m)
        held[s.table[b][p // block], p % block] = True
        p = p[at0[b]:]
        w0[s.table[b][p // block], :, p % block] = NAN                    # what others left there
    lse = np.zeros((H, s.total), np.float32)
    for b, n in enumerate(new):
        for h in range(H_kv if n else 0):
            kk, vv, qq, seen = s.rows(b, h, list(range(n)))
            lse[h * G:(h + 1) * G, s.cu[b]:s.cu[b + 1]] = P.attend_seen(qq, kk, vv, s.scale, seen)[1].reshape(n, G).T
    w = cuda(w0)
    args = (q, torch.tensor(lse, device="cuda"), k, w, table, cu, ln, s.max_q, s.max_k)
    fa.weigh_paged(*args, weighed=None if weighed is None else i32(weighed), decay=decay)
    fa.fa_sync_status()
    got = f64(w)
    for b, (n, m) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        p = np.arange(m)
        for h in range(H_kv):
            kk, _, qq, _ = s.rows(b, h, list(range(n)))
            rows = lse[h * G:(h + 1) * G, s.cu[b]:s.cu[b + 1]].T.reshape(-1).astype(np.float64)
            drawn, bound = P.weigh(qq, rows, kk, s.scale, np.repeat(np.arange(m - n, m), G))
            had = np.where(p < at0[b], np.float64(np.float32(decay)) * f64(w0)[s.table[b][p // block], h, p % block], 0)
            want = had + drawn
            x = got[s.table[b][p // block], h, p % block]
            assert (np.abs(x - want) <= bound + 2.0 ** -23 * (np.abs(want) + had)).all(), (b, h, (np.abs(x - want) / (bound + 2.0 ** -23 * want)).max())
    rest = torch.from_numpy(~held)
    assert torch.equal(w.cpu().transpose(1, 2)[rest].view(torch.int32), w0.transpose(1, 2)[rest].view(torch.int32))
    w2 = cuda(w0)
    fa.weigh_paged(*args[:3], w2, *args[4:], weighed=None if weighed is None else i32(weighed), decay=decay)
    assert torch.equal(w.view(torch.int32), w2.view(torch.int32))


def test_rows_that_see_nothing_weigh_nothing():
    require_gpu()
    s = Step([4], [200], 4, 2, 128, 64, None)
    q, k, v, table, cu, lens = s.gpu()
    lse = torch.full((4, 4), -float("inf"), device="cuda")
    w = torch.full((s.nb, 2, 64), 0.5, device="cuda")
    fa.weigh_paged(q, lse, k, w, table, cu, lens, 4, 200)
    fa.fa_sync_status()
    p = np.arange(200)
    got = f64(w)[s.table[0][p // 64], :, p % 64]
    assert (got[:196] == 0.5).all() and (got[196:] == 0).all()


def test_weights_of_many_rows_over_caches_of_no_tokens():
    require_gpu()
    q, c = cuda(normal((300, 4, 128), 1)), torch.zeros((2, 16, 1, 128), dtype=torch.bfloat16, device="cuda")
    lse, w = torch.zeros((4, 300), device="cuda"), torch.full((2, 1, 16), 7.0, device="cuda")
    fa.weigh_paged(q, lse, c, w, i32([[0], [1]]), i32([0, 0, 0]), i32([0, 0]), 300, 0)
    fa.fa_sync_status()
    fa.weigh_paged(q, lse, c, w, i32([[0], [1]]), i32([0, 300, 300]), i32([300, 0]), 300, 0)
    with pytest.raises(fa.FaError, match="invalid sequence boundaries"):
        fa.fa_sync_status()
    assert (w == 7).all()


@pytest.mark.parametrize("case", [
    ([1, 3], [300, 257], 8, 2, 128, 64), ([40, 90], [40, 1090], 4, 1, 64, 16), ([9, 31], [700, 231], 12, 4, 128, 48),     # few rows
    ([300, 1, 520], [300, 900, 1520], 4, 2, 128, 64), ([700], [700], 5, 1, 64, 32), ([530], [531], 2, 2, 128, 16),         # many
], ids=lambda c: f"{sum(c[0])}tok_H{c[2]}x{c[3]}")
@pytest.mark.parametrize("what", ["queries", "keys"])
def test_rows_that_see_nothing_weigh_nothing_whatever_they_hold(case, what):
    """An lse of -inf takes a row out, also where its queries, or keys that it would meet, are no finite numbers; the
    other rows' weights are those of a step with finite numbers there, bit for bit."""
    require_gpu()
    s = Step(*case, None)
    r = np.random.default_rng(s.total)
    q, k, v, table, cu, lens = s.gpu()
    lse = torch.tensor(r.normal(size=(s.H, s.total)) + 3, dtype=torch.float32, device="cuda")
    out = torch.tensor(r.random((s.total, s.H)) < (0.3 if s.total > 20 else 0.5), device="cuda")
    out[0, 0], out[-1, -1] = True, True
    if what == "keys":                                           # of the last token: its own row alone would see it
        out[s.cu[1:] - 1] = True
    lse[out.T] = -float("inf")

    def weights(q, k):
        w = torch.full((s.nb, s.H_kv, s.block), 0.5, device="cuda")
        fa.weigh_paged(q, lse, k, w, table, cu, lens, s.max_q, s.max_k)
        fa.fa_sync_status()
        return w

    want = weights(q, k)
    assert torch.isfinite(want).all()
    for value in (NAN, float("inf"), -float("inf")):
        q2, k2 = q.clone(), k.clone()
        if what == "queries":
            q2[out] = value
        else:
            for b, m in enumerate(s.lens):
                k2[int(s.table[b][(m - 1) // s.block]), (m - 1) % s.block] = value
        got = weights(q2, k2)
        assert torch.equal(got.view(torch.int32), want.view(torch.int32))


# --------------------------------------------------------------------------------------------
# eviction, accepted paths
# --------------------------------------------------------------------------------------------

def pool(nb, block, H_kv, d, seed):
    k, v = (torch.randint(-32768, 32767, (nb, block, H_kv, d), dtype=torch.int16, generator=torch.Generator().manual_seed(seed + i)) for i in (0, 1))
    return k, v


# (lengths, budgets, keep_first, keep_last, H_kv, d, block, weights)
EVICTS = [
    ([1], [1], 0, 0, 1, 64, 16, "normal"),
    ([1], [0], 0, 0, 1, 64, 16, "normal"),
    ([100, 0, 33, 64], [40, 5, 50, 64], 4, 10, 2, 128, 16, "normal"),
    ([1000, 1001], [1000, 1000], 0, 0, 3, 64, 48, "ties"),
    ([5000], [4000], 0, 4000, 2, 128, 64, "normal"),
    ([5000], [4000], 4000, 0, 2, 64, 64, "normal"),
    ([3000, 3000], [2000, 7], 3, 4, 2, 64, 256, "ties"),
    ([3000], [1500], 4, 64, 4, 64, 100, "strange"),
    ([2048, 17], [1, 16], 0, 1, 8, 128, 32, "zeros"),
    ([60000, 200], [30000, 110], 4, 100, 1, 64, 128, "ties"),             # more than fit on chip
    ([50000], [10], 0, 0, 1, 64, 16, "close"),
]


@pytest.mark.parametrize("case", EVICTS, ids=[f"{'_'.join(map(str, c[0]))}to{'_'.join(map(str, c[1]))}_{c[7]}" for c in EVICTS])
def test_evict(case):
    require_gpu()
    lens, budgets, first, last, H_kv, d, block, kind = case
    left = [min(x) for x in zip(lens, budgets)]
    r = np.random.default_rng(sum(lens))
    nb, both = make_pages(lens + left, block, 3, 7)
    B = len(lens)
    table, new = both[:B], both[B:, :max(1, -(-max(left) // block))]
    k, v = pool(nb, block, H_kv, d, 3)
    w = {"normal": lambda n: r.normal(size=n), "ties": lambda n: r.integers(0, 9, n) / 4, "zeros": lambda n: np.zeros(n),
         "strange": lambda n: r.choice([0.0, -0.0, 1.0, -1.0, NAN, np.inf, -np.inf, 1e-45, -1e-45], n),
         "close": lambda n: 1 + r.integers(0, 3, n) * 2.0 ** -23}[kind]((nb, H_kv, block)).astype(np.float32)
    kg, vg, wg = cuda(k), cuda(v), torch.tensor(w, device="cuda")
    max_kept = max(left)
    kept, out = fa.evict_paged(kg.view(torch.bfloat16), vg.view(torch.bfloat16), wg, i32(table), i32(new), i32(lens), i32(budgets), max(lens),
                               max_kept, keep_first=first, keep_last=last)
    fa.fa_sync_status()
    assert out.tolist() == left
    kept, kw, vw, ww = kept.cpu().numpy(), k.numpy().copy(), v.numpy().copy(), w.copy()
    for b, n in enumerate(lens):
        p = np.arange(n)
        for h in range(H_kv):
            want = np.array(P.evict(w[table[b][p // block], h, p % block], budgets[b], first, last), int)
            np.testing.assert_array_equal(kept[b, h], np.concatenate((want, np.full(max_kept - len(want), -1))))
            i = np.arange(len(want))
            to, at = (new[b][i // block], i % block), (table[b][want // block], want % block)
            kw[to[0], to[1], h], vw[to[0], to[1], h] = k.numpy()[at[0], at[1], h], v.numpy()[at[0], at[1], h]
            ww[to[0], h, to[1]] = w[at[0], h, at[1]]
    np.testing.assert_array_equal(kg.cpu().numpy(), kw)
    np.testing.assert_array_equal(vg.cpu().numpy(), vw)
    np.testing.assert_array_equal(wg.cpu().numpy().view(np.int32), ww.view(np.int32))


def test_bad_evictions_are_reported_and_left():
    require_gpu()
    lens, budgets = [100, 101, 60, -1, 50, 100], [40, 40, 10, 5, -1, 71]
    nb, both = make_pages([100, 101, 60, 1, 50, 100] + [70] * 6, 16, 2, 1)
    table, new = both[:6], both[6:, :5]
    k, v = pool(nb, 16, 2, 64, 1)
    kg, vg, wg = cuda(k), cuda(v), torch.rand((nb, 2, 16), device="cuda")
    kept, out = fa.evict_paged(kg.view(torch.bfloat16), vg.view(torch.bfloat16), wg, i32(table), i32(new), i32(lens), i32(budgets), 100, 70,
                               keep_first=20, keep_last=5)
    with pytest.raises(fa.FaError, match="invalid"):
        fa.fa_sync_status()
    assert out.tolist() == [40, 101, 60, -1, 50, 100]
    assert (kept[1:] == -1).all() and (kept[0, :, :40] >= 0).all()
    rest = np.ones(nb, bool)
    rest[new[0]] = False
    np.testing.assert_array_equal(kg.cpu().numpy()[rest], k.numpy()[rest])
    table[0, 0], new[0, 1] = nb, -5                   # a block to read from and one to write to that are not there
    fa.evict_paged(kg.view(torch.bfloat16), vg.view(torch.bfloat16), wg, i32(table[:1]), i32(new[:1]), i32([100]), i32([40]), 100, 70)
    with pytest.raises(fa.FaError, match="invalid"):
        fa.fa_sync_status()
    fa.fa_sync_status()


def test_weights_that_are_no_numbers_rank_with_the_lowest():
    """NaN counts as -inf: of equal ones the front stays, in either order, on chip and beyond it."""
    require_gpu()
    r = np.random.default_rng(8)
    for n, budget in ((200, 70), (200, 199), (60000, 20000)):
        nb, both = make_pages([n, budget], 64, 0, n)
        table, new = both[:1], both[1:, :-(-budget // 64)]
        w = r.choice([NAN, -np.inf, 1.0], (nb, 1, 64), p=[0.4, 0.4, 0.2]).astype(np.float32)
        c = torch.zeros((nb, 64, 1, 64), dtype=torch.bfloat16, device="cuda")
        kept, _ = fa.evict_paged(c, c.clone(), torch.tensor(w, device="cuda"), i32(table), i32(new), i32([n]), i32([budget]), n, budget, keep_last=3)
        fa.fa_sync_status()
        p = np.arange(n)
        np.testing.assert_array_equal(kept[0, 0].cpu().numpy(), P.evict(w[table[0][p // 64], 0, p % 64], budget, 0, 3))


def test_evictions_without_a_block_leave_out_its_tokens():
    """Tokens of a block that is not there rank behind all others and are not copied, nor is what would go to one; what is
    sound is moved, and nothing else changes."""
    require_gpu()
    lens, budgets, block, H_kv = [150, 40, 130], [60, 40, 100], 16, 2
    r = np.random.default_rng(4)
    nb, both = make_pages(lens + budgets, block, 3, 5)
    table, new = both[:3].copy(), both[3:, :7].copy()
    k, v = pool(nb, block, H_kv, 64, 6)
    w = r.normal(size=(nb, H_kv, block)).astype(np.float32)
    w[table[0][5]] = -np.inf                             # the lowest of those that have a block
    gone = {0: [2, 9], 1: [1], 2: [0, 1, 2, 3]}          # more than sequence 2 drops: some of them are kept in name
    for b, blocks in gone.items():
        table[b, blocks] = [nb, -1, nb + 7, -9][:len(blocks)]
    new[0, 1], new[2, 6] = -5, nb
    kg, vg, wg = cuda(k), cuda(v), torch.tensor(w, device="cuda")
    kept, out = fa.evict_paged(kg.view(torch.bfloat16), vg.view(torch.bfloat16), wg, i32(table), i32(new), i32(lens), i32(budgets), 150, 100,
                               keep_first=3, keep_last=4)
    with pytest.raises(fa.FaError, match="invalid"):
        fa.fa_sync_status()
    assert out.tolist() == budgets
    kept, kw, vw, ww = kept.cpu().numpy(), k.numpy().copy(), v.numpy().copy(), w.copy()
    for b, n in enumerate(lens):
        p = np.arange(n)
        there = (table[b][p // block] >= 0) & (table[b][p // block] < nb)
        for h in range(H_kv):
            # ranks in place of weights: 0 for tokens without a block, then the weights' order
            own = np.where(there, w[np.where(there, table[b][p // block], 0), h, p % block], 0)
            levels = np.unique(own[there])
            want = np.array(P.evict(np.where(there, 1.0 + np.searchsorted(levels, own), 0.0), budgets[b], 3, 4), int)
            np.testing.assert_array_equal(kept[b, h], np.concatenate((want, np.full(100 - len(want), -1))))
            for i, j in enumerate(want):
                to = new[b][i // block]
                if there[j] and 0 <= to < nb:
                    kw[to, i % block, h], vw[to, i % block, h] = k.numpy()[table[b][j // block], j % block, h], v.numpy()[table[b][j // block], j % block, h]
                    ww[to, h, i % block] = w[table[b][j // block], h, j % block]
    assert (kept[2, :, :100] // block == 1).any()     # (tokens without a block that are kept in name)
    np.testing.assert_array_equal(kg.cpu().numpy(), kw)
    np.testing.assert_array_equal(vg.cpu().numpy(), vw)
    np.testing.assert_array_equal(wg.cpu().numpy().view(np.int32), ww.view(np.int32))


def test_accept():
    require_gpu()
    new = [26, 1, 0, 7, 100, 5]
    lens = [126, 1, 30, 7, 4000, 200]
    paths = [[0, 3, 4, 11, 25], [0], [], [], list(range(1, 100, 5)), [0, 1, 2, 3, 4]]
    for H_kv, d, block in ((8, 128, 64), (1, 64, 16), (3, 64, 7), (32, 128, 48)):
        nb, table = make_pages(lens, block, 2, 5)
        k, v = pool(nb, block, H_kv, d, 2)
        kg, vg = cuda(k), cuda(v)
        deep = max(map(len, paths))
        acc = i32([p + [-7] * (deep - len(p)) for p in paths])
        out = fa.accept_paged(kg.view(torch.bfloat16), vg.view(torch.bfloat16), i32(table), i32(np.concatenate(([0], np.cumsum(new)))), i32(lens), acc,
                              i32([len(p) for p in paths]))
        fa.fa_sync_status()
        assert out.tolist() == [m - n + len(p) for m, n, p in zip(lens, new, paths)]
        kw, vw = k.numpy().copy(), v.numpy().copy()
        for b, p in enumerate(paths):
            for i, j in enumerate(p):
                x, y = lens[b] - new[b] + j, lens[b] - new[b] + i
                kw[table[b][y // block], y % block] = k.numpy()[table[b][x // block], x % block]
                vw[table[b][y // block], y % block] = v.numpy()[table[b][x // block], x % block]
        np.testing.assert_array_equal(kg.cpu().numpy(), kw)
        np.testing.assert_array_equal(vg.cpu().numpy(), vw)


def test_bad_paths_are_reported_and_left():
    require_gpu()
    new, lens = [5] * 8, [50] * 8
    paths, counts = [[0, 2], [2, 1], [1, 1], [0, 5], [-1, 0], [0, 1], [0, 1], [3, 4]], [2, 2, 2, 2, 2, 3, -1, 2]
    nb, table = make_pages(lens, 16, 2, 5)
    table[7, 3] = nb                                  # the step's tokens lie there
    k, v = pool(nb, 16, 2, 64, 9)
    kg, vg = cuda(k), cuda(v)
    out = fa.accept_paged(kg.view(torch.bfloat16), vg.view(torch.bfloat16), i32(table), i32(np.arange(0, 45, 5)), i32(lens), i32(paths), i32(counts))
    with pytest.raises(fa.FaError, match="invalid"):
        fa.fa_sync_status()
    assert out.tolist() == [47] + [50] * 7
    kw = k.numpy().copy()
    kw[table[0][46 // 16], 46 % 16] = k.numpy()[table[0][47 // 16], 47 % 16]
    np.testing.assert_array_equal(kg.cpu().numpy(), kw)


# --------------------------------------------------------------------------------------------
# positions that are not places
# --------------------------------------------------------------------------------------------

@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sizes", [([5, 0, 26], [105, 3, 26], 6, 3, 128, 32, 64), ([1500, 700, 3], [1500, 800, 30], 32, 8, 64, 64, 64)],
                         ids=["few", "many"])
def test_append_at_positions(q4, inter, sizes):
    """Appending at given positions is appending a sequence whose places are those, moved."""
    require_gpu()
    new, lens, H, H_kv, d, block, rotary = sizes
    total, cu = sum(new) + 2, np.concatenate(([0], np.cumsum(new)))
    q, k, v = (cuda(normal((total, h, d), h)) for h in (H, H_kv, H_kv))
    r = np.random.default_rng(3)
    at = r.integers(0, 5000, total)
    at[:3] = 0, 4999, 17
    cos, sin = fa.rotary_tables(5000, rotary, device="cuda")
    nb, table = make_pages(lens, block, 2, 5)

    def run(x, positions, tables):
        if q4:
            c = [torch.zeros((nb, H_kv, block, n), dtype=torch.uint8, device="cuda") for n in (d // 2, d // 16, d // 2, d // 16)]
            out = fa.append_paged_q4(x[1], x[2], *c, i32(table), i32(cu), i32(lens), q=x[0], cos=tables[0], sin=tables[1],
                                     descale_k=0.002, descale_v=0.002, interleaved=inter, positions=positions, q_out=torch.zeros_like(q))
        else:
            c = [torch.zeros((nb, block, H_kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            out = fa.append_paged(x[1], x[2], *c, i32(table), i32(cu), i32(lens), q=x[0], cos=tables[0], sin=tables[1], interleaved=inter,
                                  positions=positions, q_out=torch.zeros_like(q))
        fa.fa_sync_status()
        return [out, *c]

    got = run((q, k, v), i32(at), (cos, sin))
    # the same rotation from tables whose row p holds the angle of the token at place p: one sequence at a time
    for b, (n, m) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        rows = torch.zeros(m, dtype=torch.long, device="cuda")
        rows[m - n:] = torch.tensor(at[cu[b]:cu[b + 1]], device="cuda")
        only = np.concatenate(([0] * (b + 1), [n] * (len(new) - b)))
        x = tuple(t[cu[b]:cu[b + 1]].contiguous() for t in (q, k, v))
        if q4:
            c = [torch.zeros_like(t) for t in got[1:]]
            out = fa.append_paged_q4(x[1], x[2], *c, i32(table), i32(only), i32(lens), q=x[0], cos=cos[rows].contiguous(), sin=sin[rows].contiguous(),
                                     descale_k=0.002, descale_v=0.002, interleaved=inter)
        else:
            c = [torch.zeros_like(t) for t in got[1:]]
            out = fa.append_paged(x[1], x[2], *c, i32(table), i32(only), i32(lens), q=x[0], cos=cos[rows].contiguous(), sin=sin[rows].contiguous(),
                                  interleaved=inter)
        fa.fa_sync_status()
        assert torch.equal(out.view(torch.int16), got[0][cu[b]:cu[b + 1]].view(torch.int16))
        p = torch.arange(m - n, m)
        page, row = torch.tensor(table[b], dtype=torch.long)[p // block].cuda(), (p % block).cuda()
        for y, z in zip(c, got[1:]):
            if q4:
                assert torch.equal(y[page, :, row], z[page, :, row])
            else:
                assert torch.equal(y[page, row].view(torch.int16), z[page, row].view(torch.int16))
    assert (got[0][cu[-1]:] == 0).all()
    for bad in (5000, -1):
        at[1] = bad
        with pytest.raises(fa.FaError, match="invalid"):
            run((q, k, v), i32(at), (cos, sin))


# --------------------------------------------------------------------------------------------
# streams, graphs, and all of it together
# --------------------------------------------------------------------------------------------

def test_a_stream_of_its_own_and_two_at_once():
    require_gpu()
    a, b = Step([8, 3], [1008, 3000], 32, 8, 128, 64, "tree"), Step([70], [4000], 8, 2, 128, 64, "tree", seed=9)
    want = [a.attend(), b.attend()]
    args = [(x.gpu(), i32(x.tree), x) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (g, tree, x) in enumerate(args):
            q, k, v, table, cu, lens = g
            got[i].append(fa.forward_paged_tree(q, k, v, table, cu, lens, x.max_q, x.max_k, tree=tree, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o.view(torch.int16), want[i][0].view(torch.int16)) and torch.equal(lse, want[i][1])


def test_captured_steps_with_new_contents():
    """A step captured once and replayed with other lengths, trees, paths and budgets in the same tensors."""
    require_gpu()
    s = Step([6, 6], [500, 300], 8, 2, 128, 64, "tree")
    q, k, v, table, cu, lens = s.gpu()
    tree = i32(s.tree)
    path, count, budgets = i32([[0, 1, 2, 3]] * 2), i32([1, 1]), i32([100, 100])
    spare, fresh = make_pages([256, 256], 64, 0, 3)
    k, v = (torch.cat((x, torch.zeros((spare, 64, 2, 128), dtype=torch.bfloat16, device="cuda"))) for x in (k, v))
    fresh = i32(fresh + s.nb)
    w = torch.zeros((s.nb + spare, 2, 64), device="cuda")
    k0, v0, w0 = k.clone(), v.clone(), w.clone()

    def step():
        o, lse = fa.forward_paged_tree(q, k, v, table, cu, lens, 6, 512, tree=tree)
        o1, lse1 = fa.forward_paged_tree(q, k, v, table, cu, lens, 6, 512)
        fa.weigh_paged(q, lse1, k, w, table, cu, lens, 6, 512, weighed=zero)
        kept, left = fa.evict_paged(k, v, w, table, fresh, lens, budgets, 512, 200, keep_last=8)
        out = fa.accept_paged(k, v, table, cu, lens, path, count)
        return [o, lse, o1, lse1, kept, left, out, k, v, w]

    zero = i32([0, 0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    r = np.random.default_rng(2)
    for new_lens, p, c, bud in (([500, 300], [[0, 2, 3, 5], [1, 2, 4, 5]], [4, 2], [100, 150]), ([130, 6], [[1, 3, 4, 5]] * 2, [3, 0], [200, 9])):
        lens.copy_(i32(new_lens))
        path.copy_(i32(p))
        count.copy_(i32(c))
        budgets.copy_(i32(bud))
        tree.copy_(i32(np.concatenate([P.pack_bits(P.tree_mask(random_tree(r, 6)), 1) for _ in range(2)])))
        results = []
        for go in (graph.replay, step):
            for x, y in ((k, k0), (v, v0), (w, w0)):
                x.copy_(y)
            out = go()
            torch.cuda.synchronize()
            fa.fa_sync_status()
            results.append([x.clone() for x in (held if out is None else out)])
        for x, y in zip(*results):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


def test_masks_and_depths_on_the_device():
    """The masks that the host's make, with padding rows of any contents, and a step captured and replayed with other trees."""
    require_gpu()
    r = np.random.default_rng(3)
    sizes, pad = [26, 0, 33, 5], 6
    cu = np.concatenate(([0], np.cumsum(sizes)))
    parents, graph = i32(np.zeros(cu[-1] + pad)), torch.cuda.CUDAGraph()
    cug = i32(cu)
    fa.tree_bits(parents, cug, 33)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = fa.tree_bits(parents, cug, 33)
    for _ in range(3):
        new = np.concatenate([random_tree(r, n) for n in sizes] + [r.integers(-(1 << 31), 1 << 31, pad)])
        parents.copy_(i32(new))
        graph.replay()
        want = fa.tree_bits(torch.tensor(new, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32), 33)
        for x, y, z in zip(want, held, fa.tree_bits(parents, cug, 33)):
            assert torch.equal(x, y.cpu()) and torch.equal(x, z.cpu())


def test_serving_with_drafts_and_a_short_cache():
    """A prompt, its weights, its eviction, a drafted tree at its true positions, the accepted path, and its weights:
    every call's result against the oracle on what the cache holds."""
    require_gpu()
    H, H_kv, d, block, G = 8, 2, 128, 64, 4
    n, budget = 400, 150
    prompt, drafts = normal((n, H + 2 * H_kv, d), 1), normal((9, H + 2 * H_kv, d), 2)
    cos, sin = fa.rotary_tables(n + 20, d, device="cuda")
    nb = 20
    k, v = (torch.full((nb, block, H_kv, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.full((nb, H_kv, block), NAN, device="cuda")
    table, new = i32([[3, 17, 5, 0, 19, 8, 2]]), i32([[11, 6, 14]])

    def split(x):
        x = cuda(x)
        return x[:, :H], x[:, H:H + H_kv], x[:, H + H_kv:]

    def held(t, at, h):
        t, at = t.cpu().numpy()[0], np.asarray(at)
        return f64(k)[t[at // block], at % block, h], f64(v)[t[at // block], at % block, h]

    q, kk, vv = split(prompt)
    cu, lens = i32([0, n]), i32([n])
    q = fa.append_paged(kk, vv, k, v, table, cu, lens, q=q, cos=cos, sin=sin)
    o, lse = fa.forward_paged_tree(q, k, v, table, cu, lens, n, n)
    fa.weigh_paged(q, lse, k, w, table, cu, lens, n, n)
    kept, left = fa.evict_paged(k, v, w, table, new, lens, i32([budget]), n, budget, keep_first=4, keep_last=32)
    assert left.tolist() == [budget]
    # a drafted tree behind what is kept, at the positions behind the whole prompt
    parents = [-1, 0, 0, 1, 1, 2, 3, 3, 6]
    tree, depth = fa.tree_bits(i32(parents), i32([0, 9]), 9)
    q2, k2, v2 = split(drafts)
    cu2, lens2 = i32([0, 9]), left + 9
    q2 = fa.append_paged(k2, v2, k, v, new, cu2, lens2, q=q2, cos=cos, sin=sin, positions=n + depth)
    o2, lse2 = fa.forward_paged_tree(q2, k, v, new, cu2, lens2, 9, budget + 9, tree=tree)
    drafted = [held(new, range(budget + 9), h) for h in range(H_kv)]
    path = [0, 1, 3, 6]
    lens3 = fa.accept_paged(k, v, new, cu2, lens2, i32([path]), i32([4]))
    assert lens3.tolist() == [budget + 4]
    pick = torch.tensor(path, device="cuda")
    fa.weigh_paged(q2[pick], lse2[:, pick].contiguous(), k, w, new, i32([0, 4]), lens3, 4, budget + 4, decay=0.9)
    o4, lse4 = fa.forward_paged_tree(q2[pick], k, v, new, i32([0, 4]), lens3, 4, budget + 4)
    fa.fa_sync_status()
    # the accepted tokens' results are the tree's, now as a chain
    assert np.abs(f64(o4) - f64(o2)[path]).max() <= 2e-2 and np.abs(f64(lse4) - f64(lse2)[:, path]).max() <= 1e-4
    wg, kept = f64(w), kept.cpu().numpy()
    seen = np.ones((9, budget + 9), bool)
    seen[:, budget:] = P.tree_mask(parents)
    for h in range(H_kv):
        # weights of the prompt
        K, V = held(table, range(n), h)
        rows = f64(q)[:, h * G:(h + 1) * G].reshape(-1, d)
        want, l, bo, bl = P.attend_seen(rows, K, V, d ** -0.5, np.repeat(np.tril(np.ones((n, n), bool)), G, 0))
        assert (np.abs(f64(o)[:, h * G:(h + 1) * G].reshape(-1, d) - want) <= bo).all()
        t = np.arange(n)
        old = wg[table.cpu().numpy()[0][t // block], h, t % block]
        drawn, bound = P.weigh(rows, f64(lse)[h * G:(h + 1) * G].T.reshape(-1), K, d ** -0.5, np.repeat(t, G))
        assert (np.abs(old - drawn) <= bound).all() and abs(drawn.sum() - n * G) < 1e-2
        np.testing.assert_array_equal(kept[0, h], P.evict(old, budget, 4, 32))
        # drafts over what was kept
        K2, V2 = drafted[h]
        np.testing.assert_array_equal(K2[:budget], K[kept[0, h]])
        rows = f64(q2)[:, h * G:(h + 1) * G].reshape(-1, d)
        want, l, bo, bl = P.attend_seen(rows, K2, V2, d ** -0.5, np.repeat(seen, G, 0))
        assert (np.abs(f64(o2)[:, h * G:(h + 1) * G].reshape(-1, d) - want) <= bo).all()
        c, s = f64(cos), f64(sin)
        for i, p in enumerate(parents):               # true positions: depth behind the prompt
            pos = n + int(depth[i])
            turned = P.rotate(f64(drafts[i, H:H + H_kv]), c[pos], s[pos], False)[h]
            assert (np.abs(K2[budget + i] - turned) <= 2.0 ** -8 * np.abs(turned) + 2.0 ** -21 * 5).all()
        # accepted: in place, and their weights
        K3, _ = held(new, range(budget + 4), h)
        np.testing.assert_array_equal(K3, K2[list(range(budget)) + [budget + j for j in path]])
        rows = f64(q2)[path][:, h * G:(h + 1) * G].reshape(-1, d)
        drawn, bound = P.weigh(rows, f64(lse2)[h * G:(h + 1) * G][:, path].T.reshape(-1), K3, d ** -0.5, np.repeat(np.arange(budget, budget + 4), G))
        t = np.arange(budget + 4)
        had = np.concatenate((np.float64(np.float32(0.9)) * old[kept[0, h]], np.zeros(4)))
        got = wg[new.cpu().numpy()[0][t // block], h, t % block]
        assert (np.abs(got - had - drawn) <= bound + 2.0 ** -23 * (had + drawn + had)).all()
