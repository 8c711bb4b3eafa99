"""Refusals of the calls around the bf16 paged cache (drafted trees, weights, eviction), and their tables: without a GPU."""
import numpy as np
import pytest
import torch

import exact_io_aware_08_gb300 as fa
from exact_io_aware_08_gb300 import build as fabuild
from oracle import paged as P

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def call(fn, order, defaults, kw):
    assert set(kw) <= set(defaults)
    a = dict(defaults, **kw)
    return fn(*[a[x] for x in order.split()], None)


STEP = dict(q=FAKE, kc=FAKE, vc=FAKE, o=FAKE, lse=FAKE, tree=FAKE, words=1, cu=FAKE, lens=FAKE, table=FAKE, n_seqs=2, H=8, H_kv=2,
            total=6, max_q=4, max_blocks=8, block=64, num_blocks=16, max_k=500, d=128, scale=0.1, ws=FAKE, ws_bytes=1 << 40,
            weights=FAKE, weighed=None, decay=1.0)
TREE = ("q kc vc o lse tree words cu lens table n_seqs H H_kv total max_q max_blocks block num_blocks max_k d scale ws ws_bytes")
WEIGH = "q lse kc weights weighed cu lens table n_seqs H H_kv total max_q max_blocks block num_blocks max_k d scale decay ws ws_bytes"


@pytest.mark.parametrize("what", ["tree", "weigh"])
@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INVALID), (dict(H=0), INVALID), (dict(H=7), INVALID), (dict(H_kv=0), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(block=8), UNSUPPORTED), (dict(block=40), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(max_k=513), INVALID), (dict(max_k=-1), INVALID), (dict(max_q=-1), INVALID), (dict(max_q=7), INVALID), (dict(total=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(scale=1e-36), INVALID), (dict(scale=1e36), INVALID), (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(kc=None), INVALID),
    (dict(kc=FAKE + 8), INVALID), (dict(q=FAKE + 2), INVALID), (dict(lens=FAKE + 2), INVALID), (dict(cu=None), INVALID),
    (dict(table=None), INVALID), (dict(num_blocks=1 << 26), UNSUPPORTED), (dict(total=1 << 29), UNSUPPORTED),
    (dict(n_seqs=1 << 29, total=1 << 27), UNSUPPORTED),
])
def test_a_step_refuses(lib, what, kw, code):
    fn, order = (lib.fa_fwd_paged_tree, TREE) if what == "tree" else (lib.fa_weigh_paged, WEIGH)
    assert call(fn, order, STEP, kw) == code
    assert lib.fa_last_error_message().decode() not in ("", "no error")


@pytest.mark.parametrize("kw,code", [
    (dict(words=0), INVALID), (dict(total=40, max_q=33), INVALID), (dict(tree=FAKE + 2), INVALID), (dict(o=None), INVALID),
    (dict(vc=None), INVALID), (dict(vc=FAKE + 4), INVALID), (dict(o=FAKE + 8), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=FAKE + 8), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(total=0, max_q=0, q=None, ws=None), OK),
    (dict(max_q=0, o=None), OK), (dict(H=1031, H_kv=1, n_seqs=200000), UNSUPPORTED),
])
def test_tree_refuses_more(lib, kw, code):
    assert call(lib.fa_fwd_paged_tree, TREE, STEP, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(weights=None), INVALID), (dict(weights=FAKE + 4), INVALID), (dict(weighed=FAKE + 1), INVALID), (dict(decay=-0.1), INVALID),
    (dict(total=4000, max_q=2000, ws=None), WORKSPACE), (dict(total=4000, max_q=2000, ws_bytes=1000), WORKSPACE),
    (dict(total=4000, max_q=2000, ws=FAKE + 4), WORKSPACE), (dict(decay=1.5), INVALID), (dict(decay=NAN), INVALID), (dict(H=258), UNSUPPORTED), (dict(total=0, max_q=0, weights=None), OK),
])
def test_weigh_refuses_more(lib, kw, code):
    assert call(lib.fa_weigh_paged, WEIGH, STEP, kw) == code


def test_tree_workspace_size(lib):
    size = lib.fa_fwd_paged_tree_workspace_size
    assert size(8, 2, 1, 128) == size(8, 2, 8, 128) == 2 * 152 * 32 * 131 * 4 + 640
    assert size(8, 2, 100, 64) == size(8, 2, 100000, 64) == 2 * 152 * 256 * 67 * 4 + 640
    assert size(8, 3, 1, 128) == size(8, 2, -1, 128) == size(8, 2, 1, 96) == size(0, 1, 1, 64) == 0


def test_weigh_workspace_size(lib):
    size = lib.fa_weigh_paged_workspace_size
    assert size(8, 2, 1) == size(8, 2, 96) == 16                 # up to three tiles of rows
    assert size(8, 2, 97) == size(32, 8, 4096) == 2 * 152 * 512 * 4
    assert size(8, 3, 1) == size(130, 1, 1) == size(8, 2, -1) == size(0, 1, 1) == 0


ACCEPT = dict(kc=FAKE, vc=FAKE, out=FAKE, path=FAKE, n=FAKE, cu=FAKE, lens=FAKE + 64, table=FAKE, n_seqs=2, H_kv=2, deep=4, max_blocks=8,
              block=64, num_blocks=16, d=64)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INVALID), (dict(n_seqs=65536), UNSUPPORTED), (dict(H_kv=0), INVALID), (dict(deep=-1), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(block=0), UNSUPPORTED), (dict(kc=None), INVALID), (dict(vc=FAKE + 8), INVALID), (dict(path=None), INVALID), (dict(n=None), INVALID),
    (dict(n=FAKE + 2), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 64), INVALID), (dict(cu=None), INVALID),
    (dict(table=FAKE + 1), INVALID), (dict(num_blocks=1 << 26), UNSUPPORTED),
])
def test_accept_refuses(lib, kw, code):
    assert call(lib.fa_accept_paged, "kc vc out path n cu lens table n_seqs H_kv deep max_blocks block num_blocks d", ACCEPT, kw) == code


EVICT = dict(kc=FAKE, vc=FAKE, weights=FAKE, kept=FAKE, out=FAKE, budgets=FAKE + 128, lens=FAKE + 64, table=FAKE, new=FAKE + 256, n_seqs=2, H_kv=2,
             max_k=500, max_kept=100, first=4, last=10, max_blocks=8, new_blocks=2, block=64, num_blocks=16, d=64)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INVALID), (dict(n_seqs=65536), UNSUPPORTED), (dict(max_k=513), INVALID), (dict(max_k=-1), INVALID),
    (dict(max_kept=129), INVALID), (dict(max_kept=-1), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(new_blocks=-1), INVALID), (dict(new_blocks=1 << 26), UNSUPPORTED), (dict(d=100), UNSUPPORTED), (dict(weights=None), INVALID),
    (dict(weights=FAKE + 8), INVALID), (dict(kept=None), INVALID), (dict(new=None), INVALID), (dict(new=FAKE + 2), INVALID),
    (dict(out=None), INVALID), (dict(out=FAKE + 64), INVALID), (dict(out=FAKE + 128), INVALID), (dict(budgets=None), INVALID),
    (dict(kc=FAKE + 2), INVALID), (dict(num_blocks=1 << 26), UNSUPPORTED), (dict(new=FAKE), INVALID),
])
def test_evict_refuses(lib, kw, code):
    order = "kc vc weights kept out budgets lens table new n_seqs H_kv max_k max_kept first last max_blocks new_blocks block num_blocks d"
    assert call(lib.fa_evict_paged, order, EVICT, kw) == code


# Arrays of their own, far apart; every entry of the two tables below makes an output share memory with one that is read.
APART = {x: (i + 1) << 24 for i, x in enumerate("kc vc weights out kept path n cu lens table new budgets".split())}


@pytest.mark.parametrize("kw", [
    dict(out=APART["lens"]), dict(out=APART["n"]), dict(out=APART["cu"]), dict(out=APART["path"]), dict(out=APART["table"]),
    dict(out=APART["lens"] + 4), dict(out=APART["lens"] - 4), dict(out=APART["cu"] + 8), dict(out=APART["path"] + 4 * 2 * 4 - 4),
    dict(out=APART["table"] + 4 * 2 * 8 - 4), dict(n=APART["out"] + 4), dict(cu=APART["out"] - 8),
], ids=str)
def test_accept_refuses_lengths_in_an_array_that_is_read(lib, kw):
    order = "kc vc out path n cu lens table n_seqs H_kv deep max_blocks block num_blocks d"
    assert call(lib.fa_accept_paged, order, dict(ACCEPT, **{x: APART[x] for x in order.split() if x in APART}), kw) == INVALID
    assert b"array of their own" in lib.fa_last_error_message()


@pytest.mark.parametrize("kw", [
    dict(out=APART["lens"]), dict(out=APART["budgets"]), dict(out=APART["table"]), dict(out=APART["new"]), dict(out=APART["kept"]),
    dict(kept=APART["lens"]), dict(kept=APART["budgets"]), dict(kept=APART["table"]), dict(kept=APART["new"]),
    dict(out=APART["budgets"] + 4), dict(out=APART["kept"] + 4 * 2 * 2 * 100 - 4), dict(kept=APART["out"] + 4), dict(new=APART["out"] - 4 * 2 * 2 + 4),
    dict(lens=APART["kept"] + 4 * 2 * 2 * 100 - 8),
], ids=str)
def test_evict_refuses_outputs_in_an_array_that_is_read(lib, kw):
    order = "kc vc weights kept out budgets lens table new n_seqs H_kv max_k max_kept first last max_blocks new_blocks block num_blocks d"
    assert call(lib.fa_evict_paged, order, dict(EVICT, **{x: APART[x] for x in order.split() if x in APART}), kw) == INVALID
    assert b"of their own" in lib.fa_last_error_message() or b"of its own" in lib.fa_last_error_message()


def test_append_at_refuses(lib):
    def append(positions):
        return lib.fa_append_paged_at(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, positions, FAKE, FAKE, FAKE, 2, 8, 2, 4, 1024, 256, 256,
                                      4, 64, 8, 128, 128, 0, 100, None)
    assert append(FAKE + 2) == INVALID


def test_package_refuses_host_tensors_and_shapes(lib):
    z = torch.zeros
    c = z(3, 16, 2, 64, dtype=torch.bfloat16)
    w, q, lse = z(3, 2, 16), z(4, 8, 64, dtype=torch.bfloat16), z(8, 4)
    table, cu, lens = z(2, 2, dtype=torch.int32), z(3, dtype=torch.int32), z(2, dtype=torch.int32)
    for f in (lambda: fa.forward_paged_tree(q, c, c, table, cu, lens, 2, 16), lambda: fa.weigh_paged(q, lse, c, w, table, cu, lens, 2, 16),
              lambda: fa.accept_paged(c, c, table, cu, lens, table, lens), lambda: fa.evict_paged(c, c, w, table, table, lens, lens, 16, 8),
              lambda: fa.append_paged(q[:, :2], q[:, :2], c, c, table, cu, lens, positions=lens)):
        with pytest.raises(fa.FaError, match="CUDA tensor"):
            f()
    with pytest.raises(fa.FaError, match="k_cache must be"):
        fa.forward_paged_tree(q, c[0], c, table, cu, lens, 2, 16)
    with pytest.raises(fa.FaError, match="k_cache must be a tensor"):
        fa.weigh_paged(q, lse, None, w, table, cu, lens, 2, 16)
    with pytest.raises(fa.FaError):
        fa.fa_accept_paged(c, c, None, table, lens, cu, lens, table)
    with pytest.raises(fa.FaError):
        fa.fa_evict_paged(c, c, w, None, lens, lens, lens, table, table, 16, 8, 0, 0)


@pytest.mark.parametrize("sizes", [[1], [5, 0, 33], [64, 1, 2, 100]])
def test_tree_bits(sizes):
    r = np.random.default_rng(sum(sizes))
    trees = [[-1 if i == 0 or r.random() < 0.1 else int(r.integers(0, i)) for i in range(n)] for n in sizes]
    cu = np.concatenate(([0], np.cumsum(sizes)))
    words = -(-max(sizes) // 32)
    bits, depth = fa.tree_bits(torch.tensor(sum(trees, []), dtype=torch.int32), torch.tensor(cu, dtype=torch.int32), max(sizes))
    assert bits.dtype == torch.int32 and depth.dtype == torch.int32
    masks = [P.tree_mask(p) for p in trees]
    np.testing.assert_array_equal(bits.numpy(), np.concatenate([P.pack_bits(m, words) for m in masks]))
    np.testing.assert_array_equal(depth.numpy(), np.concatenate([m.sum(1) - 1 for m in masks if len(m)]))


@pytest.mark.parametrize("kind", ["padding", "outside", "behind", "uninitialised"])
def test_tree_bits_of_parents_that_are_none(kind):
    """Whatever stands in the parents, behind the last sequence's tokens too: what is no token in front of the own one, of
    the same sequence, makes a root, and the others keep their ancestors."""
    r = np.random.default_rng(len(kind))
    sizes, pad = [40, 0, 7, 33], 9
    trees = [[-1 if i == 0 else int(r.integers(0, i)) for i in range(n)] for n in sizes]
    parents = np.array(sum(trees, []) + [-1] * pad, np.int64)
    cu = np.concatenate(([0], np.cumsum(sizes)))
    first = np.repeat(cu[:-1], sizes)
    big = np.iinfo(np.int32)
    if kind in ("padding", "uninitialised"):
        parents[cu[-1]:] = r.choice([0, 1, 89, 1 << 30, big.max, big.min, -2], pad)
    if kind == "outside":
        parents[r.choice(cu[-1], 20, replace=False)] = r.choice([big.max, big.min, -7, 80, 1000, 1 << 24], 20)
    if kind == "behind":
        at = r.choice(cu[-1], 25, replace=False)
        parents[at] = (at - first[at]) + r.integers(0, 30, 25)             # itself, a later one, the next sequence's
    if kind == "uninitialised":
        parents[:] = r.integers(big.min, big.max, len(parents))
        parents[::3] = r.integers(-3, 90, len(parents[::3]))
    bits, depth = fa.tree_bits(torch.tensor(parents, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32), 40)
    sound = [[p if 0 <= p < i else -1 for i, p in enumerate(parents[a:b].tolist())] for a, b in zip(cu[:-1], cu[1:])]
    masks = [P.tree_mask(p) for p in sound]
    np.testing.assert_array_equal(bits.numpy()[:cu[-1]], np.concatenate([P.pack_bits(m, 2) for m in masks]))
    np.testing.assert_array_equal(depth.numpy()[:cu[-1]], np.concatenate([m.sum(1) - 1 for m in masks if len(m)]))
    assert (bits.numpy()[cu[-1]:] == 0).all() and (depth.numpy()[cu[-1]:] == 0).all()


def test_tree_bits_of_more_tokens_than_there_is_room_for():
    """Tokens behind max_seqlen_q have no bits (the attention refuses their sequence); odd boundaries index nothing."""
    parents = torch.tensor([-1, 0, 1, 2] * 12, dtype=torch.int32)
    bits, depth = fa.tree_bits(parents, torch.tensor([0, 48], dtype=torch.int32), 32)
    seen = P.tree_mask([p if p < i else -1 for i, p in enumerate(parents.tolist())])
    np.testing.assert_array_equal(bits.numpy(), P.pack_bits(seen[:, :32], 1))
    for cu in ([0, 0], [7, 48], [0, 1 << 30], [40, 9], [-5, 20], [-(1 << 20), 48], [48]):
        bits, depth = fa.tree_bits(parents, torch.tensor(cu, dtype=torch.int32), 32)
        assert bits.shape == (48, 1) and depth.shape == (48,)
    bits, depth = fa.tree_bits(parents[:0], torch.tensor([0, 0], dtype=torch.int32), 0)
    assert bits.shape == (0, 1) and depth.shape == (0,)


def test_oracle_agrees_with_torch():
    """The oracle's masked attention, weights and eviction against other ways to say them."""
    r = np.random.default_rng(5)
    q, k, v = r.normal(size=(6, 16)), r.normal(size=(20, 16)), r.normal(size=(20, 16))
    seen = r.random((6, 20)) < 0.5
    seen[2] = False
    o, lse, _, _ = P.attend_seen(q, k, v, 0.25, seen)
    s = torch.from_numpy(q @ k.T * 0.25).masked_fill(~torch.from_numpy(seen), -INF)
    want = torch.softmax(s, -1) @ torch.from_numpy(v)
    rows = [0, 1, 3, 4, 5]
    np.testing.assert_allclose(o[rows], want.numpy()[rows], atol=1e-12)
    np.testing.assert_allclose(lse[rows], torch.logsumexp(s, -1).numpy()[rows], atol=1e-12)
    assert (o[2] == 0).all() and lse[2] == -np.inf
    at = [14, 15, 16, 17, 18, 19]
    causal = np.arange(20)[None] <= np.array(at)[:, None]
    lse = P.attend_seen(q, k, v, 0.25, causal)[1]
    w, _ = P.weigh(q, lse, k, 0.25, at)
    assert abs(w.sum() - 6) < 1e-12                          # each row's weights sum to 1
    np.testing.assert_allclose(w, np.where(causal, np.exp(q @ k.T * 0.25 - lse[:, None]), 0).sum(0), atol=1e-12)
    assert P.evict(np.array([5., 1, 1, 3, np.nan, 1, 0, 2]), 5, 1, 1) == [0, 1, 2, 3, 7]
    assert P.evict(np.array([5., 1]), 2, 2, 2) == [0, 1]
    assert P.evict(np.array([-0., 0, -1, np.inf]), 2, 0, 0) == [0, 3]
