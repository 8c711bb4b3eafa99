"""The 4-bit attention at the ends of its ranges, on the GPU, against the plain oracle."""
import numpy as np
import pytest
import torch

import exact_io_aware_08_gb300 as fa
from oracle import paged as P
from tests.gpu_common import cuda, require_gpu
from tests.test_paged_q4_gpu import DK, DV, check_attention, f64, fill_cache, i32, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_splits", [0, 1, 3])
@pytest.mark.parametrize("n,d", [(1, 128), (1, 64), (4, 128), (4, 64), (20, 64), (20, 128), (80, 128)])
def test_one_key_draws_most_of_the_attention(n, d, n_splits):
    """The first key's score lies 12 to 21 above all others, its value is zero: what a row gives is
    made of weights of 2^-17 to 2^-31, as many as there are keys.  (n tokens of 4 query heads: 8 and 16
    rows a team, tiles, tiles on two SMs.)"""
    require_gpu()
    H, block, keys, descale_v = 4, 256, 33000, 0.002
    rng = np.random.default_rng(n + d)
    k, v = np.zeros((keys, 1, d), np.float32), rng.uniform(0.5, 1.5, (keys, 1, d)).astype(np.float32)
    k[1:, 0, 1] = rng.normal(0, 0.2, keys - 1)
    k[0, 0, 0], v[0] = 12.0, 0.0
    nb = -(-keys // block)
    cache, val = [], []
    for x, descale in ((k, 1.0), (v, descale_v)):
        code, scale = P.quantise_f32(x, descale)
        packed = P.pack(code)
        val.append(P.values(packed, scale, descale)[:, 0])
        for y in (packed, scale):
            pool = np.full((nb * block, y.shape[-1]), 0x7F, np.uint8)
            pool[:keys] = y[:, 0]
            cache.append(cuda(torch.from_numpy(pool.reshape(nb, 1, block, -1))))
    assert val[0][0, 0] == 12.0 and not val[1][0].any()
    # head h's scores: 12, 15, 18 and 21 for the first key, and about 0 for the rest
    q = torch.zeros(n, H, d, dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([1.0, 1.25, 1.5, 1.75])
    q[:, :, 1] = 1.0
    o, lse = fa.forward_paged_q4(cuda(q), *cache, i32(np.arange(nb)[None]), i32([0, n]), i32([keys]), n, keys, causal=False,
                                 n_splits=n_splits, scale=1.0, descale_k=1.0, descale_v=descale_v)
    fa.fa_sync_status()
    want = P.attend(f64(q[0]), *val, 1.0, [keys] * H)
    assert (np.abs(want[0]) > 2.0 ** -17).all()
    for t in range(n):
        check_attention(f64(o[t]), f64(lse[:, t]), want)


@pytest.mark.parametrize("n_splits", [0, 1, 3])
@pytest.mark.parametrize("what", ["front", "many", "end", "order", "sixty"])
@pytest.mark.parametrize("n,d", [(3, 64), (4, 128), (12, 128), (70, 64), (70, 128), (200, 128)])
def test_rows_without_a_sequence_stay_as_they_are(n, d, what, n_splits):
    """Rows in front of the first boundary and rows of a sequence whose boundaries are rejected keep what
    they held, whatever the split count and the workspace's contents; the other sequences get results."""
    require_gpu()
    H, H_kv, lens = 4, 2, [500, 900, 700]
    if what == "sixty":                                # more boundaries than a warp looks at in one step
        lens = [200 + i for i in range(60)]
    B, N = len(lens), max(lens)
    cu, max_q = np.arange(B + 1) * n, n
    total, sound = B * n, set(range(B))
    if what == "front":
        cu = cu + 5
        total += 5
    elif what == "many":
        cu[2:] += 1
        total, sound = total + 1, {0, 2}
    elif what == "end":
        cu[-1] += 1
        max_q, sound = n + 1, {0, 1}
    elif what == "order":
        cu, sound = np.array([0, n, -5, 3 * n]), {0}
        max_q = 3 * n
    else:
        cu[31:] += 1
        total, sound = total + 1, set(range(B)) - {30}
    cache, table, val = fill_cache(lens, H_kv, d, 64, 31)
    q = normal((total, H, d), 32)
    o = torch.full((total, H, d), -7.25, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, total), -7.25, device="cuda")
    ws = torch.full((fa.fa_fwd_paged_q4_workspace_size(B, H, H_kv, total, max_q, N, d, n_splits) // 4,), 3.0, device="cuda")
    fa.fa_fwd_paged_q4(cuda(q), *cache, o, lse, i32(cu), i32(lens), i32(table), max_q, N, d ** -0.5, DK, DV, True, n_splits, ws)
    if what == "front":
        fa.fa_sync_status()
    else:
        with pytest.raises(fa.FaError) as e:
            fa.fa_sync_status()
        assert e.value.status == 1
    left = np.ones(total, bool)
    for b in sorted(sound):
        mine = slice(cu[b], cu[b + 1])
        left[mine] = False
        if b % 7 < 3:
            m = cu[b + 1] - cu[b]
            for h in range(H):
                want = P.attend(f64(q[mine, h]), val["k"][b][:, h // 2], val["v"][b][:, h // 2], d ** -0.5, [lens[b] - m + i + 1 for i in range(m)])
                check_attention(f64(o[mine, h]), f64(lse[h, mine]), want)
    assert left.any() and (f64(o)[left] == -7.25).all() and (f64(lse)[:, left] == -7.25).all()


def test_flags_that_are_neither_true_nor_false():
    """Two truth values as one: refused as an argument, with nothing launched or written."""
    require_gpu()
    cache, table, _ = fill_cache([40], 2, 64, 16, 5)
    q, t, n = cuda(normal((1, 4, 64), 1)), i32(table), i32([40])
    before = [x.clone() for x in cache]
    for two in (torch.tensor([True, False]), np.array([1, 0])):
        with pytest.raises(fa.FaError, match="causal must be true or false") as e:
            fa.forward_paged_q4(q, *cache, t, i32([0, 1]), n, 1, 40, causal=two)
        assert e.value.status == 1
        with pytest.raises(fa.FaError, match="interleaved must be true or false") as e:
            fa.append_paged_q4(q[:, :2], q[:, :2], *cache, t, i32([0, 1]), n, interleaved=two)
        assert e.value.status == 1
    fa.fa_sync_status()
    assert all(torch.equal(x, y) for x, y in zip(cache, before))


def test_streams_by_their_named_handles():
    """0 and 1 are the default stream, 2 the thread's own: as in the other calls, which take any handle."""
    require_gpu()
    cache, table, _ = fill_cache([500, 90], 2, 128, 64, 21)
    q, t, n = cuda(normal((2, 8, 1, 128), 6)), i32(table), i32([500, 90])
    o, lse = fa.decode_paged_q4(q, *cache, t, n, 500, descale_k=DK, descale_v=DV)
    torch.cuda.synchronize()
    for handle in (0, 1, 2):
        o2, lse2 = fa.decode_paged_q4(q, *cache, t, n, 500, descale_k=DK, descale_v=DV, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    fa.fa_sync_status()


@pytest.mark.parametrize("H,H_kv,d,n,seqs", [(8, 4, 64, 1, 300), (32, 4, 128, 1, 270), (8, 4, 128, 3, 257), (4, 4, 128, 2, 256), (6, 3, 64, 4, 130),
                                              (16, 4, 128, 4, 270), (32, 4, 64, 4, 140)])
def test_many_row_blocks(H, H_kv, d, n, seqs):
    """More row blocks than teams, some divided between two or several of them: about as many as the rule
    between the two ways to join them leaves to one, and more.  The same as a call that divides none."""
    require_gpu()
    rng = np.random.default_rng(seqs)
    lens = np.where(rng.random(seqs) < 0.1, 0, rng.integers(0, 900, seqs)).tolist()
    lens[seqs // 2] = 6000
    new = [1 if n == 1 else int(x) for x in rng.integers(0, n + 1, seqs)]
    new[3] = n
    cu, total = np.concatenate(([0], np.cumsum(new))), sum(new) + 2
    cache, table, val = fill_cache(lens, H_kv, d, 64, 8)
    q = normal((total, H, d), 9)
    got = []
    for n_splits in (0, 1):
        o = torch.full((total, H, d), -7.25, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((H, total), -7.25, device="cuda")
        ws = torch.full((fa.fa_fwd_paged_q4_workspace_size(seqs, H, H_kv, total, n, 6000, d, n_splits) // 4,), float("nan"), device="cuda")
        fa.fa_fwd_paged_q4(cuda(q), *cache, o, lse, i32(cu), i32(lens), i32(table), n, 6000, d ** -0.5, DK, DV, True, n_splits, ws)
        fa.fa_sync_status()
        got.append((f64(o), f64(lse)))
    G = H // H_kv
    for b in sorted({seqs // 2, *range(0, seqs, 9)}):
        mine = slice(cu[b], cu[b + 1])
        seen = [lens[b] - new[b] + i + 1 for i in range(new[b])]
        for h in range(H if new[b] else 0):
            want = P.attend(f64(q[mine, h]), val["k"][b][:, h // G], val["v"][b][:, h // G], d ** -0.5, seen)
            for o, lse in got:
                check_attention(o[mine, h], lse[h, mine], want)
    (o, lse), (o1, lse1) = got
    # two results within half a bf16 step and the weights' own 2^-11 each of one another's value
    top = np.abs(val["v"][seqs // 2]).max()
    assert (np.abs(o - o1) <= 2.0 ** -7 * np.abs(o1) + 2.0 ** -9 * top).all()
    assert (np.isneginf(lse) == np.isneginf(lse1)).all() and (o[cu[-1]:] == -7.25).all() and (lse[:, cu[-1]:] == -7.25).all()
