"""The 4-bit attention at the ends of its ranges, on the GPU, against the plain oracle."""
import numpy as np
import pytest
import torch

import exact_io_aware_08_gb300 as fa
from oracle import paged as P
from tests.gpu_common import cuda, require_gpu
from tests.test_paged_q4_gpu import check_attention, f64, i32

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
