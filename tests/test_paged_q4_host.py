"""Refusals of the paged-cache operators, through the C ABI and through the package: all of them
before anything is launched, so they run without a GPU."""
import glob
import math
import os
import subprocess

import pytest
import torch

import exact_io_aware_08_gb300 as fa
from exact_io_aware_08_gb300 import build as fabuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def append(lib, q4=False, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, cos=FAKE, sin=FAKE, cu=FAKE,
             lens=FAKE, table=FAKE, n_seqs=2, H=8, H_kv=2, total=4, sq=1024, sk=256, sv=256, max_blocks=4, block=64,
             num_blocks=8, d=128, rotary=128, inter=0, n_pos=100, dk=1.0, dv=1.0)
    assert set(kw) <= set(a)
    a.update(kw)
    ints = [a[x] for x in ("n_seqs", "H", "H_kv", "total", "sq", "sk", "sv", "max_blocks", "block", "num_blocks", "d",
                           "rotary", "inter", "n_pos")]
    idx = [a[x] for x in ("cos", "sin", "cu", "lens", "table")]
    if q4:
        return lib.fa_append_paged_q4(a["q"], a["k"], a["v"], a["q_out"], a["kc"], a["ks"], a["vc"], a["vs"], *idx, *ints,
                                      a["dk"], a["dv"], None)
    return lib.fa_append_paged(a["q"], a["k"], a["v"], a["q_out"], a["kc"], a["vc"], *idx, *ints, None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INVALID), (dict(H_kv=0), INVALID), (dict(H=-1), INVALID), (dict(H=0), INVALID),
    (dict(total=-1), INVALID), (dict(d=96), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(block=0), UNSUPPORTED), (dict(rotary=48), UNSUPPORTED), (dict(rotary=-32), UNSUPPORTED),
    (dict(rotary=160), UNSUPPORTED), (dict(inter=2), INVALID), (dict(n_pos=0), INVALID),
    (dict(num_blocks=1 << 25), UNSUPPORTED), (dict(max_blocks=1 << 25), UNSUPPORTED),
    (dict(total=1 << 28, n_seqs=1), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID), (dict(kc=None), INVALID),
    (dict(cos=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(table=FAKE + 2), INVALID), (dict(k=FAKE + 8), INVALID), (dict(sin=FAKE + 4), INVALID),
    (dict(sq=1016), INVALID), (dict(sk=260), INVALID), (dict(sv=-256), INVALID), (dict(sk=1 << 41), INVALID),
])
def test_append_refuses(lib, q4, kw, code):
    assert append(lib, q4, **kw) == code
    assert lib.fa_last_error_message().decode() not in ("", "no error")


def test_append_q4_refuses_more(lib):
    assert append(lib, True, block=24) == UNSUPPORTED
    assert append(lib, True, ks=None) == INVALID
    assert append(lib, True, vs=FAKE + 4) == INVALID
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-38, 1e38):
        assert append(lib, True, dk=bad) == INVALID
        assert append(lib, True, dv=bad) == INVALID


@pytest.mark.parametrize("q4", [False, True])
def test_append_of_nothing_is_a_noop(lib, q4):
    assert append(lib, q4, total=0, k=None, v=None, kc=None, cu=None) == OK


def gather(lib, **kw):
    a = dict(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, k=FAKE, v=FAKE, cu=FAKE, lens=FAKE, table=FAKE, n_seqs=2, H_kv=2, total=4,
             max_blocks=4, block=64, num_blocks=8, d=128, dk=1.0, dv=1.0)
    a.update(kw)
    return lib.fa_gather_paged_q4(*[a[x] for x in ("kc", "ks", "vc", "vs", "k", "v", "cu", "lens", "table", "n_seqs", "H_kv",
                                                   "total", "max_blocks", "block", "num_blocks", "d", "dk", "dv")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INVALID), (dict(H_kv=-2), INVALID), (dict(total=-1), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(block=8), UNSUPPORTED), (dict(dk=0.0), INVALID), (dict(dv=float("nan")), INVALID), (dict(k=None), INVALID),
    (dict(vs=None), INVALID), (dict(kc=FAKE + 8), INVALID), (dict(cu=FAKE + 1), INVALID), (dict(total=1 << 29), UNSUPPORTED),
    (dict(total=0, k=None, v=None), OK),
])
def test_gather_refuses(lib, kw, code):
    assert gather(lib, **kw) == code


def attend(lib, fwd, **kw):
    a = dict(q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, o=FAKE, lse=FAKE, cu=FAKE, lens=FAKE, table=FAKE, n_seqs=2, H=8,
             H_kv=2, total=6, max_q=4, max_blocks=8, block=64, num_blocks=16, max_k=500, d=128, scale=0.1, dk=1.0, dv=1.0,
             causal=1, n_splits=4, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    head = [a[x] for x in ("q", "kc", "ks", "vc", "vs", "o", "lse")]
    pages = [a[x] for x in ("max_blocks", "block", "num_blocks", "max_k", "d", "scale", "dk", "dv")]
    tail = [a["n_splits"], a["ws"], a["ws_bytes"], None]
    if fwd:
        return lib.fa_fwd_paged_q4(*head, a["cu"], a["lens"], a["table"], a["n_seqs"], a["H"], a["H_kv"], a["total"],
                                   a["max_q"], *pages, a["causal"], *tail)
    return lib.fa_decode_paged_q4(*head, a["table"], a["lens"], a["n_seqs"], a["H"], a["H_kv"], *pages, *tail)


@pytest.mark.parametrize("fwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INVALID), (dict(H=0), INVALID), (dict(H=7), INVALID), (dict(H_kv=0), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(block=8), UNSUPPORTED), (dict(block=40), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(max_k=513), INVALID),
    (dict(max_k=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(dk=-1.0), INVALID),
    (dict(dv=float("inf")), INVALID), (dict(scale=1e-10, dk=1e-29), INVALID), (dict(n_splits=1025), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(ks=None), INVALID), (dict(o=FAKE + 8), INVALID),
    (dict(lens=FAKE + 2), INVALID), (dict(table=None), INVALID), (dict(num_blocks=1 << 26), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
])
def test_attention_refuses(lib, fwd, kw, code):
    assert attend(lib, fwd, **kw) == code
    assert lib.fa_last_error_message().decode() not in ("", "no error")


def test_forward_refuses_more(lib):
    assert attend(lib, True, cu=None) == INVALID
    assert attend(lib, True, max_q=7) == INVALID
    assert attend(lib, True, total=-1) == INVALID
    assert attend(lib, True, total=0, max_q=0, q=None, ws=None) == OK


def test_workspace_sizes(lib):
    assert lib.fa_decode_paged_q4_workspace_size(4, 8, 2, 1000, 128, 8) >= 4 * 8 * 8 * 130 * 4
    assert lib.fa_decode_paged_q4_workspace_size(4, 8, 3, 1000, 128, 8) == 0
    assert lib.fa_decode_paged_q4_workspace_size(4, 8, 2, 1000, 96, 8) == 0
    assert lib.fa_decode_paged_q4_workspace_size(4, 8, 2, 1000, 128, 1025) == 0
    assert lib.fa_fwd_paged_q4_workspace_size(4, 8, 2, 100, 50, 1000, 64, 2) >= 100 * 8 * 2 * 66 * 4


def tensors():
    z = torch.zeros
    return dict(q=z(4, 8, 64, dtype=torch.bfloat16), k=z(4, 2, 64, dtype=torch.bfloat16), v=z(4, 2, 64, dtype=torch.bfloat16),
                kc=z(3, 2, 16, 32, dtype=torch.uint8), ks=z(3, 2, 16, 4, dtype=torch.uint8),
                table=z(2, 2, dtype=torch.int32), cu=z(3, dtype=torch.int32), lens=z(2, dtype=torch.int32))


def test_package_refuses_host_tensors(lib):
    """No pointer of host memory, or of another device, reaches a kernel."""
    t = tensors()
    with pytest.raises(fa.FaError, match="CUDA tensor"):
        fa.append_paged_q4(t["k"], t["v"], t["kc"], t["ks"], t["kc"], t["ks"], t["table"], t["cu"], t["lens"])
    with pytest.raises(fa.FaError, match="CUDA tensor"):
        fa.append_paged(t["k"], t["v"], t["k"][None], t["k"][None], t["table"], t["cu"], t["lens"])
    with pytest.raises(fa.FaError, match="CUDA tensor"):
        fa.gather_paged_q4(t["kc"], t["ks"], t["kc"], t["ks"], t["table"], t["cu"], t["lens"], 4)
    with pytest.raises(fa.FaError, match="CUDA tensor"):
        fa.decode_paged_q4(t["q"][:2, :, None], t["kc"], t["ks"], t["kc"], t["ks"], t["table"], t["lens"], 16)
    with pytest.raises(fa.FaError, match="CUDA tensor"):
        fa.forward_paged_q4(t["q"], t["kc"], t["ks"], t["kc"], t["ks"], t["table"], t["cu"], t["lens"], 2, 16)
    with pytest.raises(fa.FaError, match="k_codes"):
        fa.decode_paged_q4(t["q"][:2, :, None].repeat(1, 1, 1, 2), t["kc"], t["ks"], t["kc"], t["ks"], t["table"], t["lens"], 16)


def test_rotary_tables_are_exact_far_out():
    cos, sin = fa.rotary_tables(100001, 64)
    for i in (0, 1, 31):
        a = 100000 * 10000.0 ** (-2 * i / 64)
        assert abs(cos[100000, i].item() - math.cos(a)) < 2 ** -24 and abs(sin[100000, i].item() - math.sin(a)) < 2 ** -24


SHARES = """
#include <cstdio>
#include <cstdlib>
#include "q4_share.h"
int main(int argc, char** argv) {
  fa::Q4Share s;
  s.set(atoll(argv[1]), atoi(argv[2]));
  printf("%d", s.n);
  for (int i = 0; i <= s.n; ++i) printf(" %lld", s.begin(i));
  printf("\\n");
  for (int a = 3; a < argc; ++a) printf("%d ", s.owner(atoll(argv[a])));
}
"""


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    at = tmp_path_factory.mktemp("shares")
    (at / "shares.cpp").write_text(SHARES)
    subprocess.run(["g++", "-std=c++17", "-I" + fabuild.CSRC, "-o", str(at / "shares"), str(at / "shares.cpp")], check=True)
    return str(at / "shares")


@pytest.mark.parametrize("total", [1, 5, 607, 608, 609, 10 ** 6 + 7, 2 ** 32 // 608, 2 ** 31 - 1, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1,
                                   2 ** 33 + 12345, 2 ** 36 + 99, 2 ** 38 - 1])
@pytest.mark.parametrize("teams", [1, 3, 456, 608])
def test_shares_cover_every_unit_once(shares, total, teams):
    """Team i has units [T i // N, T (i + 1) // N), whatever T is, and owner() names it."""
    n = max(1, min(teams, total))
    if total // n >= 2 ** 31:
        pytest.skip("more units a team than the calls allow")
    begin = [total * i // n for i in range(n + 1)]
    units = sorted({min(total - 1, max(0, b + k)) for b in begin for k in (-1, 0, 1)} | {total // 3, total // 2})
    out = subprocess.run([shares, str(total), str(teams), *map(str, units)], capture_output=True, text=True, check=True).stdout
    first, second = out.split("\n")[:2]
    assert [int(x) for x in first.split()] == [n, *begin]
    want = [next(i for i in range(n) if begin[i] <= u < begin[i + 1]) for u in units]
    assert [int(x) for x in second.split()] == want


def test_messages_hold_any_shape(lib):
    """The sizes in a refusal's text end where its room does."""
    t = tensors()
    for lead in range(8, 17):
        for digits in (1, 2, 5, 18):
            shape = (0,) + (1000,) * lead + (10 ** digits,) * 3
            wrong = torch.empty(0, dtype=torch.uint8).as_strided(shape, (0,) * len(shape))
            with pytest.raises(fa.FaError, match=r"block_size, d/2\], is \[0, 1000, .*(\.\.\.|0)\]$"):
                fa.decode_paged_q4(t["q"][:2, :, None], wrong, t["ks"], t["kc"], t["ks"], t["table"], t["lens"], 16)


def test_arrivals_in_another_cta_name_their_scope():
    """An arrival without a scope is ordered within its own CTA only, whatever CTA its barrier lies in."""
    found = 0
    for path in glob.glob(os.path.join(fabuild.CSRC, "*")):
        for line in open(path):
            if "mbarrier.arrive" in line and "shared::cluster" in line and "tcgen05" not in line:
                found += 1
                assert ".release.cluster." in line or ".relaxed.cluster." in line, (path, line)
    assert found
