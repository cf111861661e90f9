"""Refusals of the prompt, tree and page entry points and of their binding, workspace
sizes, and the oracles of their tests (fake addresses that are never dereferenced). No GPU."""
import math
import os
import shutil

import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO
from oracle import pages_oracle as PO
from oracle import prompt_oracle as O
from test_cache_host import _Fake, _fake_cache

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def tsel():
    import attention_score_vision_gb300 as t
    t.build()
    t.load_library()
    return t


@pytest.fixture(scope="module")
def lib(tsel):
    return tsel.load_library()


# ------------------------------------------------------------------ oracles

@pytest.mark.parametrize("causal", [False, True])
def test_prompt_oracle_row_by_row(causal):
    rng = np.random.default_rng(0)
    cu_q, cu_k = [0, 3, 3, 8, 9], [0, 5, 9, 11, 11]
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((11, 2, 8)), rng.standard_normal((11, 2, 8))
    out, lse, av, mag = O.prompt_attention(q, k, v, cu_q, cu_k, 0.3, causal)
    for g in range(4):
        n, m = cu_q[g + 1] - cu_q[g], cu_k[g + 1] - cu_k[g]
        for i in range(n):
            seen = max(0, m - n + i + 1) if causal else m
            rows = slice(cu_k[g], cu_k[g] + seen)
            for h in range(4):
                a = CO.attention_row(q[cu_q[g] + i, h], k[rows, h // 2], v[rows, h // 2], 0.3)
                assert np.allclose(out[cu_q[g] + i, h], a[0]) and np.allclose(av[cu_q[g] + i, h], a[2])
                assert (lse[h, cu_q[g] + i] == a[1] == -math.inf) or np.isclose(lse[h, cu_q[g] + i], a[1])
                assert np.isclose(mag[cu_q[g] + i, h], a[3])


def test_pages_oracle_keeps_counts_and_rows():
    rng = np.random.default_rng(1)
    page, pages = 4, 12
    cache = [rng.integers(0, 9, (pages, 1, page, 2)), rng.integers(0, 9, (pages, 1, page))]
    table = np.full((3, 3), -1)
    refs, lens = np.zeros(pages, int), np.zeros(3, int)
    assert PO.resize(refs, table, lens, [9, -1, -1], page) and table[0].tolist() == [0, 1, 2] and lens.tolist() == [9, 0, 0]
    PO.fork(cache, refs, table, lens, [0], [1])
    assert table[1].tolist() == [0, 1, 3] and refs[:4].tolist() == [2, 2, 1, 1] and lens[1] == 9
    assert np.array_equal(cache[0][3, :, :1], cache[0][2, :, :1])
    rows = cache[1][table[0], 0].ravel()[:9].copy()
    assert PO.compact(cache, table[:1], [2], [10], [11, 13, 16], [0, 3]).tolist() == [5]
    assert cache[1][table[0], 0].ravel()[:5].tolist() == [*rows[:2], rows[3], rows[5], rows[8]]
    assert not PO.resize(refs, table, lens, [12, 12, 40], page)        # the third finds too few
    PO.resize(refs, table, lens, [0, 0, 0], page)
    assert not refs.any()


# ------------------------------------------------------------------ C entry points

def _n(x):
    return x or None


def _prompt(lib, **over):
    a = dict(q=16, qs=0, k=16, ks=0, v=16, vs=0, cq=16, ck=16, seg=2, tq=8, tk=8, mq=4, mk=4, H=4, Hkv=2, d=64, dtype=0, scale=0.0,
             flags=1, out=16, os=0, lse=0, ws=256, wsb=1 << 26)
    a.update(over)
    return lib.tsel_prompt_attention(_n(a["q"]), a["qs"], _n(a["k"]), a["ks"], _n(a["v"]), a["vs"], _n(a["cq"]), _n(a["ck"]), a["seg"], a["tq"],
                                     a["tk"], a["mq"], a["mk"], a["H"], a["Hkv"], a["d"], a["dtype"], a["scale"], a["flags"], _n(a["out"]),
                                     a["os"], _n(a["lse"]), _n(a["ws"]), a["wsb"], None)


def test_prompt_host_checks(lib):
    assert _prompt(lib, tq=0) == 0
    for over, code in ((dict(dtype=2), 2), (dict(d=72), 2), (dict(d=256), 2), (dict(H=5), 1), (dict(H=0), 1), (dict(H=258), 1), (dict(Hkv=0), 1),
                       (dict(H=256, Hkv=1), 2), (dict(seg=-1), 1), (dict(tq=-1), 1), (dict(tk=-1), 1), (dict(mq=-1), 1), (dict(mk=-1), 1),
                       (dict(cq=0), 1), (dict(ck=0), 1), (dict(cq=18), 1), (dict(lse=18), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1),
                       (dict(out=0), 1), (dict(q=8), 1), (dict(v=24), 1), (dict(qs=64), 1), (dict(ks=132), 1), (dict(vs=100), 1), (dict(os=260), 1),
                       (dict(flags=2), 2), (dict(scale=math.nan), 1), (dict(scale=-math.inf), 1), (dict(ws=0), 1), (dict(ws=64), 3),
                       (dict(wsb=512), 3), (dict(tq=2 ** 30 + 1), 2), (dict(tk=2 ** 30 + 1), 2), (dict(mk=2 ** 30 + 1), 2),
                       (dict(tq=1, mq=1, mk=2 ** 30, tk=2 ** 30, wsb=2048), 3)):
        assert _prompt(lib, **over) == code, over


def test_prompt_workspace_size(tsel):
    size = tsel.tsel_prompt_attention_workspace_size
    assert size(1, 36973, 36973, 36973, 16, 8, 128) == 1024 and size(0, 0, 0, 0, 4, 2, 64) == 1024
    assert size(1, 142, 142, 36973, 16, 8, 128) > 2 * 142 * 16 * 128 * 4       # keys in chunks
    assert size(1, 1, 1, 2 ** 30, 1, 1, 64) > 1024
    for bad in ((-1, 4, 4, 4, 4, 2, 64), (1, -4, 4, 4, 4, 2, 64), (1, 4, -4, 4, 4, 2, 64), (1, 4, 4, -4, 4, 2, 64), (1, 4, 4, 4, 5, 2, 64),
                (1, 4, 4, 4, 4, 0, 64), (1, 4, 4, 4, 256, 1, 64), (1, 4, 4, 4, 4, 2, 72), (1, 4, 4, 4, 512, 256, 64), (1, 2 ** 30 + 1, 4, 4, 4, 2, 64),
                (1, 4, 4, 2 ** 30 + 1, 4, 2, 64), (2 ** 31, 4, 4, 4, 4, 2, 64)):
        assert size(*bad) == 0


def _tree(lib, **over):
    a = dict(q=16, qs=0, cu=16, R=2, tq=4, mn=2, par=16, kp=16, vp=16, ke=16, ve=16, pages=8, ps=16, pp=16, pl=16, mp=100, pt=16, pts=4,
             sl=16, ms=50, H=4, Hkv=2, d=64, dtype=0, scale=0.0, out=16, os=0, lse=0, ws=256, wsb=1 << 26)
    a.update(over)
    return lib.tsel_tree_attention(_n(a["q"]), a["qs"], _n(a["cu"]), a["R"], a["tq"], a["mn"], _n(a["par"]), _n(a["kp"]), _n(a["vp"]), _n(a["ke"]),
                                   _n(a["ve"]), a["pages"], a["ps"], _n(a["pp"]), _n(a["pl"]), a["mp"], _n(a["pt"]), a["pts"], _n(a["sl"]),
                                   a["ms"], a["H"], a["Hkv"], a["d"], a["dtype"], a["scale"], _n(a["out"]), a["os"], _n(a["lse"]), _n(a["ws"]),
                                   a["wsb"], None)


def test_tree_host_checks(lib, tsel):
    assert _tree(lib, tq=0) == 0 and _tree(lib, tq=0, mn=64, par=0) == 0
    for over, code in ((dict(mn=65), 2), (dict(par=0), 1), (dict(par=18), 1), (dict(mn=-1), 1), (dict(ms=0), 1), (dict(d=72), 2), (dict(pts=3), 1), (dict(q=8), 1),
                       (dict(out=0), 1), (dict(dtype=2), 2), (dict(ws=0), 1), (dict(wsb=4096), 3), (dict(kp=0), 1), (dict(mp=2 ** 30 + 1), 2)):
        assert _tree(lib, **over) == code, over
    size = tsel.tsel_tree_attention_workspace_size
    assert size(4, 32, 8, 16, 8, 128, 1228, 142) > 1024 and size(4, 32, 65, 16, 8, 128, 1228, 142) == 0
    assert size(4, 32, 8, 16, 8, 72, 1228, 142) == 0 and size(4, -32, 8, 16, 8, 128, 1228, 142) == 0


def _compact(lib, **over):
    a = dict(kp=16, vp=16, ke=16, ve=16, pages=8, ps=16, t=16, ts=4, tw=4, dt=0, ds=0, dw=0, st=0, ba=0, ki=16, cu=16, R=2, total=4, most=4,
             Hkv=2, d=64, nl=0, ws=256, wsb=1024)
    a.update(over)
    return lib.tsel_cache_compact(_n(a["kp"]), _n(a["vp"]), _n(a["ke"]), _n(a["ve"]), a["pages"], a["ps"], _n(a["t"]), a["ts"], a["tw"], _n(a["dt"]),
                                  a["ds"], a["dw"], _n(a["st"]), _n(a["ba"]), _n(a["ki"]), _n(a["cu"]), a["R"], a["total"], a["most"], a["Hkv"],
                                  a["d"], _n(a["nl"]), _n(a["ws"]), a["wsb"], None)


def test_compact_host_checks(lib):
    assert _compact(lib, R=0) == 0
    for over, code in ((dict(R=-1), 1), (dict(total=-1), 1), (dict(most=-1), 1), (dict(tw=-1), 1), (dict(dt=16, dw=-1), 1), (dict(cu=0), 1),
                       (dict(cu=18), 1), (dict(st=18), 1), (dict(ba=18), 1), (dict(nl=18), 1), (dict(ki=0), 1), (dict(ki=18), 1), (dict(t=0), 1),
                       (dict(t=18), 1), (dict(ts=3), 1), (dict(dt=16, ds=1, dw=2), 1), (dict(dt=18, ds=2, dw=2), 1), (dict(d=72), 2),
                       (dict(ps=8), 2), (dict(Hkv=0), 1), (dict(kp=0), 1), (dict(ve=8), 1), (dict(pages=2 ** 27, ps=16), 1), (dict(ws=0), 1),
                       (dict(ws=8), 3), (dict(wsb=1000), 3)):
        assert _compact(lib, **over) == code, over


def _resize(lib, **over):
    a = dict(refs=16, pages=8, ps=16, t=16, ts=4, rows=3, w=4, lens=16, new=16, ws=256, wsb=1 << 20)
    a.update(over)
    return lib.tsel_cache_resize(_n(a["refs"]), a["pages"], a["ps"], _n(a["t"]), a["ts"], a["rows"], a["w"], _n(a["lens"]), _n(a["new"]),
                                 _n(a["ws"]), a["wsb"], None)


def _fork(lib, **over):
    a = dict(kp=16, vp=16, ke=16, ve=16, Hkv=2, d=64, refs=16, pages=8, ps=16, t=16, ts=4, rows=3, w=4, lens=16, par=16, kid=16, n=2, ws=256,
             wsb=1 << 20)
    a.update(over)
    return lib.tsel_cache_fork(_n(a["kp"]), _n(a["vp"]), _n(a["ke"]), _n(a["ve"]), a["pages"], a["ps"], a["Hkv"], a["d"], _n(a["refs"]), _n(a["t"]),
                               a["ts"], a["rows"], a["w"], _n(a["lens"]), _n(a["par"]), _n(a["kid"]), a["n"], _n(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("call", [_resize, _fork])
def test_pages_host_checks(lib, call):
    assert call(lib, **(dict(rows=0) if call is _resize else dict(n=0))) == 0
    for over, code in ((dict(ps=24), 2), (dict(pages=-1), 1), (dict(pages=2 ** 27), 1), (dict(rows=-1), 1), (dict(w=-1), 1), (dict(ts=3), 1),
                       (dict(rows=2 ** 20, w=2 ** 12, ts=2 ** 12), 1), (dict(t=0), 1), (dict(t=18), 1), (dict(lens=0), 1), (dict(lens=18), 1),
                       (dict(refs=0), 1), (dict(refs=18), 1), (dict(ws=0), 1), (dict(ws=8), 3), (dict(wsb=1024), 3)):
        assert call(lib, **over) == code, over


def test_resize_and_fork_host_checks(lib, tsel):
    assert _resize(lib, new=0) == 1 and _resize(lib, new=18) == 1
    for over, code in ((dict(n=-1), 1), (dict(n=4), 1), (dict(par=0), 1), (dict(kid=18), 1), (dict(d=72), 2), (dict(Hkv=0), 1), (dict(kp=0), 1),
                       (dict(ke=8), 1)):
        assert _fork(lib, **over) == code, over
    size = tsel.tsel_cache_resize_workspace_size
    assert size(3, 4) >= 1024 + 4 * 4 + 4 * 12 and size(0, 0) >= 1024
    assert size(-1, 4) == size(3, -1) == size(2 ** 20, 2 ** 12) == size(2 ** 31, 1) == 0


# ------------------------------------------------------------------ refusals of the binding

def _ints(n):
    return _Fake((n,), I32)


def test_binding_refuses_prompts(tsel):
    q, k = _Fake((8, 4, 64), BF), _Fake((9, 2, 64), BF)
    good = dict(q=q, k=k, v=k, cu_seqlens_q=_ints(3), cu_seqlens_k=_ints(3), max_seqlen_q=4, max_seqlen_k=5)

    def refused(error, **over):
        with pytest.raises(error):
            tsel.tsel_prompt_attention(**{**good, **over})
    refused(TypeError, q=_Fake((8, 4, 64), torch.float32), k=_Fake((9, 2, 64), torch.float32), v=_Fake((9, 2, 64), torch.float32))
    refused(TypeError, k=_Fake((9, 2, 64), torch.float16))
    refused(ValueError, v=_Fake((8, 2, 64), BF))
    refused(ValueError, k=_Fake((9, 2, 80), BF), v=_Fake((9, 2, 80), BF))
    refused(ValueError, k=_Fake((9, 2, 64), BF, (256, 128, 1)))                   # heads apart
    refused(ValueError, v=_Fake((9, 2, 64), BF, (0, 64, 1)))                      # expanded
    refused(ValueError, k=_Fake((9, 2, 64), BF, device=1))
    refused(ValueError, cu_seqlens_k=_ints(4))
    refused(ValueError, cu_seqlens_q=_ints(0), cu_seqlens_k=_ints(0))
    refused(TypeError, cu_seqlens_q=_Fake((3,), torch.int64))
    refused(ValueError, max_seqlen_k=2 ** 31)
    refused(ValueError, max_seqlen_q=-1)
    refused(ValueError, out=_Fake((8, 4, 80), BF))
    refused(TypeError, lse=_Fake((4, 8), BF))
    refused(ValueError, lse=_Fake((4, 7), torch.float32))


def test_binding_refuses_trees(tsel):
    q, cache = _Fake((4, 4, 64), BF), _fake_cache(tsel)
    good = dict(q=q, cu_seqlens_q=_ints(3), max_nodes=2, parents=_ints(4), cache=cache, prefix_pages=None, prefix_len=None, max_prefix_len=0,
                page_table=_Fake((2, 4), I32), suffix_lens=_ints(2), max_suffix_len=50)

    def refused(error, **over):
        with pytest.raises(error):
            tsel.tsel_tree_attention(**{**good, **over})
    refused(ValueError, parents=None)
    refused(ValueError, parents=_ints(3))
    refused(TypeError, parents=_Fake((4,), torch.int64))
    refused(ValueError, max_prefix_len=5)
    refused(ValueError, page_table=_Fake((2, 3), I32))
    refused(ValueError, suffix_lens=_ints(3))


def test_binding_refuses_pages(tsel):
    cache, t = _fake_cache(tsel), _Fake((2, 4), I32)

    def refused(error, call, *args, **kw):
        with pytest.raises(error):
            call(*args, **kw)
    c = tsel.tsel_cache_compact
    refused(ValueError, c, cache, t, _ints(4), _ints(0), 4)
    refused(ValueError, c, cache, t, _ints(4), _ints(4), 4)                       # three requests, two rows
    refused(ValueError, c, cache, _Fake((2, 4), I32, (3, 1)), _ints(4), _ints(3), 4)
    refused(ValueError, c, cache, _Fake((2, 4), I32, (8, 2)), _ints(4), _ints(3), 4)
    refused(TypeError, c, cache, _Fake((2, 4), torch.int64), _ints(4), _ints(3), 4)
    refused(TypeError, c, cache, t, _Fake((4,), torch.int64), _ints(3), 4)
    refused(ValueError, c, cache, t, _ints(4), _ints(3), 4, starts=_ints(3))
    refused(ValueError, c, cache, t, _ints(4), _ints(3), 4, bases=_Fake((2,), I32, (2,)))
    refused(ValueError, c, cache, t, _ints(4), _ints(3), 4, dst_table=t)          # in place is said by None
    refused(ValueError, c, cache, t, _ints(4), _ints(3), 4, new_lens=_ints(3))
    refused(ValueError, c, cache, t, _ints(4), _ints(3), -1)
    r = tsel.tsel_cache_resize
    refused(TypeError, r, torch.zeros(4, dtype=I32), t, _ints(2), _ints(2), 16)          # on the host
    refused(TypeError, r, _Fake((4,), torch.int64), t, _ints(2), _ints(2), 16)
    refused(ValueError, r, _ints(4), t, _ints(3), _ints(2), 16)
    refused(ValueError, r, _ints(4), t, _ints(2), _ints(3), 16)
    refused(ValueError, r, _ints(4), t, _ints(2), _ints(2), -16)
    f = tsel.tsel_cache_fork
    refused(ValueError, f, cache, _ints(3), t, _ints(2), _ints(1), _ints(1))      # counts of another pool
    refused(ValueError, f, cache, _ints(4), t, _ints(2), _ints(1), _ints(2))
    refused(ValueError, f, cache, _ints(4), t, _ints(1), _ints(1), _ints(1))


def test_pages_oracle_lists_out_of_order():
    assert PO.good_forks([9, 6] + [0] * 6, [0, 0, 0], [5, 3, 5]) == [True, False, False]
    assert PO.good_forks([9, 6] + [0] * 6, [0, 0, 5], [5, 3, 6]) == [True, False, False]
    assert PO.good_forks([9, 6] + [0] * 6, [0, 3, 8, 1], [2, 3, 4, 5]) == [True, False, False, True]


def test_pages_oracle_shared_ends():
    refs, table, lens = np.asarray([2, 2, 1, 1, 0, 0]), np.asarray([[0, 1, 2], [0, 1, 3], [-1, -1, -1]]), np.asarray([9, 6, 0])
    assert PO.shared_end(refs, table, lens, [12, 7, 4], 4).tolist() == [False, True, False]
    assert PO.shared_end(refs, table, lens, [4, 6, -1], 4).tolist() == [False, False, False]
    assert PO.resize(refs, table, lens, [-1, 12, 4], 4) and lens.tolist() == [9, 6, 4] and refs.tolist() == [2, 2, 1, 1, 1, 0]


def test_overlapping_page_arguments(lib):
    """What a call writes and what it reads or also writes must not share memory. Every call here is
    refused before a launch."""
    def refused(call, **over):
        assert call(lib, **over) == 1 and b"overlap" in lib.tsel_last_error(), over
    # [3 rows of 4] at 4096, vectors of 2 or 3 elsewhere
    c = dict(t=4096, ki=8192, cu=12288, st=16384, ba=20480, dt=24576, ds=4, dw=4)
    for at in (16384, 16384 + 4, 16384 - 4, 20480, 20480 + 4, 8192 + 12, 8192 - 4, 12288, 12288 + 8, 4096, 4096 + 28, 24576 + 16):
        refused(_compact, **c, nl=at)
    refused(_compact, **{**c, "ts": 16, "tw": 4}, nl=4096 + 64 + 12)          # the last entry of the second row
    r = dict(refs=4096, t=8192, lens=12288, new=16384)
    for over in (dict(new=12288 + 4), dict(new=12288 - 8), dict(new=4096 + 28), dict(new=8192 + 44), dict(lens=4096), dict(lens=8192 + 16),
                 dict(t=4096 + 28)):
        refused(_resize, **{**r, **over})
    f = dict(refs=4096, t=8192, lens=12288, par=16384, kid=20480)
    for over in (dict(par=12288 + 8), dict(kid=12288), dict(par=4096 - 4), dict(kid=8192 + 44), dict(lens=4096 + 28), dict(t=12288 + 8), dict(refs=8192 + 40)):
        refused(_fork, **{**f, **over})
