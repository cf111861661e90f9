"""Rotary tables, the fp64 oracle of the cache-side operators, and the refusals
of their host checks (fake addresses that are never dereferenced). No GPU."""
import math
import shutil
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import cache_oracle as O

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

LAYOUTS = {"sectioned": 0, "interleaved": 1, "per_axis": 2}


@pytest.fixture(scope="module")
def tsel():
    import attention_score_vision_gb300 as t
    t.build()
    t.load_library()
    return t


@pytest.fixture(scope="module")
def lib(tsel):
    return tsel.load_library()


@pytest.mark.parametrize("sections,layout", [([24, 20, 20], "interleaved"), ([16, 24, 24], "sectioned"),
                                             ([0, 20, 20], "per_axis"), ([64], "sectioned"), ([14, 13, 13], "interleaved")])
def test_frequencies_match_the_oracle(tsel, sections, layout):
    f, a = tsel.tsel_rope_frequencies(1e6, sections, LAYOUTS[layout])
    f_ref, a_ref = O.rope_frequencies(1e6, sections, layout)
    assert a == a_ref.tolist()
    np.testing.assert_allclose(f, f_ref, rtol=1e-14)
    assert [a.count(i) for i in range(len(sections))] == sections


def test_table_counts_turns_to_2_to_the_minus_61(tsel):
    # 2 pi to 60 digits
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    f = [1.0, 0.8058421877614819, 1e-6, 3.7e-9, 6.5, -0.25, 123456.789, 0.0]
    t = tsel.tsel_rope_table(f, [0, 1, 2, 3, 4, 5, 6, 7], device="cpu")
    for i, (x, e) in enumerate(zip(f, t.tolist())):
        e &= 2 ** 64 - 1
        assert e & 7 == i
        off = (Fraction(e >> 3, 2 ** 61) - Fraction(x) / two_pi) % 1
        # one step of 2^-61, and 2^-106 of the turns
        assert min(off, 1 - off) <= Fraction(1, 2 ** 61) + Fraction(abs(x)) / 2 ** 104


def test_table_and_frequency_refusals(tsel, lib):
    for sections, layout in (([10, 30, 24], 1), ([4, -1], 0), ([129], 0), ([], 0), ([1] * 9, 0), ([4], 3)):
        with pytest.raises(tsel.TselError):
            tsel.tsel_rope_frequencies(1e4, sections, layout)
    for base in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(tsel.TselError):
            tsel.tsel_rope_frequencies(base, [4])
    for f, a in (([math.nan], [0]), ([2e6], [0]), ([math.inf], [0]), ([1.0], [8]), ([1.0], [-1]), ([1.0] * 129, [0] * 129)):
        with pytest.raises(tsel.TselError):
            tsel.tsel_rope_table(f, a, device="cpu")
    with pytest.raises(ValueError):
        tsel.tsel_rope_table([1.0, 2.0], [0], device="cpu")
    assert lib.tsel_rope_table(None, None, 4, None) == 1
    assert tsel.tsel_rope_table([], [], device="cpu").numel() == 0


# ------------------------------------------------------------------ the oracle itself

def test_oracle_rotation_is_orthogonal_and_inverts():
    rng = np.random.default_rng(5)
    f, a = O.rope_frequencies(1e4, [3, 2, 2], "interleaved")
    x = rng.standard_normal((9, 2, 16))
    pos = rng.integers(-50, 50, (9, 3))
    for adjacent in (False, True):
        y = O.rope(x, pos, f, a, adjacent)
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
        np.testing.assert_allclose(O.rope(y, pos, f, a, adjacent, inverse=True), x, atol=1e-13)
        assert np.array_equal(y[..., 14:], x[..., 14:])
        assert not np.allclose(y[..., :14], x[..., :14])
    # one pair by hand: a quarter turn
    y = O.rope(np.asarray([[[1.0, 2.0]]]), [[1]], np.asarray([math.pi / 2]), np.asarray([0]))
    np.testing.assert_allclose(y, [[[-2.0, 1.0]]], atol=1e-15)


def test_oracle_rotation_depends_on_position_differences_only():
    rng = np.random.default_rng(6)
    f, a = O.rope_frequencies(1e4, [4, 4], "sectioned")
    q, k = rng.standard_normal((2, 1, 1, 16))
    dots = [float((O.rope(q, [[p + 7, p - 3]], f, a) * O.rope(k, [[p, p]], f, a)).sum()) for p in (0, 5, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_oracle_quantiser_rounds_to_the_nearest_code():
    rng = np.random.default_rng(7)
    x = rng.standard_normal((200, 16)) * 2.0 ** rng.integers(-30, 30, (200, 1))
    x[3] = 0
    x[4, 2] = np.nan
    x[5, 1] = -np.inf
    codes, exps = O.quantise(x)
    y = O.dequantise(codes, exps)
    assert exps[3] == 0 and not codes[3].any()
    assert exps[4] == exps[5] == 255 and np.isnan(y[4]).all()
    ok = exps < 255
    e = 2.0 ** (exps[ok].astype(float) - 127)[:, None]
    assert np.all(np.abs(y[ok] - x[ok]) <= np.maximum(np.abs(x[ok]) / 16, e * 2.0 ** -10))
    top = np.abs(x[ok]).max(-1, keepdims=True)
    assert np.all(top <= 448 * e) and np.all((top > 224 * e) | (top == 0))
    # torch's cast agrees on the codes (448 is never passed)
    t = torch.from_numpy((x[ok] / e).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    near = (x[ok] / e).astype(np.float32).astype(np.float64) == x[ok] / e
    assert np.array_equal(t[near], codes[ok][near])


def test_oracle_attention_joins_prefix_and_suffix():
    rng = np.random.default_rng(8)
    k, v = rng.standard_normal((2, 40, 2, 8))
    q = rng.standard_normal((3, 4, 8))
    out, lse, _, _ = O.prefix_attention(q, [0, 2, 3], k, v, np.arange(10), [np.arange(10, 15), np.arange(20, 20)], 0.5)
    # row 0 of request 0 sees the prefix and suffix keys 10..13; brute force
    rows = list(range(14))
    z = 0.5 * k[rows, 1] @ q[0, 2]
    w = np.exp(z) / np.exp(z).sum()
    np.testing.assert_allclose(out[0, 2], w @ v[rows, 1], rtol=1e-12)
    np.testing.assert_allclose(lse[2, 0], np.log(np.exp(z).sum()), rtol=1e-12)
    z = 0.5 * k[:10, 0] @ q[2, 1]
    np.testing.assert_allclose(out[2, 1], np.exp(z) @ v[:10, 0] / np.exp(z).sum(), rtol=1e-12)
    # no keys at all
    out, lse, _, _ = O.prefix_attention(q, [0, 2, 3], k, v, np.arange(0), [np.arange(1), np.arange(0)], 0.5)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[:, 0])) and np.isfinite(lse[:, 1]).all()


# ------------------------------------------------------------------ refusals of the C entry points

def _rope(lib, **over):
    a = dict(q=16, qs=0, k=16, ks=0, pos=16, pd=3, table=16, pairs=32, total=4, H=4, Hkv=2, d=64, dtype=0, flags=0,
             qo=16, qos=0, ko=16, kos=0, ws=256, wsb=1024)
    a.update(over)
    return lib.tsel_rope(a["q"] or None, a["qs"], a["k"] or None, a["ks"], a["pos"] or None, a["pd"], a["table"] or None,
                         a["pairs"], a["total"], a["H"], a["Hkv"], a["d"], a["dtype"], a["flags"], a["qo"] or None, a["qos"],
                         a["ko"] or None, a["kos"], a["ws"] or None, a["wsb"], None)


def test_rope_host_checks(lib):
    assert _rope(lib, total=0) == 0                       # nothing to do
    for over, code in ((dict(dtype=3), 2), (dict(d=68), 2), (dict(d=264), 2), (dict(flags=4), 2), (dict(H=0), 1),
                       (dict(H=257), 1), (dict(Hkv=-1), 1), (dict(total=-1), 1), (dict(pairs=33), 1), (dict(pairs=-1), 1),
                       (dict(pd=9), 1), (dict(pd=0), 1), (dict(pos=0), 1), (dict(table=0), 1), (dict(pos=18), 1),
                       (dict(table=20), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(qo=0), 1), (dict(ko=0), 1), (dict(q=8), 1),
                       (dict(ko=24), 1), (dict(qs=255), 1), (dict(qs=260), 1), (dict(kos=64), 1), (dict(ws=0), 1),
                       (dict(ws=128), 3), (dict(wsb=1000), 3)):
        assert _rope(lib, **over) == code, over


def _cache(lib, what, **over):
    a = dict(k=16, ks=0, v=16, vs=0, pos=0, pd=0, table=0, pairs=0, slots=16, total=4, Hkv=2, d=64, dtype=0, flags=0,
             kp=16, vp=16, ke=16, ve=16, pages=4, ps=16, ws=256, wsb=1024)
    a.update(over)
    p = [a[n] or None for n in ("kp", "vp", "ke", "ve")]
    if what == "write":
        return lib.tsel_cache_write(a["k"] or None, a["ks"], a["v"] or None, a["vs"], a["pos"] or None, a["pd"],
                                    a["table"] or None, a["pairs"], a["slots"] or None, a["total"], a["Hkv"], a["d"],
                                    a["dtype"], a["flags"], *p, a["pages"], a["ps"], a["ws"] or None, a["wsb"], None)
    return lib.tsel_cache_read(*p, a["pages"], a["ps"], a["slots"] or None, a["total"], a["Hkv"], a["d"], a["dtype"],
                               a["k"] or None, a["ks"], a["v"] or None, a["vs"], a["ws"] or None, a["wsb"], None)


COMMON = ((dict(d=72), 2), (dict(d=256), 2), (dict(ps=8), 2), (dict(ps=48), 2), (dict(ps=256), 2), (dict(Hkv=0), 1),
          (dict(Hkv=257), 1), (dict(pages=-1), 1), (dict(pages=2 ** 27, ps=16), 1), (dict(kp=0), 1), (dict(ve=0), 1),
          (dict(kp=24), 1), (dict(ke=4), 1), (dict(dtype=7), 2), (dict(total=-1), 1), (dict(slots=0), 1), (dict(slots=18), 1),
          (dict(k=0), 1), (dict(v=8), 1), (dict(ks=100), 1), (dict(vs=132), 1), (dict(ws=0), 1), (dict(ws=8), 3), (dict(wsb=0), 3))


@pytest.mark.parametrize("what", ["write", "read"])
def test_cache_host_checks(lib, what):
    assert _cache(lib, what, total=0) == 0
    for over, code in COMMON:
        assert _cache(lib, what, **over) == code, over


def test_cache_write_rotation_checks(lib):
    for over, code in ((dict(pairs=8), 1), (dict(pairs=8, pos=16, pd=2), 1), (dict(pairs=8, pos=16, pd=0, table=16), 1),
                       (dict(pairs=33, pos=16, pd=2, table=16), 1), (dict(flags=2), 2)):
        assert _cache(lib, "write", **over) == code, over


def _attend(lib, **over):
    a = dict(q=16, qs=0, cu=16, R=2, tq=4, mq=2, kp=16, vp=16, ke=16, ve=16, pages=8, ps=16, pp=16, pl=16, mp=100, pt=16, pts=4,
             sl=16, ms=50, H=4, Hkv=2, d=64, dtype=0, scale=0.0, out=16, os=0, lse=0, ws=256, wsb=1 << 26)
    a.update(over)
    n = lambda x: x or None   # noqa: E731
    return lib.tsel_prefix_attention(n(a["q"]), a["qs"], n(a["cu"]), a["R"], a["tq"], a["mq"], n(a["kp"]), n(a["vp"]), n(a["ke"]),
                                     n(a["ve"]), a["pages"], a["ps"], n(a["pp"]), n(a["pl"]), a["mp"], n(a["pt"]), a["pts"],
                                     n(a["sl"]), a["ms"], a["H"], a["Hkv"], a["d"], a["dtype"], a["scale"], n(a["out"]), a["os"],
                                     n(a["lse"]), n(a["ws"]), a["wsb"], None)


def test_attention_host_checks(lib):
    assert _attend(lib, tq=0) == 0
    for over, code in ((dict(dtype=2), 2), (dict(d=72), 2), (dict(ps=20), 2), (dict(H=5), 1), (dict(H=0), 1), (dict(H=258), 1),
                       (dict(H=256, Hkv=1), 2), (dict(R=-1), 1), (dict(tq=-1), 1), (dict(mq=-1), 1), (dict(mp=-1), 1),
                       (dict(ms=-1), 1), (dict(cu=0), 1), (dict(pp=0), 1), (dict(pl=0), 1), (dict(pt=0), 1), (dict(sl=0), 1),
                       (dict(pts=3), 1), (dict(q=0), 1), (dict(q=8), 1), (dict(out=0), 1), (dict(qs=64), 1), (dict(os=260), 1),
                       (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(ws=0), 1), (dict(ws=64), 3), (dict(wsb=4096), 3),
                       (dict(kp=0), 1), (dict(ve=8), 1), (dict(mp=2 ** 30 + 1), 2), (dict(ms=2 ** 30 + 1, pts=2 ** 27), 2),
                       (dict(R=2 ** 31 - 1, tq=2 ** 31 - 1, mq=2 ** 31 - 1, mp=2 ** 30), 2)):
        assert _attend(lib, **over) == code, over


def test_attention_workspace_size(tsel):
    size = tsel.tsel_prefix_attention_workspace_size
    assert size(0, 0, 0, 4, 2, 64, 0, 0) == 1024
    assert size(64, 64, 1, 32, 8, 128, 40000, 1000) > 64 * 32 * 128 * 4
    for bad in ((-1, 4, 1, 4, 2, 64, 10, 10), (1, -4, 1, 4, 2, 64, 10, 10), (1, 4, 1, 5, 2, 64, 10, 10), (1, 4, 1, 4, 2, 64, -1, 10),
                (1, 4, 1, 256, 1, 64, 10, 10), (1, 4, 1, 4, 2, 72, 10, 10), (1, 4, 1, 512, 256, 64, 10, 10), (1, 4, 1, 4, 2, 64, 2 ** 30 + 1, 10),
                (1, 4, 1, 4, 2, 64, 10, 2 ** 30 + 1), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 256, 256, 128, 2 ** 30, 2 ** 30)):
        assert size(*bad) == 0
    assert size(1, 4, 1, 4, 2, 64, 2 ** 30, 2 ** 30) > 0


# ------------------------------------------------------------------ refusals of the binding

class _Fake:
    def __init__(self, shape, dtype, strides=None, device=0):
        self.shape, self.dtype, self.is_cuda, self.device = tuple(shape), dtype, True, torch.device("cuda", device)
        if strides is None:
            strides, acc = [], 1
            for n in reversed(self.shape):
                strides.insert(0, acc)
                acc *= n
        self._dense = [n for n in strides]
        self._strides = tuple(strides)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return self._strides[i]

    def get_device(self):
        return self.device.index

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        acc = 1
        for n, s in zip(reversed(self.shape), reversed(self._strides)):
            if n != 1 and s != acc:
                return False
            acc *= n
        return True

    def data_ptr(self):
        return 1 << 20


def _fake_cache(tsel, pages=4, heads=2, ps=16, d=64, **kw):
    codes = [_Fake((pages, heads, ps, d), torch.uint8, **kw) for _ in range(2)]
    return tsel.TselCache(*codes, *[_Fake((pages, heads, ps), torch.uint8, **kw) for _ in range(2)])


def test_binding_refuses_what_the_kernels_cannot_see(tsel):
    bf, i32 = torch.bfloat16, torch.int32
    q, k = _Fake((5, 4, 64), bf), _Fake((5, 2, 64), bf)
    pos, table = _Fake((5, 3), i32), _Fake((32,), torch.int64)
    slots, cache = _Fake((5,), i32), _fake_cache(tsel)
    bad = [
        lambda: tsel.tsel_rope(q, k, _Fake((4, 3), i32), table),                       # positions of other tokens
        lambda: tsel.tsel_rope(q, k, _Fake((5, 3), torch.int64), table),
        lambda: tsel.tsel_rope(q, k, _Fake((5, 3), i32, strides=(1, 5)), table),       # transposed
        lambda: tsel.tsel_rope(q, k, pos, _Fake((32,), torch.int32)),
        lambda: tsel.tsel_rope(q, _Fake((5, 2, 64), torch.float16), pos, table),       # mixed types
        lambda: tsel.tsel_rope(q, _Fake((6, 2, 64), bf), pos, table),
        lambda: tsel.tsel_rope(q, _Fake((5, 2, 64), bf, device=1), pos, table),
        lambda: tsel.tsel_rope(_Fake((5, 4, 64), bf, strides=(256, 1, 4)), k, pos, table),
        lambda: tsel.tsel_rope(q, None, pos, table, k_out=k),
        lambda: tsel.tsel_rope(_Fake((5, 4, 64), bf, strides=(0, 64, 1)), k, pos, table),   # one row, expanded
        lambda: tsel.tsel_cache_write(_Fake((5, 2, 64), bf, strides=(0, 64, 1)), k, slots, cache),
        lambda: tsel.tsel_rope(q, k, pos, table, q_out=k),
        lambda: tsel.tsel_cache_write(k, k, _Fake((4,), i32), cache),
        lambda: tsel.tsel_cache_write(k, k, _Fake((5,), torch.int64), cache),
        lambda: tsel.tsel_cache_write(k, q, slots, cache),
        lambda: tsel.tsel_cache_write(k, k, slots, _fake_cache(tsel, heads=4)),
        lambda: tsel.tsel_cache_write(k, k, slots, _fake_cache(tsel, d=80)),
        lambda: tsel.tsel_cache_write(k, k, slots, cache._replace(v_exps=_Fake((4, 2, 32), torch.uint8))),
        lambda: tsel.tsel_cache_write(k, k, slots, cache._replace(v_pages=_Fake((4, 2, 16, 64), torch.int8))),
        lambda: tsel.tsel_cache_write(k, k, slots, cache, table=table),                # no positions
        lambda: tsel.tsel_cache_read(cache, slots, dtype=torch.float64),
        lambda: tsel.tsel_cache_read(cache, slots, k_out=q),
        lambda: tsel.tsel_cache_read(_fake_cache(tsel, device=1), slots),
    ]
    cu, pp, pl = _Fake((3,), i32), _Fake((7,), i32), _Fake((1,), i32)
    pt, sl = _Fake((2, 4), i32), _Fake((2,), i32)

    def attend(q=q, cu=cu, mq=3, cache=cache, pp=pp, pl=pl, mp=100, pt=pt, sl=sl, ms=50, **kw):
        return lambda: tsel.tsel_prefix_attention(q, cu, mq, cache, pp, pl, mp, pt, sl, ms, **kw)

    bad += [attend(q=_Fake((5, 4, 64), torch.float32)), attend(cu=_Fake((3,), torch.int64)), attend(cu=_Fake((0,), i32)),
            attend(pp=None), attend(pl=None), attend(pp=_Fake((6,), i32)), attend(pt=None), attend(sl=None), attend(sl=_Fake((3,), i32)),
            attend(pt=_Fake((2, 3), i32)), attend(pt=_Fake((3, 4), i32)), attend(pt=_Fake((2, 4), i32, strides=(1, 2))),
            attend(pt=_Fake((2, 4), i32, strides=(0, 1))), attend(out=_Fake((5, 4, 64), bf, strides=(0, 64, 1))),
            attend(cache=_fake_cache(tsel, d=80)), attend(out=_Fake((4, 4, 64), bf)), attend(lse=_Fake((3, 5), torch.float32)),
            attend(pp=_Fake((7,), i32, device=1)), attend(workspace=_Fake((1 << 20,), torch.uint8, device=1))]
    for i, fn in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            fn()
            pytest.fail(f"call {i} was not refused")


def test_binding_refuses_outputs_where_autograd_records(tsel):
    """A recorded rotation returns new tensors."""
    bf = torch.bfloat16

    def fake(shape, grad):
        t = _Fake(shape, bf)
        t.requires_grad = grad
        return t

    pos, table = _Fake((5, 3), torch.int32), _Fake((32,), torch.int64)
    for grads in ((True, False, False, False), (False, True, False, False), (True, True, False, False)):
        q, k, qo, ko = (fake((5, h, 64), g) for h, g in zip((4, 2, 4, 2), grads))
        with pytest.raises(ValueError, match="autograd records"):
            tsel.tsel_rope(q, k, pos, table, q_out=qo, k_out=ko)


def test_binding_refuses_to_write_outputs_that_require_gradients(tsel):
    """... as torch refuses them."""
    bf = torch.bfloat16

    def fake(shape, dtype=bf, grad=False):
        t = _Fake(shape, dtype)
        t.requires_grad = grad
        return t

    i32, cache = torch.int32, _fake_cache(tsel)
    q, k, leaf_q, leaf_k = fake((5, 4, 64)), fake((5, 2, 64)), fake((5, 4, 64), grad=True), fake((5, 2, 64), grad=True)
    pos, table, slots = _Fake((5, 3), i32), _Fake((32,), torch.int64), _Fake((5,), i32)
    attend = (_Fake((3,), i32), 3, cache, _Fake((7,), i32), _Fake((1,), i32), 100, None, None, 0)
    for call in (lambda: tsel.tsel_rope(q, None, pos, table, q_out=leaf_q),
                 lambda: tsel.tsel_rope(q, k, pos, table, k_out=leaf_k),
                 lambda: tsel.tsel_cache_read(cache, slots, v_out=leaf_k),
                 lambda: tsel.tsel_prefix_attention(q, *attend, out=leaf_q),
                 lambda: tsel.tsel_prefix_attention(q, *attend, lse=fake((4, 5), torch.float32, True))):
        with pytest.raises(ValueError, match="autograd records"):
            call()


def test_binding_refuses_sizes_past_32_bits(tsel):
    """A foreign call would take the low 32 bits of them and work on those rows only."""
    bf, i32, far = torch.bfloat16, torch.int32, 2 ** 32 + 5
    table, cache = _Fake((32,), torch.int64), _fake_cache(tsel)
    q, cu = _Fake((5, 4, 64), bf), _Fake((3,), i32)
    pp, pl, pt, sl = _Fake((2 ** 29,), i32), _Fake((1,), i32), _Fake((2, 2 ** 29), i32), _Fake((2,), i32)
    ws = _Fake((1 << 20,), torch.uint8)
    for call in (lambda: tsel.tsel_rope(_Fake((far, 1, 64), bf), None, _Fake((far, 2), i32), table, workspace=ws),
                 lambda: tsel.tsel_rope(_Fake((2 ** 31, 1, 64), bf), None, _Fake((2 ** 31, 2), i32), table, workspace=ws),
                 lambda: tsel.tsel_rope(_Fake((1, far, 64), bf), None, _Fake((1, 2), i32), table, workspace=ws),
                 lambda: tsel.tsel_rope(q, _Fake((5, far, 64), bf), _Fake((5, 2), i32), table, workspace=ws),
                 lambda: tsel.tsel_rope(q, None, _Fake((5, far), i32), table, workspace=ws),
                 lambda: tsel.tsel_rope(q, None, _Fake((5, 2), i32), _Fake((2 ** 32,), torch.int64), workspace=ws),
                 lambda: tsel.tsel_cache_write(*[_Fake((far, 2, 64), bf)] * 2, _Fake((far,), i32), cache, workspace=ws),
                 lambda: tsel.tsel_cache_write(*[_Fake((1, 2, 64), bf)] * 2, _Fake((1,), i32), _fake_cache(tsel, pages=far), workspace=ws),
                 lambda: tsel.tsel_cache_read(cache, _Fake((far,), i32), workspace=ws),
                 lambda: tsel.tsel_prefix_attention(_Fake((far, 4, 64), bf), cu, 3, cache, pp, pl, 100, pt, sl, 50, workspace=ws),
                 lambda: tsel.tsel_prefix_attention(q, cu, 2 ** 32, cache, pp, pl, 100, pt, sl, 50, workspace=ws),
                 lambda: tsel.tsel_prefix_attention(q, cu, 2 ** 32 + 3, cache, pp, pl, 100, pt, sl, 50, workspace=ws),
                 lambda: tsel.tsel_prefix_attention(q, cu, -1, cache, pp, pl, 100, pt, sl, 50, workspace=ws),
                 lambda: tsel.tsel_prefix_attention(q, cu, 3, cache, pp, pl, far, pt, sl, 50, workspace=ws),
                 lambda: tsel.tsel_prefix_attention(q, cu, 3, cache, pp, pl, 100, pt, sl, far, workspace=ws)):
        with pytest.raises(ValueError, match="past 2"):
            call()
    size = tsel.tsel_prefix_attention_workspace_size
    ok = [1, 4, 4, 4, 2, 64, 10, 10]
    assert size(*ok) > 0
    for i in range(8):
        assert size(*[n + 2 ** 32 if j == i else n for j, n in enumerate(ok)]) == 0


def test_binding_refuses_expanded_and_strided_workspaces(tsel):
    """An expanded workspace has fewer bytes behind its pointer than entries."""
    bf, i32 = torch.bfloat16, torch.int32
    q, k, pos, table, slots = _Fake((5, 4, 64), bf), _Fake((5, 2, 64), bf), _Fake((5, 3), i32), _Fake((32,), torch.int64), _Fake((5,), i32)
    cache = _fake_cache(tsel)
    q.requires_grad = k.requires_grad = False
    for stride in (0, 2):
        ws = _Fake((1 << 20,), torch.uint8, strides=(stride,))
        for call in (lambda: tsel.tsel_rope(q, k, pos, table, workspace=ws),
                     lambda: tsel.tsel_cache_write(k, k, slots, cache, workspace=ws),
                     lambda: tsel.tsel_cache_read(cache, slots, workspace=ws),
                     lambda: tsel.tsel_prefix_attention(q, _Fake((3,), i32), 3, cache, _Fake((7,), i32), _Fake((1,), i32), 100,
                                                        None, None, 0, workspace=ws)):
            with pytest.raises(ValueError, match="workspace must be contiguous"):
                call()


def test_attention_unit_counts_past_64_bits(tsel, lib):
    """Sizes whose units, times their chunks, wrap around 64 bits are too large, not small."""
    size, far = tsel.tsel_prefix_attention_workspace_size, 2 ** 31 - 1
    for bad in ((far, 1, far, 256, 2, 64, 0, 2 ** 30), (2 ** 30, 1, far, 256, 256, 64, 0, 2 ** 30), (far, 1, far, 256, 256, 64, 0, 1024),
                (2 ** 30, 4, 2 ** 30, 128, 1, 64, 64, 2 ** 20)):
        assert size(*bad) == 0
        R, tq, mq, H, Hkv, d, mp, ms = bad
        assert _attend(lib, R=R, tq=tq, mq=mq, H=H, Hkv=Hkv, d=d, mp=mp, ms=ms, pts=2 ** 27, wsb=2 ** 40) == 2


def test_rope_host_helpers_refuse_numbers_past_32_bits(tsel):
    """... whose low 32 bits would be a valid section or axis; and no buffer grows with a refused section."""
    for sections in ([2 ** 32 + 4, 4], [2 ** 31, 4], [-2 ** 32 + 4]):
        with pytest.raises(ValueError, match="sections past 32 bits"):
            tsel.tsel_rope_frequencies(1e4, sections)
    with pytest.raises(tsel.TselError):
        tsel.tsel_rope_frequencies(1e4, [2 ** 31 - 1])
    for axis in (2 ** 32, 2 ** 32 + 1, -2 ** 32):
        with pytest.raises(ValueError, match="axis past 32 bits"):
            tsel.tsel_rope_table([1.0], [axis], device="cpu")
    f, a = tsel.tsel_rope_frequencies(1e4, [128])
    assert len(f) == len(a) == 128
