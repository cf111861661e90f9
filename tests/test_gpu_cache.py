"""GPU: rotary positions with several axes, the quantised paged cache, and
attention over a shared prefix, against the fp64 oracle.

Tolerances. Rotation: the angle is within 2^-24 rad, sine and cosine within
2^-23, two fp32 products and one sum, so a column is within (|a| + |b|) * 2^-21
before its one rounding to the output type (half a step: eps / 2 of the value).
Cache: exact on given rows. Attention: with A = sum_j p_j |v_j| (columnwise) and
delta the error of a logit (fp32 sums of d products, 2^-23 of their absolute sum
each, at most d of them), the probabilities are within delta + 2^-11 (fp16) +
2^-20 (exp2, sums, joining), so out is within A * (2 delta + 2^-11 + 2^-19) plus
n * 2^-31 max|v| for probabilities below fp16's range (its smallest step, 2^-24,
halved, against 2^6 at the row's reference, which is at most its maximum) plus half a step of the
output; lse within delta + 2^-20 + |lse| 2^-22."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import i32
from oracle import cache_oracle as O

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NAMES = {"sectioned": 0, "interleaved": 1, "per_axis": 2}


@pytest.fixture(scope="module")
def tsel():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attention_score_vision_gb300 as t
    t.build()
    t.load_library()
    return t


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _np(t):
    return t.detach().double().cpu().numpy()


def _table(tsel, sections, layout, base=1e6):
    f, a = tsel.tsel_rope_frequencies(base, sections, NAMES[layout])
    return tsel.tsel_rope_table(f, a), *O.rope_frequencies(base, sections, layout)


def _close_rotation(got, x, pos, f, a, adjacent, inverse, dtype):
    ref = O.rope(x, pos, f, a, adjacent, inverse)
    n = len(f)
    mag = np.abs(x).copy()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    both = mag[..., first] + mag[..., second]
    mag[..., first] = mag[..., second] = both
    tol = mag * 2.0 ** -21
    tol[..., 2 * n:] = 0
    tiny = float(torch.finfo(dtype).smallest_normal) * torch.finfo(dtype).eps / 2   # below the normal range
    tol += (np.abs(ref) + tol) * (_half(dtype) if dtype != FP else 0) + tiny
    assert np.all(np.abs(_np(got) - ref) <= tol)


# ------------------------------------------------------------------ rotation

ROPE = [
    # tokens, H, Hkv, d, sections, layout, dtype, adjacent, inverse
    (1, 1, 1, 64, [11, 11, 10], "interleaved", BF, False, False),
    (1, 16, 8, 128, [24, 20, 20], "interleaved", BF, False, False),
    (33, 4, 2, 80, [0, 20, 20], "per_axis", BF, False, False),
    (7, 3, 1, 72, [12, 12, 12], "sectioned", HF, False, True),       # pairs in halves of four
    (129, 2, 2, 96, [24, 24], "sectioned", FP, True, False),
    (50, 5, 1, 128, [16, 24, 24], "sectioned", FP, False, True),
    (19, 2, 1, 112, [10, 9, 9], "interleaved", BF, False, False),    # 28 of 56 pairs, the rest copied
    (19, 2, 1, 64, [7], "sectioned", FP, False, False),              # an odd count of pairs: single elements
    (19, 2, 1, 64, [5, 4, 4], "sectioned", BF, True, False),
    (5, 1, 0, 256, [128], "sectioned", BF, False, False),            # no K, the widest head
    (5, 3, 2, 248, [31, 31, 31, 31], "interleaved", HF, False, False),
    (6, 2, 1, 8, [1], "sectioned", BF, False, False),
    (40, 2, 1, 64, [32], "sectioned", HF, True, True),
    (3000, 12, 4, 80, [14, 13, 13], "interleaved", BF, False, False),
]


@pytest.mark.parametrize("case", ROPE, ids=[str(c[:4]) + c[5][:4] + str(c[6])[6:] for c in ROPE])
def test_rope_matches_the_oracle(tsel, case):
    T, H, Hkv, d, sections, layout, dtype, adjacent, inverse = case
    rng = np.random.default_rng(100 + T + d)
    table, f, a = _table(tsel, sections, layout)
    q = torch.from_numpy(rng.standard_normal((T, H, d))).to(dtype).cuda()
    k = torch.from_numpy(rng.standard_normal((T, Hkv, d))).to(dtype).cuda() if Hkv else None
    pos = rng.integers(-5000, 200000, (T, len(sections))).astype(np.int32)
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    flags = (tsel.TSEL_ROPE_ADJACENT if adjacent else 0) | (tsel.TSEL_ROPE_INVERSE if inverse else 0)
    qo, ko = tsel.tsel_rope(q, k, i32(pos), table, flags=flags, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    _close_rotation(qo, _np(q), pos, f, a, adjacent, inverse, dtype)
    if Hkv:
        _close_rotation(ko, _np(k), pos, f, a, adjacent, inverse, dtype)
    else:
        assert ko is None
    # in place gives the same bits
    q2, k2 = q.clone(), None if k is None else k.clone()
    tsel.tsel_rope(q2, k2, i32(pos), table, flags=flags, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))


def test_rope_far_positions_lose_nothing(tsel):
    table, f, a = _table(tsel, [11, 11, 10], "interleaved", base=1e4)
    pos = np.asarray([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1], [-1, 0, 1], [2 ** 24 + 1, 2 ** 25 + 3, -2 ** 29 + 7]], np.int32)
    x = np.random.default_rng(3).standard_normal((3, 2, 64))
    q = torch.from_numpy(x).to(FP).cuda()
    qo, _ = tsel.tsel_rope(q, None, i32(pos), table)
    _close_rotation(qo, _np(q), pos, f, a, False, False, FP)


def test_rope_strided_rows_and_empty(tsel):
    table, f, a = _table(tsel, [0, 20, 20], "per_axis")
    rng = np.random.default_rng(4)
    packed = torch.from_numpy(rng.standard_normal((21, 3 * 4 * 80))).to(BF).cuda()   # a packed QKV row
    q = packed[:, :320].unflatten(1, (4, 80))
    k = packed[:, 320:640].unflatten(1, (4, 80))
    pos = rng.integers(0, 64, (21, 3)).astype(np.int32)
    before = packed[:, 640:].clone()
    qo, ko = tsel.tsel_rope(q, k, i32(pos), table)
    _close_rotation(qo, _np(q), pos, f, a, False, False, BF)
    _close_rotation(ko, _np(k), pos, f, a, False, False, BF)
    tsel.tsel_rope(q, k, i32(pos), table, q_out=q, k_out=k)      # in place in the packed rows
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(packed[:, 640:], before)
    e, _ = tsel.tsel_rope(q[:0], k[:0], i32(pos[:0]).view(0, 3), table)
    assert e.shape == (0, 4, 80)


def test_rope_axis_without_positions_is_flagged_and_copied(tsel):
    table, f, a = _table(tsel, [8, 8, 16], "sectioned")
    q = torch.randn(5, 2, 64, device="cuda")
    pos = np.random.default_rng(1).integers(0, 99, (5, 2)).astype(np.int32)   # axis 2 is missing
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    qo, _ = tsel.tsel_rope(q, None, i32(pos), table, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_POSITIONS
    assert torch.equal(qo[..., 16:32], q[..., 16:32]) and torch.equal(qo[..., 48:], q[..., 48:])
    assert not torch.equal(qo[..., :16], q[..., :16])


def test_rope_inverse_is_the_gradient(tsel):
    """<g, R(x + h u)> differenced in fp64 against <R^-1(g), u>."""
    table, f, a = _table(tsel, [6, 5, 5], "interleaved", base=1e4)
    rng = np.random.default_rng(11)
    x, g, u = rng.standard_normal((3, 4, 2, 40))
    pos = rng.integers(0, 500, (4, 3)).astype(np.int32)
    gq = torch.from_numpy(g).to(FP).cuda()
    gi, _ = tsel.tsel_rope(gq, None, i32(pos), table, flags=tsel.TSEL_ROPE_INVERSE)
    h = 1e-3
    diff = (np.sum(_np(gq) * O.rope(x + h * u, pos, f, a)) - np.sum(_np(gq) * O.rope(x - h * u, pos, f, a))) / (2 * h)
    terms = np.abs(_np(gq)).sum() * np.abs(u).max() * 2
    assert abs(diff - np.sum(_np(gi) * u)) <= terms * 2.0 ** -20


# ------------------------------------------------------------------ cache

def _slots(rng, pages, ps, n):
    return rng.permutation(pages * ps)[:n].astype(np.int32)


def _poisoned(tsel, pages, ps, hkv, d):
    """A cache whose unwritten rows are NaN codes and NaN scales."""
    c = tsel.tsel_cache_new(pages, ps, hkv, d)
    for t in (c.k_pages, c.v_pages):
        t.fill_(0x7F)
    for t in (c.k_exps, c.v_exps):
        t.fill_(255)
    return c


def _cells(cache, slots, ps):
    s = torch.from_numpy(slots.astype(np.int64)).cuda()
    return [t[s // ps, :, s % ps].cpu().numpy() for t in cache]


CACHE = [(1, 1, 64, 16, BF), (1, 8, 128, 128, HF), (37, 2, 80, 16, BF), (130, 3, 96, 32, FP), (65, 5, 112, 64, HF), (513, 4, 128, 64, BF),
         (2000, 1, 64, 128, BF)]


@pytest.mark.parametrize("case", CACHE, ids=str)
def test_cache_write_is_exact_and_reads_back(tsel, case):
    T, hkv, d, ps, dtype = case
    rng = np.random.default_rng(7 * T + d)
    pages = -(-T // ps) + 3
    slots = _slots(rng, pages, ps, T)
    big = 8 if dtype == HF else 90
    x = [torch.from_numpy(rng.standard_normal((T, hkv, d)) * 2.0 ** rng.integers(-big, big, (T, hkv, 1))).to(dtype).cuda() for _ in range(2)]
    x[0][0, 0] = 0                                          # a row of zeros
    x[1][T // 2, hkv - 1, 1:] = 0                           # one nonzero element
    x[0][T - 1, hkv - 1, 3] = 448.0                         # the border of an exponent
    cache = _poisoned(tsel, pages, ps, hkv, d)
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    tsel.tsel_cache_write(x[0], x[1], i32(slots), cache, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    kc, vc, ke, ve = _cells(cache, slots, ps)
    for codes, exps, src in ((kc, ke, x[0]), (vc, ve, x[1])):
        c_ref, e_ref = O.quantise(_np(src))
        assert np.array_equal(exps, e_ref)
        assert np.array_equal(codes, c_ref)
    # nothing else was written
    rest = np.setdiff1d(np.arange(pages * ps), slots)
    for t, fill in zip(_cells(cache, rest, ps), (0x7F, 0x7F, 255, 255)):
        assert np.all(t == fill)
    for out in (FP, BF):
        for got, codes, exps in zip(tsel.tsel_cache_read(cache, i32(slots), dtype=out, workspace=ws), (kc, vc), (ke, ve)):
            ref = torch.from_numpy(O.dequantise(codes, exps)).to(out)
            assert torch.equal(got.cpu(), ref)
    assert tsel.tsel_read_device_status(ws) == 0


@pytest.mark.parametrize("d,sections,adjacent,dtype", [(128, [24, 20, 20], False, BF), (80, [20], False, HF), (80, [13, 13, 14], True, FP),
                                                       (64, [7], False, BF), (112, [9, 9], False, FP), (96, [16, 16, 16], True, BF),
                                                       (64, [16, 15], False, FP), (128, [2], False, BF)])
def test_cache_write_rotates_k_on_its_way(tsel, d, sections, adjacent, dtype):
    T, hkv, ps = 45, 3, 16
    rng = np.random.default_rng(d + len(sections))
    table, f, a = _table(tsel, sections, "sectioned", base=1e4)
    pos = rng.integers(0, 3000, (T, 3)).astype(np.int32)
    k, v = (torch.from_numpy(rng.standard_normal((T, hkv, d)) * 2.0 ** rng.integers(-5, 5, (T, hkv, 1))).to(dtype).cuda() for _ in range(2))
    slots = _slots(rng, 5, ps, T)
    cache = _poisoned(tsel, 5, ps, hkv, d)
    flags = tsel.TSEL_ROPE_ADJACENT if adjacent else 0
    tsel.tsel_cache_write(k, v, i32(slots), cache, pos=i32(pos), table=table, flags=flags)
    kr, vr = tsel.tsel_cache_read(cache, i32(slots), dtype=FP)
    assert torch.equal(vr.cpu(), torch.from_numpy(O.dequantise(*O.quantise(_np(v)))).float())
    ref = O.rope(_np(k), pos, f, a, adjacent)
    # half a code (2^-4 of the value, 2^-10 of the scale below the normal codes; the scale may be the
    # next one where the largest element is at the border) after an error of (|a| + |b|) 2^-21
    scale = 2.0 ** (O.quantise(ref)[1].astype(float) - 127)[..., None]
    slack = 2 * np.abs(_np(k)).max(-1, keepdims=True) * 2.0 ** -21
    tol = np.maximum((np.abs(ref) + slack) * 2.0 ** -4, 2 * scale * 2.0 ** -10) + slack
    assert np.all(np.abs(_np(kr) - ref) <= tol)
    # and the codes are those of the rotated rows wherever that row is not at a border
    n = len(f)
    same = _cells(cache, slots, ps)[0] == O.quantise(ref)[0]
    assert same.mean() > 0.999
    assert np.array_equal(_np(kr)[..., 2 * n:], O.dequantise(*O.quantise(ref))[..., 2 * n:])


def test_cache_skips_padding_and_flags_bad_slots_and_nan(tsel):
    cache = _poisoned(tsel, 3, 16, 2, 64)
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    k = torch.randn(6, 2, 64, device="cuda")
    v = torch.randn(6, 2, 64, device="cuda")
    slots = np.asarray([5, -1, 47, -2 ** 31, 0, 1], np.int32)
    tsel.tsel_cache_write(k, v, i32(slots), cache, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    kr, vr = tsel.tsel_cache_read(cache, i32(slots), dtype=FP, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    assert not kr[[1, 3]].any() and not vr[[1, 3]].any()
    assert torch.equal(kr[[0, 2, 4, 5]].cpu().double(), torch.from_numpy(O.dequantise(*O.quantise(_np(k)[[0, 2, 4, 5]]))))
    assert torch.isnan(tsel.tsel_cache_read(cache, i32([7]), dtype=FP)[0]).all()         # never written
    # a slot past the last page
    before = [t.clone() for t in cache]
    tsel.tsel_cache_write(k[:2], v[:2], i32([48, 2 ** 31 - 1]), cache, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_PAGES
    assert all(torch.equal(x, y) for x, y in zip(before, cache))
    tsel.tsel_clear_device_status(ws)
    kr, _ = tsel.tsel_cache_read(cache, i32([48, 5]), dtype=FP, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_PAGES
    assert not kr[0].any() and kr[1].any()
    # NaN and infinities
    tsel.tsel_clear_device_status(ws)
    k[0, 1, 9] = float("nan")
    v[1, 0, 0] = float("-inf")
    tsel.tsel_cache_write(k[:2], v[:2], i32([8, 9]), cache, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_NAN
    kr, vr = tsel.tsel_cache_read(cache, i32([8, 9, 8]), dtype=BF)
    assert torch.isnan(kr[0, 1]).all() and torch.isfinite(kr[0, 0]).all() and torch.isfinite(kr[1]).all()
    assert torch.isnan(vr[1, 0]).all() and torch.isfinite(vr[0]).all()
    assert torch.equal(kr[0, 0], kr[2, 0])                                               # the same slot twice


def test_cache_offsets_past_32_bits(tsel):
    """A pool of 4.8 GB of codes: the last page lies past 2^32 bytes."""
    pages, ps, hkv, d = 36800, 128, 8, 128
    cache = tsel.TselCache(*[torch.empty(pages, hkv, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2)],
                           *[torch.empty(pages, hkv, ps, dtype=torch.uint8, device="cuda") for _ in range(2)])
    slots = np.asarray([pages * ps - 1, 0, pages * ps - 128, 2 ** 22 + 5], np.int32)
    k, v = torch.randn(2, 4, hkv, d, device="cuda").unbind(0)
    tsel.tsel_cache_write(k, v, i32(slots), cache)
    kr, vr = tsel.tsel_cache_read(cache, i32(slots), dtype=FP)
    assert torch.equal(kr.cpu().double(), torch.from_numpy(O.dequantise(*O.quantise(_np(k)))))
    assert torch.equal(vr.cpu().double(), torch.from_numpy(O.dequantise(*O.quantise(_np(v)))))
    # attention over the last page
    q = torch.randn(1, hkv, d, device="cuda").to(BF)
    out, _ = tsel.tsel_prefix_attention(q, i32([0, 1]), 1, cache, None, None, 0, i32([[pages - 1]]), i32([1]), 128)
    s2 = np.asarray([(pages - 1) * ps], np.int32)
    _, v1 = tsel.tsel_cache_read(cache, i32(s2), dtype=BF)
    assert torch.equal(out[0], v1[0])                       # one key: its V


def test_attention_offsets_past_32_bits_with_many_rows(tsel):
    pages, ps, hkv, d = 36800, 128, 8, 128
    cache = tsel.TselCache(*[torch.empty(pages, hkv, ps, d, dtype=torch.uint8, device="cuda") for _ in range(2)],
                           *[torch.empty(pages, hkv, ps, dtype=torch.uint8, device="cuda") for _ in range(2)])
    slots = np.arange((pages - 1) * ps, (pages - 1) * ps + 100).astype(np.int32)
    k, v = torch.randn(2, 100, hkv, d, device="cuda").unbind(0)
    tsel.tsel_cache_write(k, v, i32(slots), cache)
    q = torch.randn(40, hkv, d, device="cuda").to(BF)
    out, lse = tsel.tsel_prefix_attention(q, i32([0, 40]), 40, cache, i32([pages - 1]), i32([100]), 128, None, None, 0)
    kr, vr = tsel.tsel_cache_read(cache, i32(slots), dtype=FP)
    ref, lref, av, mag = O.prefix_attention(_np(q), [0, 40], _np(kr), _np(vr), np.arange(100), [np.zeros(0, np.int64)], d ** -0.5)
    delta = d * 2.0 ** -23 * mag + 2.0 ** -22
    tol = av * (2 * delta[..., None] + 2.0 ** -11 + 2.0 ** -19) + 100 * 2.0 ** -31 * float(vr.abs().max())
    assert np.all(np.abs(_np(out) - ref) <= tol + (np.abs(ref) + tol) * 2.0 ** -8)
    assert np.all(np.abs(_np(lse) - lref) <= delta.T + 2.0 ** -20 + np.abs(lref) * 2.0 ** -22)


# ------------------------------------------------------------------ attention

class Batch:
    """A cache with a prefix and suffixes at random pages; unwritten rows are poisoned."""

    def __init__(self, tsel, seed, rows, lens, prefix, H, Hkv, d, ps, dtype, spread=2, k_rows=None, v_rows=None, pad=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.tsel, self.ps, self.H, self.Hkv, self.d, self.dtype = tsel, ps, H, Hkv, d, dtype
        self.R, self.prefix, self.lens = len(rows), prefix, list(lens)
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.max_q, self.max_s = max(list(rows) + [0]), max(list(lens) + [0])
        npg, spg = -(-prefix // ps), -(-self.max_s // ps)
        pages = npg + self.R * spg + 2
        order = rng.permutation(pages)
        self.prefix_pages = order[:npg].astype(np.int32)
        self.table = order[npg:npg + self.R * spg].reshape(self.R, spg).astype(np.int32)
        self.prefix_rows = (self.prefix_pages[np.arange(prefix) // ps] * ps + np.arange(prefix) % ps).astype(np.int64)
        self.suffix_rows = [(self.table[r][np.arange(n) // ps] * ps + np.arange(n) % ps).astype(np.int64) for r, n in enumerate(lens)]
        slots = np.concatenate([self.prefix_rows] + self.suffix_rows)
        n = len(slots)
        k, v = (rng.standard_normal((n, Hkv, d)) * 2.0 ** rng.integers(-spread, spread + 1, (n, Hkv, 1)) for _ in range(2))
        if k_rows is not None:
            k_rows(k)
        if v_rows is not None:
            v_rows(v)
        self.cache = _poisoned(tsel, pages, ps, Hkv, d)
        if n:
            tsel.tsel_cache_write(torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda(), i32(slots), self.cache)
        codes = [t.cpu().numpy() for t in self.cache]
        flat = lambda c: np.ascontiguousarray(np.moveaxis(c, 1, 2)).reshape((-1, Hkv) + c.shape[3:])   # noqa: E731
        self.k = O.dequantise(flat(codes[0]), flat(codes[2]))
        self.v = O.dequantise(flat(codes[1]), flat(codes[3]))
        T = int(self.cu[-1]) + pad
        self.q = torch.from_numpy(rng.standard_normal((T, H, d)) * qscale).to(dtype).cuda()

    def args(self, max_p=None, max_s=None):
        p = self.prefix if max_p is None else max_p
        s = self.max_s if max_s is None else max_s
        pages = self.prefix_pages
        if len(pages) * self.ps < p:        # room for a longer prefix: pages that do not exist must not be read
            pages = np.concatenate([pages, np.full(-(-p // self.ps) - len(pages), 2 ** 30)])
        table = self.table
        if table.shape[1] * self.ps < s:
            table = np.concatenate([table, np.full((self.R, -(-s // self.ps) - table.shape[1]), -7)], 1)
        return (i32(self.cu), self.max_q, self.cache, i32(pages), i32([self.prefix]), p, i32(table), i32(self.lens), s)

    def run(self, max_p=None, max_s=None, status=0, **kw):
        a = self.args(max_p, max_s)
        ws = torch.zeros(self.tsel.tsel_prefix_attention_workspace_size(self.R, self.q.shape[0], self.max_q, self.H, self.Hkv, self.d, a[5], a[8]),
                         dtype=torch.uint8, device="cuda")
        ws[1024:].fill_(0xFF)               # whatever an earlier call left there
        out, lse = self.tsel.tsel_prefix_attention(self.q, *a, workspace=ws, **kw)
        assert self.tsel.tsel_read_device_status(ws) == status
        return out, lse

    def check(self, out, lse, scale=None):
        s = self.d ** -0.5 if scale is None else scale
        T = int(self.cu[-1])
        ref, lref, av, mag = O.prefix_attention(_np(self.q)[:T], self.cu, self.k, self.v, self.prefix_rows, self.suffix_rows, s)
        delta = self.d * 2.0 ** -23 * mag + 2.0 ** -22
        vmax = np.nanmax(np.abs(self.v)) if np.isfinite(self.v).any() else 0.0
        n = self.prefix + max(self.lens + [0])
        tol = av * (2 * delta[..., None] + 2.0 ** -11 + 2.0 ** -19) + n * 2.0 ** -31 * vmax
        tol = tol + (np.abs(ref) + tol) * _half(self.dtype)
        got, gl = _np(out)[:T], _np(lse)[:, :T]
        fin = np.isfinite(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        bad = np.abs(got - ref)[fin] - tol[fin]
        assert bad.max(initial=-1) <= 0, (bad.max(), np.unravel_index(np.argmax(np.where(fin, np.abs(got - ref) - tol, -1)), ref.shape))
        ok = np.isfinite(lref)
        assert np.array_equal(np.isneginf(gl), np.isneginf(lref)) and np.array_equal(np.isnan(gl), np.isnan(lref))
        assert np.all(np.abs(gl - lref)[ok] <= (delta.T + 2.0 ** -20 + np.abs(np.where(ok, lref, 0)) * 2.0 ** -22)[ok])


ATT = [
    # rows, suffix lens, prefix, H, Hkv, d, page, type
    ([1], [1], 0, 1, 1, 64, 16, BF),
    ([1], [0], 1, 1, 1, 128, 16, BF),
    ([1], [5], 127, 2, 1, 128, 16, HF),
    ([1], [0], 128, 4, 2, 128, 64, BF),
    ([1, 1], [129, 17], 129, 4, 2, 80, 16, BF),
    ([1, 1, 1], [1, 128, 300], 1000, 8, 2, 96, 32, HF),
    ([3, 1, 7], [40, 1, 7], 333, 6, 2, 112, 128, BF),
    ([2, 0, 5, 1], [2, 50, 130, 0], 260, 5, 1, 64, 16, BF),
    ([9], [4], 70, 2, 2, 64, 32, HF),                    # more rows than suffix keys: the first rows see none of it
    ([4], [2], 0, 2, 1, 80, 16, BF),                     # ... and nothing at all
    ([130], [140], 200, 1, 1, 64, 16, BF),               # two row tiles, prefix and suffix
    ([40, 60], [45, 300], 515, 4, 1, 128, 64, BF),
    ([1] * 70, [1 + 3 * i for i in range(70)], 400, 4, 2, 64, 16, BF),
    ([1, 2], [33, 64], 150, 128, 1, 64, 16, HF),         # 128 query heads on one KV head
    ([1, 2], [33, 64], 150, 12, 4, 128, 16, BF),
    ([1, 3], [33, 64], 150, 7, 1, 80, 32, BF),           # heads that do not divide the tile
    ([300], [300], 0, 2, 1, 128, 128, HF),               # causal from the start
    ([1], [4000], 0, 1, 1, 64, 32, BF),                  # one row, split over many units
]


@pytest.mark.parametrize("case", ATT, ids=[str(i) for i in range(len(ATT))])
def test_attention_matches_the_oracle(tsel, case):
    rows, lens, prefix, H, Hkv, d, ps, dtype = case
    b = Batch(tsel, 50 + prefix + d, rows, lens, prefix, H, Hkv, d, ps, dtype)
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("max_p,max_s", [(1, 0), (5000, 3000), (9000, 9000)])
def test_attention_bounds_above_the_lengths(tsel, max_p, max_s):
    """The launch is cut for the bounds; chunks past the lengths are empty."""
    b = Batch(tsel, 3, [1, 4, 2], [20, 150, 2], 700 if max_p > 1 else 1, 4, 2, 128, 32, BF)
    out, lse = b.run(max_p=max_p, max_s=max(max_s, 150))
    b.check(out, lse)


@pytest.mark.parametrize("rows", [1, 90])
def test_attention_large_moving_logits(tsel, rows):
    """Logits that climb through the keys by hundreds (every tile moves the
    reference and rescales), and V rows whose scales grow and shrink by 2^16."""
    def climb(k):
        k[:, :, 0] = 0.4 * np.arange(len(k))[:, None]

    def grow(v):
        v *= 2.0 ** (16 * np.sin(np.arange(len(v)) / 60.0))[:, None, None]

    b = Batch(tsel, 9, [rows], [rows + 30], 900, 4, 2, 64, 16, BF, spread=0, k_rows=climb, v_rows=grow)
    with torch.no_grad():
        b.q[:, 0, 0] = 8.0                # one head climbs
        b.q[:, 1, 0] = -8.0               # one falls
    out, lse = b.run()
    b.check(out, lse)


def test_attention_scale_and_sink(tsel):
    def sink(k):
        k[0] *= 12.0

    b = Batch(tsel, 10, [1, 1], [10, 200], 2500, 8, 4, 128, 64, BF, k_rows=sink)
    for s in (0.01, 0.5):
        out, lse = b.run(softmax_scale=s)
        b.check(out, lse, scale=float(np.float32(s)))


def test_attention_widely_spread_scales(tsel):
    """K rows down to 2^-20 of their tile's largest, V rows down to 2^-18, keep their codes."""
    b = Batch(tsel, 12, [1, 2], [60, 90], 600, 4, 2, 96, 16, HF, spread=9)
    out, lse = b.run()
    b.check(out, lse)


def test_attention_nan_rows_reach_those_that_see_them(tsel):
    """NaN K and V of a drafted token, later ones in the same tile: earlier rows
    of the request and other requests stay finite."""
    def nan_at(i):
        def f(x):
            x[i, 0, 3] = np.nan
        return f

    for which in ("k_rows", "v_rows"):
        # suffix of request 0 starts at row 100; its 4 query rows see 17, 18, 19, 20 keys
        b = Batch(tsel, 13, [4, 1], [20, 20], 100, 4, 2, 64, 16, BF, **{which: nan_at(100 + 18)})
        T = b.q.shape[0]
        assert T == 5
        out, lse = b.run()
        got = torch.isnan(out).any(-1)
        want = torch.zeros(5, 4, dtype=torch.bool)
        want[2:4, :2] = True                              # rows that see key 18, heads of KV head 0
        assert torch.equal(got.cpu(), want), which
        assert torch.equal(torch.isnan(out).all(-1).cpu(), want)
        if which == "k_rows":
            assert torch.equal(torch.isnan(lse).T.cpu(), want)
        else:
            assert torch.isfinite(lse).all()
        b.k, b.v = np.nan_to_num(b.k), np.nan_to_num(b.v)
        keep = [0, 1, 4]
        ref, _, av, mag = O.prefix_attention(_np(b.q), b.cu, b.k, b.v, b.prefix_rows, b.suffix_rows, 0.125)
        tol = av * (2 * 64 * 2.0 ** -23 * mag[..., None] + 2.0 ** -10) + np.abs(ref) * 2.0 ** -8
        assert np.all(np.abs(_np(out) - ref)[keep] <= tol[keep] + 1e-9)


def test_attention_inf_and_nan_queries_stay_in_their_rows(tsel):
    b = Batch(tsel, 14, [1, 1, 1], [9, 9, 9], 200, 4, 2, 64, 16, BF)
    clean, lse0 = b.run()
    b.q[1, 2, 5] = float("nan")
    b.q[2, 0, 1] = float("inf")
    out, lse = b.run()
    touched = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    touched[1, 2] = touched[2, 0] = True
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[2, 1])
    assert torch.equal(out[~touched], clean[~touched]) and torch.equal(lse.T[~touched], lse0.T[~touched])
    assert not torch.isfinite(out[2, 0]).all()


def test_attention_strided_padded_and_partial_outputs(tsel):
    """Q and out as views of wider rows; rows past the last request are left as they are."""
    b = Batch(tsel, 15, [2, 1], [30, 7], 140, 4, 2, 80, 16, BF, pad=6)
    T = b.q.shape[0]
    wide = torch.full((T, 3 * 320), float("nan"), dtype=BF, device="cuda")
    wide[:3, :320] = b.q[:3].flatten(1)
    ref, lref = b.run()
    b.check(ref, lref)
    b.q = wide[:, :320].unflatten(1, (4, 80))
    buf = torch.full((T, 640), 7.0, dtype=BF, device="cuda")
    lse = torch.full((4, T), 9.0, device="cuda")
    out, _ = b.run(out=buf[:, 320:].unflatten(1, (4, 80)), lse=lse)
    assert torch.equal(out[:3], ref[:3]) and torch.equal(lse[:, :3], lref[:, :3])
    assert torch.all(buf[:, :320] == 7) and torch.all(buf[3:] == 7) and torch.all(lse[:, 3:] == 9)
    out, none = b.run(want_lse=False)
    assert none is None and torch.equal(out[:3], ref[:3])


def test_attention_empty_batches(tsel):
    b = Batch(tsel, 16, [2, 1], [30, 7], 140, 4, 2, 64, 16, BF)
    out, lse = tsel.tsel_prefix_attention(b.q[:0], i32([0]), 0, b.cache, i32(b.prefix_pages), i32([140]), 140, None, None, 0)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    # requests without rows, and neither prefix nor suffix
    buf = torch.full_like(b.q, 3.0)
    tsel.tsel_prefix_attention(b.q, i32([0, 0, 0]), 5, b.cache, i32(b.prefix_pages), i32([140]), 140, i32(b.table), i32([3, 4]), 32, out=buf)
    assert torch.all(buf == 3)
    out, lse = tsel.tsel_prefix_attention(b.q, i32(b.cu), 2, b.cache, None, None, 0, None, None, 0)
    assert not out.any() and torch.all(torch.isneginf(lse))
    # rows without a request's suffix see the prefix alone: a bound but no lengths
    out, lse = tsel.tsel_prefix_attention(b.q, i32(b.cu), 2, b.cache, i32(b.prefix_pages), i32([0]), 140, i32(b.table), i32([0, 0]), 30)
    assert not out.any() and torch.all(torch.isneginf(lse))


def test_attention_bad_lengths_and_pages_are_flagged(tsel):
    b = Batch(tsel, 17, [2, 1], [30, 7], 140, 4, 2, 64, 16, BF)
    cu, mq, cache, pp, pl, mp, pt, sl, ms = b.args()
    ws = torch.zeros(tsel.tsel_prefix_attention_workspace_size(2, 3, 2, 4, 2, 64, mp, ms), dtype=torch.uint8, device="cuda")

    def status(**kw):
        a = dict(cu=cu, mq=mq, pp=pp, pl=pl, pt=pt, sl=sl)
        a.update(kw)
        tsel.tsel_clear_device_status(ws)
        tsel.tsel_prefix_attention(b.q, a["cu"], a["mq"], cache, a["pp"], a["pl"], mp, a["pt"], a["sl"], ms, workspace=ws)
        return tsel.tsel_read_device_status(ws)

    assert status() == 0
    S, P = tsel.TSEL_DEV_SEQLENS, tsel.TSEL_DEV_PAGES
    for bad in ([0, 2, 4], [0, -1, 3], [1, 2, 3], [0, 3, 3], [0, 2, -2], [0, 2, 2 ** 30], [0, 3, 2]):
        assert status(cu=i32(bad)) & S, bad
    assert status(pl=i32([141])) & S and status(pl=i32([-1])) & S
    assert status(sl=i32([31, 7])) & S and status(sl=i32([30, -1])) & S
    bad_pp = b.prefix_pages.copy()
    bad_pp[3] = b.cache.k_pages.shape[0]
    assert status(pp=i32(bad_pp)) == P
    bad_pp[3] = -1
    assert status(pp=i32(bad_pp)) == P
    bad_pt = b.table.copy()
    bad_pt[0, 1] = 2 ** 30
    assert status(pt=i32(bad_pt)) == P
    bad_pt = b.table.copy()
    bad_pt[1, 1] = 2 ** 30                                  # past request 1's seven keys: never read
    assert status(pt=i32(bad_pt)) == 0


def test_attention_is_deterministic_and_runs_on_other_streams(tsel):
    b = Batch(tsel, 18, [1] * 9, [40 * i + 1 for i in range(9)], 3000, 8, 2, 128, 16, BF)
    out, lse = b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        o, l = b.run() if i % 2 else b.run(stream=side)
        side.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_attention_in_captured_graphs_that_share_a_workspace(tsel):
    """Two captured steps with one workspace, replayed in turn with lengths and
    rows changed in place between replays."""
    b = Batch(tsel, 19, [1, 1, 1], [40, 3, 77], 500, 4, 2, 64, 16, BF)
    cu, mq, cache, pp, pl, mp, pt, sl, ms = b.args()
    q = [b.q.clone(), b.q.flip(0).contiguous()]
    ws = torch.zeros(tsel.tsel_prefix_attention_workspace_size(3, 3, 1, 4, 2, 64, mp, ms), dtype=torch.uint8, device="cuda")
    tsel.tsel_prefix_attention(q[0], cu, 1, cache, pp, pl, mp, pt, sl, ms, workspace=ws)   # kernel attributes set before capture
    graphs, outs = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tsel.tsel_prefix_attention(x, cu, 1, cache, pp, pl, mp, pt, sl, ms, workspace=ws))
        graphs.append(g)
    for lens, prefix in (([40, 3, 77], 500), ([1, 0, 60], 500), ([40, 3, 77], 17), ([0, 0, 0], 0)):
        sl.copy_(i32(lens))
        pl.fill_(prefix)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert tsel.tsel_read_device_status(ws) == 0
        for x, (o, l) in zip(q, outs):
            eo, el = tsel.tsel_prefix_attention(x, cu, 1, cache, pp, pl, mp, pt, sl, ms)
            assert torch.equal(o, eo) and torch.equal(l, el)


WIDE = [
    # more than 32 rows of a KV head: 128-row products; suffixes of both kinds beside them
    ([33], [33], 513, 2, 2, 96, 64, HF),                 # one row more than the few-row kernel takes
    ([45, 1, 20], [300, 1, 45], 700, 3, 1, 64, 16, HF),  # three heads: 42 tokens to a tile
    ([50, 3], [64, 3], 1300, 4, 2, 80, 16, BF),
    ([64, 70], [64, 900], 900, 2, 1, 112, 128, BF),
    ([35], [500], 2100, 5, 1, 128, 32, HF),
    ([150], [150], 100, 1, 1, 96, 16, BF),               # causal within and across key tiles
    ([257], [257], 129, 1, 1, 80, 32, HF),               # three row tiles, the last of one row
    ([1, 300, 2], [5, 310, 2], 0, 7, 7, 64, 64, BF),     # no prefix
    ([1] * 40, [7] * 40, 1000, 4, 4, 128, 16, BF),       # prefix wide, suffixes of one row each
    ([5] * 9, [33 * i for i in range(9)], 300, 6, 2, 112, 16, HF),   # suffixes of 15 rows
    ([2, 1, 2], [90, 1, 30], 260, 10, 2, 96, 32, BF),    # prefix 25 rows, suffixes 10: two to a unit, both
    ([1, 1, 1], [90, 1, 30], 260, 10, 2, 80, 32, HF),    # prefix 15 rows, suffixes 5 in its launch
]


@pytest.mark.parametrize("case", WIDE, ids=[str(i) for i in range(len(WIDE))])
def test_attention_row_counts_of_both_kernels(tsel, case):
    rows, lens, prefix, H, Hkv, d, ps, dtype = case
    b = Batch(tsel, 90 + prefix + d, rows, lens, prefix, H, Hkv, d, ps, dtype)
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("rows", [7, 8, 9, 15, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("d,dtype", [(64, HF), (128, BF)])
def test_attention_around_the_row_limits(tsel, rows, d, dtype):
    b = Batch(tsel, 200 + rows, [rows], [rows + 40], 270, 2, 2, d, 16, dtype)
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("rows", [16, 17])
def test_attention_few_rows_over_a_long_prefix(tsel, rows):
    b = Batch(tsel, 230 + rows, [rows], [20], 17000, 1, 1, 64, 64, BF)
    out, lse = b.run()
    b.check(out, lse)


def test_attention_two_launches_of_the_few_row_kernel(tsel):
    """Prefix units of 16 rows, and suffixes with room for too many keys to join their launch."""
    b = Batch(tsel, 44, [1, 1, 1], [90, 1, 300], 260, 10, 2, 80, 32, HF)
    out, lse = b.run(max_s=25600)
    b.check(out, lse)


def _subset(b, out, lse, rows):
    """Checks some rows of a batch of one request without a suffix."""
    b.q, b.cu = b.q[rows], np.asarray([0, len(rows)], np.int32)
    b.check(out[rows], lse[:, rows])


def test_attention_chunks_of_the_longest_page_lists(tsel):
    """76 row-tile pairs over 16,384 keys in pages of 16: two chunks of 512 pages."""
    b = Batch(tsel, 31, [4864], [0], 16384, 4, 4, 64, 16, BF)
    out, lse = b.run()
    _subset(b, out, lse, [0, 127, 128, 255, 256, 2500, 4863])


def test_attention_over_a_million_keys(tsel):
    """More partial results to a row than one round of the joining warps takes."""
    b = Batch(tsel, 32, [33], [0], 8192 * 130, 1, 1, 64, 128, BF, qscale=3.0)
    out, lse = b.run()
    _subset(b, out, lse, [0, 13, 32])


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_smallest_scales(tsel, rows):
    """K and V rows whose scale is the least there is, 2^-127, under large queries."""
    def tiny(x):
        x *= 2.0 ** -122
        x[::3] *= 16.0

    b = Batch(tsel, 42, [rows], [rows + 50], 200, 4, 2, 64, 16, BF, spread=0, k_rows=tiny, qscale=2.0 ** 119)
    assert (b.cache.k_exps.cpu().numpy() == 0).any()
    out, lse = b.run()
    b.check(out, lse)

    def small(x):                                           # of one sign: outputs stay normal numbers
        x[:] = (1 + np.abs(x)) * 2.0 ** -121

    b = Batch(tsel, 43, [rows], [rows + 50], 200, 4, 2, 64, 16, BF, spread=0, v_rows=small)
    assert (b.cache.v_exps.cpu().numpy() == 0).any()
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("which", ["k_rows", "v_rows"])
def test_attention_nan_rows_with_many_rows(tsel, which):
    def nan_row(x):
        x[100 + 40, 0, 3] = np.nan

    # request 0: its row i sees 21 + i suffix keys, key 40 from i = 20 on
    b = Batch(tsel, 33, [40, 2], [60, 20], 100, 4, 2, 80, 16, BF, **{which: nan_row})
    out, lse = b.run()
    want = torch.zeros(42, 4, dtype=torch.bool)
    want[20:40, :2] = True
    assert torch.equal(torch.isnan(out).any(-1).cpu(), want) and torch.equal(torch.isnan(out).all(-1).cpu(), want)
    assert torch.equal(torch.isnan(lse).T.cpu(), want if which == "k_rows" else torch.zeros_like(want))
    b.k, b.v = np.nan_to_num(b.k), np.nan_to_num(b.v)
    ref, _, av, mag = O.prefix_attention(_np(b.q), b.cu, b.k, b.v, b.prefix_rows, b.suffix_rows, 80 ** -0.5)
    tol = av * (2 * 80 * 2.0 ** -23 * mag[..., None] + 2.0 ** -10) + np.abs(ref) * 2.0 ** -8 + 1e-9
    ok = ~want.numpy()
    assert np.all(np.abs(_np(out) - ref)[ok] <= tol[ok])


@pytest.mark.parametrize("rows", [[2, 1], [70, 2]])
def test_attention_bad_pages_reach_their_request_only(tsel, rows):
    b = Batch(tsel, 34, rows, [90, 20], 200, 4, 2, 64, 16, BF)
    out, lse = b.run()
    b.table[0, 2] = -5
    b.table[0, 4] = 2 ** 30
    got, gl = b.run(status=tsel.TSEL_DEV_PAGES)
    n = rows[0]
    assert torch.equal(got[n:], out[n:]) and torch.equal(gl[:, n:], lse[:, n:])
    assert torch.isfinite(got).all()                        # the pages' keys are zeros


def test_attention_into_q(tsel):
    for rows in ([3, 1], [60, 1]):
        b = Batch(tsel, 35, rows, [70, 9], 300, 4, 2, 128, 32, BF)
        out, lse = b.run()
        again, _ = b.run(out=b.q)
        assert again.data_ptr() == b.q.data_ptr() and torch.equal(again, out)


def test_calls_on_their_own_streams_at_once(tsel):
    """Calls that run beside one another, with workspaces and outputs that the
    calls allocate on the stream they are given."""
    made = []
    for i, rows in enumerate(([1] * 6, [90, 3], [4], [200])):
        b = Batch(tsel, 36 + i, rows, [60] * len(rows) if max(rows) < 60 else [300] * len(rows), 3000, 8, 2, 128, 16, BF)
        made.append((b, b.args(), b.run()))
    x = torch.randn(500, 8, 128, device="cuda").to(BF)
    pos = torch.arange(1000, dtype=torch.int32, device="cuda").view(500, 2)
    table, _, _ = _table(tsel, [32, 32], "sectioned")
    turned, _ = tsel.tsel_rope(x, None, pos, table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        got = []
        for st, (b, a, _) in zip(streams, made):
            handle = st if len(got) % 2 else st.cuda_stream
            y, _ = tsel.tsel_rope(x, None, pos, table, stream=handle)
            got.append((y, *tsel.tsel_prefix_attention(b.q, *a, stream=handle)))
        torch.cuda.synchronize()
        for (y, o, l), (b, _, (out, lse)) in zip(got, made):
            assert torch.equal(y, turned) and torch.equal(o, out) and torch.equal(l, lse)


def test_attention_graphs_of_many_rows(tsel):
    """A captured batch whose prefix takes the wide kernel and whose suffixes the
    few-row one, and one of two wide parts, replayed in turn in one workspace
    while lengths change in place."""
    made = []
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    for rows, lens in (([1] * 50, [5 * i for i in range(50)]), ([40, 60, 1], [50, 77, 1])):
        b = Batch(tsel, 40, rows, lens, 900, 4, 2, 96, 16, HF)
        a = b.args()
        tsel.tsel_prefix_attention(b.q, *a, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = tsel.tsel_prefix_attention(b.q, *a, workspace=ws)
        made.append((b, a, g, got, list(lens)))
    for prefix, cut in ((900, 0), (130, 3), (0, 10), (899, 0)):
        for b, a, g, got, lens in made:
            b.prefix, b.lens = prefix, [max(n - cut, 0) for n in lens]
            a[4].fill_(prefix)
            a[7].copy_(i32(b.lens))
        for b, a, g, got, lens in made:
            g.replay()
        torch.cuda.synchronize()
        assert tsel.tsel_read_device_status(ws) == 0
        for b, a, g, (out, lse), lens in made:
            o, l = tsel.tsel_prefix_attention(b.q, *a)
            assert torch.equal(o, out) and torch.equal(l, lse)
            full, rows_full = b.prefix_rows, b.suffix_rows
            b.prefix_rows, b.suffix_rows = full[:prefix], [r[:n] for r, n in zip(rows_full, b.lens)]
            b.check(out, lse)
            b.prefix_rows, b.suffix_rows = full, rows_full


def test_expanded_tensors_are_refused(tsel):
    b = Batch(tsel, 41, [1, 1], [9, 9], 40, 4, 2, 64, 16, BF)
    a = b.args()
    one = b.q[:1].expand(2, 4, 64)
    table, _, _ = _table(tsel, [32], "sectioned")
    for call in (lambda: tsel.tsel_prefix_attention(one, *a),
                 lambda: tsel.tsel_prefix_attention(b.q, *a, out=one),
                 lambda: tsel.tsel_rope(one, None, i32([[1], [2]]), table),
                 lambda: tsel.tsel_cache_write(one[:, :2], one[:, :2], i32([0, 1]), b.cache)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ together

def test_the_path_from_scoring_to_answers(tsel):
    """Rotate, score, select and compact image tokens with their positions; write
    their K and V rotated to the cache; let three users ask about them; score the
    cached keys again for one question."""
    rng = np.random.default_rng(77)
    T, H, Hkv, d, ps = 600, 4, 2, 64, 16
    cu = [0, 256, 400, 600]
    pos = np.stack([np.repeat([0, 1, 2], [256, 144, 200]), np.arange(T) // 16, np.arange(T) % 16], 1).astype(np.int32)
    mk = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(BF).cuda()   # noqa: E731
    q, k = mk(T, H, d), mk(T, H, d)
    vt, vf, va = _table(tsel, [0, 16, 16], "per_axis", 1e4)
    qr, kr = tsel.tsel_rope(q, k, i32(pos), vt)
    B = tsel.tsel_keep_count(T, 600)
    scores, _, keep, _ = tsel.tsel_score_select(qr, kr, i32(cu), i32(cu), 256, 256, i32([0, T]), i32([B]), B)
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)       # noqa: E731
    _, s_ref = oracle.importance(bits(qr), bits(kr), cu, cu)
    assert np.max(np.abs(scores.cpu().numpy() - s_ref) / s_ref) <= 2e-3
    hidden = mk(T, Hkv * d * 2)
    rows, kept_pos, _, _ = tsel.tsel_gather_compact(hidden, i32(pos), i32(cu), keep)
    assert torch.equal(rows, hidden[keep.long()]) and torch.equal(kept_pos, i32(pos)[keep.long()])
    # the language model's K and V of the kept tokens, rotated by their own positions
    lt, lf, la = _table(tsel, [12, 10, 10], "interleaved")
    npg, spg = -(-B // ps), 3
    order = rng.permutation(npg + 3 * spg).astype(np.int32)
    cache = _poisoned(tsel, len(order), ps, Hkv, d)
    slots = order[:npg][np.arange(B) // ps] * ps + np.arange(B) % ps
    kv = rows.view(B, 2, Hkv, d)
    tsel.tsel_cache_write(kv[:, 0], kv[:, 1], i32(slots), cache, pos=kept_pos, table=lt)
    # three users: 5 + 1 + 9 question tokens, written after the prefix and asked at once
    n = [5, 1, 9]
    qcu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    qt, kt, vt2 = mk(15, H, d), mk(15, Hkv, d), mk(15, Hkv, d)
    tpos = np.repeat((1000 + np.concatenate([np.arange(x) for x in n]))[:, None], 3, 1).astype(np.int32)
    table = order[npg:].reshape(3, spg)
    where = np.concatenate([table[r][np.arange(x) // ps] * ps + np.arange(x) % ps for r, x in enumerate(n)]).astype(np.int32)
    qq, _ = tsel.tsel_rope(qt, None, i32(tpos), lt)
    tsel.tsel_cache_write(kt, vt2, i32(where), cache, pos=i32(tpos), table=lt)
    out, lse = tsel.tsel_prefix_attention(qq, i32(qcu), 9, cache, i32(order[:npg]), i32([B]), B, i32(table), i32(n), spg * ps)
    # the oracle on the values that the cache stands for
    kc, vc = (np.zeros((len(order) * ps, Hkv, d)) for _ in range(2))
    every = np.concatenate([slots, where]).astype(np.int32)
    kb, vb = tsel.tsel_cache_read(cache, i32(every), dtype=FP)
    kc[every], vc[every] = _np(kb), _np(vb)
    ref_k = O.rope(_np(kv[:, 0]), kept_pos.cpu().numpy(), lf, la)
    assert np.all(np.abs(kc[slots] - ref_k) <= np.abs(ref_k) * 2.0 ** -4 + np.abs(ref_k).max(-1, keepdims=True) * 2.0 ** -14)
    ref, lref, av, mag = O.prefix_attention(_np(qq), qcu, kc, vc, slots, [where[qcu[r]:qcu[r + 1]] for r in range(3)], 0.125)
    tol = av * (2 * 64 * 2.0 ** -23 * mag[..., None] + 2.0 ** -10) + np.abs(ref) * 2.0 ** -8
    assert np.all(np.abs(_np(out) - ref) <= tol)
    assert np.all(np.abs(_np(lse) - lref) <= 64 * 2.0 ** -23 * mag.T + 2.0 ** -18 + np.abs(lref) * 2.0 ** -22)
    # the third question scores the cached keys
    kb16, _ = tsel.tsel_cache_read(cache, i32(slots))
    s2, _ = tsel.tsel_importance(qq[6:], kb16, i32([0, 9]), i32([0, B]), 9, B)
    _, s2_ref = oracle.importance(bits(qq[6:].contiguous()), bits(kb16), [0, 9], [0, B])
    assert np.max(np.abs(s2.cpu().numpy() - s2_ref) / s2_ref) <= 2e-3


def test_attention_reads_what_the_calls_before_it_wrote(tsel):
    """Decoding steps one right behind another: Q rotated in place, each
    request's last cached token overwritten, then attention whose prefix takes
    the wide kernel and whose suffixes the few-row one, all in the same memory.
    Without a pause, and from one graph, every step is what it is when each call
    is waited for."""
    R, steps = 48, 12
    b = Batch(tsel, 50, [1] * R, [20 + 3 * i for i in range(R)], 700, 8, 4, 128, 16, BF)
    a = b.args()
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(51)
    k, v = (torch.from_numpy(rng.standard_normal((steps, R, 4, 128))).to(BF).cuda() for _ in range(2))
    slots = i32([r[-1] for r in b.suffix_rows])
    pos = i32(rng.integers(0, 999, (R, 2)))
    table, _, _ = _table(tsel, [32, 32], "sectioned")
    q0 = b.q.clone()
    out, lse = (torch.empty((steps,) + s, dtype=t, device="cuda") for s, t in (((R, 8, 128), BF), ((8, R), FP)))

    def run(pause):
        b.q.copy_(q0)
        for i in range(steps):
            for call in (lambda: tsel.tsel_rope(b.q, None, pos, table, q_out=b.q, workspace=ws),
                         lambda: tsel.tsel_cache_write(k[i], v[i], slots, b.cache, workspace=ws),
                         lambda: tsel.tsel_prefix_attention(b.q, *a, out=out[i], lse=lse[i], workspace=ws)):
                call()
                if pause:
                    torch.cuda.synchronize()

    run(True)
    want = out.clone(), lse.clone()
    assert all(not torch.equal(out[i], out[i + 1]) for i in range(steps - 1))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(False)
    for again in (lambda: run(False), g.replay, lambda: run(False), g.replay):
        out.zero_()
        lse.zero_()
        again()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert tsel.tsel_read_device_status(ws) == 0


@pytest.mark.parametrize("rows,prefix", [([1], 300), ([1], 9000), ([2] * 40, 300), ([90], 9000)])
def test_attention_nan_row_under_far_larger_logits(tsel, rows, prefix):
    """A NaN V row makes NaN of every row that sees it, also where another chunk
    holds logits so much higher that its own chunk's weight is 0 in fp32."""
    def high(k):
        k[prefix - 1] = 40.0                   # q is positive: 40 * 64 * mean q / 8, some 250 above the rest
        k[:prefix - 1] = np.minimum(k[:prefix - 1], 1.0)

    def nan_row(v):
        v[3, 0, 7] = np.nan

    b = Batch(tsel, 60, rows, [n + 5 for n in rows], prefix, 4, 2, 64, 16, BF, spread=0, k_rows=high, v_rows=nan_row)
    b.q = b.q.abs() + 0.25
    out, lse = b.run()
    assert torch.isnan(out[:, :2]).all() and torch.isfinite(out[:, 2:]).all() and torch.isfinite(lse).all()
    b.check(out, lse)


@pytest.mark.parametrize("rows", [[1], [2] * 40])
def test_attention_nan_row_of_a_suffix_under_a_far_larger_prefix(tsel, rows):
    """... between a request's suffix and the prefix: the other requests stay finite."""
    def high(k):
        k[9] = 40.0
        k[300:] = np.minimum(k[300:], 1.0)

    def nan_row(v):
        v[300, 1, 0] = np.nan                  # the first suffix key of request 0

    b = Batch(tsel, 61, rows, [n + 5 for n in rows], 300, 4, 2, 64, 16, BF, spread=0, k_rows=high, v_rows=nan_row)
    b.q = b.q.abs() + 0.25
    out, lse = b.run()
    want = torch.zeros(len(b.q), 4, dtype=torch.bool)
    want[:rows[0], 2:] = True
    assert torch.equal(torch.isnan(out).any(-1).cpu(), want) and torch.isfinite(lse).all()


def _reread(b):
    """The batch's cache as values, after a test wrote to its pages itself."""
    codes = [t.cpu().numpy() for t in b.cache]
    flat = lambda c: np.ascontiguousarray(np.moveaxis(c, 1, 2)).reshape((-1, b.Hkv) + c.shape[3:])   # noqa: E731
    b.k, b.v = O.dequantise(flat(codes[0]), flat(codes[2])), O.dequantise(flat(codes[1]), flat(codes[3]))


def _at(b, slot):
    return int(slot) // b.ps, int(slot) % b.ps


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("which", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("where", ["prefix", "suffix"])
def test_attention_scale_byte_255_is_nan_whatever_the_codes(tsel, rows, which, where):
    """A visible row whose byte is 255 while its codes are ordinary ones makes NaN
    of the rows that see it, in both kernels, as the cache read has it."""
    b = Batch(tsel, 62, [rows, 2], [rows + 20, 30], 200, 4, 2, 64, 16, BF, spread=0)
    page, off = _at(b, b.prefix_rows[150] if where == "prefix" else b.suffix_rows[0][3])
    b.cache[2 + which][page, 1, off] = 255
    assert b.cache[which][page, 1, off].any()
    _reread(b)
    out, lse = b.run()
    b.check(out, lse)
    want = torch.zeros(rows + 2, 4, dtype=torch.bool)
    want[:None if where == "prefix" else rows, 2:] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want)
    assert torch.equal(torch.isnan(lse).T.cpu(), want if which == 0 else torch.zeros_like(want))
    got = tsel.tsel_cache_read(b.cache, i32([page * 16 + off]))[which]
    assert torch.isnan(got[0, 1]).all() and torch.isfinite(got[0, 0]).all()


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("byte", [247, 252, 253, 254])
def test_attention_largest_scale_bytes_of_v(tsel, rows, byte):
    """V rows of the largest scales, values of 2^118 to 2^126, beside ordinary ones."""
    b = Batch(tsel, 63, [rows], [rows + 20], 200, 4, 2, 64, 16, BF, spread=0)
    rng = np.random.default_rng(64)
    for slot in (b.prefix_rows[7], b.prefix_rows[160], b.suffix_rows[0][0]):
        page, off = _at(b, slot)
        b.cache.v_pages[page, :, off] = torch.from_numpy(rng.integers(1, 48, (2, 64)).astype(np.uint8)).cuda()   # 2^-9 to 0.47
        b.cache.v_exps[page, :, off] = byte
    _reread(b)
    out, lse = b.run()
    assert torch.isfinite(out).all() and (out[:, :, :].abs() > 2.0 ** (byte - 150)).any()
    b.check(out, lse)


@pytest.mark.parametrize("rows", [[4, 1], [40, 2]])
@pytest.mark.parametrize("code", [0x7F, 0xFF, 0x7E, 0x00])
def test_attention_hidden_rows_of_byte_255_never_reach(tsel, rows, code):
    """Drafted keys marked as NaN by their scale byte, whatever their codes (E4M3's
    NaN among them): rows of the request that do not see them stay as they were."""
    b = Batch(tsel, 65, rows, [n + 20 for n in rows], 100, 4, 2, 64, 16, BF, spread=1)
    clean, lse0 = b.run()
    n = rows[0]
    page, off = _at(b, b.suffix_rows[0][20 + n // 2])       # seen from row n // 2 on
    for t in b.cache[:2]:
        t[page, 0, off] = code
    for t in b.cache[2:]:
        t[page, 0, off] = 255
    _reread(b)
    out, lse = b.run()
    want = torch.zeros(len(b.q), 4, dtype=torch.bool)
    want[n // 2:n, :2] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)
    assert torch.equal(torch.isnan(lse).T.cpu(), want)
    b.check(out, lse)


@pytest.mark.parametrize("rows", [[4, 1], [40, 2]])
def test_attention_nan_codes_under_an_ordinary_byte(tsel, rows):
    """E4M3's NaN as a code, which the cache write never leaves: rows that see the
    key are NaN (in that column for V, whole for K). A K row reaches no others, a
    V row no other request, no other KV head and no other column."""
    for which in (0, 1):
        b = Batch(tsel, 66, rows, [n + 20 for n in rows], 100, 4, 2, 64, 16, BF, spread=1)
        clean, lse0 = b.run()
        n = rows[0]
        page, off = _at(b, b.suffix_rows[0][20 + n // 2])
        b.cache[which][page, 0, off, 5] = 0x7F
        out, lse = b.run()
        nan = torch.isnan(out).cpu()
        assert nan[n // 2:n, :2, 5].all()
        if which == 0:
            assert nan[n // 2:n, :2].all() and not nan[:n // 2].any() and not nan[n:].any() and not nan[:, 2:].any()
            hidden = torch.cat([out[:n // 2], out[n:]]).float(), torch.cat([clean[:n // 2], clean[n:]]).float()
            assert torch.allclose(*hidden, rtol=2.0 ** -6, atol=2.0 ** -6)
        else:
            assert torch.equal(out[n:], clean[n:]) and torch.equal(out[:n, 2:], clean[:n, 2:]) and torch.equal(lse, lse0)
            rest = torch.arange(64) != 5
            assert torch.equal(out[..., rest], clean[..., rest])


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("kexp,qexp", [(112, -110), (100, -100), (-100, 105)])
def test_attention_far_scales_of_k_and_q(tsel, rows, kexp, qexp):
    """Some K rows of 2^112 under queries of 2^-110: the logits are ordinary numbers
    although a product of codes and scale alone passes fp32's range; and the other way round."""
    def far(k):
        k[::3] *= 2.0 ** kexp

    b = Batch(tsel, 67, [rows], [rows + 40], 260, 4, 2, 64, 16, BF, spread=0, k_rows=far if kexp > 0 else lambda k: np.multiply(k, 2.0 ** kexp, out=k),
              qscale=2.0 ** qexp)
    out, lse = b.run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    b.check(out, lse)


@pytest.mark.parametrize("rows", [1, 40])
def test_attention_largest_scale_bytes_of_k(tsel, rows):
    b = Batch(tsel, 68, [rows], [rows + 20], 200, 4, 2, 64, 16, BF, spread=0, qscale=2.0 ** -114)
    rng = np.random.default_rng(69)
    for i, byte in ((7, 254), (60, 253), (160, 250), (199, 248)):
        page, off = _at(b, b.prefix_rows[i])
        codes = rng.integers(1, 8, (2, 64)) | np.where(rng.random((2, 64)) < 0.5, 128, 0)     # +-2^-9 to 2^-6.2
        b.cache.k_pages[page, :, off] = torch.from_numpy(codes.astype(np.uint8)).cuda()
        b.cache.k_exps[page, :, off] = byte
    _reread(b)
    out, lse = b.run()
    b.check(out, lse)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_small_angles_keep_their_bits(tsel, adjacent):
    """Sines and cosines alone (pairs (0, 1) and (1, 0)), relative to their own size:
    2^-24 for the phase as fp32, an ulp (2^-23) for the function, and the table's
    2^-61 of a turn per step of position (a frequency is rounded in two parts)."""
    for f, a in (O.rope_frequencies(1e6, [24, 20, 20], "interleaved"), O.rope_frequencies(1e4, [64, 0, 0], "sectioned"),
                 (np.asarray([1e-6, 1e-5, 3e-8, 1.3e-4, 6.283185, 3.1415927, 1.5707964, -1e-3]), np.zeros(8, np.int64))):
        table = tsel.tsel_rope_table(f.tolist(), a.tolist())
        n = len(f)
        pos = np.concatenate([np.arange(-8, 65), [1000, 4095, 65537, 10 ** 6, -10 ** 7]])[:, None].repeat(3, 1).astype(np.int32)
        x = np.zeros((len(pos), 2, 128), np.float32)
        first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
        x[:, 0, second] = 1                    # -> (-sin, cos)
        x[:, 1, first] = 1                     # -> (cos, sin)
        got, _ = tsel.tsel_rope(torch.from_numpy(x).cuda(), None, i32(pos), table, flags=tsel.TSEL_ROPE_ADJACENT if adjacent else 0)
        ref = O.rope(x, pos, f, a, adjacent)
        step = np.abs(pos[:, :1, None].astype(np.float64)) * 2 * np.pi * 2.0 ** -61
        assert np.all(np.abs(_np(got) - ref) <= np.abs(ref) * 4 * 2.0 ** -24 + step)


def test_rope_carries_gradients(tsel):
    """Where autograd records, the rotation is part of the graph: gradients of
    shared, expanded and partly needed inputs against the formula's, and through
    the backward pass itself."""
    table, f, a = _table(tsel, [6, 5, 5], "interleaved", base=1e4)
    rng = np.random.default_rng(70)
    x, y, gx, gy = (torch.from_numpy(rng.standard_normal((9, h, 40))).float().cuda() for h in (4, 2, 4, 2))
    pos = rng.integers(0, 500, (9, 3)).astype(np.int32)
    for flags, inverse in ((0, False), (tsel.TSEL_ROPE_INVERSE, True)):
        q, k = x.clone().requires_grad_(), y.clone().requires_grad_()
        qo, ko = tsel.tsel_rope(q, k, i32(pos), table, flags=flags)
        plain = tsel.tsel_rope(x, y, i32(pos), table, flags=flags)
        assert torch.equal(qo, plain[0]) and torch.equal(ko, plain[1]) and not plain[0].requires_grad
        ((qo * gx).sum() + (ko * gy).sum()).backward()
        _close_rotation(q.grad, _np(gx), pos, f, a, False, not inverse, FP)
        _close_rotation(k.grad, _np(gy), pos, f, a, False, not inverse, FP)
    q = x.clone().requires_grad_()
    qo, ko = tsel.tsel_rope(q, y, i32(pos), table)          # K needs none
    assert qo.requires_grad and not ko.requires_grad
    qo.sum().backward()                                     # an expanded gradient
    _close_rotation(q.grad, np.ones((9, 4, 40)), pos, f, a, False, True, FP)
    q.grad = None
    qo, none = tsel.tsel_rope(q, None, i32(pos), table)
    g, = torch.autograd.grad((qo ** 2).sum(), q, create_graph=True)
    assert none is None and torch.allclose(g, 2 * q, atol=1e-5)    # the rotation keeps lengths
    h, = torch.autograd.grad((g * gx).sum(), q)
    assert torch.allclose(h, 2 * gx, atol=1e-5)
    with torch.no_grad():
        assert not tsel.tsel_rope(q, None, i32(pos), table)[0].requires_grad


def test_rope_gradients_in_a_captured_graph(tsel):
    table, f, a = _table(tsel, [16, 16], "sectioned")
    rng = np.random.default_rng(71)
    pos = i32(rng.integers(0, 99, (7, 2)))
    q = torch.from_numpy(rng.standard_normal((7, 2, 64))).float().cuda().requires_grad_()
    g = torch.from_numpy(rng.standard_normal((7, 2, 64))).float().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            got, = torch.autograd.grad(tsel.tsel_rope(q, None, pos, table)[0], q, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, = torch.autograd.grad(tsel.tsel_rope(q, None, pos, table)[0], q, g)
    for seed in (1, 2):
        g.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((7, 2, 64))))
        graph.replay()
        want, _ = tsel.tsel_rope(g, None, pos, table, flags=tsel.TSEL_ROPE_INVERSE)
        assert torch.equal(out, want)


def test_autograd_notices_what_is_written_in_place(tsel):
    table, _, _ = _table(tsel, [32], "sectioned")
    x = torch.randn(3, 2, 64, device="cuda")
    w = torch.randn(3, 2, 64, device="cuda", requires_grad=True)
    pos = i32([[1], [2], [3]])
    for k in (None, x):
        saved = (w * x).sum()                               # keeps x for w's gradient
        q = x if k is None else torch.randn(3, 2, 64, device="cuda")
        tsel.tsel_rope(q, k, pos, table, q_out=q, k_out=k)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.backward()
    for call in (lambda: tsel.tsel_rope(w, None, pos, table, q_out=w),
                 lambda: tsel.tsel_rope(w, None, pos, table, q_out=x),
                 lambda: tsel.tsel_rope(x, w, pos, table, k_out=torch.empty_like(x)),
                 lambda: tsel.tsel_rope(x, None, pos, table, q_out=w * 1.0)):
        with pytest.raises(ValueError):
            call()
    b = Batch(tsel, 73, [2], [9], 40, 4, 2, 64, 16, BF)
    for name, shape in (("out", (2, 4, 64)), ("lse", (4, 2))):
        t = torch.ones(shape, dtype=BF if name == "out" else FP, device="cuda")
        saved = (torch.ones_like(t).requires_grad_() * t).sum()
        b.run(**{name: t})
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.backward()
    with torch.no_grad():
        tsel.tsel_rope(w, None, pos, table, q_out=w)        # as torch has it
    with torch.inference_mode():
        y = torch.randn(3, 2, 64, device="cuda")
        tsel.tsel_rope(y, None, pos, table, q_out=y)
    tsel.tsel_rope(y, None, pos, table, q_out=x)            # an inference tensor read outside


def test_attention_row_counts_past_their_bound_are_flagged(tsel):
    """More rows than num_req * max_seqlen_q: flagged also where no suffix kernel
    runs to look at the requests one by one."""
    b = Batch(tsel, 72, [2, 1], [30, 7], 140, 4, 2, 64, 16, BF)
    cu, mq, cache, pp, pl, mp, pt, sl, ms = b.args()
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")

    def status(*a):
        tsel.tsel_clear_device_status(ws)
        tsel.tsel_prefix_attention(b.q, *a, workspace=ws)
        return tsel.tsel_read_device_status(ws)

    S = tsel.TSEL_DEV_SEQLENS
    assert status(cu, 0, cache, pp, pl, mp, pt, sl, ms) == S          # suffixes, but no rows by the bound
    assert status(cu, 0, cache, pp, pl, mp, None, None, 0) == S
    assert status(cu, 1, cache, pp, pl, mp, None, None, 0) == S
    assert status(cu, 1, cache, None, None, 0, None, None, 0) == S
    assert status(i32([3]), 2, cache, pp, pl, mp, None, None, 0) == S   # rows of no request
    assert status(i32([0, 0, 0]), 0, cache, pp, pl, mp, pt, sl, ms) == 0
    assert status(cu, 2, cache, pp, pl, mp, None, None, 0) == 0
    assert status(i32([0]), 0, cache, pp, pl, mp, None, None, 0) == 0


@pytest.mark.parametrize("rows,prefix", [([1], 9000), ([1], 300), ([90], 9000)])
def test_attention_mean_past_fp32_under_far_larger_logits(tsel, rows, prefix):
    """V values that E4M3 rounds up to 2^128, in a chunk whose weight is 0: nothing
    of them is left, where 0 times the chunk's infinite mean would be NaN."""
    def high(k):
        k[prefix - 1] = 40.0
        k[:prefix - 1] = np.minimum(k[:prefix - 1], 1.0)

    def huge(v):
        v[:20, 0, 7] = float(torch.finfo(BF).max)

    b = Batch(tsel, 74, rows, [n + 5 for n in rows], prefix, 4, 2, 64, 16, BF, spread=0, k_rows=high, v_rows=huge)
    b.q = b.q.abs() + 0.25
    assert np.nanmax(b.v) == 2.0 ** 128
    out, lse = b.run()
    assert torch.isfinite(out).all()
    b.v[b.v > 1e30] = 0.0                      # their weight is e^-250: 2^-233 of an ordinary value
    b.check(out, lse)


@pytest.mark.parametrize("rows,prefix", [([1], 9000), ([2] * 20, 9000), ([90], 9000), ([1], 200)])
def test_attention_nan_key_among_keys_far_below(tsel, rows, prefix):
    """A NaN K row makes NaN of the log-sum-exp too, also where the partial results
    around it are far below others (eight, two and one warps to a row of the join)."""
    def high(k):
        k[prefix // 2] = 40.0
        k[:prefix // 2] = np.minimum(k[:prefix // 2], 1.0)
        k[prefix // 2 + 1:] = np.minimum(k[prefix // 2 + 1:], 1.0)
        k[nan_at, 1, 9] = np.nan

    for nan_at in (0, prefix // 3, prefix - 1):
        b = Batch(tsel, 75, rows, [n + 5 for n in rows], prefix, 4, 2, 64, 16, BF, spread=0, k_rows=high)
        b.q = b.q.abs() + 0.25
        out, lse = b.run()
        assert torch.isnan(out[:, 2:]).all() and torch.isnan(lse[2:]).all()
        assert torch.isfinite(out[:, :2]).all() and torch.isfinite(lse[:2]).all()
