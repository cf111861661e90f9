"""GPU: cached tokens moved together, pages shared, given out and back, against a
plain simulation. Everything here is moved or counted, so results are exact."""
import numpy as np
import pytest
import torch

from gpu_util import i32
from oracle import pages_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsel():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attention_score_vision_gb300 as t
    t.build()
    t.load_library()
    return t


def _cache(tsel, rng, pages, page, Hkv, d):
    """A cache of random bytes and its host copy."""
    host = [rng.integers(0, 256, (pages, Hkv, page, d), dtype=np.uint8) for _ in range(2)]
    host += [rng.integers(0, 256, (pages, Hkv, page), dtype=np.uint8) for _ in range(2)]
    return tsel.TselCache(*[torch.from_numpy(a.copy()).cuda() for a in host]), host


def _same(cache, host):
    for a, b in zip(cache, host):
        assert np.array_equal(a.cpu().numpy(), b)


def _ws(tsel, n=1024):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


COMPACT = [
    # kept counts, page, Hkv, d, start, span of positions, in place
    ([1], 16, 1, 64, 0, 1, True),
    ([0, 3, 0], 16, 2, 80, 7, 20, True),
    ([6, 1, 4, 6], 64, 8, 128, 100, 32, True),
    ([400], 16, 8, 128, 0, 700, True),              # one request: few CTAs, many chunks
    ([900, 2, 333], 32, 1, 96, 5, 1100, True),
    ([57] * 40, 128, 3, 112, 130, 64, True),
    ([700, 1, 0, 250], 16, 4, 128, 3, 900, False),
    ([1500], 64, 1, 64, 0, 1501, False),
    ([5], 32, 40, 128, 0, 8, False),                # more heads than a CTA takes
    ([33, 33], 32, 40, 128, 1, 40, True),
    ([1300], 16, 1, 64, 0, 5000, True),
    ([2500], 128, 2, 80, 11, 2500, True),           # nothing moves
]


@pytest.mark.parametrize("case", COMPACT, ids=[str(i) for i in range(len(COMPACT))])
def test_compact(tsel, case):
    counts, page, Hkv, d, start, span, in_place = case
    rng = np.random.default_rng(len(counts) * 1000 + page + d)
    R = len(counts)
    starts = np.asarray([start + r for r in range(R)], np.int32)
    bases = np.asarray([1000 * r for r in range(R)], np.int32)
    keep = np.concatenate([np.sort(rng.permutation(span)[:n]) + b for n, b in zip(counts, bases)]).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    width = -(-(start + R + span) // page)
    order = rng.permutation(2 * R * width + 2).astype(np.int32)
    table = order[:R * width].reshape(R, width)
    to = None if in_place else order[R * width:2 * R * width].reshape(R, width)
    cache, host = _cache(tsel, rng, len(order), page, Hkv, d)
    ws = _ws(tsel)
    lens = tsel.tsel_cache_compact(cache, i32(table), i32(keep), i32(cu), max(counts), starts=i32(starts), bases=i32(bases),
                                   dst_table=None if to is None else i32(to), workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    want = O.compact(host, table, starts, bases, keep, cu, to)
    assert np.array_equal(lens.cpu().numpy(), want)
    _same(cache, host)


def test_compact_chains_of_moves_in_place(tsel):
    """Every token's destination is the next one's source: the hardest order."""
    rng = np.random.default_rng(5)
    n, page = 3000, 16
    width = -(-(n + 1) // page)
    table = rng.permutation(width).astype(np.int32)[None]
    for Hkv, d in ((1, 64), (8, 128)):
        cache, host = _cache(tsel, rng, width, page, Hkv, d)
        keep = np.arange(1, n + 1, dtype=np.int32)
        tsel.tsel_cache_compact(cache, i32(table), i32(keep), i32([0, n]), n)
        O.compact(host, table, [0], [0], keep, [0, n])
        _same(cache, host)


def test_compact_flags_and_skips(tsel):
    rng = np.random.default_rng(6)
    page, width = 16, 4
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    cache, host = _cache(tsel, rng, 12, page, 2, 64)
    ws = _ws(tsel)
    bits = lambda: (tsel.tsel_read_device_status(ws), tsel.tsel_clear_device_status(ws))[0]

    def call(keep, cu, most=8, starts=None, table=table):
        return tsel.tsel_cache_compact(cache, i32(table), i32(keep), i32(cu), most, starts=None if starts is None else i32(starts), workspace=ws)
    # not ascending: the second of the equal two is skipped, the others move
    call([1, 3, 3, 9], [0, 0, 4, 4])
    assert bits() == tsel.TSEL_DEV_KEEP_IDX
    for p, k in ((1, 0), (3, 1), (9, 3)):
        for a in host:
            a[4, :, k] = a[4, :, p]
    _same(cache, host)
    # past the pages, and below its own place
    call([63, 64], [0, 0, 0, 2])
    assert bits() == tsel.TSEL_DEV_KEEP_IDX
    for a in host:
        a[8, :, 0] = a[11, :, 15]
    _same(cache, host)
    call([-1], [0, 1, 1, 1])
    assert bits() == tsel.TSEL_DEV_KEEP_IDX
    # counts that are no counts
    for cu, most in (([0, 2, 1, 1], 8), ([1, 1, 1, 1], 8), ([0, 5, 5, 5], 4), ([0, 0, 0, 3], 8)):
        call([1, 2], cu, most)
        assert bits() & tsel.TSEL_DEV_REQUESTS
    call([0], [0, 1, 1, 1], starts=[-1, 0, 0])
    assert bits() & tsel.TSEL_DEV_REQUESTS
    call([0], [0, 1, 1, 1], starts=[64, 0, 0])
    assert bits() & tsel.TSEL_DEV_REQUESTS
    torch.cuda.synchronize()
    # pages that are none
    bad = table.copy()
    bad[0, 1], bad[1, 2] = -3, 12
    before = [a.clone() for a in cache]
    call([20, 40], [0, 1, 2, 2], table=bad)
    assert bits() == tsel.TSEL_DEV_PAGES
    for a, b in zip(cache, before):
        assert torch.equal(a, b)


def test_compact_of_nothing(tsel):
    rng = np.random.default_rng(7)
    cache, host = _cache(tsel, rng, 2, 16, 1, 64)
    lens = tsel.tsel_cache_compact(cache, i32([[0], [1]]), i32([]), i32([0, 0, 0]), 0, starts=i32([3, 9]))
    assert lens.tolist() == [3, 9]
    assert tsel.tsel_cache_compact(cache, i32(np.zeros((0, 1))), i32([]), i32([0]), 0).numel() == 0
    _same(cache, host)


# ------------------------------------------------------------------ pages

def _state(rng, rows, width, pages, page, lens):
    """Rows that hold pages of their own."""
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((rows, width), -1, np.int32)
    refs, at = np.zeros(pages, np.int32), 0
    for r, n in enumerate(lens):
        k = -(-n // page)
        table[r, :k] = order[at:at + k]
        refs[order[at:at + k]] = 1
        at += k
    return table, refs, np.asarray(lens, np.int32)


@pytest.mark.parametrize("rows,width,pages,page", [(1, 3, 5, 16), (7, 20, 150, 32), (300, 9, 20000, 128), (1500, 4, 3000, 16), (3, 5000, 40000, 16)])
def test_resize(tsel, rows, width, pages, page):
    rng = np.random.default_rng(rows + pages)
    some = min(width, pages // (2 * rows))
    table, refs, lens = _state(rng, rows, width, pages, page, rng.integers(0, some * page + 1, rows).tolist())
    dev = [i32(x) for x in (refs, table, lens)]
    ws = _ws(tsel, tsel.tsel_cache_resize_workspace_size(rows, width))
    for step in range(6):
        new = rng.integers(-1 if step else 0, width * page + 1 if step % 2 else some * page + 1, rows).astype(np.int32)
        new[rng.random(rows) < 0.3] = -1
        tsel.tsel_cache_resize(dev[0], dev[1], dev[2], i32(new), page, workspace=ws)
        ok = O.resize(refs, table, lens, new, page)
        assert tsel.tsel_read_device_status(ws) == (0 if ok else tsel.TSEL_DEV_PAGES)
        tsel.tsel_clear_device_status(ws)
        for a, b in zip(dev, (refs, table, lens)):
            assert np.array_equal(a.cpu().numpy(), b)
    tsel.tsel_cache_resize(dev[0], dev[1], dev[2], i32(np.zeros(rows)), page, workspace=ws)
    assert not dev[0].any() and not dev[2].any()


def test_resize_flags(tsel):
    refs, table, lens = i32([1, 0, 0, 1]), i32([[0, -1], [3, 9]]), i32([16, 32])
    ws = _ws(tsel, tsel.tsel_cache_resize_workspace_size(2, 2))
    tsel.tsel_cache_resize(refs, table, lens, i32([33, -1]), 16, workspace=ws)   # past the row
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_REQUESTS
    tsel.tsel_clear_device_status(ws)
    assert lens.tolist() == [16, 32] and refs.tolist() == [1, 0, 0, 1]
    tsel.tsel_cache_resize(refs, table, lens, i32([-1, 0]), 16, workspace=ws)    # page 9 is none
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_PAGES
    tsel.tsel_clear_device_status(ws)
    assert lens.tolist() == [16, 0] and refs.tolist() == [1, 0, 0, 0]
    lens.fill_(16)
    tsel.tsel_cache_resize(refs, table, lens, i32([-1, 0]), 16, workspace=ws)    # page 3 is free already
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_PAGES
    assert refs.tolist() == [1, 0, 0, 0]


@pytest.mark.parametrize("lens,children,page,Hkv,d", [([1], 1, 16, 1, 64), ([48, 17, 0, 160], 3, 16, 2, 80), ([1370] * 5, 9, 64, 8, 128), ([127, 129, 128], 40, 128, 3, 96)])
def test_fork_grow_and_end(tsel, lens, children, page, Hkv, d):
    rng = np.random.default_rng(len(lens) + children + page)
    P = len(lens)
    kids = P * children
    width = -(-(max(lens) + 2 * page) // page)
    pages = sum(-(-n // page) for n in lens) + 4 * kids
    table, refs, lens = _state(rng, P + kids, width, pages, page, lens + [0] * kids)
    cache, host = _cache(tsel, rng, pages, page, Hkv, d)
    parents = np.asarray([i % P for i in range(kids)], np.int32)
    kid = np.arange(P, P + kids, dtype=np.int32)
    dev = [i32(x) for x in (refs, table, lens)]
    ws = _ws(tsel, tsel.tsel_cache_resize_workspace_size(P + kids, width))

    def check():
        assert tsel.tsel_read_device_status(ws) == 0
        _same(cache, host)
        for a, b in zip(dev, (refs, table, lens)):
            assert np.array_equal(a.cpu().numpy(), b)
    tsel.tsel_cache_fork(cache, *dev, i32(parents), i32(kid), workspace=ws)
    O.fork(host, refs, table, lens, parents, kid)
    check()
    new = np.where(np.arange(P + kids) < P, -1, lens + rng.integers(0, 2 * page, P + kids)).astype(np.int32)
    tsel.tsel_cache_resize(*dev, i32(new), page, workspace=ws)
    assert O.resize(refs, table, lens, new, page)
    check()
    new = np.where(np.arange(P + kids) % 2 == 0, 0, -1).astype(np.int32)     # some parents end before their children
    tsel.tsel_cache_resize(*dev, i32(new), page, workspace=ws)
    O.resize(refs, table, lens, new, page)
    check()
    tsel.tsel_cache_resize(*dev, i32(np.zeros(P + kids)), page, workspace=ws)
    assert not dev[0].any()


def test_fork_refuses_and_runs_out(tsel):
    rng = np.random.default_rng(9)
    table, refs, lens = _state(rng, 5, 3, 6, 16, [20, 32, 0, 0, 0])      # two free pages
    cache, host = _cache(tsel, rng, 6, 16, 1, 64)
    dev = [i32(x) for x in (refs, table, lens)]
    ws = _ws(tsel, tsel.tsel_cache_resize_workspace_size(5, 3))
    bits = lambda: (tsel.tsel_read_device_status(ws), tsel.tsel_clear_device_status(ws))[0]

    def unchanged():
        _same(cache, host)
        for a, b in zip(dev, (refs, table, lens)):
            assert np.array_equal(a.cpu().numpy(), b)
    for parents, children in (([5], [2]), ([-1], [2]), ([0], [5]), ([0], [1]), ([0], [0]), ([2], [2])):
        tsel.tsel_cache_fork(cache, *dev, i32(parents), i32(children), workspace=ws)
        assert bits() == tsel.TSEL_DEV_REQUESTS
        unchanged()
    # the same child twice: the second is refused; a child that is a parent too: refused
    tsel.tsel_cache_fork(cache, *dev, i32([1, 0]), i32([2, 2]), workspace=ws)
    assert bits() == tsel.TSEL_DEV_REQUESTS
    O.fork(host, refs, table, lens, [1], [2])
    unchanged()
    tsel.tsel_cache_fork(cache, *dev, i32([3, 1]), i32([3, 4]), workspace=ws)
    assert bits() == tsel.TSEL_DEV_REQUESTS
    O.fork(host, refs, table, lens, [1], [4])
    unchanged()
    # three children, two pages
    table, refs, lens = _state(rng, 5, 3, 6, 16, [20, 32, 0, 0, 0])
    dev = [i32(x) for x in (refs, table, lens)]
    tsel.tsel_cache_fork(cache, *dev, i32([0, 0, 0]), i32([2, 3, 4]), workspace=ws)
    assert bits() == tsel.TSEL_DEV_PAGES
    O.fork(host, refs, table, lens, [0, 0, 0], [2, 3, 4])
    assert lens.tolist() == [20, 32, 20, 20, 0]
    unchanged()


def _dev_state(tsel, rng, rows, width, pages, page, lens):
    """Rows with pages of their own (counts, table, lengths), here and on the device, and a workspace."""
    table, refs, lens = _state(rng, rows, width, pages, page, lens)
    host = [refs, table, lens]
    return host, [i32(x) for x in host], _ws(tsel, tsel.tsel_cache_resize_workspace_size(rows, width))


def _status(tsel, ws):
    bits = tsel.tsel_read_device_status(ws)
    tsel.tsel_clear_device_status(ws)
    return bits


def _equal(dev, host):
    for a, b in zip(dev, host):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("parents,children", [([0, 0, 0], [5, 3, 5]), ([0, 0, 5], [5, 3, 6]), ([1, 0, 1, 0], [2, 6, 4, 6]),
                                              ([0, 1, 6, 0], [3, 6, 4, 7]), ([0, 0, 1], [2, 99, 5]), ([0, 1, 0], [-4, 2, 2])])
def test_fork_lists_out_of_order(tsel, parents, children):
    """An entry that is not above all those before it is refused, and a parent is found among the children
    whatever the order."""
    rng = np.random.default_rng(22)
    host, dev, ws = _dev_state(tsel, rng, 8, 4, 30, 16, [40, 33, 0, 0, 0, 0, 0, 0])
    cache, bytes_ = _cache(tsel, rng, 30, 16, 2, 64)
    tsel.tsel_cache_fork(cache, *dev, i32(parents), i32(children), workspace=ws)
    assert _status(tsel, ws) == tsel.TSEL_DEV_REQUESTS
    good = O.good_forks(host[2], parents, children)
    assert 0 < sum(good) < len(good)
    O.fork(bytes_, *host, [p for p, g in zip(parents, good) if g], [c for c, g in zip(children, good) if g])
    _equal(dev, host)
    _same(cache, bytes_)


def test_fork_lists_out_of_order_in_many_rows(tsel):
    """Lists longer than a round of the planning CTA."""
    rng = np.random.default_rng(23)
    page, rows, pages = 16, 5000, 12000
    host, dev, ws = _dev_state(tsel, rng, rows, 3, pages, page, [int(n) for n in rng.integers(0, 40, 50)] + [0] * (rows - 50))
    cache, bytes_ = _cache(tsel, rng, pages, page, 1, 64)
    children = np.sort(rng.permutation(np.arange(50, rows))[:3500]).astype(np.int32)
    parents = rng.integers(0, 50, 3500).astype(np.int32)
    some = rng.permutation(3500)[:60]
    children[some[:30]] += rng.integers(-60, 60, 30).astype(np.int32)   # out of order; an early one may reach rows that hold tokens
    parents[some[30:]] = rng.integers(-1, rows + 1, 30)      # some of them children
    good = np.asarray(O.good_forks(host[2], parents, children))
    assert 30 < good.sum() < 3500
    tsel.tsel_cache_fork(cache, *dev, i32(parents), i32(children), workspace=ws)
    assert _status(tsel, ws) == tsel.TSEL_DEV_REQUESTS
    O.fork(bytes_, *host, parents[good], children[good])
    _equal(dev, host)
    _same(cache, bytes_)


def test_growth_behind_a_shared_page_is_refused(tsel):
    """What is written behind a row's length must not land in a page that another row holds too."""
    rng = np.random.default_rng(20)
    page, rows, width, pages = 16, 6, 5, 24
    host, dev, ws = _dev_state(tsel, rng, rows, width, pages, page, [40, 0, 0, 20, 0, 0])
    cache, bytes_ = _cache(tsel, rng, pages, page, 2, 64)

    def resize(new, bits=0):
        tsel.tsel_cache_resize(*dev, i32(new), page, workspace=ws)
        ok = O.resize(*host, new, page)
        assert _status(tsel, ws) == bits and ok
        _equal(dev, host)

    def fork(parents, children):
        tsel.tsel_cache_fork(cache, *dev, i32(parents), i32(children), workspace=ws)
        O.fork(bytes_, *host, parents, children)
        assert _status(tsel, ws) == 0
        _equal(dev, host)
        _same(cache, bytes_)
    fork([0, 0], [1, 2])                                     # pages 0 and 1 of row 0 are held three times
    resize([-1, 24, -1, -1, -1, -1])                         # row 1 rolls back into the second of them: read only
    assert host[2].tolist() == [40, 24, 40, 20, 0, 0]
    for then in (25, 32, 33, 80):                            # row 3 grows in the same calls
        was = host[2][3]
        resize([-1, then, -1, was + 9, -1, -1], tsel.TSEL_DEV_REQUESTS)
        assert host[2][1] == 24 and host[2][3] == was + 9
    resize([-1, 24, -1, -1, -1, -1])                         # the length that it has
    resize([-1, 17, -1, -1, -1, -1])                         # further back
    resize([20, -1, -1, -1, -1, -1])                         # the parent as well
    resize([21, -1, -1, -1, -1, -1], tsel.TSEL_DEV_REQUESTS)
    # a fork copies the rows in use: that row can grow and be written, no other sees it
    fork([1], [4])
    resize([-1, 0, -1, -1, 30, -1])
    at = [int(host[1][4, p // page]) * page + p % page for p in range(17, 30)]
    k = torch.from_numpy(rng.standard_normal((13, 2, 64))).to(torch.bfloat16).cuda()
    before = [a[host[1][2, :3]].copy() for a in bytes_]
    tsel.tsel_cache_write(k, k, i32(at), cache, workspace=ws)
    for a, b in zip(cache, before):
        assert np.array_equal(a.cpu().numpy()[host[1][2, :3]], b)
    bytes_ = [a.cpu().numpy() for a in cache]
    # at a whole page's end a row gets a page of its own
    resize([16, -1, -1, -1, -1, -1])
    resize([19, -1, -1, -1, -1, -1])
    # counts when the call begins decide: row 2 gives back what row 5 holds too, row 5 grows one call later
    fork([2], [5])
    resize([-1, -1, -1, -1, -1, 18])
    resize([-1, -1, 0, -1, -1, 19], tsel.TSEL_DEV_REQUESTS)
    assert host[2][2] == 0 and host[2][5] == 18
    resize([-1, -1, -1, -1, -1, 19])
    resize([0] * rows)
    assert not dev[0].any()


def test_growth_behind_shared_pages_in_many_rows(tsel):
    rng = np.random.default_rng(21)
    page, rows, width, pages, parents = 16, 1500, 6, 20000, 40
    host, dev, ws = _dev_state(tsel, rng, rows, width, pages, page, [int(n) for n in rng.integers(1, 80, parents)] + [0] * (rows - parents))
    cache, bytes_ = _cache(tsel, rng, pages, page, 1, 64)
    src, kids = rng.integers(0, parents, rows - parents).astype(np.int32), np.arange(parents, rows, dtype=np.int32)
    tsel.tsel_cache_fork(cache, *dev, i32(src), i32(kids), workspace=ws)
    O.fork(bytes_, *host, src, kids)
    _equal(dev, host)
    refused = []
    for _ in range(6):
        new = rng.integers(-1, width * page + 1, rows).astype(np.int32)
        refused.append(O.shared_end(*host, new, page).sum())
        tsel.tsel_cache_resize(*dev, i32(new), page, workspace=ws)
        assert O.resize(*host, new, page) and _status(tsel, ws) == (tsel.TSEL_DEV_REQUESTS if refused[-1] else 0)
        _equal(dev, host)
    assert refused[0] == 0 and max(refused) > 10             # a fork's own last page can be written
    tsel.tsel_cache_resize(*dev, i32([0] * rows), page, workspace=ws)
    assert not dev[0].any()


def test_lengths_of_refused_requests(tsel):
    """-1, which tsel_cache_resize takes as a row to leave alone, also in a length tensor of the call's own."""
    rng = np.random.default_rng(24)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    for to in (None, table + 12):
        cache, host = _cache(tsel, rng, 24, 16, 2, 64)
        for starts, keep, cu, most, want in (([9, -1, 5], [1, 2], [0, 1, 1, 2], 8, [10, -1, 6]), ([0, 0, 0], [1, 2, 3], [0, 1, 3, 3], 1, [1, -1, 0]),
                                             ([64, 60, 0], [0, 0], [0, 0, 2, 1], 8, [64, 62, -1]), ([62, 0, 0], [0, 1, 2], [0, 3, 3, 9], 8, [-1, 0, -1])):
            ws = _ws(tsel)
            for given in (None, torch.full((3,), 77, dtype=torch.int32, device="cuda")):
                new = tsel.tsel_cache_compact(cache, i32(table), i32(keep), i32(cu), most, starts=i32(starts), new_lens=given,
                                              dst_table=None if to is None else i32(to), workspace=ws)
                assert new.tolist() == want and _status(tsel, ws) & tsel.TSEL_DEV_REQUESTS


def test_overlapping_lengths(tsel):
    """Results among the inputs are refused; lengths that stay, and tensors side by side, are taken."""
    rng = np.random.default_rng(25)
    cache, host = _cache(tsel, rng, 12, 16, 1, 64)
    both = i32([3, 4, 5, 6])
    table = i32(np.arange(12).reshape(3, 4))
    for kw in (dict(starts=both[:3], new_lens=both[1:]), dict(bases=both[1:], new_lens=both[1:]), dict(bases=both[1:], new_lens=both[:3]),
               dict(new_lens=table[1, :3])):
        with pytest.raises(tsel.TselError, match="overlap"):
            tsel.tsel_cache_compact(cache, table, i32([0, 1, 2]), i32([0, 1, 2, 3]), 1, **kw)
    buf = i32([0] * 6)
    new = tsel.tsel_cache_compact(cache, table, i32([0, 0, 0]), i32([0, 1, 2, 3]), 1, starts=buf[:3], new_lens=buf[3:])
    assert new.tolist() == [1, 1, 1]
    _same(cache, host)
    # a table whose rows leave room for the lengths between them
    state = torch.zeros(3, 8, dtype=torch.int32, device="cuda")
    state[:, :4] = table
    new = tsel.tsel_cache_compact(cache, state[:, :4], i32([0, 0, 0]), i32([0, 1, 2, 3]), 1, new_lens=state[1, 4:7])
    assert new.tolist() == [1, 1, 1] and torch.equal(state[:, :4], table)
    refs, lens = i32([1] * 12), i32([64, 64, 64])
    tsel.tsel_cache_resize(refs, table, lens, lens, 16)      # every row keeps its length
    assert lens.tolist() == [64] * 3 and refs.tolist() == [1] * 12


def test_pools_past_32_bits_of_bytes(tsel):
    """Pages whose bytes lie past 2^32: moved in place and elsewhere, copied by a fork, given out and back."""
    rng = np.random.default_rng(26)
    page, Hkv, d, pages = 128, 8, 128, 40000                 # 5.2 GB of codes in K and in V
    free = torch.cuda.mem_get_info()[0]
    if free < 14 << 30:
        pytest.skip("needs 14 GB")
    cache = tsel.TselCache(*[torch.zeros(pages, Hkv, page, *x, dtype=torch.uint8, device="cuda") for x in ([d], [d], [], [])])
    rows, width, lens = 3, 4, [500, 300, 0]
    order = (pages - 1 - rng.permutation(12)).astype(np.int32)
    first = int(order.min())                                 # the last twelve pages, from `first` on
    host = [rng.integers(0, 256, (12, Hkv, page, *x), dtype=np.uint8) for x in ([d], [d], [], [])]
    for t, a in zip(cache, host):
        t[first:] = torch.from_numpy(a).cuda()
    table = np.full((rows, width), -1, np.int32)
    table[0], table[1, :3] = order[:4], order[4:7]
    refs = np.ones(pages, np.int32)                          # the free pages lie at the end
    refs[order[7:]] = 0
    state = [refs, table, np.asarray(lens, np.int32)]
    dev = [i32(x) for x in state]
    small = lambda: [refs[first:], np.where(table < 0, table, table - first), state[2]]   # noqa: E731
    ws = _ws(tsel, tsel.tsel_cache_resize_workspace_size(rows, width))

    def check():
        assert _status(tsel, ws) == 0
        _equal(dev, state)
        for t, a in zip(cache, host):
            assert np.array_equal(t[first:].cpu().numpy(), a)
            assert not bool(t[:first:997].any())
    # in place, and to two of the free pages
    keep, cu = np.sort(rng.permutation(500)[:333]).astype(np.int32), [0, 333]
    tsel.tsel_cache_compact(cache, dev[1][:1], i32(keep), i32(cu), 333, workspace=ws)
    O.compact(host, small()[1][:1], [0], [0], keep, cu)
    check()
    keep, cu, to = np.sort(rng.permutation(300)[:200]).astype(np.int32), [0, 200], order[None, 8:10]
    tsel.tsel_cache_compact(cache, dev[1][1:2], i32(keep), i32(cu), 200, dst_table=i32(to), workspace=ws)
    O.compact(host, small()[1][1:2], [0], [0], keep, cu, to - first)
    check()
    tsel.tsel_cache_fork(cache, *dev, i32([0]), i32([2]), workspace=ws)
    s = small()
    O.fork(host, *s, [0], [2])
    table[:] = np.where(s[1] < 0, s[1], s[1] + first)
    check()
    for new in ([-1, 0, 512], [0, -1, 0]):
        tsel.tsel_cache_resize(*dev, i32(new), page, workspace=ws)
        assert O.resize(*state, new, page)
        check()


@pytest.mark.parametrize("Hkv,d,page", [(4, 112, 32), (1, 112, 16), (8, 80, 128), (3, 96, 64)])
def test_compact_long_and_short_requests_in_place(tsel, Hkv, d, page):
    """Requests of many chunks beside ones that stop in their first, second or third."""
    rng = np.random.default_rng(27)
    counts = [4000, 3, 1700, 0, 130, 900, 2600, 64]
    R, span = len(counts), 5000
    starts = np.asarray([7 * r for r in range(R)], np.int32)
    keep = np.concatenate([np.sort(rng.permutation(span if r % 2 == 0 else 2 * n + 1)[:n]) for r, n in enumerate(counts)]).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    width = -(-(span + 7 * R) // page)
    table = rng.permutation(R * width).astype(np.int32).reshape(R, width)
    cache, host = _cache(tsel, rng, R * width, page, Hkv, d)
    ws = _ws(tsel)
    for _ in range(2):                                       # the second call moves what the first one left behind
        lens = tsel.tsel_cache_compact(cache, i32(table), i32(keep), i32(cu), max(counts), starts=i32(starts), workspace=ws)
        assert tsel.tsel_read_device_status(ws) == 0
        assert np.array_equal(lens.cpu().numpy(), O.compact(host, table, starts, [0] * R, keep, cu))
        _same(cache, host)
