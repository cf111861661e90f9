"""GPU: the prompt, tree and page operators together, as a serving program uses them:
prefill, scoring with the attention's log-sum-exps, pruning, the cache, forked
answers, drafted trees, accepted tokens moved together, pages given back."""
import numpy as np
import pytest
import torch

from gpu_util import i32
from oracle import cache_oracle as CO
from oracle import pages_oracle as PO

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def tsel():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import attention_score_vision_gb300 as t
    t.build()
    t.load_library()
    return t


def _np(t):
    return t.detach().double().cpu().numpy()


def test_from_prompt_to_accepted_drafts(tsel):
    rng = np.random.default_rng(11)
    H, Hkv, d, page, images = 4, 2, 64, 16, 3
    T, keep = 40 * images, 70
    draw = lambda n, h: torch.from_numpy(rng.standard_normal((n, h, d))).to(BF).cuda()
    # prefill of one request of three images; the scoring takes its log-sum-exps
    q, k, v = draw(T, H), draw(T, Hkv), draw(T, Hkv)
    cu = i32([40 * i for i in range(images + 1)])
    _, lse = tsel.tsel_prompt_attention(q, k, v, cu, cu, 40, 40)
    scores, _ = tsel.tsel_importance(q, k, cu, cu, 40, 40, flags=tsel.TSEL_IMP_LSE_PROVIDED, lse=lse)
    idx, cu_keep = tsel.tsel_select_topk(scores, i32([0, T]), i32([keep]), keep)
    # the whole prompt is cached, then pruned in its pages
    rows, width, pages = 4, 12, 40
    cache = tsel.tsel_cache_new(pages, page, Hkv, d)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")

    def resize(new):
        tsel.tsel_cache_resize(refs, table, lens, i32(new), page)

    def slots(row, positions):
        p = torch.as_tensor(positions, device="cuda")
        return (table[row].long()[p // page] * page + p % page).to(torch.int32)
    resize([T, -1, -1, -1])
    tsel.tsel_cache_write(k, v, slots(0, range(T)), cache)
    kept = tsel.tsel_cache_compact(cache, table[:1], idx, cu_keep, keep)
    assert kept.tolist() == [keep]
    resize([keep, -1, -1, -1])
    assert int(refs.sum()) == -(-keep // page)
    fresh = tsel.tsel_cache_new(pages, page, Hkv, d)
    tsel.tsel_cache_write(k[idx.long()], v[idx.long()], slots(0, range(keep)), fresh)
    for a, b in zip(tsel.tsel_cache_read(cache, slots(0, range(keep))), tsel.tsel_cache_read(fresh, slots(0, range(keep)))):
        assert torch.equal(a, b)
    # three answers start from it; each drafts a tree of its own
    tsel.tsel_cache_fork(cache, refs, table, lens, i32([0, 0, 0]), i32([1, 2, 3]))
    assert lens.tolist() == [keep] * 4
    nodes = [5, 1, 4]
    parents = [-1, 0, 0, 1, 3, -1, -1, -1, 1, 0]
    resize([-1] + [keep + n for n in nodes])
    kd, vd, qd = draw(sum(nodes), Hkv), draw(sum(nodes), Hkv), draw(sum(nodes), H)
    at = torch.cat([slots(r + 1, range(keep, keep + n)) for r, n in enumerate(nodes)])
    tsel.tsel_cache_write(kd, vd, at, cache)
    cu_n = i32([0, 5, 6, 10])
    out, _ = tsel.tsel_tree_attention(qd, cu_n, 5, i32(parents), cache, None, None, 0, table[1:], lens[1:], keep + 5)
    kv = [_np(t) for t in tsel.tsel_cache_read(cache, torch.arange(pages * page, dtype=torch.int32, device="cuda"), dtype=torch.float32)]
    for t in range(10):
        r = int(np.searchsorted([5, 6, 10], t, side="right"))
        first = [0, 5, 6][r]
        seen, i = list(range(keep)), t - first
        while i >= 0:
            seen.append(keep + i)
            i = parents[first + i]
        rows_ = slots(r + 1, seen).cpu().numpy()
        for h in range(H):
            ref, _, av, mag = CO.attention_row(_np(qd[t, h]), kv[0][rows_, h // 2], kv[1][rows_, h // 2], d ** -0.5)
            tol = av * (2.0 ** -22 * d * mag + 2.0 ** -11 + 2.0 ** -19) + (np.abs(ref) + av * 2.0 ** -10) * 2.0 ** -8
            assert np.all(np.abs(_np(out[t, h]) - ref) <= tol)
    # accepted: 0, 1, 3, 4 of the first tree, nothing of the second, 0 and 3 of the third
    accepted, cu_a = [0, 1, 3, 4, 0, 3], [0, 4, 4, 6]
    starts = lens[1:] - i32(nodes)
    new = tsel.tsel_cache_compact(cache, table[1:], i32(accepted), i32(cu_a), 4, starts=starts)
    assert new.tolist() == [keep + 4, keep, keep + 2]
    tsel.tsel_cache_resize(refs, table, lens, torch.cat([i32([-1]), new]), page)
    # one more token each: the same as from a cache that had the accepted tokens alone
    q1 = draw(3, H)
    got, _ = tsel.tsel_prefix_attention(q1, i32([0, 1, 2, 3]), 1, cache, None, None, 0, table[1:], lens[1:], keep + 5)
    plain = tsel.tsel_cache_new(3 * 6, page, Hkv, d)
    own = torch.arange(18, dtype=torch.int32, device="cuda").view(3, 6)
    for r, acc in enumerate(([0, 1, 3, 4], [], [0, 3])):
        src = [[0, 5, 6][r] + a for a in acc]
        kk, vv = torch.cat([k[idx.long()], kd[src]]), torch.cat([v[idx.long()], vd[src]])
        p = torch.arange(len(kk), device="cuda")
        tsel.tsel_cache_write(kk, vv, (own[r].long()[p // page] * page + p % page).to(torch.int32), plain)
    want, _ = tsel.tsel_prefix_attention(q1, i32([0, 1, 2, 3]), 1, plain, None, None, 0, own, new, keep + 5)
    assert torch.equal(got, want)
    # all end: every page is free again
    resize([0] * rows)
    assert not refs.any()


def test_a_step_of_drafts_in_a_captured_graph(tsel):
    """Tree attention, accepted tokens moved and pages given back, replayed with other lengths."""
    rng = np.random.default_rng(12)
    H, Hkv, d, page, R, n = 2, 1, 64, 16, 3, 6
    width, pages = 8, 30
    cache = tsel.tsel_cache_new(pages, page, Hkv, d)
    for t in cache[:2]:
        t.copy_(torch.from_numpy(rng.integers(0, 120, t.shape, dtype=np.uint8)))
    for t in cache[2:]:
        t.fill_(120)
    order = rng.permutation(pages)[:R * width].astype(np.int32).reshape(R, width)
    table, lens, refs = i32(order), i32([0] * R), torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[torch.from_numpy(order.ravel()).long().cuda()] = 1
    q, cu, parents = torch.from_numpy(rng.standard_normal((R * n, H, d))).to(BF).cuda(), i32([0, n, 2 * n, 3 * n]), i32([-1, 0, 0, 1, 2, 4] * R)
    starts, keep, cu_a, new = i32([0] * R), i32([0] * (R * n)), i32([0] * (R + 1)), i32([0] * R)
    out = torch.empty_like(q)
    ws = torch.zeros(max(tsel.tsel_tree_attention_workspace_size(R, R * n, n, H, Hkv, d, 0, width * page),
                         tsel.tsel_cache_resize_workspace_size(R, width)), dtype=torch.uint8, device="cuda")

    def step():
        tsel.tsel_tree_attention(q, cu, n, parents, cache, None, None, 0, table, lens, width * page, out=out, want_lse=False, workspace=ws)
        tsel.tsel_cache_compact(cache, table, keep, cu_a, n, starts=starts, new_lens=new, workspace=ws)
        tsel.tsel_cache_resize(refs, table, lens, new, page, workspace=ws)
    before = [t.clone() for t in cache]
    lens.copy_(i32([n] * R))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        for base, acc in (([30, 0, 100], [[0, 1, 3], [0], [0, 2, 4, 5]]), ([17, 90, 4], [[], [0, 2], [0, 1, 3]])):
            for t, b in zip(cache, before):
                t.copy_(b)
            host = [t.cpu().numpy().copy() for t in cache]
            counts = np.zeros(pages, np.int32)
            L = [b + n for b in base]
            for r in range(R):
                counts[order[r, :-(-L[r] // page)]] = 1
            refs.copy_(torch.from_numpy(counts))
            lens.copy_(i32(L))
            starts.copy_(i32(base))
            flat = sum(acc, [])
            c = [0]
            for a in acc:
                c.append(c[-1] + len(a))
            keep[:len(flat)].copy_(i32(flat))
            cu_a.copy_(i32(c))
            want, _ = tsel.tsel_tree_attention(q, cu, n, parents, cache, None, None, 0, table, lens, width * page)
            g.replay()
            s.synchronize()
            assert torch.equal(out, want)
            got = PO.compact(host, order, base, [0] * R, flat, c)
            lens_h = np.asarray(L)
            PO.resize(counts, order.copy(), lens_h, got, page)
            assert np.array_equal(lens.cpu().numpy(), got) and np.array_equal(refs.cpu().numpy(), counts)
            for t, h in zip(cache, host):
                assert np.array_equal(t.cpu().numpy(), h)
    assert tsel.tsel_read_device_status(ws) == 0
