"""GPU: attention of drafted trees over the cache against the fp64 oracle.

Tolerances as for attention over a shared prefix: with A = sum_j p_j |v_j| and delta
the error of a logit (fp32 sums of d products, 2^-23 of their absolute sum each, at
most d of them), out is within A * (2 delta + 2^-11 + 2^-19) (probabilities in fp16;
exp2, sums, joining) plus n * 2^-31 max|v| (probabilities below fp16's range) plus half
a step of the output; lse within delta + 2^-20 + |lse| 2^-22."""
import numpy as np
import pytest
import torch

from gpu_util import i32
from oracle import cache_oracle as O

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


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


def _tree(rng, n, shape):
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "roots":
        return [-1] * n
    if shape == "star":
        return [-1] + [0] * (n - 1)
    return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]


class Batch:
    """A cache, a shared prefix and requests whose last keys are their trees'."""

    def __init__(self, tsel, seed, nodes, own, prefix, H, Hkv, d, page, dtype, shape="any"):
        rng = np.random.default_rng(seed)
        R = len(nodes)
        self.H, self.Hkv, self.d, self.dtype = H, Hkv, d, dtype
        self.nodes, self.lens = nodes, [a + b for a, b in zip(nodes, own)]
        self.max_nodes, self.prefix, self.max_suffix = max(nodes, default=0), prefix, max(self.lens, default=0)
        width, pw = -(-max(1, self.max_suffix) // page), -(-max(1, prefix) // page)
        order = rng.permutation(R * width + pw + 2).astype(np.int32)
        self.table, self.prefix_pages = order[pw:pw + R * width].reshape(R, width), order[:pw]
        k, v = (torch.from_numpy(rng.standard_normal((len(order) * page, Hkv, d)) * 2.0 ** rng.integers(-3, 4, (len(order) * page, Hkv, 1))).float().cuda()
                for _ in range(2))
        self.cache = tsel.tsel_cache_new(len(order), page, Hkv, d)
        slots = torch.arange(len(order) * page, dtype=torch.int32, device="cuda")
        tsel.tsel_cache_write(k, v, slots, self.cache)
        self.k, self.v = (_np(t) for t in tsel.tsel_cache_read(self.cache, slots, dtype=torch.float32))
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.q = torch.from_numpy(rng.standard_normal((int(self.cu[-1]), H, d))).to(dtype).cuda()
        self.parents = sum([_tree(rng, n, shape) for n in nodes], [])
        self.slot = lambda pages, j: pages[j // page] * page + j % page

    def rows(self, r, i):
        """Slots that node i of request r sees."""
        n, m = self.nodes[r], self.lens[r]
        seen = list(range(m - n))
        up = []
        while i >= 0:
            up.append(m - n + i)
            i = self.parents[self.cu[r] + i]
        return [self.slot(self.prefix_pages, j) for j in range(self.prefix)] + [self.slot(self.table[r], j) for j in seen + up[::-1]]

    def call(self, tsel, ws=None, **kw):
        pre = (i32(self.prefix_pages), i32([self.prefix]), self.prefix) if self.prefix else (None, None, 0)
        return tsel.tsel_tree_attention(self.q, i32(self.cu), self.max_nodes, i32(self.parents), self.cache, *pre,
                                        i32(self.table), i32(self.lens), self.max_suffix, workspace=ws, **kw)

    def close(self, out, lse):
        half = torch.finfo(self.dtype).eps / 2
        G = self.H // self.Hkv
        vmax = np.abs(self.v).max()
        out, lse = _np(out), _np(lse)
        for r, n in enumerate(self.nodes):
            for i in range(n):
                rows, t = self.rows(r, i), self.cu[r] + i
                for h in range(self.H):
                    ref, ref_lse, av, mag = O.attention_row(_np(self.q[t, h]), self.k[rows, h // G], self.v[rows, h // G], self.d ** -0.5)
                    delta = 2.0 ** -23 * self.d * mag
                    tol = av * (2 * delta + 2.0 ** -11 + 2.0 ** -19) + len(rows) * 2.0 ** -31 * vmax
                    tol += (np.abs(ref) + tol) * half + (2.0 ** -25 if self.dtype is HF else 0)
                    assert np.all(np.abs(out[t, h] - ref) <= tol), (r, i, h)
                    assert abs(lse[h, t] - ref_lse) <= delta + 2.0 ** -20 + abs(ref_lse) * 2.0 ** -22


CASES = [
    # nodes, own keys before the tree, prefix, H, Hkv, d, page, dtype, shape
    ([1], [0], 0, 1, 1, 64, 16, BF, "any"),
    ([8], [13], 0, 2, 1, 128, 16, BF, "any"),
    ([5, 0, 7, 1], [140, 3, 0, 16], 200, 4, 2, 80, 32, HF, "any"),        # 8 rows a unit
    ([16, 9], [300, 17], 130, 2, 2, 128, 64, BF, "any"),                   # 16 rows a unit
    ([16, 15, 3], [100, 50, 250], 0, 8, 4, 112, 16, HF, "any"),            # 32 rows: two units of 16
    ([33], [95], 77, 1, 1, 96, 128, BF, "any"),                            # the wide kernel, a tree over two tiles
    ([64, 40], [70, 0], 150, 4, 1, 128, 16, BF, "any"),
    ([64], [40], 0, 1, 1, 64, 32, HF, "chain"),
    ([64, 64], [63, 65], 0, 2, 1, 80, 16, BF, "roots"),
    ([61, 2, 17], [333, 5, 120], 300, 3, 1, 128, 64, HF, "star"),          # three heads: 126 rows a tile
    ([12], [2000], 0, 1, 1, 128, 16, BF, "any"),                           # chunks, the tree at the end of the last
    ([13], [1], 0, 2, 2, 64, 16, BF, "chain"),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_matches_the_oracle(tsel, case):
    b = Batch(tsel, 50 + sum(case[0]), *case)
    ws = torch.zeros(tsel.tsel_tree_attention_workspace_size(len(b.nodes), int(b.cu[-1]), b.max_nodes, b.H, b.Hkv, b.d, b.prefix, b.max_suffix),
                     dtype=torch.uint8, device="cuda")
    out, lse = b.call(tsel, ws)
    assert tsel.tsel_read_device_status(ws) == 0
    b.close(out, lse)
    again, lse2 = b.call(tsel, ws)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("nodes,H,Hkv", [([4, 8, 1], 2, 2), ([16, 3], 2, 1), ([40, 64], 2, 1)])
def test_a_chain_gives_the_prefix_attention_bit_for_bit(tsel, nodes, H, Hkv):
    b = Batch(tsel, 3, nodes, [100] * len(nodes), 140, H, Hkv, 128, 16, BF, "chain")
    out, lse = b.call(tsel)
    out2, lse2 = tsel.tsel_prefix_attention(b.q, i32(b.cu), b.max_nodes, b.cache, i32(b.prefix_pages), i32([b.prefix]), b.prefix,
                                            i32(b.table), i32(b.lens), b.max_suffix)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("nodes,H", [([8], 1), ([16], 1), ([16], 2), ([64], 2)])
def test_hidden_nodes_never_reach_a_row(tsel, nodes, H):
    """Rows of NaN (scale byte 255) in keys and values of a node reach its descendants only."""
    b = Batch(tsel, 8, nodes, [21], 0, H, 1, 64, 16, BF)
    n = nodes[0]
    poisoned = n // 2
    slot = int(b.slot(b.table[0], b.lens[0] - n + poisoned))
    clean, _ = b.call(tsel)
    for exps in (b.cache.k_exps, b.cache.v_exps):
        old = exps[slot // 16, 0, slot % 16].clone()
        exps[slot // 16, 0, slot % 16] = 255
        out, _ = b.call(tsel)
        exps[slot // 16, 0, slot % 16] = old
        for i in range(n):
            sees = slot in b.rows(0, i)
            assert bool(torch.isnan(out[i]).all()) == sees and (sees or torch.equal(out[i], clean[i]))


def test_bad_trees_are_flagged(tsel):
    for nodes, H in (([6], 1), ([40], 1)):
        b = Batch(tsel, 9, nodes, [30], 0, H, 1, 64, 16, BF)
        ws = torch.zeros(tsel.tsel_tree_attention_workspace_size(1, nodes[0], nodes[0], H, 1, 64, 0, b.max_suffix), dtype=torch.uint8, device="cuda")
        for at, parent in ((3, 3), (2, 5), (1, -2), (0, 0), (4, 1 << 30)):
            good, b.parents[at] = b.parents[at], parent
            out, lse = b.call(tsel, ws)
            assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_PARENTS
            tsel.tsel_clear_device_status(ws)
            b.parents[at] = -1        # what it is taken for
            b.close(out, lse)
            b.parents[at] = good
        # fewer keys than nodes
        out, _ = tsel.tsel_tree_attention(b.q, i32(b.cu), nodes[0], i32(b.parents), b.cache, None, None, 0, i32(b.table), i32([nodes[0] - 1]),
                                          b.max_suffix, workspace=ws)
        assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_SEQLENS


@pytest.mark.parametrize("nodes,prefix,H", [([5, 3], 0, 2), ([5, 3], 200, 1), ([40, 9], 30, 2)])
def test_padding_rows_and_given_results(tsel, nodes, prefix, H):
    """Rows past the last request are left alone, their parents are not read as a tree, and
    results may go to q itself."""
    b = Batch(tsel, 21, nodes, [33, 50], prefix, H, 1, 64, 16, BF)
    clean, clean_lse = b.call(tsel)
    n = b.q.shape[0]
    q = torch.cat([b.q, torch.full_like(b.q[:7], float("nan"))])
    parents = i32(list(b.parents) + [99] * 7)
    out, lse = torch.full_like(q, 3.0), torch.full((H, n + 7), 4.0, device="cuda")
    ws = torch.zeros(tsel.tsel_tree_attention_workspace_size(2, n + 7, b.max_nodes, H, 1, 64, prefix, b.max_suffix), dtype=torch.uint8, device="cuda")
    pre = (i32(b.prefix_pages), i32([prefix]), prefix) if prefix else (None, None, 0)
    for target in (out, q):
        tsel.tsel_tree_attention(q, i32(b.cu), b.max_nodes, parents, b.cache, *pre, i32(b.table), i32(b.lens), b.max_suffix, out=target,
                                 lse=lse, workspace=ws)
        assert tsel.tsel_read_device_status(ws) == 0
        b.close(target[:n], lse[:, :n])
    assert bool((out[n:] == 3).all()) and bool((lse[:, n:] == 4).all()) and bool(torch.isnan(q[n:]).all())
    b.close(clean, clean_lse)


def test_trees_on_two_streams_at_once(tsel):
    b = Batch(tsel, 22, [16, 9, 30], [300, 40, 7], 150, 2, 2, 80, 32, HF)
    want, _ = b.call(tsel)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [b.call(tsel, stream=s)[0] for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
