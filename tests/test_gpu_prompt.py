"""GPU: attention over whole prompts against the fp64 oracle.

Tolerances. With A = sum_j p_j |v_j| (columnwise), h half a step of the type (bf16
2^-8, fp16 2^-11, relative) and delta the error of a logit (an fp32 sum of d
products, 2^-23 of their absolute sum each, at most d of them): a probability is
within delta + h (rounded to the type) + 2^-20 (exp2, sums, joining), so out is within
A * (2 delta + h + 2^-19), plus n * 2^-31 max|v| in fp16 for probabilities below its
range (its smallest step, 2^-24, halved, against 2^6 at the row's reference, which is
at most its maximum), plus h of the output; lse within delta + 2^-20 + |lse| 2^-22."""
import numpy as np
import pytest
import torch

from gpu_util import i32
from oracle import prompt_oracle as O

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


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _close(out, lse, q, k, v, cu_q, cu_k, scale, causal, dtype):
    ref, ref_lse, av, mag = O.prompt_attention(_np(q), _np(k), _np(v), cu_q, cu_k, scale, causal)
    half = torch.finfo(dtype).eps / 2
    n = max([0] + list(np.diff(cu_k)))
    delta = (2.0 ** -23 * q.shape[2] * mag)
    tol = av * (2 * delta[..., None] + half + 2.0 ** -19) + (np.abs(ref) + av * half) * half
    if dtype is HF:
        tol += n * 2.0 ** -31 * np.abs(_np(v)).max(initial=0.0) + 2.0 ** -25   # and the output's own range
    T = cu_q[-1]
    err = np.abs(_np(out) - ref)[:T]
    assert np.all(err <= tol[:T]), (err - tol[:T]).max()
    if lse is not None:
        got, want, d = _np(lse)[:, :T], ref_lse[:, :T], delta.T[:, :T]
        empty = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), empty)
        fine = np.where(empty, 0.0, want)
        assert np.all(np.abs(np.where(empty, 0.0, got) - fine) <= d + 2.0 ** -20 + np.abs(fine) * 2.0 ** -22)


def _inputs(rng, tq, tk, H, Hkv, d, dtype, spread=1.0):
    q = torch.from_numpy(rng.standard_normal((tq, H, d)) * spread).to(dtype).cuda()
    k, v = (torch.from_numpy(rng.standard_normal((tk, Hkv, d))).to(dtype).cuda() for _ in range(2))
    return q, k, v


CASES = [
    # query lengths, key lengths (None: the same), H, Hkv, d, dtype, causal
    ([1], None, 1, 1, 64, BF, False),
    ([1], [1], 4, 2, 128, BF, True),
    ([64], None, 1, 1, 128, BF, False),
    ([65], None, 2, 1, 128, HF, True),
    ([128], None, 2, 2, 64, BF, True),
    ([129], None, 1, 1, 80, BF, True),
    ([256], None, 4, 4, 64, BF, False),
    ([257], [391], 2, 2, 128, BF, True),
    ([300], None, 5, 1, 96, HF, True),                    # five heads a row tile: 125 rows of it
    ([200], [77], 2, 1, 112, BF, True),                   # rows that see nothing
    ([40], [0], 2, 2, 64, BF, False),                     # no keys at all
    ([0, 5, 0, 190, 1, 0], [3, 5, 0, 190, 700, 64], 4, 2, 80, HF, True),
    ([31, 64, 200, 3], [64, 128, 65, 1], 8, 2, 128, BF, False),
    ([7], [1000], 128, 1, 64, BF, True),                  # 128 heads: one token a row tile
    ([9, 2], [300, 130], 48, 2, 64, HF, False),
    ([1], [5000], 8, 2, 128, BF, True),                   # a single token, keys in chunks
    ([142], [2900], 4, 2, 128, BF, True),                 # a question after many keys, in chunks
    ([3, 1, 2], [1500, 10, 0], 4, 4, 80, BF, True),       # chunks that some segments do not reach
    ([513], None, 1, 1, 64, HF, True),
    ([1025], [1100], 1, 1, 128, BF, True),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) + "-" + "x".join(map(str, c[2:5])) + str(c[5])[6:] for i, c in enumerate(CASES)])
def test_matches_the_oracle(tsel, case):
    nq, nk, H, Hkv, d, dtype, causal = case
    nk = nq if nk is None else nk
    rng = np.random.default_rng(sum(nq) + sum(nk) + d)
    q, k, v = _inputs(rng, sum(nq), sum(nk), H, Hkv, d, dtype)
    cu_q, cu_k = _cu(nq), _cu(nk)
    ws = torch.zeros(tsel.tsel_prompt_attention_workspace_size(len(nq), sum(nq), max(nq), max(nk), H, Hkv, d), dtype=torch.uint8, device="cuda")
    flags = tsel.TSEL_ATT_CAUSAL if causal else 0
    out, lse = tsel.tsel_prompt_attention(q, k, v, i32(cu_q), i32(cu_k), max(nq), max(nk), flags=flags, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    _close(out, lse, q, k, v, cu_q, cu_k, d ** -0.5, causal, dtype)
    again, lse2 = tsel.tsel_prompt_attention(q, k, v, i32(cu_q), i32(cu_k), max(nq), max(nk), flags=flags, workspace=ws)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


def _run(tsel, q, k, v, nq, nk, causal, **kw):
    cu_q, cu_k = _cu(nq), _cu(nk)
    ws = kw.pop("workspace", None)
    if ws is None:
        ws = torch.zeros(tsel.tsel_prompt_attention_workspace_size(len(nq), q.shape[0], max(nq), max(nk), q.shape[1], k.shape[1], q.shape[2]),
                         dtype=torch.uint8, device="cuda")
    out, lse = tsel.tsel_prompt_attention(q, k, v, i32(cu_q), i32(cu_k), max(nq), max(nk), flags=tsel.TSEL_ATT_CAUSAL if causal else 0,
                                          workspace=ws, **kw)
    assert tsel.tsel_read_device_status(ws) == 0
    return out, lse, cu_q, cu_k


@pytest.mark.parametrize("segments,most,H,Hkv", [(300, 40, 4, 4), (256, 33, 4, 2), (40, 300, 16, 16), (700, 3, 2, 1)])
def test_many_units(tsel, segments, most, H, Hkv):
    """Units from the counter, sorted segments and more than are sorted."""
    rng = np.random.default_rng(segments)
    nq = rng.integers(0, most + 1, segments).tolist()
    nk = [n + int(rng.integers(0, 9)) for n in nq]
    q, k, v = _inputs(rng, sum(nq), sum(nk), H, Hkv, 64, BF)
    out, lse, cu_q, cu_k = _run(tsel, q, k, v, nq, nk, True)
    _close(out, lse, q, k, v, cu_q, cu_k, 64 ** -0.5, True, BF)


def test_views_of_a_packed_tensor_and_results_in_place(tsel):
    rng = np.random.default_rng(1)
    for H, Hkv, d, dtype in ((4, 2, 80, BF), (2, 2, 128, HF)):
        nq = [130, 1, 77]
        packed = torch.from_numpy(rng.standard_normal((sum(nq), H + 2 * Hkv, d))).to(dtype).cuda()
        q, k, v = packed[:, :H], packed[:, H:H + Hkv], packed[:, H + Hkv:]
        out, lse, cu, _ = _run(tsel, q, k, v, nq, nq, True)
        _close(out, lse, q, k, v, cu, cu, d ** -0.5, True, dtype)
        kv = packed[:, H:].clone()
        _run(tsel, q, k, v, nq, nq, True, out=q, want_lse=False)
        assert torch.equal(q, out) and torch.equal(packed[:, H:], kv)


@pytest.mark.parametrize("nq,nk,H", [([150, 3], [150, 200], 2), ([5], [2000], 1)])
def test_padding_rows_are_left_alone(tsel, nq, nk, H):
    rng = np.random.default_rng(2)
    q, k, v = _inputs(rng, sum(nq) + 9, sum(nk) + 70, H, 1, 64, BF)
    clean, _, cu_q, cu_k = _run(tsel, q, k, v, nq, nk, True)
    for t, n in ((q, sum(nq)), (k, sum(nk)), (v, sum(nk))):
        t[n:] = float("nan")
    out, lse = torch.full_like(q, 7.0), torch.full((H, q.shape[0]), 5.0, device="cuda")
    _run(tsel, q, k, v, nq, nk, True, out=out, lse=lse)
    n = sum(nq)
    assert torch.equal(out[:n], clean[:n]) and bool((out[n:] == 7).all()) and bool((lse[:, n:] == 5).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("nq,nk", [([200], [200]), ([70, 90], [100, 90]), ([3], [3000])])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_infinities_and_nan_reach_only_rows_that_see_them(tsel, dtype, nq, nk, value):
    rng = np.random.default_rng(3)
    q, k, v = _inputs(rng, sum(nq), sum(nk), 2, 1, 80, dtype)
    clean, clean_lse, cu_q, cu_k = _run(tsel, q, k, v, nq, nk, True)
    key = nk[0] - 2                        # the last row but one of the first segment and the last see it
    sees = torch.zeros(sum(nq), dtype=torch.bool, device="cuda")
    sees[nq[0] - 2:nq[0]] = True
    v2 = v.clone()
    v2[key, 0, 5] = value
    out, lse, _, _ = _run(tsel, q, k, v2, nq, nk, True)
    assert torch.equal(lse, clean_lse)
    hit = out[sees][..., 5].float()
    assert bool((torch.isnan(hit) if value != value else hit == value).all())
    out[sees, :, 5] = clean[sees, :, 5]
    assert torch.equal(out, clean)
    k2 = k.clone()
    k2[key, 0, 7] = value
    out, lse, _, _ = _run(tsel, q, k2, v, nq, nk, True)
    assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[:, ~sees], clean_lse[:, ~sees])
    if value != value:
        assert bool(torch.isnan(out[sees]).all()) and bool(torch.isnan(lse[:, sees]).all())


def test_infinities_in_whole_steps_and_nan_queries(tsel):
    rng = np.random.default_rng(4)
    q, k, v = _inputs(rng, 140, 256, 1, 1, 64, BF)
    clean, _, _, _ = _run(tsel, q, k, v, [140], [256], False)
    v[3, 0, 9] = float("nan")
    out, _, _, _ = _run(tsel, q, k, v, [140], [256], False)
    assert bool(torch.isnan(out[..., 9]).all())
    out[..., 9] = clean[..., 9]
    assert torch.equal(out, clean)
    v[3, 0, 9] = 0.25
    q[17] = float("nan")
    again, _, _, _ = _run(tsel, q, k, v, [140], [256], False)
    q[17] = 0.5
    ref, _, _, _ = _run(tsel, q, k, v, [140], [256], False)
    assert bool(torch.isnan(again[17]).all())
    keep = torch.arange(140, device="cuda") != 17
    assert torch.equal(again[keep], ref[keep])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_logits_that_climb(tsel, dtype):
    """References move late and far: keys grow along the sequence."""
    rng = np.random.default_rng(5)
    q, k, v = _inputs(rng, 300, 700, 2, 1, 64, dtype)
    k *= torch.linspace(0.1, 40, 700, device="cuda").to(dtype)[:, None, None]
    out, lse, cu_q, cu_k = _run(tsel, q, k, v, [300], [700], True)
    _close(out, lse, q, k, v, cu_q, cu_k, 64 ** -0.5, True, dtype)
    out, lse, _, _ = _run(tsel, q, k, v, [300], [700], False, softmax_scale=0.02)
    _close(out, lse, q, k, v, cu_q, cu_k, 0.02, False, dtype)


def test_bad_lengths_are_flagged(tsel):
    rng = np.random.default_rng(6)
    q, k, v = _inputs(rng, 60, 80, 1, 1, 64, BF)
    good, _, _, _ = _run(tsel, q, k, v, [20, 40], [30, 50], True)
    ws = torch.zeros(tsel.tsel_prompt_attention_workspace_size(2, 60, 40, 50, 1, 1, 64), dtype=torch.uint8, device="cuda")

    def call(cu_q, cu_k, max_q=40, max_k=50):
        out = torch.zeros_like(q)
        tsel.tsel_prompt_attention(q, k, v, i32(cu_q), i32(cu_k), max_q, max_k, flags=tsel.TSEL_ATT_CAUSAL, out=out, workspace=ws)
        bits = tsel.tsel_read_device_status(ws)
        tsel.tsel_clear_device_status(ws)
        return out, bits
    for cu_q, cu_k, kw in (([0, 20, 61], [0, 30, 80], {}), ([0, 20, 60], [0, 30, 81], {}), ([0, 20, 10], [0, 30, 80], {}),
                           ([0, 20, 60], [0, 30, 29], {}), ([0, 20, 60], [0, 30, 80], {"max_q": 39}), ([0, 20, 60], [0, 30, 80], {"max_k": 49}),
                           ([0, 20, -5], [0, 30, 80], {}), ([0, 20, 1 << 30], [0, 30, 1 << 30], {})):
        out, bits = call(cu_q, cu_k, **kw)
        assert bits == tsel.TSEL_DEV_SEQLENS
        assert torch.equal(out[:20], good[:20])          # the other segment
    for cu_q, cu_k in (([1, 20, 60], [0, 30, 80]), ([0, 20, 60], [2, 30, 80])):
        assert call(cu_q, cu_k)[1] == tsel.TSEL_DEV_SEQLENS


def test_nothing_to_do(tsel):
    q = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    out, lse = tsel.tsel_prompt_attention(q, q, q, i32([0]), i32([0]), 0, 0)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    q = torch.ones(3, 2, 64, dtype=BF, device="cuda")
    out, lse = tsel.tsel_prompt_attention(q, q[:0], q[:0], i32([0, 3]), i32([0, 0]), 3, 0)
    assert not out.any() and bool(torch.isneginf(lse).all())
    out = torch.full_like(q, 3.0)
    tsel.tsel_prompt_attention(q, q, q, i32([0]), i32([0]), 0, 0, out=out)      # no segments
    assert bool((out == 3).all())


def test_scores_from_the_log_sum_exps(tsel):
    """The importance scoring takes the attention's LSE, as the two-pass scoring computes its own."""
    rng = np.random.default_rng(7)
    nq = [300, 41]
    q, k, v = _inputs(rng, sum(nq), sum(nq), 4, 2, 80, BF)
    _, lse, cu, _ = _run(tsel, q, k, v, nq, nq, False)
    scores, own = tsel.tsel_importance(q, k, i32(cu), i32(cu), 300, 300)
    given, _ = tsel.tsel_importance(q, k, i32(cu), i32(cu), 300, 300, flags=tsel.TSEL_IMP_LSE_PROVIDED, lse=lse)
    assert torch.allclose(lse, own, rtol=1e-5, atol=1e-5) and torch.allclose(given, scores, rtol=2e-3, atol=0)


def test_graphs_share_a_workspace_and_replay_with_other_lengths(tsel):
    rng = np.random.default_rng(8)
    H, Hkv, d, T = 8, 8, 64, 900
    q, k, v = _inputs(rng, T, T, H, Hkv, d, BF)
    few = [torch.from_numpy(rng.standard_normal((n, H, d))).to(BF).cuda() for n in (4, T)]
    lens = [[500, 400], [899, 1], [3, 600]]
    ws = torch.zeros(max(tsel.tsel_prompt_attention_workspace_size(90, T, 900, 900, H, Hkv, d),
                         tsel.tsel_prompt_attention_workspace_size(1, 4, 4, T, H, Hkv, d)), dtype=torch.uint8, device="cuda")
    # 90 segments make units enough for the counter; the other graph's keys come in chunks
    cu = torch.zeros(91, dtype=torch.int32, device="cuda")
    cu1, cuk = i32([0, 4]), i32([0, T])
    outs = torch.empty_like(q), torch.empty_like(few[0])
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for which in (0, 1):
            def call():
                if which == 0:
                    tsel.tsel_prompt_attention(q, k, v, cu, cu, 900, 900, flags=tsel.TSEL_ATT_CAUSAL, out=outs[0], want_lse=False, workspace=ws)
                else:
                    tsel.tsel_prompt_attention(few[0], k, v, cu1, cuk, 4, T, out=outs[1], want_lse=False, workspace=ws)
            call()
            g = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(g, stream=s):
                call()
            graphs.append(g)
        for a in lens:
            full = np.concatenate([_cu(a), np.full(91 - len(a) - 1, sum(a))]).astype(np.int32)
            cu.copy_(torch.from_numpy(full))
            outs[0].fill_(9)
            graphs[0].replay()
            graphs[1].replay()
            s.synchronize()
            n = sum(a)
            # the same sizes called, not replayed (two segments alone would come in chunks)
            want, lse = tsel.tsel_prompt_attention(q, k, v, i32(full), i32(full), 900, 900, flags=tsel.TSEL_ATT_CAUSAL)
            assert torch.equal(outs[0][:n], want[:n]) and bool((outs[0][n:] == 9).all())
            _close(want[:n], lse[:, :n], q[:n], k[:n], v[:n], _cu(a), _cu(a), d ** -0.5, True, BF)
            want, _, _, _ = _run(tsel, few[0], k, v, [4], [T], False)
            assert torch.equal(outs[1], want)
    assert tsel.tsel_read_device_status(ws) == 0


def test_calls_on_two_streams_at_once(tsel):
    rng = np.random.default_rng(9)
    q, k, v = _inputs(rng, 1500, 1500, 4, 4, 80, BF)
    want, _, _, _ = _run(tsel, q, k, v, [1500], [1500], True)
    cu = i32([0, 1500])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for s in streams:
            outs.append(tsel.tsel_prompt_attention(q, k, v, cu, cu, 1500, 1500, flags=tsel.TSEL_ATT_CAUSAL, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_offsets_past_32_bits(tsel):
    """Keys whose elements lie past 2^31, and a key count in the millions."""
    rng = np.random.default_rng(10)
    n = (1 << 24) + 700
    k = torch.zeros(n, 1, 128, dtype=BF, device="cuda")
    v = torch.zeros(n, 1, 128, dtype=BF, device="cuda")
    for t in (k, v):
        t[-700:] = torch.from_numpy(rng.standard_normal((700, 1, 128))).to(BF).cuda()
    q = torch.from_numpy(rng.standard_normal((90, 2, 128))).to(BF).cuda()
    ws = torch.zeros(tsel.tsel_prompt_attention_workspace_size(2, 90, 90, n, 2, 1, 128), dtype=torch.uint8, device="cuda")
    out, lse = tsel.tsel_prompt_attention(q, k, v, i32([0, 0, 90]), i32([0, n - 700, n]), 90, n, flags=tsel.TSEL_ATT_CAUSAL, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == 0
    _close(out, lse, q, k[-700:], v[-700:], _cu([90]), _cu([700]), 128 ** -0.5, True, BF)
    # One row over all of them: zero keys weigh 1 each, values 0. Their sums are whole
    # numbers below 2^24 in a chunk, so exact; P and the output are rounded once each.
    out, lse = tsel.tsel_prompt_attention(q[:1], k, v, i32([0, 1]), i32([0, n]), 1, n)
    z = _np(q[0]) @ _np(k[-700:, 0]).T * 128 ** -0.5
    total = (n - 700) + np.exp(z).sum(-1)
    assert np.allclose(_np(lse)[:, 0], np.log(total), rtol=2.0 ** -19, atol=0)
    ref = np.exp(z) @ _np(v[-700:, 0]) / total[:, None]
    av = np.exp(z) @ np.abs(_np(v[-700:, 0])) / total[:, None]
    assert np.all(np.abs(_np(out)[0] - ref) <= av * 2.0 ** -7)


def _redone(rng, rows, keys, d, dtype):
    """Logits that climb by some 20 with every 64 keys, past the 15 ln 2 at which a step is done again."""
    q = torch.from_numpy(np.abs(rng.standard_normal((rows, 2, d)))).to(dtype).cuda()
    k = torch.from_numpy(np.abs(rng.standard_normal((keys, 1, d)))).to(dtype).cuda()
    k *= torch.linspace(0, keys / 16, keys, device="cuda").to(dtype)[:, None, None]
    v = torch.from_numpy(rng.standard_normal((keys, 1, d))).to(dtype).cuda()
    return q, k, v


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 80, 128])
def test_every_step_done_again(tsel, dtype, d):
    """Each step's probabilities are stored twice, the first time past fp16's range."""
    rng = np.random.default_rng(d)
    scale = 8.0 / d                        # the mean of a logit, 0.64 d scale times a key's factor, grows alike for every d
    for rows, keys in ((256, 1280), (5, 1280), (129, 333)):
        q, k, v = _redone(rng, rows, keys, d, dtype)
        for causal in (False, True):
            out, lse, cu_q, cu_k = _run(tsel, q, k, v, [rows], [keys], causal, softmax_scale=scale)
            _close(out, lse, q, k, v, cu_q, cu_k, scale, causal, dtype)
            again, lse2, _, _ = _run(tsel, q, k, v, [rows], [keys], causal, softmax_scale=scale)
            assert torch.equal(again, out) and torch.equal(lse2, lse)


BAD_LENGTHS = [
    # cu_q, cu_k, max_q, max_k, the good segment, rows of no segment
    ([0, 20, 61], [0, 600, 1300], 40, 700, 0, []),
    ([0, 20, 60], [0, 600, 1301], 40, 700, 0, []),
    ([0, 20, 10], [0, 600, 1300], 40, 700, 0, [30, 59]),
    ([0, 20, 60], [0, 600, 599], 40, 700, 0, []),
    ([0, 20, 60], [0, 600, 1300], 30, 700, 0, []),
    ([0, 20, 60], [0, 600, 1300], 40, 650, 0, []),
    ([0, 20, -5], [0, 600, 1300], 40, 700, 0, [30, 59]),
    ([0, 20, 1 << 30], [0, 600, 1 << 30], 40, 700, 0, []),
    ([0, 45, 60], [0, 600, 1300], 40, 700, 1, []),
    ([0, 20, 60], [2, 600, 1300], 40, 700, 1, []),
    ([0, 35, 50], [0, 800, 1300], 20, 700, 1, [50, 59]),
]


@pytest.mark.parametrize("case", range(len(BAD_LENGTHS)))
def test_bad_lengths_spare_the_other_segment_in_chunks(tsel, case):
    cu_q, cu_k, max_q, max_k, good, free = BAD_LENGTHS[case]
    rng = np.random.default_rng(14)
    q, k, v = _inputs(rng, 60, 1300, 2, 1, 64, BF)
    size = tsel.tsel_prompt_attention_workspace_size(2, 60, max_q, max_k, 2, 1, 64)
    assert size > 4 * 60 * 2 * 64 * 2      # at least two chunks
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((2, 60), 5.0, device="cuda")
    tsel.tsel_prompt_attention(q, k, v, i32(cu_q), i32(cu_k), max_q, max_k, flags=tsel.TSEL_ATT_CAUSAL, out=out, lse=lse, workspace=ws)
    assert tsel.tsel_read_device_status(ws) == tsel.TSEL_DEV_SEQLENS
    a, b, c, e = cu_q[good], cu_q[good + 1], cu_k[good], cu_k[good + 1]
    _close(out[a:b], lse[:, a:b], q[a:b], k[c:e], v[c:e], [0, b - a], [0, e - c], 64 ** -0.5, True, BF)
    if free:
        assert bool((out[free[0]:free[1] + 1] == 7).all()) and bool((lse[:, free[0]:free[1] + 1] == 5).all())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows,keys,H", [(60, 128, 2), (300, 700, 1), (3, 2000, 2), (3, 20000, 2), (700, 20000, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_infinities_under_a_weight_that_underflows(tsel, dtype, rows, keys, H, value):
    """A row that sees an infinite V gives an infinity or NaN of its column however small the key's weight,
    in one chunk (the first case) and in several."""
    rng = np.random.default_rng(13)
    q, k, v = torch.ones(rows, H, 64, device="cuda"), torch.zeros(keys, 1, 64, device="cuda"), rng.standard_normal((keys, 1, 64))
    k[:keys // 3] = -20.0                 # logits 160 below the others': 2^-230 of their weight
    q, k, v = q.to(dtype), k.to(dtype), torch.from_numpy(v).to(dtype).cuda()
    clean, clean_lse, _, _ = _run(tsel, q, k, v, [rows], [keys], False)
    v[5, 0, 33] = value
    out, lse, _, _ = _run(tsel, q, k, v, [rows], [keys], False)
    assert not bool(torch.isfinite(out[..., 33]).any()) and torch.equal(lse, clean_lse)
    out[..., 33] = clean[..., 33]
    assert torch.equal(out, clean)
