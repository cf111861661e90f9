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
