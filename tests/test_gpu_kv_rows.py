"""Attention over the 4-bit cache: what a row's result may depend on.  Scores anywhere in the range of binary32,
rows beside others whose scores grow, and the weights' precision by the number of stacked rows."""
import numpy as np
import pytest
import torch

from bit_quantized_dit_amd import w4a4 as B
from tests import kv_ref as R
from tests.test_gpu_kv import BF16, Setup

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634
FEW_ROWS = 64      # W4A4_KV_FEW_ROWS
F32_MAX = float(np.finfo(np.float32).max)


def _attend(s, rows, q, causal=True, scale=1.0, qt=BF16):
    n, Hq = q.shape[:2]
    b = s.batch(rows)
    O = torch.full((n, Hq, s.D), 7.0, dtype=BF16, device="cuda")
    B.w4a4_kv_attention(torch.from_numpy(q).cuda().to(qt), b, s.cache, O, B.alloc_workspace_kv(n, b, Hq, s.cache), scale=scale, causal=causal)
    torch.cuda.synchronize()
    return O


# (rows, tokens, key/value heads, channels): one row, several, ranges that are joined, many rows by four wavefronts, many by eight
FORMS = [(1, 300, 1, 64), (9, 300, 2, 64), (30, 300, 1, 128), (50, 300, 1, 64), (1, 5000, 1, 64), (9, 5000, 1, 128), (80, 300, 1, 64),
         (80, 300, 1, 200), (70, 5000, 1, 64), (300, 400, 130, 32)]


def _one_channel(rows, n, H, D, ks, q0):
    """Keys and queries with one channel that is not zero, so that a score is one exact product q0 ks[t]."""
    def edit(s):
        s.K[:] = 0
        s.K[:, :, 0] = np.float32(ks)[:, None]
    s = Setup([n], H, D, 16, edit=edit)
    assert np.array_equal(s.values(0, [0])[0][:, 0, 0], np.float64(ks))      # codes hold them
    q = np.zeros((rows, 2 * H, D), np.float32)
    q[:, :, 0] = q0
    return s, q


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("q0,grid", [(2.0 ** 24, [1, 2, 3]), (2.0 ** 33, [1, 2, 3]), (2.0 ** 60, [1.5, 3, 6]), (-2.0 ** 33, [1.5, 3, 6]), (-2.0 ** 60, [1, 2, 4]),
                                     (1.375 * 2.0 ** 125, [1, 2, 3, 4]), (-1.25 * 2.0 ** 125, [4, 6]), (-1.375 * 2.0 ** 125, [4])])
def test_scores_of_any_size(form, q0, grid):
    """Scores so large that the weights are those of the largest ones alone, up to the ends of binary32: the
    mean of their values.  A weight of 1 and sums of at most 5000 values in binary32 (2 L + 16 roundings, as in the oracle's
    bound), then bf16.  Scaled scores below binary32 are -Inf, as the 4 of -1.25 2^127 is beside the 6."""
    rows, n, H, D = form
    ks = np.random.default_rng(1).choice(grid, n)
    ks[0], ks[n // 2] = grid[0], grid[-1]
    s, q = _one_channel(rows, n, H, D, ks, q0)
    x = ks * q0 * LOG2E
    assert (x <= F32_MAX).all() and (x >= -F32_MAX).any()
    O = _attend(s, [rows], q, causal=False).double().cpu().numpy()
    best = x == x.max()
    for h in [0, H - 1]:
        v = s.values(0, [h])[1][best, 0]
        want, mag = v.mean(0), np.abs(v).mean(0)
        tol = (2 * n + 16) * 2.0 ** -23 * mag
        tol = tol + R.BF16_U * (np.abs(want) + tol)
        for j in (2 * h, 2 * h + 1):
            assert (np.abs(O[:, j] - want[None]) <= tol[None]).all(), (h, j, float(np.abs(O[:, j] - want[None]).max()))


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_scores_past_binary32(form):
    """A scaled score above the largest number is +Inf and makes its row NaN; all of them below the lowest are -Inf: zero."""
    rows, n, H, D = form
    ks = np.full(n, 1.0)
    ks[n // 3] = 4.0
    s, q = _one_channel(rows, n, H, D, ks, 1.5 * 2.0 ** 125)
    assert bool(torch.isnan(_attend(s, [rows], q, causal=False)).all())
    q[:] = 0
    q[rows // 2, 1, 0] = 1.5 * 2.0 ** 125      # one row of many
    nan = torch.isnan(_attend(s, [rows], q, causal=False))
    assert bool(nan[rows // 2, 1].all()) and int(nan.sum()) == D
    s, q = _one_channel(rows, n, H, D, np.full(n, 4.0), -1.5 * 2.0 ** 125)
    assert not bool(_attend(s, [rows], q, causal=False).any())


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("where", ["first", "last"])
def test_far_scores_beside_ordinary_ones(form, where):
    """One block of tokens far below all others (weight zero, in whichever order they come), or one token far above (all of the weight)."""
    rows, n, H, D = form
    rng = np.random.default_rng(2)
    ks = rng.choice([-1.0, -0.5, 0.5, 1.0], n)
    far = slice(0, 37) if where == "first" else slice(n - 37, n)
    ks[far] = -2.0 ** 44
    s, q = _one_channel(rows, n, H, D, ks, 2.0)
    O = _attend(s, [rows], q, causal=False).double().cpu()
    keep = np.ones(n, bool)
    keep[far] = False
    qd = torch.from_numpy(q).double()
    for h in [0, H - 1]:
        k, v = (x[keep, 0] for x in s.values(0, [h]))
        o, tol, _ = R.attention(qd[:, 2 * h], k, v, 1.0, np.zeros(rows, int), np.full(rows, int(keep.sum())), rows * 2 <= 32)
        assert bool(((O[:, 2 * h] - o).abs() <= tol).all())
    at = 3 if where == "first" else n - 3
    ks[far] = 0.5
    ks[at] = 2.0 ** 44
    s, q = _one_channel(rows, n, H, D, ks, 2.0)
    O = _attend(s, [rows], q, causal=False).double().cpu().numpy()
    for h in [0, H - 1]:
        want = s.values(0, [h])[1][at, 0]
        assert (np.abs(O[:, 2 * h] - want) <= R.BF16_U * np.abs(want) * (1 + 2.0 ** -14)).all()


@pytest.mark.parametrize("D", [64, 72, 128, 200])
@pytest.mark.parametrize("rows,H,Hq", [(8, 2, 4), (16, 1, 2), (40, 1, 1), (100, 2, 2), (200, 1, 1), (100, 260, 260)])
def test_rows_do_not_move_each_other(rows, H, Hq, D):
    """Bits of a row are the same whatever the tokens hold that it does not see, and whatever the rows beside it hold."""
    if H > 100 and D == 200:      # eight wavefronts share a tile up to 128 channels
        D = 31
    n, last = 260, 5
    rng = np.random.default_rng(4)
    q = (rng.standard_normal((rows, Hq, D)) * 2).astype(np.float32)
    base = _attend(Setup([n], H, D, 16), [rows], q, scale=D ** -0.5)
    for factor in (20.0, 2.0 ** 40, np.nan):
        def edit(s): s.K[n - last:] *= factor
        s = Setup([n], H, D, 16, edit=edit)
        got = _attend(s, [rows], q, scale=D ** -0.5)
        assert torch.equal(got[:rows - last], base[:rows - last]), f"tokens of {factor}"
    for factor in (20.0, 2.0 ** 40, np.inf):
        p = q.copy()
        p[1::2] *= factor
        got = _attend(Setup([n], H, D, 16), [rows], p, scale=D ** -0.5)
        assert torch.equal(got[::2], base[::2]), f"rows of {factor}"


def two_terms(max_rows, ratio, D):
    """Whether the header promises weights of two bf16 terms."""
    return max_rows * ratio <= (FEW_ROWS if R.d_pad(D) <= 128 else FEW_ROWS // 2)


@pytest.mark.parametrize("D", [31, 64, 96, 97, 100, 127, 128, 130])
@pytest.mark.parametrize("rows,H,Hq,lens", [([33], 2, 2, [700]), ([8, 3], 1, 8, [900, 40]), ([64, 1, 20], 1, 1, [64, 30, 333]), ([12], 2, 10, [5000]),
                                            ([1, 1], 1, 64, [3000, 17]), ([40], 260, 260, [90])])
def test_weights_of_up_to_64_stacked_rows(D, rows, H, Hq, lens):
    """33 to 64 stacked rows within the bound of weights in two bf16 terms (2^-16 of themselves) up to 128 channels, of one term above,
    every output and the root mean square; causal, windowed and not."""
    s = Setup(lens, H, D, 16)
    n, ratio = sum(rows), Hq // H
    few = two_terms(max(rows), ratio, D)
    assert few == (D <= 128)
    q = (np.random.default_rng(7).standard_normal((n, Hq, D)) * 2).astype(np.float32)
    b = s.batch(rows)
    Q = torch.from_numpy(q).cuda().bfloat16()
    heads = [0, 1, H - 1] if H > 2 else list(range(H))
    for causal, window in ((True, 0), (True, 100), (False, 0)):
        O = torch.empty(n, Hq, D, dtype=BF16, device="cuda")
        B.w4a4_kv_attention(Q, b, s.cache, O, B.alloc_workspace_kv(n, b, Hq, s.cache), causal=causal, window=window)
        at, err2, var, count = 0, 0.0, 0.0, 0
        for i, r in enumerate(rows):
            k, v = s.values(i, heads)
            pos = np.arange(lens[i] - r, lens[i])
            lo = np.maximum(pos - window + 1, 0) if window else np.zeros(r, np.int64)
            hi = pos + 1 if causal else np.full(r, lens[i])
            for e, h in enumerate(heads):
                for j in range(h * ratio, (h + 1) * ratio):
                    o, tol, va = R.attention(Q[at:at + r, j].double().cpu(), k[:, e], v[:, e], D ** -0.5, lo, hi, few)
                    d = (O[at:at + r, j].double().cpu() - o).abs()
                    assert bool((d <= tol).all()), (i, j)
                    err2, var, count = err2 + float((d ** 2).sum()), var + float(va.sum()), count + d.numel()
            at += r
        assert err2 <= 1.21 * var or count < 4000, (err2 ** 0.5, var ** 0.5)
