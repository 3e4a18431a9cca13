"""The forward-pass operators on the GPU where the values or the sizes are awkward: keys and values that are not
finite at positions that only some rows see, fp32 steps of every row count, norms of odd widths over many rows.

Tolerances are those of the sibling module of the operators' tests, derived there.  Where the 64-bit form gives NaN
or an infinity the operator has to give the same; everywhere else it has to be finite and within tolerance.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import test_gpu_forward_ops as ops  # noqa: E402
from transformer_sharding_affinity_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, U, E = ops.BF, ops.F32, ops.U, ops.E


def _put(case, pool, dev, b, key, value, col=None):
    """Writes `value` to own key `key` of sequence b, all groups, in the host's and the device's pool."""
    page, at = case.ids[b][key // case.page], key % case.page
    for p in (pool, dev):
        if col is None:
            p[page, :, at] = value
        else:
            p[page, :, at, col] = value


def _check(case):
    H, G, d = case.heads
    out = torch.full((case.T, H, d), 77.0, dtype=case.dtype, device="cuda")
    lse = torch.full((case.T, H), 77.0, device="cuda")
    B.prefix_attention(case.q.cuda(), case.cache, case.step, d ** -0.5, out, lse, case.plan)
    assert B.device_status(case.plan) == B.AFF_OK
    ref, rlse, mag, dots = case.attend(d ** -0.5)
    got = out.cpu().double()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isinf(), ref.isinf()) and (got[ref.isinf()] == ref[ref.isinf()]).all()
    fine = ref.isfinite()
    score = (d + 4) * E * dots
    keys = case.prefix + max(case.kv_lens)
    if case.dtype == BF:
        tol = U * ref.abs() + 1.05 * (U + score)[..., None] * mag
    else:
        tol = 2 * (score + (keys + 16) * E)[..., None] * mag
    assert ((got - ref).abs()[fine] <= tol[fine]).all()
    assert torch.equal(lse.cpu().isnan(), rlse.isnan())
    return out


STEPS = [([1, 5, 3], [200, 131, 3], 0), ([5, 2, 8, 3], [140, 20, 8, 257], 150), ([150, 40], [150, 300], 77),
         ([300], [300], 0), ([2, 1, 0, 4], [1500, 1, 7, 900], 0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64), (6, 2, 96), (3, 1, 72), (8, 1, 80)])
@pytest.mark.parametrize("q_lens,kv_lens,prefix", STEPS)
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, heads, q_lens, kv_lens, prefix):
    if dtype == F32 and heads[2] % 4:
        pytest.skip("rows of whole 16-byte pieces")
    case = ops.Case(heads, q_lens, kv_lens, prefix, dtype=dtype, seed=41)
    d = heads[2]
    first = None
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        if n < 2:
            continue
        at = sorted({length - 1, length - (n + 1) // 2, max(length - n, 1)})
        for i, key in enumerate(at):
            value = (math.nan, math.inf, -math.inf)[i % 3]
            _put(case, case.v, case.vd, b, key, value, col=(3 + 31 * i) % d)
            _put(case, case.v, case.vd, b, key, math.inf, col=d - 1)
    first = _check(case)
    # the plan is as it was: a second call gives the same
    again = _check(case)
    assert torch.equal(first.isnan(), again.isnan()) and torch.equal(first.nan_to_num(), again.nan_to_num())


@pytest.mark.parametrize("prefix", [0, 40])
def test_many_items_with_values_that_are_not_finite(prefix):
    """Every CTA has several items to put back; a call over finite values on the same plan afterwards."""
    n = 90
    lens = [(64, 5, 130, 20)[i % 4] for i in range(n)]
    case = ops.Case((4, 4, 64), lens, [k + 9 * (i % 3) for i, k in enumerate(lens)], prefix, seed=43)
    clean = (case.v.clone(), case.vd.clone())
    for b in range(n):
        _put(case, case.v, case.vd, b, case.kv_lens[b] - 2, math.inf, col=b % 64)
        _put(case, case.v, case.vd, b, case.kv_lens[b] - 1, math.nan, col=(b + 7) % 64)
    _check(case)
    case.v.copy_(clean[0])
    case.vd.copy_(clean[1])
    case.check_attention()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_lens,kv_lens,prefix", STEPS)
def test_keys_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, q_lens, kv_lens, prefix):
    case = ops.Case((4, 2, 64), q_lens, kv_lens, prefix, dtype=dtype, seed=42)
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        if n > 1:
            _put(case, case.k, case.kd, b, length - 1, math.nan)
            _put(case, case.v, case.vd, b, length - 1, math.nan)
    _check(case)


@pytest.mark.parametrize("heads", [(8, 4, 128), (4, 2, 96), (5, 5, 72), (4, 2, 64)])
@pytest.mark.parametrize("page", [8, 24, 40, 64, 104, 128, 136, 200, 256])
def test_single_tokens_over_pages_that_do_not_fill_a_tile(heads, page):
    """Several tiles to an item, so that tiles lie next to each other while they are worked on; one to eight tokens."""
    case = ops.Case(heads, [1, 1, 4, 1, 8, 0, 1], [900, 411, 640, 128, 1300, 50, 24 * 5], 130, page=page, seed=page)
    first = case.check_attention()
    for _ in range(4):
        again = case.check_attention()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("heads", [(4, 2, 128), (2, 2, 64), (8, 1, 80), (5, 5, 72), (4, 4, 16)])
@pytest.mark.parametrize("q,kv,B_,prefix", [(1, 300, 3, 0), (2, 131, 2, 0), (3, 70, 5, 260), (7, 9, 2, 1), (17, 400, 2, 0),
                                            (40, 41, 3, 130), (70, 70, 1, 0), (131, 200, 2, 64), (9, 9, 9, 500)])
def test_fp32_rows(heads, q, kv, B_, prefix):
    """From one row of an item to several row tiles, with the prefix apart and not."""
    ops.Case(heads, [q] * B_, [kv] * B_, prefix, page=24, dtype=F32, seed=q).check_attention()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D", [(1300, 65), (1300, 130), (1250, 333), (1300, 894), (1217, 1802), (1220, 2047), (1218, 2050)])
@pytest.mark.parametrize("post,gate,pre", [(True, "rows", True), (False, "token", True), (True, None, False)])
def test_norms_of_odd_widths_over_many_rows(dtype, T, D, post, gate, pre):
    ops.test_block_norm(dtype, T, D, post, gate, pre)
