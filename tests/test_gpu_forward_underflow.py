"""Values that are not finite behind scores whose probabilities underflow to 0: they reach every row that sees their
key, in one part or in several, in a tile that all its rows see or only some; and no other row or column.
Elsewhere the output is that of the 64-bit form with the value left out (its weight is below 1e-100)."""
import math

import pytest

torch = pytest.importorskip("torch")

import test_gpu_forward_ops as ops  # noqa: E402
from test_gpu_forward_mixed import Mixed  # noqa: E402
from transformer_sharding_affinity_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, U, E = ops.BF, ops.F32, ops.U, ops.E


def _slot(c, b, key):
    ids = c.prefix_ids if b is None else c.ids[b]
    return ids[key // c.page], key % c.page


# (query tokens, own keys, prefix, [(sequence or None for the prefix, key of the value, low keys from, to)])
STEPS = [([1], [9000], 0, [(0, 100, 0, 6000)]),                            # single token, a part of low keys alone
         ([1, 1, 1], [5000, 300, 40], 0, [(0, 4990, 3000, 4995), (1, 250, 200, 300)]),
         ([1, 1], [600, 50], 4000, [(None, 70, 0, 4000), (1, 3, 2, 9)]),   # the whole prefix is low
         ([4], [9], 0, [(0, 6, 6, 7)]),                                    # seen by some rows of the tile
         ([40, 1], [300, 900], 0, [(0, 280, 275, 285), (1, 500, 0, 800)]),
         ([200], [200], 0, [(0, 30, 20, 40), (0, 150, 140, 152)]),
         ([130, 1], [4200, 9000], 0, [(0, 10, 0, 3000), (1, 8000, 5000, 9000 - 4)]),
         ([70, 90], [70, 100], 200, [(None, 199, 0, 200), (1, 60, 50, 70)])]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128), (2, 2, 96), (3, 1, 80)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q_lens,kv_lens,prefix,marks", STEPS)
def test_values_behind_probabilities_of_zero(dtype, heads, value, q_lens, kv_lens, prefix, marks):
    H, G, d = heads
    c = Mixed(heads, q_lens, kv_lens, prefix, 16, dtype=dtype, seed=61)
    c.q.abs_().clamp_(min=0.5)               # a score of a low key is -400 sqrt(d) / 8 or less below the others' zero mean
    hit = torch.zeros(c.T, H, d, dtype=torch.bool)
    for n, (b, key, lo, hi) in enumerate(marks):
        for j in range(lo, hi):
            page, at = _slot(c, b, j)
            c.kd[page, :, at] = -100.0
        page, at = _slot(c, b, key)
        col = (5 + 37 * n) % d
        c.vd[page, :, at, col] = 0.0
        for s in range(len(q_lens)):
            if b is None or s == b:
                for i in range(q_lens[s]):
                    if b is None or kv_lens[s] - q_lens[s] + i >= key:
                        hit[c.starts[s] + i, :, col] = True
    scale = d ** -0.5
    ref, rlse, mag, dots = c.attend(scale)
    for n, (b, key, _, _) in enumerate(marks):
        page, at = _slot(c, b, key)
        c.vd[page, :, at, (5 + 37 * n) % d] = value
    out, lse = torch.empty(c.T, H, d, dtype=dtype, device="cuda"), torch.empty(c.T, H, device="cuda")
    B.prefix_attention(c.q, c.cache, c.step, scale, out, lse, c.plan)
    assert B.device_status(c.plan) == B.AFF_OK
    got = out.cpu().double()
    assert torch.equal(~got.isfinite(), hit)
    score, keys = (d + 4) * E * dots, prefix + max(kv_lens)
    if dtype == BF:
        tol = U * ref.abs() + 1.05 * (U + score)[..., None] * mag
    else:
        tol = 2 * (score + (keys + 16) * E)[..., None] * mag
    assert ((got - ref).abs()[~hit] <= tol[~hit]).all()
    ltol = 2 * (score + (keys + 16) * E) + 4 * E * rlse.abs()
    assert ((lse.cpu().double() - rlse).abs() <= ltol).all()
