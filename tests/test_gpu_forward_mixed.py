"""Steps that mix prompts and single tokens, in which some jobs are cut and others are not, and steps of more
sequences than the planner holds at a time.  Every partial row has one item that writes it, every key tile of a row
is in one item, and attention is that of the 64-bit form (tolerances as derived in test_gpu_forward_ops.py).
"""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import test_gpu_forward_ops as ops  # noqa: E402
from transformer_sharding_affinity_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = ops.BF, ops.F32


class Mixed(ops.Case):
    """As ops.Case, with the pools filled and the 64-bit form computed on the GPU: for thousands of tokens."""

    def __init__(self, heads, q_lens, kv_lens, prefix=0, page=16, dtype=BF, seed=0):
        H, G, d = self.heads = heads
        self.q_lens, self.kv_lens, self.prefix, self.page, self.dtype = q_lens, kv_lens, prefix, page, dtype
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T = sum(q_lens)
        counts = [-(-n // page) for n in kv_lens]
        n_pre = -(-prefix // page)
        n_pages = n_pre + sum(counts) + 2
        order = torch.randperm(n_pages, generator=g, device="cuda").cpu().tolist()
        self.prefix_ids, at, self.ids = order[:n_pre], n_pre, []
        for n in counts:
            self.ids.append(order[at:at + n])
            at += n
        width = max(counts + [1])
        table = torch.tensor([i + [-7] * (width - len(i)) for i in self.ids], dtype=torch.int32)
        # what is not a valid token is NaN
        self.kd, self.vd = (torch.full((n_pages, G, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2))
        for ids, n in [(self.prefix_ids, prefix)] + list(zip(self.ids, kv_lens)):
            if n:
                j = torch.arange(n, device="cuda")
                where = torch.tensor(ids, device="cuda")[j // page]
                for pool in (self.kd, self.vd):
                    pool[where, :, j % page] = torch.randn(n, G, d, generator=g, device="cuda").to(dtype)
        self.k, self.v = self.kd, self.vd
        self.q = torch.randn(self.T, H, d, generator=g, device="cuda").to(dtype)
        self.starts = [0]
        for n in q_lens:
            self.starts.append(self.starts[-1] + n)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.dev = {"q_start": ints(self.starts), "kv_len": ints(kv_lens), "pages": table.cuda(),
                    "prefix_pages": ints(self.prefix_ids) if n_pre else None}
        self.cache = B.kv_cache(self.kd, self.vd)
        self.step = B.step(self.T, H, prefix_len=prefix, **self.dev)
        self.plan = torch.empty(B.step_plan_size(self.step, self.cache), dtype=torch.uint8, device="cuda")
        B.step_plan(self.step, self.cache, self.plan)

    def attend(self, scale):
        H, G, d = self.heads
        R = H // G
        out = torch.zeros(self.T, H, d, dtype=torch.float64, device="cuda")
        mag, dots = torch.zeros_like(out), torch.zeros(self.T, H, dtype=torch.float64, device="cuda")
        lse = torch.full((self.T, H), -math.inf, dtype=torch.float64, device="cuda")
        kp, vp = (self.rows(p, self.prefix_ids, self.prefix).cuda() for p in (self.kd, self.vd))
        for b, (n, length) in enumerate(zip(self.q_lens, self.kv_lens)):
            if not n:
                continue
            ks, vs = (torch.cat([pre, self.rows(p, self.ids[b], length).cuda()])
                      for pre, p in ((kp, self.kd), (vp, self.vd)))
            t0 = self.starts[b]
            own = length - n + torch.arange(n, device="cuda")
            hidden = torch.arange(self.prefix + length, device="cuda")[None] > self.prefix + own[:, None]
            for h in range(H):
                k, v, q = ks[:, h // R], vs[:, h // R], self.q[t0:t0 + n, h].double()
                s = (q @ k.T * scale).masked_fill_(hidden, -math.inf)
                m = s.amax(1, keepdim=True)
                p = (s - m).exp_()
                total = p.sum(1, keepdim=True)
                out[t0:t0 + n, h] = p @ v / total
                mag[t0:t0 + n, h] = p @ v.abs() / total
                lse[t0:t0 + n, h] = (m + total.log())[:, 0]
                dots[t0:t0 + n, h] = (q.abs() @ k.abs().T).masked_fill_(hidden, 0).amax(1) * scale
        return out.cpu(), lse.cpu(), mag.cpu(), dots.cpu()

    def items(self):
        """The plan's work items [n, 12]: row0, nrows, group, seq, t0, n0, n1, part_row, own_off, own_len, alt, np."""
        up = lambda n: (n + 255) // 256 * 256
        at = 256 + up(16 * self.T) + up(32 * len(self.q_lens))
        n = int(self.plan[4:8].view(torch.int32))
        return self.plan[at:at + 48 * n].view(torch.int32).reshape(n, 12).cpu()

    def check_items(self):
        """No two items write the same partial row, all lie in the buffer, and a row tile's items share out its key
        tiles."""
        it = self.items().tolist()
        assert it and B.device_status(self.plan) == B.AFF_OK
        parts = sorted((i[7], i[7] + i[1]) for i in it if i[7] >= 0)
        assert all(a[1] <= b[0] for a, b in zip(parts, parts[1:]))
        assert not parts or parts[-1][1] * 4 * (1 + self.heads[2]) <= self.plan.numel()
        runs = {}
        for row0, nrows, group, seq, t0, n0, n1, part, _, _, alt, _ in it:
            runs.setdefault((seq, row0, group, nrows), []).append((t0, max(n0, n1) if alt == 0 else n0 + n1, part))
        for run in runs.values():
            run.sort()
            assert run[0][0] == 0 and all(a[0] + a[1] == b[0] for a, b in zip(run, run[1:]))
            assert len(run) == 1 or all(p >= 0 for _, _, p in run)


# (heads, query tokens, own keys, prefix, page): prompts of several row tiles that are cut, beside single tokens
# behind many keys; R = 1, 2, 4, 8, 16 query heads to a group
STEPS = [((16, 8, 128), [1026, 1, 1], [1026, 14828, 15544], 0, 16), ((16, 1, 128), [1, 289], [9567, 4521], 0, 8),
         ((8, 8, 128), [1, 613, 1, 217, 1], [11815, 793, 19056, 493, 14721], 1028, 8),
         ((8, 8, 96), [922, 1, 1, 279], [1078, 19928, 9769, 2188], 0, 24),
         ((2, 1, 128), [525, 519, 1], [1006, 760, 7017], 5124, 16), ((4, 1, 64), [224, 794, 96], [547, 975, 535], 5619, 8),
         ((8, 1, 128), [346, 117], [559, 196], 8743, 16), ((1, 1, 64), [396, 161, 294], [852, 184, 388], 7196, 8),
         ((4, 1, 72), [600, 1, 1, 2], [600, 9000, 1, 8000], 0, 16), ((32, 8, 128), [700, 1, 1, 1], [1500, 5000, 12000, 40], 3000, 64),
         ((6, 2, 96), [1500, 3, 1], [1500, 7000, 6000], 700, 24)]


@pytest.mark.parametrize("heads,q_lens,kv_lens,prefix,page", STEPS)
def test_prompts_beside_single_tokens_with_many_keys(heads, q_lens, kv_lens, prefix, page):
    c = Mixed(heads, q_lens, kv_lens, prefix, page, seed=51)
    c.check_items()
    first = c.check_attention()
    for _ in range(3):
        again = c.check_attention()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("heads,q_lens,kv_lens,prefix,page", STEPS[1:6])
def test_the_same_in_fp32(heads, q_lens, kv_lens, prefix, page):
    c = Mixed(heads, q_lens, kv_lens, prefix, page, dtype=F32, seed=52)
    c.check_items()
    c.check_attention()


@pytest.mark.parametrize("seed", range(8))
def test_plans_of_many_mixed_steps(seed):
    """Plans alone, of steps like those above."""
    rng = random.Random(seed)
    for _ in range(40):
        G, R, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8, 16]), 16
        n = rng.choice([1, 2, 3, 4, 6, 40])
        q = [rng.choice([0, 1, 1, rng.randint(2, 300), rng.randint(300, 1800)]) for _ in range(n)]
        q[0] = max(q[0], 1)
        kv = [k + rng.choice([0, rng.randint(0, 500), rng.randint(0, 20000)]) for k in q]
        Mixed((G * R, G, d), q, kv, rng.choice([0, rng.randint(1, 9000)]), rng.choice([8, 16, 24, 64, 128, 200]),
              dtype=rng.choice([BF, BF, F32]), seed=seed).check_items()


@pytest.mark.parametrize("n", [1024, 1025, 2300])
@pytest.mark.parametrize("prefix", [0, 150])
def test_more_sequences_than_the_planner_holds_at_a_time(n, prefix):
    q = [(1, 0, 2, 1, 30, 1, 1)[i % 7] for i in range(n)]
    kv = [q[i] + (13 * i) % 60 + (3000 if i % 700 == 5 else 0) for i in range(n)]
    c = Mixed((4, 2, 64), q, kv, prefix, 16, seed=53)
    c.check_items()
    c.check_attention()


@pytest.mark.parametrize("heads", [(4, 4, 128), (8, 4, 64), (4, 2, 96)])
def test_items_of_output_rows_before_items_of_partial_rows(heads):
    """Every CTA goes from items that write whole output rows, by bulk copies, to items that write partial rows from
    the same staging buffer, and back; short items, so that the one follows close behind the other."""
    R = heads[0] // heads[1]
    q = [128 // R if i % 3 else 20 for i in range(180)]
    kv = [n if i % 3 else 9000 - 17 * i for i, n in enumerate(q)]
    c = Mixed(heads, q, kv, 0, 64, seed=54)
    c.check_items()
    kinds = [i[7] >= 0 for i in c.items().tolist()]
    assert 100 < sum(kinds) < len(kinds) - 100
    first = c.check_attention()
    for _ in range(20):
        out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
        B.prefix_attention(c.q, c.cache, c.step, heads[2] ** -0.5, out, lse, c.plan)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
