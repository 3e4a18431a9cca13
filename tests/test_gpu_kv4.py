"""The cache in 4 bits on the GPU: appends against the 64-bit quantiser's codes, reading back, and attention against a
64-bit form over the same codes.

Tolerances, derived from the formats (u = 2^-8: half a unit of bf16's last place, relative; e = 2^-24: of fp32's; a
tensor-core sum is taken to cut off 2 e of its running value with each 16 terms):
  codes, scales     equal: the rounding is that of the exact value
  queries           u |ref| + 16 e (|terms|) for bf16, 16 e (|terms|) for fp32
  attention, bf16   each probability is rounded to 11 bits (2^-11 relative, below 2^-21 of the largest 2^-32 of it), the
                    output once: u |out| + (2^-11 + score + sum) mag + keys 2^-31 max|v|, mag = sum p|v| / sum p
  attention, fp32   (2^-20 + score + sum) mag + keys 2^-31 max|v|: queries and probabilities of 22 bits (2^-22 each, twice
                    over), fp32 sums of 16 keys at a time
  score             (2 d + 16) e max_j sum_i |q_i k_ji| scale, and 2^-22 of it for fp32 queries in two parts; the
                    argument of the exponential is rounded where it is largest: 4 e of the same bound
  sum               (keys + 32) 2 e
"""
import math

import numpy as np
import pytest

from oracle import kv4 as K

torch = pytest.importorskip("torch")

from transformer_sharding_affinity_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


class Case:
    """A step and its cache in 4 bits: page tables in random order, every byte that is no valid token's 0xFF."""

    def __init__(self, heads, q_lens, kv_lens, prefix=0, page=16, dtype=BF, pad=0, seed=0, k_scale=1.0, v_scale=0.25,
                 extra_pages=2, page_major=True):
        H, G, d = self.heads = heads
        self.q_lens, self.kv_lens, self.prefix, self.page, self.dtype = q_lens, kv_lens, prefix, page, dtype
        self.scales = k_scale, v_scale
        rng = self.rng = np.random.default_rng(seed)
        self.T = sum(q_lens) + pad
        counts = [-(-n // page) for n in kv_lens]
        n_pre = -(-prefix // page)
        n_pages = n_pre + sum(counts) + extra_pages
        order = rng.permutation(n_pages).tolist()
        self.prefix_ids = order[:n_pre]
        self.ids, at = [], n_pre
        for n in counts:
            self.ids.append(order[at:at + n])
            at += n
        width = max(counts + [1])
        table = torch.tensor([i + [-7] * (width - len(i)) for i in self.ids], dtype=torch.int32)
        nb = K.page_bytes(page, d)
        self.pools = [np.full((n_pages, G, nb), 0xFF, dtype=np.uint8) for _ in range(2)]
        nc = -(-d // 32)
        for pool, g in zip(self.pools, self.scales):
            for ids, n in [(self.prefix_ids, prefix)] + list(zip(self.ids, kv_lens)):
                for p0, pid in enumerate(ids):
                    m = min(page, n - p0 * page)
                    codes, sc = K.quantise(rng.standard_normal((m, G, d)) * 1.3, g)
                    full = np.zeros((m, G, 32 * nc), dtype=np.uint8)
                    full[..., :d] = codes
                    pool[pid, :, :m * 16 * nc] = (full[..., 0::2] | full[..., 1::2] << 4).transpose(1, 0, 2).reshape(G, -1)
                    for t in range(m):
                        a = page * 16 * nc + t // 4 * 8 * nc + t % 4
                        pool[pid, :, a:a + 4 * (d // 16):4] = sc[t]
                        pool[pid, :, a + 4 * (d // 16):a + 8 * nc:4] = 0
        self.q = torch.tensor(rng.standard_normal((self.T, H, d))).to(dtype)
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.dev = {"q_start": torch.tensor(starts, dtype=torch.int32).cuda(),
                    "kv_len": torch.tensor(kv_lens, dtype=torch.int32).cuda(), "pages": table.cuda(),
                    "prefix_pages": torch.tensor(self.prefix_ids, dtype=torch.int32).cuda() if n_pre else None}
        self.upload(page_major)

    def upload(self, page_major=True):
        up = [torch.tensor(p).cuda() for p in self.pools]
        if not page_major:      # [group][page]
            up = [p.transpose(0, 1).contiguous().transpose(0, 1) for p in up]
        self.kd, self.vd = up
        self.cache = B.kv4_cache(self.kd, self.vd, self.page, self.heads[2], self.dtype, *self.scales)
        self.step = B.step(self.T, self.heads[0], prefix_len=self.prefix, **self.dev)
        self.plan = torch.empty(B.step_plan_size(self.step, self.cache), dtype=torch.uint8, device="cuda")
        B.step_plan(self.step, self.cache, self.plan)

    def rows(self, which, ids, n):
        """[n, G, d] in 64 bits."""
        G, d = self.heads[1:]
        if n == 0:
            return torch.zeros(0, G, d, dtype=torch.float64)
        v = K.values(*K.get(self.pools[which][ids], self.page, d), self.scales[which])
        return torch.tensor(v.transpose(0, 2, 1, 3).reshape(-1, G, d)[:n])

    def attend(self, scale):
        """(out, lse, mag, max_j sum_i |q_i k_ji| scale) in 64 bits."""
        H, G, d = self.heads
        R = H // G
        out = torch.zeros(self.T, H, d, dtype=torch.float64)
        mag, dots = torch.zeros_like(out), torch.zeros(self.T, H, dtype=torch.float64)
        lse = torch.full((self.T, H), -math.inf, dtype=torch.float64)
        kp, vp = (self.rows(w, self.prefix_ids, self.prefix) for w in (0, 1))
        for b, (n, length) in enumerate(zip(self.q_lens, self.kv_lens)):
            ko, vo = (torch.cat([x, self.rows(w, self.ids[b], length)]) for w, x in ((0, kp), (1, vp)))
            for i in range(n):
                t, seen = self.starts[b] + i, self.prefix + length - n + i + 1
                if length - n + i < 0:
                    continue
                q = self.q[t].double().view(G, R, d)
                k, v = ko[:seen].transpose(0, 1), vo[:seen].transpose(0, 1)
                s = torch.einsum("grd,gkd->grk", q, k) * scale
                m = s.amax(-1, keepdim=True)
                p = (s - m).exp()
                z = p.sum(-1, keepdim=True)
                out[t] = (p @ v / z).reshape(H, d)
                mag[t] = (p @ v.abs() / z).reshape(H, d)
                lse[t] = (m + z.log()).reshape(H)
                dots[t] = (torch.einsum("grd,gkd->grk", q.abs(), k.abs()).amax(-1) * scale).reshape(H)
        return out, lse, mag, dots

    def run(self, scale=None, q=None, **kw):
        H, G, d = self.heads
        out = torch.full((self.T, H, d), math.nan, dtype=self.dtype, device="cuda")
        lse = torch.full((self.T, H), math.nan, device="cuda")
        B.kv4_attention(self.q.cuda() if q is None else q, self.cache, self.step, d ** -0.5 if scale is None else scale, out,
                        lse, self.plan, **kw)
        assert B.device_status(self.plan) == B.AFF_OK
        return out, lse

    def bounds(self, ref, rlse, mag, dots):
        d, keys = self.heads[2], self.prefix + max(self.kv_lens + [1])
        vmax = max([float(self.rows(1, i, n).abs().max()) for i, n in [(self.prefix_ids, self.prefix)] +
                    list(zip(self.ids, self.kv_lens)) if n] + [0.0])
        score = (2 * d + 20) * E * dots
        sums = (keys + 32) * 2 * E
        if self.dtype == BF:
            tol = U * ref.abs() + (2.0 ** -11 + score + sums)[..., None] * mag * (1 + U) + keys * 2.0 ** -31 * vmax
        else:
            score = score + 2.0 ** -22 * dots
            tol = (2.0 ** -20 + score + sums)[..., None] * mag + keys * 2.0 ** -31 * vmax
        return tol, score + sums + 8 * E * (1 + rlse.abs())

    def check(self, scale=None, q=None, **kw):
        scale = self.heads[2] ** -0.5 if scale is None else scale
        out, lse = self.run(scale, q, **kw)
        ref, rlse, mag, dots = self.attend(scale)
        tol, ltol = self.bounds(ref, rlse, mag, dots)
        err = (out.cpu().double() - ref).abs()
        assert not torch.isnan(err).any()
        assert (err <= tol).all(), ((err - tol).max(), (err / tol.clamp(min=1e-30)).max())
        got = lse.cpu().double()
        assert torch.equal(torch.isinf(got), torch.isinf(rlse))
        seen = ~torch.isinf(rlse)
        assert ((got - rlse).abs()[seen] <= ltol[seen]).all()
        return out, lse


# ---------------------------------------------------------------- attention

HEADS = [(4, 2, 128), (2, 2, 64), (6, 2, 96), (3, 1, 80), (4, 4, 16), (8, 1, 48), (10, 2, 32), (9, 1, 112)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("prefix", [0, 1, 130])
def test_single_tokens(heads, prefix):
    """Decoding: sequences of one token to a few tiles, one of them without a query."""
    Case(heads, [1, 1, 1, 0, 1, 1], [1, 16, 17, 5, 128, 300], prefix).check()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("prefix,page", [(0, 16), (128, 8), (77, 24)])
def test_prompts(heads, prefix, page):
    """Whole and continued prompts of odd lengths, several row tiles, a sequence with no key at all."""
    Case(heads, [150, 1, 0, 33, 20], [150, 140, 9, 64, 21], prefix, page, seed=1).check()


@pytest.mark.parametrize("page", [8, 40, 64, 128, 136, 200, 256])
@pytest.mark.parametrize("page_major", [False, True])
def test_page_sizes_and_orders(page, page_major):
    Case((4, 2, 128), [1, 3, 130], [200, 129, 131], 70, page, seed=2, page_major=page_major).check()


def test_long_keys_are_cut_and_joined():
    """Few rows, many keys: items along the keys, partial rows, the join."""
    Case((4, 2, 64), [1, 2], [3001, 2500], 0, seed=3).check()
    Case((4, 2, 64), [1, 2, 1], [701, 90, 1], 4100, page=64, seed=4).check()
    Case((2, 1, 128), [140], [2000], 1000, page=64, seed=5).check()


def test_many_sequences_share_a_prefix():
    """More rows than a row tile behind one prefix: row tiles run across sequences."""
    n = 150
    Case((8, 2, 64), [1] * n, [1 + (7 * i) % 40 for i in range(n)], 260, seed=6).check()


@pytest.mark.parametrize("prefix", [0, 300])
def test_many_items_of_every_kind(prefix):
    """Every CTA takes several items in turn: single rows, a few tokens, more than one row tile; short and long keys."""
    n = 170
    q = [(1, 1, 20, 1, 9, 150, 1)[i % 7] if i % 31 else 0 for i in range(n)]
    kv = [max(q[i], 1 + (37 * i) % 400) for i in range(n)]
    c = Case((4, 4, 64), q, kv, prefix, page=24, seed=30)
    first = c.check()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run()))


@pytest.mark.parametrize("few", [True, False])
def test_a_long_prompt_among_single_tokens(few):
    """Items of few rows and of whole row tiles in one step, on either side of the rule on rows a sequence."""
    n = 60 if few else 4
    Case((4, 2, 128), [400] + [1] * n, [430] + [1 + (11 * i) % 300 for i in range(n)], 50, page=16, seed=31).check()


def test_padding_rows_are_zero():
    """Queries before the first key, tokens past the last sequence, sequences without keys."""
    for dtype in (BF, F32):
        for prefix in (0, 40):
            c = Case((4, 2, 64), [3, 2, 1], [2, 0, 9], prefix, pad=5, seed=7, dtype=dtype)
            out, lse = c.check()
            for t in (0, 3, 4, 6, 10):
                assert not out[t].any() and torch.isinf(lse[t]).all()
        c = Case((4, 2, 64), [0], [4], 20, pad=2, seed=8, dtype=dtype)
        out, _ = c.check()
        assert not out.any()
        Case((2, 2, 64), [300], [200], 0, pad=300, seed=9, dtype=dtype).check()


@pytest.mark.parametrize("heads", [(4, 2, 128), (6, 2, 96), (4, 2, 16), (3, 1, 64)])
@pytest.mark.parametrize("q_lens,kv_lens,prefix", [([1, 1, 0, 1], [1, 17, 3, 300], 0), ([1, 1, 1], [5, 64, 130], 200),
                                                   ([70, 3, 0, 20], [70, 129, 9, 21], 45), ([2], [2500], 0)])
def test_fp32(heads, q_lens, kv_lens, prefix):
    Case(heads, q_lens, kv_lens, prefix, dtype=F32, seed=10).check()


def test_strided_queries_and_scale():
    c = Case((4, 2, 64), [5, 1], [9, 30], 20, seed=11)
    wide = torch.zeros(c.T, 4 * 64 + 64, dtype=BF, device="cuda")
    wide[:, 64:] = c.q.flatten(1).cuda()
    c.check(q=wide[:, 64:].unflatten(1, (4, 64)))
    c.check(scale=0.7)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [40, 70]), ([140, 3], [150, 60])])
@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 60, 2.0 ** -20])
def test_queries_of_any_size(dtype, q_lens, kv_lens, factor):
    """Far outside fp16's range; the scale brings the scores back."""
    c = Case((4, 2, 64), q_lens, kv_lens, 33, dtype=dtype, seed=12)
    c.q = (c.q.float() * factor).to(dtype)
    c.check(scale=float(np.float32(0.125 / factor)))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sharp_and_growing_scores(dtype):
    """Scores that grow from tile to tile by more than the rescaling step, and one-hot rows."""
    c = Case((2, 1, 64), [2, 140], [700, 640], 0, seed=13, dtype=dtype)
    for ids, n in zip(c.ids, c.kv_lens):
        for j in range(n):
            page = c.pools[0][ids[j // 16], 0]
            codes, scales = (x[j % 16] for x in K.get(page, 16, 64))
            K.put(page, j % 16, 16, *K.quantise(K.values(codes, scales, 1.0) * (1 + j / 64) * 4, 1.0))
    c.upload()
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_lens,kv_lens,prefix", [([1, 20], [30, 20], 30), ([150], [200], 0), ([4], [300], 0)])
def test_nan_in_the_cache_reaches_the_rows_that_see_it(dtype, q_lens, kv_lens, prefix):
    """A block of NaN values makes its 16 columns NaN in the rows that see the key, a block of NaN keys the whole row;
    the other rows are as without it."""
    c = Case((4, 2, 64), q_lens, kv_lens, prefix, dtype=dtype, seed=14)
    clean, _ = c.check()
    for which, token in [(1, kv_lens[-1] - 3), (0, kv_lens[-1] - 2), (1, kv_lens[-1] - q_lens[-1])]:
        b = len(q_lens) - 1
        kept = c.pools[which].copy()
        page = c.pools[which][c.ids[b][token // 16], 1]          # of group 1: heads 2 and 3
        at = 16 * 32 + token % 16 // 4 * 16 + 2 * 4 + token % 4   # block 2: columns 32 .. 47
        page[at] = 0x7F
        c.upload()
        out, _ = c.run()
        c.pools[which] = kept
        sees = torch.zeros(c.T, dtype=torch.bool)
        for i in range(q_lens[b]):
            sees[c.starts[b] + i] = kv_lens[b] - q_lens[b] + i >= token
        cols = slice(32, 48) if which else slice(0, 64)
        assert torch.isnan(out[sees][:, 2:, cols]).all()
        want = clean.clone()
        want[sees.nonzero().flatten().cuda()[:, None], torch.tensor([2, 3]).cuda(), cols] = 0
        out[sees.nonzero().flatten().cuda()[:, None], torch.tensor([2, 3]).cuda(), cols] = 0
        assert torch.equal(out, want)


def test_a_nan_in_the_prefix_reaches_every_row():
    for q_lens, kv_lens in [([1, 1, 1], [5, 9, 300]), ([140, 1], [150, 20])]:
        c = Case((4, 2, 64), q_lens, kv_lens, 100, seed=15)
        page = c.pools[1][c.prefix_ids[3], 0]
        page[16 * 32 + 1 * 4] = 0x7F                # token 48, block 1
        c.upload()
        out, _ = c.run()
        assert torch.isnan(out[:, :2, 16:32]).all()
        assert not torch.isnan(out[:, 2:]).any() and not torch.isnan(out[:, :2, :16]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_and_nan_queries_stay_in_their_rows(dtype):
    c = Case((2, 1, 64), [20, 1], [20, 40], 30, seed=16, dtype=dtype)
    clean, _ = c.check()
    q = c.q.cuda().clone()
    q[7, 1, 3], q[20, 0, 5] = math.nan, math.nan
    out, _ = c.run(q=q)
    assert torch.isnan(out[7, 1]).all() and torch.isnan(out[20, 0]).all()
    out[7, 1], out[20, 0] = clean[7, 1], clean[20, 0]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("q_lens,kv_lens,prefix", [([4], [300], 0), ([3, 1], [1, 40], 0), ([150], [200], 0), ([140], [100], 30),
                                                   ([1] * 9, [70] * 9, 200)])
def test_rows_with_an_infinity_are_nan(q_lens, kv_lens, prefix, dtype):
    """Whatever the signs of the keys' elements: no row is taken for one that sees nothing.  Rows that see nothing stay so."""
    c = Case((4, 2, 64), q_lens, kv_lens, prefix, seed=18, dtype=dtype)
    clean, lse = c.check()
    for value in (math.inf, -math.inf):
        q = c.q.cuda().clone()
        rows = [(0, 1), (c.T - 1, 0), (c.T - 1, 3)]
        for t, h in rows:
            q[t, h, 5] = value
            q[t, h, 6] = 1e30
        out, got = c.run(q=q)
        for t, h in rows:
            if math.isinf(lse[t, h]):
                assert not out[t, h].any() and math.isinf(got[t, h])
            else:
                assert torch.isnan(out[t, h]).all() and math.isnan(got[t, h])
            out[t, h], got[t, h] = clean[t, h], lse[t, h]
        assert torch.equal(out, clean) and torch.equal(got, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("prefix", [0, 40])
def test_items_of_few_and_of_more_rows_one_after_the_other(dtype, prefix):
    """2, 4, 6 and 8 rows, several items to every CTA, from one key to some hundred."""
    rng = np.random.default_rng(19)
    q_lens = rng.choice([0, 1, 2, 3, 4], 500).tolist()
    kv_lens = [n + int(rng.integers(0, 5) if i % 3 else rng.integers(0, 200)) for i, n in enumerate(q_lens)]
    Case((8, 4, 32), q_lens, kv_lens, prefix, page=16, seed=31, dtype=dtype).check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_results_repeat_bit_for_bit(dtype):
    c = Case((4, 2, 128), [1, 40, 1], [900, 200, 3], 1500, seed=17, dtype=dtype)
    first = c.run()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, c.run()))


# ---------------------------------------------------------------- appends and reading back

def _append(c, rot, interleaved=False, norm=True, eps=1e-6, x=None, n_pos=None):
    """Runs an append; checks every byte of the pools, the queries and what is read back."""
    H, G, d = c.heads
    rng = c.rng
    n_pos = n_pos or c.prefix + max(c.kv_lens)
    ang = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    cos, sin = (torch.tensor(f(ang), dtype=F32) for f in (np.cos, np.sin))
    qkv = torch.tensor(rng.standard_normal((c.T, (H + 2 * G) * d))).to(c.dtype) if x is None else x
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([H * d, G * d, G * d], 1))
    gains = [torch.tensor(1 + 0.2 * rng.standard_normal(d)).to(c.dtype) if norm else None for _ in range(2)]
    dev = qkv.cuda()
    dq, dk, dv = (t.unflatten(1, (-1, d)) for t in dev.split([H * d, G * d, G * d], 1))
    r = B.rotary(cos.cuda(), sin.cuda(), interleaved, *[t.cuda() if norm else None for t in gains], eps)
    out = torch.full((c.T, H, d), math.nan, dtype=c.dtype, device="cuda")
    B.kv4_append(dq, dk, dv, c.cache, c.step, r, out, c.plan)
    kb, vb = (torch.full((c.T, G, d), 7.0, dtype=c.dtype, device="cuda") for _ in range(2))
    B.kv4_read(c.cache, c.step, kb, vb, c.plan)
    assert B.device_status(c.plan) == B.AFF_OK
    want = [p.copy() for p in c.pools]
    back = [np.zeros((c.T, G, d)) for _ in range(2)]
    ref_q, terms = np.zeros((c.T, H, d)), np.zeros((c.T, H, d))
    g64 = [None if t is None else t.double().numpy() for t in gains]
    cos, sin = cos.numpy(), sin.numpy()
    for b, (n, length) in enumerate(zip(c.q_lens, c.kv_lens)):
        own = np.arange(length - n, length)
        at = np.arange(c.starts[b], c.starts[b + 1])[own >= 0]
        own = own[own >= 0]
        if not len(own):
            continue
        pos = own + c.prefix
        ref_q[at] = K.turned(q[at].double().numpy(), pos, cos, sin, g64[0], eps, interleaved)
        terms[at] = K.turned(np.abs(q[at].double().numpy()), pos, np.abs(cos), -np.abs(sin),
                             None if g64[0] is None else np.abs(g64[0]), eps, interleaved) if rot else np.abs(ref_q[at])
        terms[at] = np.maximum(np.abs(terms[at]), np.abs(K.turned(np.abs(q[at].double().numpy()), pos, np.abs(cos),
                                                                   np.abs(sin), None if g64[0] is None else np.abs(g64[0]),
                                                                   eps, interleaved))) if rot else terms[at]
        keys = K.turned(k[at].double().numpy(), pos, cos, sin, g64[1], eps, interleaved)
        for w, rows in ((0, keys), (1, v[at].double().numpy())):
            codes, scales = K.quantise(rows, c.scales[w])
            back[w][at] = K.values(codes, scales, c.scales[w])
            for j, o in enumerate(own):
                for h in range(G):
                    K.put(want[w][c.ids[b][o // c.page], h], o % c.page, c.page, codes[j, h], scales[j, h])
    got = out.cpu().double().numpy()
    assert (np.abs(got - ref_q) <= (U if c.dtype == BF else 0) * np.abs(ref_q) + 16 * E * terms).all()
    for w, pool in enumerate((c.kd, c.vd)):
        new = pool.cpu().numpy()
        # the sign of a code that stands for 0 is free
        zero = lambda p: [np.where(x & 7 == 0, 0, x) for x in K.get(p, c.page, d)[:1]][0]
        assert (K.get(new, c.page, d)[1] == K.get(want[w], c.page, d)[1]).all()
        assert (zero(new) == zero(want[w])).all()
        nc = -(-d // 32)
        if d % 32:
            pad = lambda p: p[..., :c.page * 16 * nc].reshape(-1, 16 * nc)[:, d // 2:]
            assert (pad(new) == pad(want[w])).all()
        ref = torch.tensor(back[w]).to(c.dtype).double().numpy()
        assert np.array_equal((kb, vb)[w].cpu().double().numpy() + 0.0, ref + 0.0, equal_nan=True)
    return out


@pytest.mark.parametrize("heads,rot", [((4, 2, 128), 128), ((4, 2, 128), 64), ((6, 2, 96), 96), ((6, 3, 96), 48), ((5, 5, 80), 80),
                                       ((3, 1, 80), 32), ((4, 4, 16), 16), ((2, 2, 16), 0), ((2, 1, 256), 256), ((7, 1, 112), 112),
                                       ((4, 2, 48), 48), ((3, 1, 208), 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved,norm", [(False, True), (True, False), (True, True), (False, False)])
def test_append(heads, rot, dtype, interleaved, norm):
    c = Case(heads, [5, 1, 0, 33], [5, 40, 3, 50], 19, page=24, dtype=dtype, seed=20, k_scale=0.5)
    _append(c, rot, interleaved, norm)


@pytest.mark.parametrize("page", [8, 16, 64, 200])
def test_append_pages_and_padding(page):
    """Single tokens, queries before the first key, tokens past the last sequence."""
    c = Case((4, 2, 64), [1, 3, 2, 1], [9, 2, 0, page + 1], 0, page=page, pad=5, seed=21)
    out = _append(c, 64)
    for t in (1, 4, 5, 7, 11):
        assert not out[t].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_no_key_falls_on_the_wrong_side_of_a_border(dtype, interleaved):
    """4 million rotated and normalised elements, some hundred of them nearer to a border than fp32 is sure of."""
    c = Case((8, 8, 128), [4096], [4096], 0, page=64, dtype=dtype, seed=22, k_scale=0.25)
    _append(c, 128, interleaved)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k_scale", [2.0 ** -30, 2.0 ** -28, 2.0 ** -26, 2.0 ** 30])
def test_keys_far_from_the_caches_scale(dtype, k_scale):
    """fp32's errors are whole codes where every block saturates, and nothing where every block is zero."""
    for norm, interleaved in [(True, False), (False, False), (True, True)]:
        c = Case((2, 2, 64), [64], [64], 0, page=64, dtype=dtype, seed=28, k_scale=k_scale)
        _append(c, 64, interleaved, norm)


@pytest.mark.parametrize("interleaved", [False, True])
def test_blocks_whose_rotation_cancels(interleaved):
    """The block is 2^-24 to 2^-8 of the products that it is the difference of: fp32 is sure of nothing, of some codes, of most."""
    c = Case((2, 2, 64), [340], [340], 0, page=40, dtype=F32, seed=29, k_scale=2.0 ** -12)
    rng = np.random.default_rng(30)
    ang = np.arange(340)[:, None] * 100.0 ** (-np.arange(32) / 32)
    co, si = (f(ang)[:, None] for f in (np.cos, np.sin))
    size = rng.standard_normal((340, 6, 32)) * 2.0 ** -rng.uniform(8, 24, (340, 6, 1))
    far = 1 + rng.random((340, 6, 32))
    if interleaved:                                # (whole blocks of neighbours: both of a pair)
        size[..., 1::2] = size[..., ::2]
    # z = (size, far) where it is turned back: x = z turned by the opposite angle
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    x = np.zeros((340, 6, 64))
    z = (size, size * 0.7) if interleaved else (size, far)
    x[..., a], x[..., b] = z[0] * co + z[1] * si, z[1] * co - z[0] * si
    _append(c, 64, interleaved, norm=False, x=torch.tensor(x.reshape(340, 384)).to(F32), n_pos=340)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_are_those_of_the_exact_values(dtype):
    """Elements and maxima on the borders, at position 0 (not turned at all), past the rotated part and in values."""
    for norm, rot in [(False, 64), (False, 16), (False, 0)]:
        c = Case((2, 2, 64), [64], [64], 0, page=64, dtype=dtype, seed=23, k_scale=1.0)
        rng = np.random.default_rng(24)
        grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
        x = rng.choice(grid, (64, 6 * 64)) * rng.choice([-1, 1], (64, 6 * 64))
        tops = rng.choice([6, 6 * 1.0625, 6 * 1.1875, 6 * 0.9375, 6 * 2.0 ** -9, 9 * 2.0 ** -9], (64, 6 * 4))
        x = x.reshape(64, 24, 16)
        x[:, :, 3] = tops
        x *= np.where(tops < 1, 2.0 ** -9, 1.0)[..., None]
        x[:, :, 3] = tops
        _append(c, rot, norm=norm, x=torch.tensor(x.reshape(64, 384)).to(dtype), n_pos=64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", [False, True])
def test_zeros_small_large_and_not_finite(dtype, norm):
    c = Case((2, 2, 64), [32], [32], 0, page=32, dtype=dtype, seed=25, k_scale=2.0 ** -10, v_scale=2.0 ** 10)
    rng = np.random.default_rng(26)
    x = rng.standard_normal((32, 6, 64)) * 2.0 ** rng.integers(-40, 40, (32, 6, 1))
    x[3] = 0
    x[4, :, 16:32] = 0
    x = torch.tensor(x.reshape(32, 384)).to(dtype)
    _append(c, 0, norm=norm, x=x)
    if not norm:
        c.upload()
        x.view(32, 6, 64)[5, 4:, 7], x.view(32, 6, 64)[6, 2:, 33], x.view(32, 6, 64)[7, 5, 60] = math.inf, math.nan, -math.inf
        q, k, v = (t.cuda().unflatten(1, (2, 64)) for t in x.split(128, 1))
        kb, vb = (torch.empty(32, 2, 64, dtype=dtype, device="cuda") for _ in range(2))
        one = torch.ones(32, 0, device="cuda")
        B.kv4_append(q, k, v, c.cache, c.step, B.rotary(one, one), torch.empty_like(q), c.plan)
        B.kv4_read(c.cache, c.step, kb, vb, c.plan)
        for name, got, src in (("k", kb, k), ("v", vb, v)):
            bad = ~torch.isfinite(src).unflatten(-1, (4, 16)).all(-1)
            assert bad.any() and torch.equal(torch.isnan(got).unflatten(-1, (4, 16)).all(-1), bad), name


def test_a_step_over_a_whole_sequence_reads_it():
    c = Case((4, 2, 96), [1], [150], 0, page=24, seed=27)
    whole = B.step(150, 4, torch.tensor([0, 150], dtype=torch.int32).cuda(), c.dev["kv_len"], c.dev["pages"])
    plan = torch.empty(B.step_plan_size(whole, c.cache), dtype=torch.uint8, device="cuda")
    B.step_plan(whole, c.cache, plan)
    for dtype in (BF,):
        k, v = (torch.empty(150, 2, 96, dtype=dtype, device="cuda") for _ in range(2))
        B.kv4_read(c.cache, whole, k, v, plan)
        assert B.device_status(plan) == B.AFF_OK
        assert torch.equal(k.cpu(), c.rows(0, c.ids[0], 150).to(dtype)) and torch.equal(v.cpu(), c.rows(1, c.ids[0], 150).to(dtype))


# ---------------------------------------------------------------- together, streams, graphs, plans

def test_append_attend_append_attend():
    """A prompt and three single tokens of four sequences, as they would be served; attention reads what was appended."""
    H, G, d, page = 4, 2, 64, 16
    g = torch.Generator().manual_seed(28)
    lens, more = [40, 7, 100, 1], 3
    n_pages = 40
    kp, vp = (torch.full((n_pages, G, B.kv4_page_bytes(page, d)), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = B.kv4_cache(kp, vp, page, d, BF, 0.5, 0.5)
    table = torch.tensor([[10 * b + i for i in range(10)] for b in range(4)], dtype=torch.int32).cuda()
    ang = torch.arange(200)[:, None] * 10.0 ** (-torch.arange(d // 2) / 8)
    r = B.rotary(ang.cos().float().cuda(), ang.sin().float().cuda())
    done = [0] * 4
    for new in [lens] + [[1] * 4] * more:
        done = [a + b for a, b in zip(done, new)]
        starts = np.cumsum([0] + new).tolist()
        s = B.step(starts[-1], H, torch.tensor(starts, dtype=torch.int32).cuda(), torch.tensor(done, dtype=torch.int32).cuda(), table)
        plan = torch.empty(B.step_plan_size(s, cache), dtype=torch.uint8, device="cuda")
        B.step_plan(s, cache, plan)
        q, k, v = (torch.randn(starts[-1], h, d, generator=g).to(BF).cuda() for h in (H, G, G))
        B.kv4_append(q, k, v, cache, s, r, q, plan)
        out = torch.empty_like(q)
        B.kv4_attention(q, cache, s, 0.125, out, None, plan)
        assert B.device_status(plan) == B.AFF_OK
        c = Case.__new__(Case)
        c.heads, c.q_lens, c.kv_lens, c.prefix, c.page, c.dtype, c.scales = (H, G, d), new, done, 0, page, BF, (0.5, 0.5)
        c.T, c.starts, c.prefix_ids, c.ids, c.q = starts[-1], starts, [], table.tolist(), q.cpu()
        c.pools = [kp.cpu().numpy(), vp.cpu().numpy()]
        ref, rlse, mag, dots = c.attend(0.125)
        assert ((out.cpu().double() - ref).abs() <= c.bounds(ref, rlse, mag, dots)[0]).all()


def test_another_stream_and_a_graph():
    c = Case((4, 2, 64), [1, 4, 40], [100, 30, 60], 50, seed=29)
    want, _ = c.run()
    q, out = c.q.cuda(), torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.step_plan(c.step, c.cache, c.plan, stream=s)
    B.kv4_attention(q, c.cache, c.step, 0.125, out, None, c.plan, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.step_plan(c.step, c.cache, c.plan)
        B.kv4_attention(q, c.cache, c.step, 0.125, out, None, c.plan)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_calls_in_a_row_take_and_leave_what_stands_between_them():
    """Single tokens behind a prefix: both of the attention's kernels, side by side at the first one's end.  Queries are written
    just before each call, outputs and partial rows just after; each result is that of the call by itself."""
    rng = np.random.default_rng(34)
    own = rng.integers(1, 400, 200).tolist()
    c = Case((8, 2, 128), [1] * 200, own, 5000, page=64, seed=35)
    base = c.q.cuda()
    factors = [1.0, -0.5, 2.0, 0.25, -1.5, 0.75]
    want = []
    for f in factors:
        q = base * f
        torch.cuda.synchronize()
        out, lse = c.run(q=q)
        torch.cuda.synchronize()
        want.append((out.clone(), lse.clone()))
    q = torch.empty_like(base)
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    got = [(torch.empty_like(out), torch.empty_like(lse)) for _ in factors]

    def chain():
        for f, (o, l) in zip(factors, got):
            torch.mul(base, f, out=q)
            B.kv4_attention(q, c.cache, c.step, 128 ** -0.5, out, lse, c.plan)
            o.copy_(out)
            l.copy_(lse)

    def same():
        torch.cuda.synchronize()
        assert B.device_status(c.plan) == B.AFF_OK
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            a[0].zero_()
            a[1].zero_()

    for _ in range(5):
        chain()
        same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(5):
        graph.replay()
        same()


def test_a_plan_of_the_other_kind_or_of_a_malformed_step_is_reported():
    c = Case((4, 2, 64), [2, 1], [20, 9], 0, seed=32)
    k = torch.zeros(c.kd.shape[0], 2, 16, 64, dtype=BF, device="cuda")
    other = B.kv_cache(k, k.clone())
    plan = torch.empty(max(B.step_plan_size(c.step, other), B.step_plan_size(c.step, c.cache)), dtype=torch.uint8, device="cuda")
    q, out = c.q.cuda(), torch.full((c.T, 4, 64), 3.0, dtype=BF, device="cuda")
    one = torch.ones(64, 0, device="cuda")
    calls = [lambda: B.kv4_attention(q, c.cache, c.step, 0.125, out, None, plan),
             lambda: B.kv4_append(q, q[:, :2].contiguous(), q[:, :2].contiguous(), c.cache, c.step, B.rotary(one, one), out,
                                  plan),
             lambda: B.kv4_read(c.cache, c.step, out[:, :2].contiguous(), out[:, 2:].contiguous(), plan)]
    B.step_plan(c.step, other, plan)
    before = [c.kd.clone(), c.vd.clone()]
    for f in calls:
        f()
        assert B.device_status(plan) == B.AFF_ERR_INVALID_ARG
    c.dev["kv_len"].copy_(torch.tensor([20, 10 ** 6], dtype=torch.int32))
    B.step_plan(c.step, c.cache, plan)
    assert B.device_status(plan) == B.AFF_ERR_RANGE
    for f in calls:
        f()
        assert B.device_status(plan) == B.AFF_ERR_RANGE
    assert (out == 3).all() and torch.equal(before[0], c.kd) and torch.equal(before[1], c.vd)


def test_pages_outside_the_pool_are_reported():
    c = Case((4, 2, 64), [1, 1], [40, 300], 0, seed=33)
    c.dev["pages"][1, 3] = c.kd.shape[0]
    B.step_plan(c.step, c.cache, c.plan)
    out = torch.empty(c.T, 4, 64, dtype=BF, device="cuda")
    B.kv4_attention(c.q.cuda(), c.cache, c.step, 0.125, out, None, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    c.dev["pages"][1, 3] = -1
    c.dev["pages"][1, -1] = 10 ** 6            # of the token itself
    B.step_plan(c.step, c.cache, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    before = c.kd.clone()
    q = c.q.cuda()
    one = torch.ones(512, 0, device="cuda")
    k = q[:, :2].contiguous()
    kb, vb = torch.ones_like(k), torch.ones_like(k)
    last = c.ids[0][39 // 16]
    B.kv4_append(q, k, k, c.cache, c.step, B.rotary(one, one), q, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    changed = (before != c.kd).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [last]
    B.kv4_read(c.cache, c.step, kb, vb, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    assert not kb[1].any() and kb[0].any()


def test_positions_past_the_rotary_table_are_reported_and_not_stored():
    c = Case((4, 2, 64), [2], [20], 0, seed=34)
    before = c.kd.clone()
    one = torch.ones(19, 32, device="cuda")
    q = c.q.cuda()
    B.kv4_append(q, q[:, :2].contiguous(), q[:, :2].contiguous(), c.cache, c.step, B.rotary(one, one), q, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    rows = K.get(c.kd.cpu().numpy(), 16, 64)[0]
    old = K.get(before.cpu().numpy(), 16, 64)[0]
    page, at = c.ids[0][1], 19 % 16
    assert (rows[page, :, at] == old[page, :, at]).all() and (rows[page, :, 18 % 16] != old[page, :, 18 % 16]).any()
