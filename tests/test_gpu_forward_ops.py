"""The forward-pass operators on the GPU against plain 64-bit forms: appending to a paged cache, attention over it
behind a shared prefix, and the norms around a block.

Tolerances, derived from the formats (u = 2^-8: half a unit of bf16's last place, relative; e = 2^-24: of fp32's):
  attention, bf16   each probability is rounded to bf16 once and the output once:
                    |err| <= u |out| + (u + score error) sum_j p_j |v_j| / sum_j p_j, with 5 % on top
  attention, fp32   score error + (keys + 16) e, times the same sum, twice over
  score error       (d + 4) e max_j sum_i |q_i k_ji| scale, the bound of a d-term fp32 dot product
  append, norms     u |ref| + 16 e (|terms|) for bf16, 16 e (|terms|) for fp32: a sum of squares in fp32, a
                    reciprocal root and up to four products
"""
import math

import pytest

torch = pytest.importorskip("torch")

from transformer_sharding_affinity_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- a step and its plain forms

class Case:
    """A step with its cache: page tables in random order, everything that is not a valid token NaN."""

    def __init__(self, heads, q_lens, kv_lens, prefix=0, page=16, dtype=BF, token_major=False, pad=0, seed=0,
                 garbage=math.nan, extra_pages=2):
        H, G, d = self.heads = heads
        self.q_lens, self.kv_lens, self.prefix, self.page, self.dtype = q_lens, kv_lens, prefix, page, dtype
        g = torch.Generator().manual_seed(seed)
        self.T = sum(q_lens) + pad
        counts = [-(-n // page) for n in kv_lens]
        n_pre = -(-prefix // page)
        n_pages = n_pre + sum(counts) + extra_pages
        order = torch.randperm(n_pages, generator=g).tolist()
        self.prefix_ids = order[:n_pre]
        self.ids, at = [], n_pre
        for n in counts:
            self.ids.append(order[at:at + n])
            at += n
        width = max(counts + [1])
        table = torch.tensor([i + [-7] * (width - len(i)) for i in self.ids], dtype=torch.int32)
        shape = (n_pages, page, G, d) if token_major else (n_pages, G, page, d)
        pools = [torch.full(shape, garbage, dtype=dtype) for _ in range(2)]
        self.k, self.v = [p.transpose(1, 2) if token_major else p for p in pools]
        for ids, n in [(self.prefix_ids, prefix)] + list(zip(self.ids, kv_lens)):
            for j in range(n):
                self.k[ids[j // page], :, j % page] = torch.randn(G, d, generator=g).to(dtype)
                self.v[ids[j // page], :, j % page] = torch.randn(G, d, generator=g).to(dtype)
        self.q = torch.randn(self.T, H, d, generator=g).to(dtype)
        self.gen = g
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.dev = {"q_start": torch.tensor(starts, dtype=torch.int32).cuda(),
                    "kv_len": torch.tensor(kv_lens, dtype=torch.int32).cuda(), "pages": table.cuda(),
                    "prefix_pages": torch.tensor(self.prefix_ids, dtype=torch.int32).cuda() if n_pre else None}
        self.kd, self.vd = [p.cuda().transpose(1, 2) if token_major else p.cuda() for p in pools]
        self.cache = B.kv_cache(self.kd, self.vd)
        self.step = B.step(self.T, H, prefix_len=prefix, **self.dev)
        self.plan = torch.empty(B.step_plan_size(self.step, self.cache), dtype=torch.uint8, device="cuda")
        B.step_plan(self.step, self.cache, self.plan)

    def rows(self, pool, ids, n):
        """[n, G, d] in 64 bits."""
        if n == 0:
            return torch.zeros(0, pool.shape[1], pool.shape[3], dtype=torch.float64)
        return pool[ids].transpose(1, 2).flatten(0, 1)[:n].double()

    def attend(self, scale):
        """(out, lse, sum p|v| / sum p, max_j sum_i |q_i k_ji| scale) in 64 bits."""
        H, G, d = self.heads
        out = torch.zeros(self.T, H, d, dtype=torch.float64)
        mag, dots = torch.zeros_like(out), torch.zeros(self.T, H, dtype=torch.float64)
        lse = torch.full((self.T, H), -math.inf, dtype=torch.float64)
        kp, vp = self.rows(self.k, self.prefix_ids, self.prefix), self.rows(self.v, self.prefix_ids, self.prefix)
        for b, (n, length) in enumerate(zip(self.q_lens, self.kv_lens)):
            ko, vo = self.rows(self.k, self.ids[b], length), self.rows(self.v, self.ids[b], length)
            for i in range(n):
                t, own = self.starts[b] + i, length - n + i
                if own < 0:
                    continue
                ks, vs = torch.cat([kp, ko[:own + 1]]), torch.cat([vp, vo[:own + 1]])
                for h in range(H):
                    q, k, v = self.q[t, h].double(), ks[:, h // (H // G)], vs[:, h // (H // G)]
                    s = k @ q * scale
                    m = s.max()
                    p = (s - m).exp()
                    out[t, h] = p @ v / p.sum()
                    mag[t, h] = p @ v.abs() / p.sum()
                    lse[t, h] = m + p.sum().log()
                    dots[t, h] = (k.abs() @ q.abs()).max() * scale
        return out, lse, mag, dots

    def check_attention(self, scale=None, q=None):
        H, G, d = self.heads
        scale = d ** -0.5 if scale is None else scale
        out = torch.full((self.T, H, d), math.nan, dtype=self.dtype, device="cuda")
        lse = torch.full((self.T, H), math.nan, device="cuda")
        B.prefix_attention(self.q.cuda() if q is None else q, self.cache, self.step, scale, out, lse, self.plan)
        assert B.device_status(self.plan) == B.AFF_OK
        ref, rlse, mag, dots = self.attend(scale)
        keys = self.prefix + max(self.kv_lens + [1])
        score = (d + 4) * E * dots
        if self.dtype == BF:
            tol = U * ref.abs() + 1.05 * (U + score)[..., None] * mag
        else:
            tol = 2 * (score + (keys + 16) * E)[..., None] * mag
        err = (out.cpu().double() - ref).abs()
        assert not torch.isnan(err).any()
        assert (err <= tol).all(), (err - tol).max()
        got = lse.cpu().double()
        assert torch.equal(torch.isinf(got), torch.isinf(rlse))
        seen = ~torch.isinf(rlse)
        ltol = 2 * (score + (keys + 16) * E) + 4 * E * rlse.abs()
        assert ((got - rlse).abs()[seen] <= ltol[seen]).all()
        return out, lse


# ---------------------------------------------------------------- attention

HEADS = [(4, 2, 128), (2, 2, 64), (6, 2, 96), (3, 1, 72), (4, 4, 16), (8, 1, 80)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("prefix", [0, 1, 130])
def test_single_tokens(heads, prefix):
    """Decoding: sequences of one token to a few tiles, one of them without a query."""
    Case(heads, [1, 1, 1, 0, 1, 1], [1, 16, 17, 5, 128, 300], prefix).check_attention()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("prefix,page", [(0, 16), (128, 8), (77, 24)])
def test_prompts(heads, prefix, page):
    """Whole and continued prompts of odd lengths, several row tiles, a sequence with no key at all."""
    Case(heads, [150, 1, 0, 33, 20], [150, 140, 9, 64, 21], prefix, page, seed=1).check_attention()


@pytest.mark.parametrize("page", [8, 40, 64, 128, 136, 200, 256])
@pytest.mark.parametrize("token_major", [False, True])
def test_page_sizes_and_orders(page, token_major):
    Case((4, 2, 128), [1, 3, 130], [200, 129, 131], 70, page, token_major=token_major, seed=2).check_attention()


def test_long_keys_are_cut_and_joined():
    """Few rows, many keys: items along the keys, partial rows, the join."""
    Case((4, 2, 64), [1, 2], [3001, 2500], 0, seed=3).check_attention()
    Case((4, 2, 64), [1, 2, 1], [701, 90, 1], 4100, page=64, seed=4).check_attention()
    Case((2, 1, 128), [140], [2000], 1000, page=64, seed=5).check_attention()


def test_many_sequences_share_a_prefix():
    """More rows than a row tile behind one prefix: row tiles run across sequences."""
    n = 150
    Case((8, 2, 64), [1] * n, [1 + (7 * i) % 40 for i in range(n)], 260, seed=6).check_attention()


@pytest.mark.parametrize("prefix", [0, 300])
def test_many_items_of_every_kind(prefix):
    """Every CTA takes several items in turn: single rows, a few tokens, more than one row tile; short and long keys."""
    n = 170
    q = [(1, 1, 20, 1, 9, 150, 1)[i % 7] if i % 31 else 0 for i in range(n)]
    kv = [max(q[i], 1 + (37 * i) % 400) for i in range(n)]
    c = Case((4, 4, 64), q, kv, prefix, page=24, seed=30)
    first = c.check_attention()
    for _ in range(3):
        out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
        B.prefix_attention(c.q.cuda(), c.cache, c.step, 0.125, out, lse, c.plan)
        assert B.device_status(c.plan) == B.AFF_OK
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_padding_rows_are_zero():
    """Queries before the first key, tokens past the last sequence, sequences without keys."""
    for prefix in (0, 40):
        c = Case((4, 2, 64), [3, 2, 1], [2, 0, 9], prefix, pad=5, seed=7)
        out, lse = c.check_attention()
        for t in (0, 3, 4, 6, 10):
            assert not out[t].any() and torch.isinf(lse[t]).all()
    c = Case((4, 2, 64), [0], [4], 20, pad=2, seed=8)
    out, _ = c.check_attention()
    assert not out.any()
    Case((2, 2, 64), [300], [200], 0, pad=300, seed=9).check_attention()


@pytest.mark.parametrize("heads", [(4, 2, 128), (6, 2, 96), (4, 2, 16), (3, 1, 20)])
@pytest.mark.parametrize("q_lens,kv_lens,prefix", [([1, 1, 0, 1], [1, 17, 3, 300], 0), ([1, 1, 1], [5, 64, 130], 200),
                                                   ([70, 3, 0, 20], [70, 129, 9, 21], 45), ([2], [2500], 0)])
def test_fp32(heads, q_lens, kv_lens, prefix):
    Case(heads, q_lens, kv_lens, prefix, dtype=F32, seed=10).check_attention()


def test_strided_queries_and_scale():
    c = Case((4, 2, 64), [5, 1], [9, 30], 20, seed=11)
    wide = torch.zeros(c.T, 4 * 64 + 64, dtype=BF, device="cuda")
    wide[:, 64:] = c.q.flatten(1).cuda()
    c.check_attention(q=wide[:, 64:].unflatten(1, (4, 64)))
    c.check_attention(scale=0.7)


def test_sharp_and_growing_scores():
    """Scores that grow from tile to tile by more than the rescaling step, and one-hot rows."""
    c = Case((2, 1, 64), [2, 140], [700, 640], 0, seed=12)
    for ids, n in zip(c.ids, c.kv_lens):
        for j in range(n):
            f = (1 + j / 64) * 4
            c.k[ids[j // c.page], :, j % c.page] *= f
            c.kd[ids[j // c.page], :, j % c.page] *= f
    c.check_attention()


def test_infinite_and_nan_inputs_stay_in_their_rows():
    """A NaN query row gives a NaN row and leaves its tile mates alone."""
    c = Case((2, 1, 64), [20], [20], 30, seed=13)
    q = c.q.cuda().clone()
    q[7, 1, 3] = math.nan
    out = torch.empty(c.T, 2, 64, dtype=BF, device="cuda")
    B.prefix_attention(q, c.cache, c.step, 0.125, out, None, c.plan)
    assert torch.isnan(out[7, 1]).all()
    out[7, 1] = 0
    ref = c.attend(0.125)[0].cuda()
    ref[7, 1] = 0
    assert torch.allclose(out.double(), ref, rtol=0.02, atol=0.02)


def test_results_repeat_bit_for_bit():
    c = Case((4, 2, 128), [1, 40, 1], [900, 200, 3], 1500, seed=14)
    first = c.check_attention()
    again = c.check_attention()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_another_stream_and_a_graph():
    c = Case((4, 2, 64), [1, 4], [100, 30], 50, seed=15)
    want, _ = c.check_attention()
    q, out = c.q.cuda(), torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.step_plan(c.step, c.cache, c.plan, stream=s)
    B.prefix_attention(q, c.cache, c.step, 0.125, out, None, c.plan, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.step_plan(c.step, c.cache, c.plan)
        B.prefix_attention(q, c.cache, c.step, 0.125, out, None, c.plan)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_device_checks_latch_a_status():
    c = Case((4, 2, 64), [1, 1], [20, 30], 0, seed=16)
    q, out = c.q.cuda(), torch.empty(2, 4, 64, dtype=BF, device="cuda")
    # a plan made for another step
    other = B.step(1, 4, c.dev["q_start"][:2].contiguous(), c.dev["kv_len"][:1].contiguous(),
                   c.dev["pages"][:1].contiguous())
    B.prefix_attention(q[:1], c.cache, other, 0.125, out[:1], None, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_INVALID_ARG
    for name, value in (("q_start", [0, 2, 1]), ("kv_len", [-1, 4]), ("kv_len", [5, 1000])):
        bad = dict(c.dev)
        bad[name] = torch.tensor(value, dtype=torch.int32).cuda()
        s = B.step(2, 4, **bad)
        B.step_plan(s, c.cache, c.plan)
        B.prefix_attention(q, c.cache, s, 0.125, out, None, c.plan)
        assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    bad = dict(c.dev)
    bad["pages"] = torch.full_like(c.dev["pages"], 999)
    s = B.step(2, 4, **bad)
    B.step_plan(s, c.cache, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE


# ---------------------------------------------------------------- append

def _turn(z, cos, sin, rot, interleaved):
    z = z.clone()
    a = list(range(0, rot, 2)) if interleaved else list(range(rot // 2))
    b = list(range(1, rot, 2)) if interleaved else list(range(rot // 2, rot))
    x, y = z[..., a].clone(), z[..., b].clone()
    z[..., a], z[..., b] = x * cos - y * sin, x * sin + y * cos
    return z


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads,rot", [((4, 2, 128), 128), ((6, 2, 96), 48), ((3, 1, 72), 36), ((2, 1, 16), 2),
                                       ((2, 2, 256), 256), ((2, 1, 64), 0), ((2, 1, 80), 80)])
@pytest.mark.parametrize("interleaved,norm", [(False, True), (True, False)])
def test_append(dtype, heads, rot, interleaved, norm):
    H, G, d = heads
    c = Case(heads, [1, 7, 0, 3, 4], [1, 30, 5, 3, 2], 11, page=8, dtype=dtype, token_major=rot % 3 == 0, pad=2,
             seed=20, garbage=5.0)
    g = torch.Generator().manual_seed(21)
    qkv = torch.randn(c.T, (H + 2 * G) * d, generator=g).to(dtype)
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([H * d, G * d, G * d], 1))
    dev = qkv.cuda()
    qd, kd, vd = (t.unflatten(1, (-1, d)) for t in dev.split([H * d, G * d, G * d], 1))
    n_pos = 11 + 30
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * 0.3 ** torch.arange(rot // 2, dtype=torch.float64)[None]
    cos, sin = ang.cos().float(), ang.sin().float()
    gains = [(1 + 0.2 * torch.randn(d, generator=g)).to(dtype) for _ in range(2)] if norm else [None, None]
    rot_args = B.rotary(cos.cuda(), sin.cuda(), interleaved, *[x.cuda() if x is not None else None for x in gains])
    out = torch.full((c.T, H, d), math.nan, dtype=dtype, device="cuda")
    B.kv_append(qd, kd, vd, c.cache, c.step, rot_args, out, c.plan)
    assert B.device_status(c.plan) == B.AFF_OK
    want_q = torch.zeros(c.T, H, d, dtype=torch.float64)
    want_k, want_v = c.k.double(), c.v.double()
    mag_q, mag_k = torch.zeros_like(want_q), torch.zeros_like(want_k)

    def norm_of(z, gain):
        z = z.double()
        return z if gain is None else z / (z.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gain.double()

    for b, (n, length) in enumerate(zip(c.q_lens, c.kv_lens)):
        for i in range(n):
            t, own = c.starts[b] + i, length - n + i
            if own < 0:
                continue
            cs, sn = cos[11 + own].double(), sin[11 + own].double()
            zq, zk = norm_of(q[t], gains[0]), norm_of(k[t], gains[1])
            want_q[t] = _turn(zq, cs, sn, rot, interleaved)
            mag_q[t] = zq.abs().amax(-1, keepdim=True)
            page, off = c.ids[b][own // 8], own % 8
            want_k[page, :, off] = _turn(zk, cs, sn, rot, interleaved)
            mag_k[page, :, off] = zk.abs().amax(-1, keepdim=True)
            want_v[page, :, off] = v[t].double()
    half = U if dtype == BF else 0.0
    assert ((out.cpu().double() - want_q).abs() <= half * want_q.abs() + 32 * E * mag_q).all()
    assert ((c.kd.cpu().double() - want_k).abs() <= half * want_k.abs() + 32 * E * mag_k).all()
    assert torch.equal(c.vd.cpu().double(), want_v)
    # in place
    B.kv_append(qd, kd, vd, c.cache, c.step, rot_args, qd, c.plan)
    assert torch.equal(qd, out)


def test_append_latches_positions_past_the_table():
    c = Case((2, 1, 64), [3], [30], 0, seed=22)
    cos = torch.ones(20, 32, device="cuda")
    q = torch.randn(3, 4, 64, device="cuda").to(BF)
    out = torch.empty(3, 2, 64, dtype=BF, device="cuda")
    before = c.kd.clone()
    B.kv_append(q[:, :2], q[:, 2:3], q[:, 3:], c.cache, c.step, B.rotary(cos, cos), out, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    assert torch.equal(torch.nan_to_num(c.kd), torch.nan_to_num(before)) and not out.any()


# ---------------------------------------------------------------- norms

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 8), (5, 31), (7, 264), (2, 1000), (130, 1024), (3, 1536), (2, 4096),
                                 (2, 4100), (1, 8200), (2, 16384), (1, 16383)])
@pytest.mark.parametrize("post,gate,pre", [(True, "rows", True), (False, None, True), (True, "token", False),
                                           (False, "channel", False)])
def test_block_norm(dtype, T, D, post, gate, pre):
    g = torch.Generator().manual_seed(T * 7 + D)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)
    x, f = rnd(T, D) * 3, rnd(T, D)
    pg, qg = (1 + 0.1 * rnd(D)).to(dtype), (1 + 0.1 * rnd(D)).to(dtype)
    per = {"rows": 2, "token": 1, "channel": T, None: 1}[gate]
    gt = rnd(-(-T // per), D) if gate else None
    fd, xd = f.double(), x.double()
    rms = lambda z: (z.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    u = fd / rms(fd) * pg.double() if post else fd
    if gate:
        u = u * gt.double()[torch.arange(T) // per]
    y = xd + 0.3 * u
    h = y / rms(y) * qg.double()
    dev = lambda t: None if t is None else t.cuda()
    yo = torch.full((T, D), math.nan, dtype=dtype, device="cuda")
    ho = torch.full_like(yo, math.nan) if pre else None
    kw = dict(post_gain=dev(pg) if post else None, pre_gain=dev(qg) if pre else None, gate=dev(gt), rows_per_gate=per,
              scale=0.3)
    B.block_norm(x.cuda(), f.cuda(), yo, ho, **kw)
    half = U if dtype == BF else 0.0
    # a sum of D squares in fp32 over at most 1024 threads: D / 32 + 16 roundings on a path, halved by the root
    path = (16 + D / 64) * E
    ytol = half * y.abs() + 4 * E * xd.abs() + path * 4 * (0.3 * u).abs()
    assert ((yo.cpu().double() - y).abs() <= ytol).all()
    if pre:
        rel = path * 4 * (1 + (xd.abs() + (0.3 * u).abs()))
        htol = half * h.abs() + rel * qg.double().abs() / rms(y) * 2 + path * 4 * h.abs()
        assert ((ho.cpu().double() - h).abs() <= htol).all()
    # in place: the residual over x, the normalised row over f
    x2, f2 = x.cuda(), f.cuda()
    B.block_norm(x2, f2, x2, f2 if pre else None, **kw)
    assert torch.equal(x2, yo) and (not pre or torch.equal(f2, ho))


def test_block_norm_strided_rows_and_zero_rows():
    wide = torch.randn(9, 300, device="cuda")
    x, f = wide[:, 4:132], wide[:, 140:268]
    y, h = torch.empty(9, 128, device="cuda"), torch.empty(9, 128, device="cuda")
    ones = torch.ones(128, device="cuda")
    B.block_norm(x, f, y, h, post_gain=ones, pre_gain=ones)
    r = lambda z: z / (z.square().mean(1, keepdim=True) + 1e-6).sqrt()
    want = x.double() + r(f.double())
    assert torch.allclose(y.double(), want, rtol=1e-5, atol=1e-5)
    assert torch.allclose(h.double(), r(want), rtol=1e-5, atol=1e-5)
    z = torch.zeros(2, 128, device="cuda")
    B.block_norm(z, z, y[:2], h[:2], post_gain=ones, pre_gain=ones, eps=1e-6)
    assert not y[:2].any() and not h[:2].any()
