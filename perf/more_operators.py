"""Cases of the operators of a paged cache held in 4 bits: appending a step to it (per-head norms, rotation and
quantising on the way), reading a step's tokens back, and attention of a batch that shares a prefix over it.

The format.  16 neighbouring elements of a head row share a scale: element = code * scale * g, with 4-bit codes (sign,
two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), 8-bit scales (e4m3) and one power of two g for each
pool.  scale is max |x| / (6 g) and a code x / (scale g), each rounded to nearest, ties to even, saturating.  A page of
one group holds its tokens' codes, ceil(d / 32) runs of 16 bytes for each (element j in nibble j, the low one of a byte
first), and then the scales, by four tokens: [page_size / 4][2 ceil(d / 32)][4].

Every case can be run in a plain form (``own = False``: elementary torch operations in 32 bits, in 64 where values lie
next to a border of the rounding) and through the library's calls (``own = True``); ``exact`` evaluates the definitions
in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
K_SCALE, V_SCALE = 0.5, 0.125       # the pools' powers of two

# ---------------------------------------------------------------- the cases

# Head layouts (query heads, KV groups, head width) of the Qwen3-0.6B, Danube3-500M, Llama-3-8B and tiny layers.
QWEN, DANUBE, LLAMA, TINY = (16, 8, 128), (16, 8, 96), (32, 8, 128), (4, 2, 16)


def _append(name, heads, B, q, own_len, prefix, page, dtype, ragged=0, norm=True, rot=0, interleaved=False):
    H, G, d = heads
    return {"name": name, "op": "append", "H": H, "G": G, "d": d, "B": B, "q": q, "own": own_len, "prefix": prefix,
            "page": page, "dtype": dtype, "ragged": ragged, "norm": norm, "rot": rot or d, "interleaved": interleaved}


def _read(name, heads, B, q, own_len, page, dtype, ragged=0):
    H, G, d = heads
    return {"name": name, "op": "read", "H": H, "G": G, "d": d, "B": B, "q": q, "own": own_len, "prefix": 0,
            "page": page, "dtype": dtype, "ragged": ragged}


def _attend(name, heads, B, q, own_len, prefix, page, dtype, ragged=0):
    H, G, d = heads
    return {"name": name, "op": "attend", "H": H, "G": G, "d": d, "B": B, "q": q, "own": own_len, "prefix": prefix,
            "page": page, "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # a decoding step of eight sequences: one token each, latency alone
        _append("append4_decode_8", QWEN, 8, 1, 700, 1024, 16, "bf16"),
        # the calibration set as one step: 64 sequences of 1024 tokens, Qwen3-shaped heads with their q/k norms
        _append("append4_calibration_64x1024", QWEN, 64, 1024, 1024, 0, 64, "bf16"),
        # ragged prompts behind a shared prefix, no norms, half of each head rotated in neighbouring pairs, fp32
        _append("append4_ragged_fp32", DANUBE, 37, 613, 613, 333, 24, "fp32", ragged=5, norm=False, rot=48,
                interleaved=True),
        # one sequence taken out of the cache, as its owner moves it
        _read("read4_one_1000", QWEN, 1, 1000, 1000, 16, "bf16"),
        # the calibration set's keys and values, ragged
        _read("read4_ragged_64x1500", LLAMA, 64, 1500, 1500, 64, "bf16", ragged=6),
        # one sequence, one token: the smallest step
        _attend("attend4_decode_1", QWEN, 1, 1, 1000, 0, 16, "bf16"),
        # 64 sequences decoding behind one long system prompt
        _attend("attend4_decode_64_prefix_8k", QWEN, 64, 1, 1500, 8192, 16, "bf16", ragged=1),
        # a large serving batch with Llama-3-shaped heads: long prefix, ragged answers
        _attend("attend4_decode_256_prefix_32k", LLAMA, 256, 1, 2048, 32768, 64, "bf16", ragged=2),
        # the calibration set's attention outputs in one call
        _attend("attend4_calibration_64x1024", QWEN, 64, 1024, 1024, 0, 64, "bf16"),
        # one long prompt
        _attend("attend4_prompt_8k", LLAMA, 1, 8192, 8192, 0, 128, "bf16"),
        # ragged prompts behind a shared prefix that ends inside a page, head width 96
        _attend("attend4_ragged_prefix_1500", DANUBE, 23, 777, 911, 1500, 24, "bf16", ragged=3),
        # fp32 queries: a few tokens for each of some sequences
        _attend("attend4_few_fp32", (12, 4, 64), 9, 5, 1900, 100, 16, "fp32", ragged=4),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges: steps of single tokens, of a few and of whole prompts; odd sizes; both
    types; with and without a shared prefix."""
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    while True:
        heads = rng.choice([QWEN, DANUBE, LLAMA, TINY, (12, 4, 64), (5, 5, 48), (14, 2, 80)])
        page = rng.choice([8, 16, 24, 64, 128, 200])
        kind = rng.choice(["one", "few", "prompt"])
        if kind == "one":
            q, B, own_len = 1, _spread(rng, 1, 256), _spread(rng, 1, 4096)
        elif kind == "few":
            q, B, own_len = rng.randint(2, 17), _spread(rng, 1, 64), _spread(rng, 20, 3000)
        else:
            q, B = _spread(rng, 20, 4096), _spread(rng, 1, 64)
            own_len = q + rng.choice([0, rng.randint(1, 1000)])
        prefix = rng.choice([0, _spread(rng, 1, 32768)])
        ragged = rng.choice([0, rng.randint(1, 10 ** 6)])
        H, G, d = heads
        if op == "append":
            case = _append("", heads, B, q, own_len, prefix, page, dtype, ragged, norm=rng.random() < 0.6,
                           rot=rng.choice([d, d // 32 * 16 or d]), interleaved=rng.random() < 0.4)
        elif op == "read":
            case = _read("", heads, B, q, own_len, page, dtype, ragged)
        else:
            case = _attend("", heads, B, q, own_len, prefix, page, dtype, ragged)
        cells = H * B * q * (prefix + own_len)      # padded scores: what the plain form holds
        bound = 1.5e9 if dtype == "bf16" else 6e7   # fp32 is for small shapes
        if op != "attend":
            if B * q * (H + 2 * G) * d <= 65536 * 32 * 128 // (2 if dtype == "fp32" else 1):
                break
        elif cells <= bound and (B * own_len + prefix) * G * d <= 256 * 2048 * 8 * 128:
            break
    del case["name"]
    return case


def _lengths(case):
    """(query tokens, own tokens in the cache) of each sequence; equal ones, or ragged ones that hold the largest,
    sequences without a query and, for prompts, sequences of every length."""
    B, q, own_len = case["B"], case["q"], case["own"]
    if not case["ragged"]:
        return [q] * B, [own_len] * B
    r = random.Random(case["ragged"])
    owns = [own_len] + [r.randint(1, own_len) for _ in range(B - 1)]
    qs = [q] + [min(n, r.randint(0, q)) if q > 1 else int(r.random() > 0.05) for n in owns[1:]]
    order = list(range(B))
    r.shuffle(order)
    return [qs[i] for i in order], [owns[i] for i in order]


# ---------------------------------------------------------------- what a program has in hand

def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _filled_pool(g, n_pages, G, page, d, scale):
    """A pool [n_pages, G, page_bytes] of keys or values as appends have left them: rows drawn from 16384 quantised
    ones (values of a unit variance, a few strong channels)."""
    nc = -(-d // 32)
    x = torch.randn(16384, d, generator=g, device="cuda")
    x[:, ::max(1, d // 3)] *= 4
    codes, scales = _quantise(x.double(), scale)
    at = torch.randint(0, 16384, (n_pages, G, page), generator=g, device="cuda")
    pool = torch.empty(n_pages, G, page * nc * 18, dtype=torch.uint8, device="cuda")
    pool[..., :page * nc * 16] = _pack(codes, nc)[at].flatten(2)
    s = torch.zeros(16384, 2 * nc, dtype=torch.uint8, device="cuda")
    s[:, :d // 16] = scales
    pool[..., page * nc * 16:] = s[at].unflatten(2, (page // 4, 4)).transpose(3, 4).flatten(2)
    return pool


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    st = {"case": case}
    H, G, d, B, page, prefix = (case[k] for k in ("H", "G", "d", "B", "page", "prefix"))
    qs, owns = _lengths(case)
    T = max(sum(qs), 1)       # a step of no token at all keeps one row of padding
    n_prefix = -(-prefix // page)
    counts = [-(-n // page) for n in owns]
    width = max(max(counts), 1)
    n_pages = n_prefix + sum(counts) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").cpu().tolist()
    st["prefix_pages"] = torch.tensor(order[:n_prefix], dtype=torch.int32, device="cuda") if n_prefix else None
    table, at = [], n_prefix
    for n in counts:
        table.append(order[at:at + n] + [0] * (width - n))
        at += n
    st["pages"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    starts = [0]
    for n in qs:
        starts.append(starts[-1] + n)
    st["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(owns, dtype=torch.int32, device="cuda")
    st["qs"], st["owns"], st["T"] = qs, owns, T
    st["k_pool"] = _filled_pool(g, n_pages, G, page, d, K_SCALE)
    st["v_pool"] = _filled_pool(g, n_pages, G, page, d, V_SCALE)
    if case["op"] == "append":
        # a step's fused projection: queries, keys and values of a token side by side
        qkv = _randn(g, T, (H + 2 * G) * d, dtype=dtype)
        st["q"] = qkv[:, :H * d].unflatten(1, (H, d))
        st["k"] = qkv[:, H * d:(H + G) * d].unflatten(1, (G, d))
        st["v"] = qkv[:, (H + G) * d:].unflatten(1, (G, d))
        n_pos, half = prefix + max(owns), case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv[None]
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["q_gain"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dtype) if case["norm"] else None
        st["k_gain"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dtype) if case["norm"] else None
    elif case["op"] == "attend":
        st["q"] = _randn(g, T, H, d, dtype=dtype)     # scores of a few units: neither flat nor one-hot
        st["scale"] = d ** -0.5
    if own:
        from transformer_sharding_affinity_gb300 import binding as Bd
        st["B"] = Bd
        st["cache"] = Bd.kv4_cache(st["k_pool"], st["v_pool"], page, d, dtype, K_SCALE, V_SCALE)
        st["step"] = Bd.step(T, H, st["q_start"], st["kv_len"], st["pages"], st["prefix_pages"], prefix)
        st["plan"] = torch.empty(Bd.step_plan_size(st["step"], st["cache"]), dtype=torch.uint8, device="cuda")
        Bd.step_plan(st["step"], st["cache"], st["plan"])
        if case["op"] != "read":
            st["out"] = torch.empty(T, H, d, dtype=dtype, device="cuda")
        if case["op"] == "append":
            st["rotary"] = Bd.rotary(st["cos"], st["sin"], case["interleaved"], st["q_gain"], st["k_gain"], EPS)
        if case["op"] == "attend":
            st["lse"] = torch.empty(T, H, dtype=torch.float32, device="cuda")
        else:
            st["k_out"] = torch.empty(T, G, d, dtype=dtype, device="cuda")
            st["v_out"] = torch.empty(T, G, d, dtype=dtype, device="cuda")
    _indices(st)
    return st


def _indices(st):
    """Where each token of the step stands: its sequence, its row there and its own index."""
    qs, owns = st["qs"], st["owns"]
    seq = [b for b, n in enumerate(qs) for _ in range(n)]
    row = [i for n in qs for i in range(n)]
    idx = [owns[b] - qs[b] + i for b, n in enumerate(qs) for i in range(n)]
    st["seq"], st["row"], st["idx"] = (torch.tensor(v, dtype=torch.int64, device="cuda") for v in (seq, row, idx))


def run(st):
    if own:
        return _own(st)
    return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[st["case"]["op"]](st)


# ---------------------------------------------------------------- the library's calls

def _own(st):
    op, Bd = st["case"]["op"], st["B"]
    if op == "attend":
        Bd.kv4_attention(st["q"], st["cache"], st["step"], st["scale"], st["out"], st["lse"], st["plan"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "append":
        Bd.kv4_append(st["q"], st["k"], st["v"], st["cache"], st["step"], st["rotary"], st["out"], st["plan"])
    # what an append has put into 4 bits is returned as the values it stands for
    Bd.kv4_read(st["cache"], st["step"], st["k_out"], st["v_out"], st["plan"])
    back = {"k": st["k_out"], "v": st["v_out"]}
    return back if op == "read" else {"q": st["out"], **back}


# ---------------------------------------------------------------- plain forms

def _round_to(x, grid, even):
    """Index of the value of the rising `grid` next to each x >= 0; halfway, the index whose parity is `even`."""
    mid = (grid[1:] + grid[:-1]) / 2
    below, above = torch.bucketize(x, mid), torch.bucketize(x, mid, right=True)
    # x on a border: `below` is the index under it, `above` the one over it
    return torch.where((below != above) & (below % 2 != even), above, below)


def _grids(dev, dtype):
    codes = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=dev)
    scales = torch.arange(127, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).to(dtype)
    return codes, scales


def _quantise(x, g):
    """Codes [n, d] and scale bytes [n, d / 16] of rows x [n, d], as uint8."""
    grid, scale_grid = _grids(x.device, x.dtype)
    blocks = x.unflatten(-1, (-1, 16))
    odd = ~torch.isfinite(blocks).all(-1)
    top = blocks.abs().amax(-1).masked_fill(odd, 0)
    s = _round_to(top / (6 * g), scale_grid, 0)
    step = scale_grid[s] * g
    size = torch.where((step > 0)[..., None], blocks.abs().nan_to_num(0, 0, 0) / step.clamp(min=1e-30)[..., None], 0)
    codes = _round_to(size, grid, 0) + 8 * (blocks < 0)
    return codes.masked_fill(odd[..., None], 0).flatten(-2).to(torch.uint8), s.masked_fill(odd, 127).to(torch.uint8)


def _pack(codes, nc):
    """Codes [n, d] to bytes [n, 16 nc]."""
    full = torch.zeros(codes.shape[0], 32 * nc, dtype=torch.uint8, device=codes.device)
    full[:, :codes.shape[1]] = codes
    return full[:, 0::2] | full[:, 1::2] << 4


def _values(codes, scales, d, g):
    """fp32 [..., d] of packed codes [..., 16 nc] and scale bytes [..., 2 nc]."""
    grid = _grids(codes.device, torch.float32)[0]
    grid = torch.cat([grid, -grid])
    x = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * g
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)[..., :d]


def _split(pool, page, d):
    """A pool's codes [n, G, page, 16 nc] and scales [n, G, page, 2 nc] (views of it)."""
    nc = -(-d // 32)
    codes = pool[..., :page * nc * 16].unflatten(2, (page, 16 * nc))
    return codes, pool[..., page * nc * 16:].unflatten(2, (page // 4, 2 * nc, 4))


def _token_scales(scales, page):
    """[n, G, page / 4, 2 nc, 4] to [n, G, page, 2 nc]."""
    return scales.transpose(3, 4).flatten(2, 3)


def _plain_read(st):
    c = st["case"]
    page_of = st["pages"].long()[st["seq"], st["idx"] // c["page"]]
    slot, n = st["idx"] % c["page"], st["seq"].numel()
    back = {}
    for name, g in (("k", K_SCALE), ("v", V_SCALE)):
        codes, scales = _split(st[name + "_pool"], c["page"], c["d"])
        x = _values(codes[page_of, :, slot], scales[page_of, :, slot // 4, :, slot % 4], c["d"], g)
        back[name] = torch.zeros(st["T"], c["G"], c["d"], dtype=TYPES[c["dtype"]], device=x.device)
        back[name][:n] = x.to(TYPES[c["dtype"]])
    return back


def _plain_rotate(v, c, s, rot, interleaved):
    r, rest = v[..., :rot], v[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([r, rest], -1)


def _plain_append(st):
    c = st["case"]
    n, dtype = st["seq"].numel(), TYPES[c["dtype"]]
    # keys in 64 bits: what is next to a border of the rounding would fall on either side of it in 32
    q, k, v = st["q"][:n].float(), st["k"][:n].double(), st["v"][:n].double()
    if st["q_gain"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * st["q_gain"].float()
        k = k / torch.sqrt(k.square().mean(-1, keepdim=True) + torch.tensor(EPS).double().item()) * st["k_gain"].double()
    pos = st["idx"] + c["prefix"]
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    q = _plain_rotate(q, cos, sin, c["rot"], c["interleaved"])
    k = _plain_rotate(k, cos.double(), sin.double(), c["rot"], c["interleaved"])
    page_of = st["pages"].long()[st["seq"], st["idx"] // c["page"]]
    slot, nc = st["idx"] % c["page"], -(-c["d"] // 32)
    for name, x, g in (("k", k, K_SCALE), ("v", v, V_SCALE)):
        codes, scales = _split(st[name + "_pool"], c["page"], c["d"])
        new, s = _quantise(x.flatten(0, 1), g)
        codes[page_of, :, slot] = _pack(new, nc).view(n, c["G"], 16 * nc)
        scales[page_of, :, slot // 4, :c["d"] // 16, slot % 4] = s.view(n, c["G"], -1)
    out = torch.zeros(st["T"], c["H"], c["d"], dtype=dtype, device="cuda")
    out[:n] = q.to(dtype)
    return {"q": out, **_plain_read(st)}


def _plain_attend(st):
    c = st["case"]
    B, H, G, d, Lp, page = (c[k] for k in ("B", "H", "G", "d", "prefix", "page"))
    R, n, qmax = H // G, st["seq"].numel(), max(max(st["qs"]), 1)
    dev, dtype = st["q"].device, st["q"].dtype

    def rows(pool, ids, g):
        """Values of the pages ids, [..., pages, G, page, d]."""
        codes, scales = _split(pool[ids.flatten()], page, d)
        return _values(codes, _token_scales(scales, page), d, g).unflatten(0, ids.shape)

    q = torch.zeros(B, qmax, H, d, device=dev)
    q[st["seq"], st["row"]] = st["q"][:n].float()
    # rows of one KV group together: [B, G, qmax * R, d]
    q = q.view(B, qmax, G, R, d).permute(0, 2, 1, 3, 4).reshape(B, G, qmax * R, d) * st["scale"]
    pages = st["pages"].long()
    ko = rows(st["k_pool"], pages, K_SCALE).transpose(1, 2).flatten(2, 3)
    vo = rows(st["v_pool"], pages, V_SCALE).transpose(1, 2).flatten(2, 3)
    s = q @ ko.transpose(2, 3)
    row = torch.arange(qmax, device=dev)
    lens, counts = st["kv_len"].long(), (st["q_start"][1:] - st["q_start"][:-1]).long()
    last = lens[:, None] - counts[:, None] + row[None]                  # own index of each query
    seen = torch.arange(ko.shape[2], device=dev)[None, None] <= last[:, :, None]
    seen = seen & (row[None] < counts[:, None])[:, :, None]
    seen = seen.repeat_interleave(R, 1)[:, None]
    s = s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    if Lp:
        at = st["prefix_pages"].long()
        kp = rows(st["k_pool"], at, K_SCALE).transpose(0, 1).flatten(1, 2)[:, :Lp]
        vp = rows(st["v_pool"], at, V_SCALE).transpose(0, 1).flatten(1, 2)[:, :Lp]
        # one product for the whole batch: [G, B * qmax * R, Lp]
        sp = (q.transpose(0, 1).reshape(G, -1, d) @ kp.transpose(1, 2)).view(G, B, qmax * R, Lp)
        m = torch.maximum(m, sp.amax(-1, keepdim=True).transpose(0, 1))
    m = m.masked_fill(m == -math.inf, 0.0)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = p @ vo
    del s, p
    if Lp:
        sp = sp.sub_(m.transpose(0, 1)).exp_()
        total = total + sp.sum(-1, keepdim=True).transpose(0, 1)
        o = o + (sp.view(G, -1, Lp) @ vp).view(G, B, qmax * R, d).transpose(0, 1)
    lse = (m + total.log()).squeeze(-1)
    o = o / total
    back = lambda t: t.unflatten(2, (qmax, R)).transpose(1, 2).flatten(2, 3)[st["seq"], st["row"]]
    out = torch.zeros(st["T"], H, d, dtype=dtype, device=dev)
    out[:n] = back(o).to(dtype)
    full = torch.full((st["T"], H), -math.inf, device=dev)
    full[:n] = back(lse)
    return {"out": out, "lse": full}


# ---------------------------------------------------------------- definitions, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "read":
        return _exact_read(case, st)
    if 8.0 * case["H"] * case["d"] * case["B"] * case["q"] * (case["prefix"] + case["own"]) > 4e12:
        return None
    return _exact_attend(case, st)


def _decoded(pool, ids, page, d, g):
    """[tokens of the listed pages, G, d] in 64 bits, from the bits: code (-1)^s 2^(e-1) (1 + m/2), m/2 where e is 0;
    scale 2^(E-7) (1 + M/8), 2^-6 M/8 where E is 0."""
    nc, data = -(-d // 32), pool[ids.long()]
    n, G = data.shape[:2]
    j = torch.arange(d, device=pool.device)
    byte = data[:, :, :page * nc * 16].view(n, G, page, nc * 16)[..., j // 2].long()
    nib = byte >> (4 * (j % 2)) & 15
    e, m = nib >> 1 & 3, (nib & 1).double()
    size = torch.where(e > 0, torch.ldexp(1 + m / 2, e - 1), m / 2)
    value = torch.where(nib > 7, -size, size)
    t = torch.arange(page, device=pool.device)
    at = page * nc * 16 + (t // 4)[:, None] * 8 * nc + (j // 16)[None] * 4 + (t % 4)[:, None]
    sb = data[:, :, at.flatten()].view(n, G, page, d).long()
    E, M = sb >> 3, (sb & 7).double()
    s = torch.where(E > 0, torch.ldexp(1 + M / 8, E - 7), M / 512)
    return (value * s * g).transpose(1, 2).flatten(0, 1)


def _exact_read(case, st):
    back = {}
    for name, g in (("k", K_SCALE), ("v", V_SCALE)):
        out = torch.zeros(st["T"], case["G"], case["d"], dtype=torch.float64, device="cuda")
        t = 0
        for b, (n, length) in enumerate(zip(st["qs"], st["owns"])):
            if n:
                used = st["pages"][b][:-(-length // case["page"])]
                out[t:t + n] = _decoded(st[name + "_pool"], used, case["page"], case["d"], g)[length - n:length]
                t += n
        back[name] = out
    return back


def _rms(v):
    return (torch.einsum("...i,...i->...", v, v) / v.shape[-1] + float(torch.tensor(EPS))).sqrt()[..., None]


def _nearest(x, step_of):
    """x >= 0 rounded to the nearest multiple of step_of(x), ties to even."""
    step = step_of(x)
    return torch.round(x / step) * step


def _exact_quantised(x, g):
    """What x [..., d] reads back as: both roundings as roundings to multiples of a binade's step."""
    b = x.unflatten(-1, (-1, 16))
    binade = lambda v, least: torch.floor(torch.log2(v.clamp(min=least)))
    scale = _nearest(b.abs().amax(-1, keepdim=True) / (6 * g),
                     lambda v: torch.exp2(binade(v, 2.0 ** -6) - 3)).clamp(max=448)
    size = torch.where(scale > 0, b.abs() / (scale * g), 0)
    size = _nearest(size, lambda v: torch.exp2(binade(v, 1.0) - 1)).clamp(max=6)
    return (torch.sign(b) * size * scale * g).flatten(-2)


def _exact_append(case, st):
    H, G, d, Lp, rot = (case[k] for k in ("H", "G", "d", "prefix", "rot"))
    T = st["T"]
    q, k, v = (torch.zeros(T, h, d, dtype=torch.float64, device="cuda") for h in (H, G, G))
    if case["interleaved"]:
        first, second = list(range(0, rot, 2)), list(range(1, rot, 2))
    else:
        first, second = list(range(rot // 2)), list(range(rot // 2, rot))

    def turned(x, gain, pos):
        x = x.double()
        if gain is not None:
            x = x / _rms(x) * gain.double()
        z = torch.complex(x[..., first], x[..., second])
        z = z * torch.complex(st["cos"][pos].double(), st["sin"][pos].double())[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    t = 0
    for n, length in zip(st["qs"], st["owns"]):
        if n:
            pos = torch.arange(length - n, length, device="cuda") + Lp
            q[t:t + n] = turned(st["q"][t:t + n], st["q_gain"], pos)
            k[t:t + n] = _exact_quantised(turned(st["k"][t:t + n], st["k_gain"], pos), K_SCALE)
            v[t:t + n] = _exact_quantised(st["v"][t:t + n].double(), V_SCALE)
            t += n
    return {"q": q, "k": k, "v": v}


def _exact_attend(case, st):
    H, G, d, Lp, page = (case[k] for k in ("H", "G", "d", "prefix", "page"))
    out = torch.zeros(st["T"], H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((st["T"], H), -math.inf, dtype=torch.float64, device="cuda")
    none = torch.zeros(0, G, d, dtype=torch.float64, device="cuda")
    kp = _decoded(st["k_pool"], st["prefix_pages"], page, d, K_SCALE)[:Lp] if Lp else none
    vp = _decoded(st["v_pool"], st["prefix_pages"], page, d, V_SCALE)[:Lp] if Lp else none
    t = 0
    for b, (n, length) in enumerate(zip(st["qs"], st["owns"])):
        if not n:
            continue
        used = st["pages"][b][:-(-length // page)]
        keys = torch.cat([kp, _decoded(st["k_pool"], used, page, d, K_SCALE)[:length]])
        vals = torch.cat([vp, _decoded(st["v_pool"], used, page, d, V_SCALE)[:length]])
        last = Lp + length - n + torch.arange(n, device="cuda")
        hidden = torch.arange(Lp + length, device="cuda")[None] > last[:, None]
        for g in range(G):
            heads = slice(g * (H // G), (g + 1) * (H // G))
            s = torch.einsum("thd,kd->htk", st["q"][t:t + n, heads].double(), keys[:, g]) * st["scale"]
            s[:, hidden] = -math.inf
            z = torch.logsumexp(s, -1)
            lse[t:t + n, heads] = z.T
            out[t:t + n, heads] = torch.einsum("htk,kd->thd", (s - z[..., None]).exp(), vals[:, g])
        t += n
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, G, d, Lp = (case[k] for k in ("H", "G", "d", "prefix"))
    row4 = d // 2 + d // 16       # a head row in 4 bits with its scales
    qs, owns = _lengths(case)
    T = max(sum(qs), 1)
    if case["op"] == "read":
        return {"bytes": 2 * T * G * (row4 + d * e), "flops": 4 * T * G * d}
    if case["op"] == "append":
        # queries, keys and values read once; queries, the cache and its values back written once; a row of cosines and
        # sines for each position
        table = min(Lp + max(owns), T) * case["rot"] * 4
        return {"bytes": T * (2 * H + 2 * G) * d * e + 2 * T * G * (2 * row4 + d * e) + table,
                "flops": T * (H + G) * (3 * case["rot"] + 4 * d * case["norm"]) + 12 * T * G * d}
    pairs = sum(n * (Lp + length - n) + n * (n + 1) // 2 for n, length in zip(qs, owns))
    read = (Lp if sum(qs) else 0) + sum(length for n, length in zip(qs, owns) if n)
    return {"bytes": 2 * T * H * d * e + 4 * T * H + 2 * read * G * row4, "flops": 4 * d * H * max(pairs, 1)}
