"""``forward.Forward``: the appends, the attention and the norms together, as calibration uses them, against the
64-bit layer of the oracle.

Tolerances.  fp32: every value is a chain of sums of at most n = D + I + H d_head + keys terms, so normwise off by at
most n e (e = 2^-24) per product, times what the steps after it multiply it by; 64 n e per layer of the largest
element bounds that with room for gains of up to 8 on two paths.  bf16: twelve roundings of u = 2^-8 per layer (q, k, v,
a, the four projections' outputs, the norms' outputs, the residual), independent, so sqrt(12 layers) u of the root mean
square, times 2 for what is amplified.
"""
import numpy as np
import pytest

from oracle import layer_forward as LF
from transformer_sharding_affinity_gb300 import forward as FW

torch = pytest.importorskip("torch")

D, I, H, G, DH, N = 64, 96, 4, 2, 16, 3


def _layers(seed, qk_norm=True):
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(N):
        w = {"g_attn": 1 + 0.1 * rng.standard_normal(D), "gamma": 1 + 0.1 * rng.standard_normal(D),
             "Wq": rng.standard_normal((H * DH, D)), "Wk": rng.standard_normal((G * DH, D)),
             "Wv": rng.standard_normal((G * DH, D)), "Wo": rng.standard_normal((D, H * DH)),
             "Wg": rng.standard_normal((I, D)), "Wu": rng.standard_normal((I, D)), "Wd": rng.standard_normal((D, I))}
        for k in w:
            if k[0] == "W":
                w[k] = w[k] / np.sqrt(w[k].shape[1])
        if qk_norm:
            w["qn"], w["kn"] = 1 + 0.1 * rng.standard_normal(DH), 1 + 0.1 * rng.standard_normal(DH)
        out.append(w)
    return out


def _rounded(layers, dtype):
    """The layers on the GPU and, in 64 bits, as they are there."""
    dev = [{k: torch.tensor(v, dtype=dtype, device="cuda") for k, v in w.items()} for w in layers]
    return dev, [{k: v.double().cpu().numpy() for k, v in w.items()} for w in dev]


def _oracle(x, layers):
    """(a, x entering the FFN) of every layer and the output, for one sequence from its first token."""
    a_x = []
    for w in layers:
        w = dict(w, g_ffn=w["gamma"])
        a = LF.attention_heads(x, w, H, G, DH).reshape(len(x), H * DH)
        a_x.append((a, x + a @ w["Wo"].T))
        x = LF.layer_forward(x, w, H, G, DH)
    return a_x, x


def _check(got, ref, dtype, layers_done, keys=80):
    got = got.double().cpu().numpy()
    if dtype == torch.float32:
        assert np.abs(got - ref).max() <= 64 * (D + I + H * DH + keys) * 2.0 ** -24 * layers_done * np.abs(ref).max()
    else:
        assert np.sqrt(np.mean((got - ref) ** 2)) <= 2 * np.sqrt(12 * layers_done) * 2.0 ** -8 * np.sqrt(np.mean(ref ** 2))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("qk_norm", [True, False])
def test_prompts_behind_a_prefix_then_single_tokens(dtype, qk_norm):
    dev, layers = _rounded(_layers(3, qk_norm), dtype)
    fwd = FW.Forward(dev, H, G, DH, n_pages=40, n_pos=128, page_size=8)
    g = torch.Generator().manual_seed(5)
    n_pre, lengths, more = 21, [17, 1, 30], 3
    head = torch.randn(n_pre, D, generator=g).to(dtype)
    tails = [torch.randn(n + more, D, generator=g).to(dtype) for n in lengths]
    full = [_oracle(torch.cat([head, t]).double().numpy(), layers) for t in tails]

    prefix = fwd.new_sequence()
    y = fwd.run(head.cuda(), [prefix])
    _check(y, full[0][1][:n_pre], dtype, N)
    seqs = [fwd.new_sequence() for _ in lengths]
    x = torch.cat([t[:n] for t, n in zip(tails, lengths)]).cuda()
    kept = x.clone()
    for i, a, res in fwd.blocks(x, seqs, lengths, prefix):
        ref_a = np.concatenate([f[0][i][0][n_pre:n_pre + n] for f, n in zip(full, lengths)])
        ref_x = np.concatenate([f[0][i][1][n_pre:n_pre + n] for f, n in zip(full, lengths)])
        _check(a, ref_a, dtype, i + 1)
        _check(res, ref_x, dtype, i + 1)
    assert not torch.equal(x, kept)
    for j in range(more):
        x = torch.stack([t[n + j] for t, n in zip(tails, lengths)]).cuda()
        y = fwd.run(x, seqs, prefix=prefix)
        _check(y, np.stack([f[1][n_pre + n + j] for f, n in zip(full, lengths)]), dtype, N)
    pages = len(fwd.free)
    fwd.release(seqs[2])
    assert len(fwd.free) == pages + -(-(30 + more) // 8) and seqs[2].length == 0


@pytest.mark.gpu
def test_calibration_reads_the_forward_pass(tmp_path):
    """calibrate_stack fed by the forward pass gives the scores of the 64-bit forward pass's a and x."""
    from transformer_sharding_affinity_gb300 import binding as B, stack as ST
    dev, layers = _rounded(_layers(4), torch.float32)
    g = torch.Generator().manual_seed(6)
    lengths = [25, 40, 16]
    tails = [torch.randn(n, D, generator=g) for n in lengths]
    full = [_oracle(t.double().numpy(), layers) for t in tails]
    d = B.dims(sum(lengths), D, H, G, DH, I, dtype=B.AFF_FP32)

    def from_oracle(i):
        t = {"a": torch.tensor(np.concatenate([f[0][i][0] for f in full]), dtype=torch.float32).cuda(),
             "x": torch.tensor(np.concatenate([f[0][i][1] for f in full]), dtype=torch.float32).cuda()}
        t.update({k: dev[i][k] for k in ("Wo", "gamma", "Wg", "Wu", "Wd")})
        if i + 1 < N:
            t.update(gamma_next=dev[i + 1]["g_attn"], Wq_next=dev[i + 1]["Wq"], Wk_next=dev[i + 1]["Wk"],
                     Wv_next=dev[i + 1]["Wv"])
        return t

    ref_up, ref_down = ST.calibrate_stack(from_oracle, N, d)
    x = torch.cat(tails).cuda()

    def run(checkpoint_dir=None):
        fwd = FW.Forward(dev, H, G, DH, n_pages=16, n_pos=64, page_size=16)
        return ST.calibrate_stack(fwd.layer_inputs(x, [fwd.new_sequence() for _ in lengths], lengths), N, d,
                                  checkpoint_dir=checkpoint_dir)

    up, down = run(str(tmp_path))
    # squares of products of the above: twice its relative error, and once more for the scores' own sums
    bound = 4 * 64 * (D + I + H * DH + 40) * 2.0 ** -24 * N
    for got, ref in list(zip(up, ref_up)) + list(zip(down, ref_down)):
        assert np.abs(got - ref).max() <= bound * np.abs(ref).max()
    # a run that resumes goes through the layers whose scores it already has
    (tmp_path / "layer_002.npz").unlink()
    up2, _ = run(str(tmp_path))
    assert all(np.array_equal(a, b) for a, b in zip(up, up2))


class _Fake:
    """What Forward's own checks need, without a GPU."""
    layers, H, G, d, page_size, n_pos, eps = [], 4, 2, 16, 8, 32, 1e-6

    def __init__(self, free):
        self.free = list(range(free))

    _grow, blocks = FW.Forward._grow, FW.Forward.blocks


def test_refusals_leave_the_sequences_as_they_were():
    fwd, seqs = _Fake(3), [FW.CachedSequence(), FW.CachedSequence([7], 5)]
    x = torch.zeros(6, 64)
    for bad, lengths, prefix in [(seqs, [3, 2], None), (seqs, [7, -1], None), (seqs, [6], None),
                                 ([seqs[0], seqs[0]], [3, 3], None), (seqs, [3, 3], seqs[1])]:
        with pytest.raises(ValueError):
            next(fwd.blocks(x, bad, lengths, prefix))
    with pytest.raises(ValueError, match="pages"):
        next(fwd.blocks(torch.zeros(40, 64), seqs, [9, 31]))
    with pytest.raises(ValueError, match="n_pos"):
        next(fwd.blocks(torch.zeros(20, 64), seqs, [20, 0], FW.CachedSequence([1, 2], 13)))
    with pytest.raises(ValueError, match="lengths"):
        next(fwd.blocks(torch.zeros(5, 64), seqs))
    assert [s.length for s in seqs] == [0, 5] and len(fwd.free) == 3
    assert [len(s.pages) for s in seqs] == [0, 1]


def test_rotary_tables_are_those_of_the_oracle():
    x = np.random.default_rng(0).standard_normal((7, 2, 16))
    cos, sin = (t.double().numpy()[:, None] for t in FW.rotary_tables(7, 16, device="cpu"))
    a, b = x[..., :8], x[..., 8:]
    got = np.concatenate([a * cos - b * sin, a * sin + b * cos], -1)
    np.testing.assert_allclose(got, LF.rope(x), atol=4 * 2.0 ** -24 * np.abs(x).max())
