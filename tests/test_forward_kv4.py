"""``forward.Forward`` over a cache in 4 bits: appends, attention and reading back together, as a served model and its
calibration use them.

Tolerances.  The attention is checked against a 64-bit one over what the cache holds (`cached`), from the layer's own
input: in fp32 the queries are chains of at most D terms and a norm, off by D e (e = 2^-24) of their largest terms, which
moves a score by as much relative to sum |q k| (of a few units here: factor 8), and the rest is test_gpu_kv4's; 64 (D + keys) e
of the largest value covers it.  bf16: the queries are rounded twice (projection, append) and the output once, 3 u
(u = 2^-8) of the largest value, scores of a few units again turning a relative error of the queries into as many of the probabilities:
8 times that.  A held element is at most one step from the exact one: the largest step is 2 of 6, half of it 1/6 of
the block's maximum, the scale's rounding 1/16 more, and in bf16 the projection's and the norm's roundings beside it.
"""
import numpy as np
import pytest

from oracle import kv4 as K
from transformer_sharding_affinity_gb300 import binding as B
from transformer_sharding_affinity_gb300 import forward as FW

torch = pytest.importorskip("torch")

D, I, H, G, DH, N = 64, 96, 4, 2, 32, 3


def _layers(seed, dtype, qk_norm=True):
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
        out.append({k: torch.tensor(v, dtype=dtype, device="cuda") for k, v in w.items()})
    return out


def _f64(t):
    return t.double().cpu().numpy()


def _projected(x, w, pos, fwd):
    """Queries, keys and values of a layer's input x in 64 bits."""
    h = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6) * _f64(w["g_attn"])
    cos, sin = (_f64(t) for t in fwd.rotaries[0].keep)
    q, k, v = ((h @ _f64(w[n]).T).reshape(len(x), -1, DH) for n in ("Wq", "Wk", "Wv"))
    gains = [_f64(w[n]) if n in w else None for n in ("qn", "kn")]
    return K.turned(q, pos, cos, sin, gains[0], 1e-6), K.turned(k, pos, cos, sin, gains[1], 1e-6), v


def _attend(q, k, v, first):
    """Causal attention of rows q, the first of which sees keys 0 .. first."""
    out = np.zeros_like(q)
    for t in range(len(q)):
        for h in range(H):
            s = k[:first + t + 1, h // (H // G)] @ q[t, h] * DH ** -0.5
            p = np.exp(s - s.max())
            out[t, h] = p @ v[:first + t + 1, h // (H // G)] / p.sum()
    return out.reshape(len(q), H * DH)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("qk_norm", [True, False])
def test_prompts_behind_a_prefix_then_single_tokens(dtype, qk_norm):
    layers = _layers(1, dtype, qk_norm)
    fwd = FW.Forward(layers, H, G, DH, n_pages=40, n_pos=128, page_size=8, cache_bits=4, k_scale=0.5, v_scale=0.25)
    g = torch.Generator().manual_seed(2)
    n_pre, lengths, more = 21, [17, 1, 30], 2
    head = torch.randn(n_pre, D, generator=g).to(dtype).cuda()
    prefix = fwd.new_sequence()
    fwd.run(head, [prefix])
    seqs = [fwd.new_sequence() for _ in lengths]
    e, u = 2.0 ** -24, 2.0 ** -8
    for new in [lengths] + [[1] * 3] * more:
        x = torch.randn(sum(new), D, generator=g).to(dtype).cuda()
        inputs, seen = [_f64(x)], []
        for i, a, res in fwd.blocks(x, seqs, new, prefix):
            seen.append((_f64(a), _f64(res)))
        # every layer's input is what its own block was given: rebuilt from the residual before the layer
        for i in range(N):
            w = layers[i]
            kp, vp = (_f64(t) for t in fwd.cached(prefix, i))
            at = 0
            x_in = inputs[0] if i == 0 else _next_input(seen[i - 1][1], layers[i - 1])
            for s, n in zip(seqs, new):
                k, v = (_f64(t) for t in fwd.cached(s, i))
                q, k_new, v_new = _projected(x_in[at:at + n], w, n_pre + np.arange(s.length - n, s.length), fwd)
                ref = _attend(q, np.concatenate([kp, k]), np.concatenate([vp, v]), n_pre + s.length - n)
                vmax = max(np.abs(vp).max(), np.abs(v).max())
                tol = (64 * (D + 128) * e if dtype == torch.float32 else 24 * u) * vmax * (1 if i == 0 else 4)
                assert np.abs(seen[i][0][at:at + n] - ref).max() <= tol, i
                for got, exact in ((k[s.length - n:], k_new), (v[s.length - n:], v_new)):
                    top = np.abs(exact).reshape(n, G, -1, 16).max(-1).repeat(16, -1)
                    slack = (1 / 6) * (1 + 1 / 16) + (1e-4 if dtype == torch.float32 else (4 if i == 0 else 16) * u)
                    assert (np.abs(got - exact) <= slack * top).all()
                at += n
    assert sum(s.length for s in seqs) == sum(lengths) + 3 * more


def _next_input(res, w):
    """The residual entering the next layer, from the one entering the FFN."""
    h = res / np.sqrt((res * res).mean(1, keepdims=True) + 1e-6) * _f64(w["gamma"])
    a = h @ _f64(w["Wg"]).T
    return res + (a / (1 + np.exp(-a)) * (h @ _f64(w["Wu"]).T)) @ _f64(w["Wd"]).T


@pytest.mark.gpu
def test_calibration_reads_the_forward_pass():
    """calibrate_stack fed by a 4-bit forward pass gives the scores of the a and x that the pass yields."""
    from transformer_sharding_affinity_gb300 import stack as ST
    layers = _layers(3, torch.float32)
    g = torch.Generator().manual_seed(4)
    lengths = [25, 40, 16]
    x = torch.randn(sum(lengths), D, generator=g).cuda()
    d = B.dims(sum(lengths), D, H, G, DH, I, dtype=B.AFF_FP32)

    def forward():
        fwd = FW.Forward(layers, H, G, DH, n_pages=16, n_pos=64, page_size=16, cache_bits=4)
        return fwd, [fwd.new_sequence() for _ in lengths]

    fwd, seqs = forward()
    up, down = ST.calibrate_stack(fwd.layer_inputs(x, seqs, lengths), N, d)
    fwd, seqs = forward()
    kept = [{"a": a.clone(), "x": r.clone()} for _, a, r in fwd.blocks(x.clone(), seqs, lengths)]

    def inputs(i):
        t = dict(kept[i], **{k: layers[i][k] for k in ("Wo", "gamma", "Wg", "Wu", "Wd")})
        if i + 1 < N:
            t.update(gamma_next=layers[i + 1]["g_attn"], Wq_next=layers[i + 1]["Wq"], Wk_next=layers[i + 1]["Wk"],
                     Wv_next=layers[i + 1]["Wv"])
        return t

    ref_up, ref_down = ST.calibrate_stack(inputs, N, d)
    for got, ref in list(zip(up, ref_up)) + list(zip(down, ref_down)):
        assert np.array_equal(np.asarray(got), np.asarray(ref)) and np.isfinite(np.asarray(got)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [None, 4])
def test_cached_reads_what_the_layers_hold(bits):
    layers = _layers(5, torch.bfloat16)
    fwd = FW.Forward(layers, H, G, DH, n_pages=16, n_pos=64, page_size=8, cache_bits=bits)
    a, b = fwd.new_sequence(), fwd.new_sequence()
    x = torch.randn(33, D, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    fwd.run(x, [a, b], [20, 13])
    for seq, at in ((a, 0), (b, 20)):
        k, v = fwd.cached(seq, 0)
        assert k.shape == v.shape == (seq.length, G, DH) and k.dtype == torch.bfloat16
        _, k_ref, v_ref = _projected(_f64(x[at:at + seq.length]), layers[0], np.arange(seq.length), fwd)
        slack = 4 * 2.0 ** -8 + (0 if bits is None else 17 / 96)
        for got, ref in ((k, k_ref), (v, v_ref)):
            top = np.abs(ref).reshape(seq.length, G, -1, 16).max(-1).repeat(16, -1) if bits else np.abs(ref).max()
            assert (np.abs(_f64(got) - ref) <= slack * top).all()
    empty = fwd.new_sequence()
    assert fwd.cached(empty, 0)[0].shape == (0, G, DH)
    steps = fwd.blocks(x, [a, b], [20, 13])
    next(steps)
    with pytest.raises(ValueError):
        fwd.cached(a, 0)


def test_other_widths_of_a_cache_are_refused():
    w = {"Wq": torch.zeros(4, 4)}
    for bits in (8, 16, 0, "4"):
        with pytest.raises(ValueError, match="cache_bits"):
            FW.Forward([w], 1, 1, 16, 4, 16, cache_bits=bits)


def test_heads_that_4_bits_do_not_take_are_refused():
    import os
    from transformer_sharding_affinity_gb300 import build as BUILD
    if not os.path.exists(B.LIB_PATH):
        BUILD.build()
    with pytest.raises(B.AffinityError) as e:
        FW.Forward([{"Wq": torch.zeros(4, 4)}], 1, 1, 24, 4, 16, page_size=8, cache_bits=4)
    assert e.value.status == B.AFF_ERR_UNSUPPORTED_SHAPE
