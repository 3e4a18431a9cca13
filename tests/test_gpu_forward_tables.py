"""Page tables that change in place between steps, dense ones and parts of a wider one, on two streams and in a graph."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_forward_mixed import Mixed  # noqa: E402
from transformer_sharding_affinity_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["current", "stream", "raw stream", "graph"])
@pytest.mark.parametrize("wider", [0, 5])
def test_a_table_changed_in_place_counts_from_the_next_plan(how, wider):
    c = Mixed((4, 2, 64), [1, 3, 20], [40, 90, 33], 20, 16, seed=71)
    n = c.dev["pages"].shape[1]
    wide = torch.full((3, n + wider), -7, dtype=torch.int32, device="cuda")
    wide[:, :n] = c.dev["pages"]
    # the same tokens on other pages
    order = list(range(c.kd.shape[0]))
    order = order[1:] + order[:1]
    k2, v2 = torch.empty_like(c.kd), torch.empty_like(c.vd)
    k2[order], v2[order] = c.kd, c.vd
    moved = dict(c.dev, pages=torch.tensor([[order[i] if i >= 0 else i for i in r] for r in c.dev["pages"].tolist()],
                                           dtype=torch.int32, device="cuda"),
                 prefix_pages=torch.tensor([order[i] for i in c.prefix_ids], dtype=torch.int32, device="cuda"))
    want, _ = c.check_attention()
    pre = c.dev["prefix_pages"].clone()
    step = B.step(c.T, 4, c.dev["q_start"], c.dev["kv_len"], wide[:, :n], pre, c.prefix)
    caches, outs = [c.cache, B.kv_cache(k2, v2)], [torch.zeros_like(want), torch.zeros_like(want)]
    side = torch.cuda.Stream()
    stream = {"current": None, "stream": side, "raw stream": side.cuda_stream, "graph": None}[how]

    def go(cache, out):
        B.step_plan(step, cache, c.plan, stream=stream)
        B.prefix_attention(c.q, cache, step, 0.125, out, None, c.plan, stream=stream)

    graphs = []
    if how == "graph":
        for cache, out in zip(caches, outs):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                go(cache, out)
    for i in range(2):
        if i:
            wide[:, :n] = moved["pages"]
            pre.copy_(moved["prefix_pages"])
        side.wait_stream(torch.cuda.current_stream())
        if graphs:
            graphs[i].replay()
        else:
            go(caches[i], outs[i])
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fault", ["starts", "length", "page"])
def test_every_call_on_a_malformed_step_says_so(dtype, fault):
    """The status word is cleared when it is read; the step is no better for it."""
    c = Mixed((4, 2, 64), [1, 3, 2], [40, 90, 33], 0, 16, dtype=dtype, seed=72)
    bad = {"starts": dict(q_start=torch.tensor([0, 4, 1, 6], dtype=torch.int32, device="cuda")),
           "length": dict(kv_len=torch.tensor([40, 9000, 33], dtype=torch.int32, device="cuda")),
           "page": dict(pages=torch.full_like(c.dev["pages"], 999))}[fault]
    step = B.step(c.T, 4, **dict(c.dev, **bad))
    B.step_plan(step, c.cache, c.plan)
    assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    cos = torch.ones(200, 32, device="cuda")
    kv = torch.randn(c.T, 2, 64, device="cuda").to(dtype)
    pools = c.kd.clone(), c.vd.clone()
    out = torch.empty_like(c.q)
    for _ in range(2):
        B.kv_append(c.q, kv, kv, c.cache, step, B.rotary(cos, cos), out, c.plan)
        assert B.device_status(c.plan) == B.AFF_ERR_RANGE
        B.prefix_attention(c.q, c.cache, step, 0.125, out, None, c.plan)
        assert B.device_status(c.plan) == B.AFF_ERR_RANGE
    assert torch.equal(c.kd.nan_to_num(), pools[0].nan_to_num()) and torch.equal(c.vd.nan_to_num(), pools[1].nan_to_num())
    B.step_plan(c.step, c.cache, c.plan)
    c.check_attention()
