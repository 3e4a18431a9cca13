"""The binding of the forward-pass operators: what it refuses before a call is made, and what it passes on.  Host
tensors; nothing here is launched."""
import pytest

torch = pytest.importorskip("torch")

from transformer_sharding_affinity_gb300 import binding as B


def _pool(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("gain", [_pool(64, 2)[:, 0], _pool(128)[::2], _pool(1).expand(64), _pool(1, 64), _pool(64, 1)])
def test_gains_that_are_not_dense_vectors_are_refused(gain):
    """They would be read as dense ones, the expanded one past its storage."""
    cos = torch.ones(8, 32)
    for kw in (dict(q_gain=gain), dict(k_gain=gain), dict(q_gain=_pool(64), k_gain=gain)):
        with pytest.raises(ValueError, match="dense"):
            B.rotary(cos, cos, **kw)
    r = B.rotary(cos, cos, q_gain=_pool(2, 64)[1], k_gain=_pool(64))
    assert r.q_gain and r.k_gain


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32)


class _Reached(Exception):
    pass


class _NoLaunch:
    """Stands in for the library: whatever a wrapper would launch is reported instead."""

    def __getattr__(self, name):
        if name == "affinity_step_plan_size":
            return self._size
        raise _Reached(name)

    @staticmethod
    def _size(s, c, n):
        return B.AFF_OK


@pytest.fixture
def no_launch(monkeypatch):
    monkeypatch.setattr(B, "load", _NoLaunch)


def _elsewhere(t, device):
    """A host tensor that says it lies on `device` (a GPU's index)."""
    class T(torch.Tensor):
        def get_device(self):
            return device
    return t.as_subclass(T)


def _calls(place):
    """Every call of the forward pass with its tensors made by place(name, tensor)."""
    pool = lambda n: place(n, _pool(4, 2, 16, 64))
    c = lambda: B.kv_cache(pool("pool"), pool("pool"))
    s = lambda: B.step(3, 4, place("q_start", _ints(0, 1, 3)), place("kv_len", _ints(1, 2)),
                       place("pages", torch.zeros(2, 1, dtype=torch.int32)), place("prefix_pages", _ints(3)), 5)
    cos = lambda n: place(n, torch.ones(8, 32))
    gain = lambda n: place(n, _pool(64))
    r = lambda: B.rotary(cos("cos"), cos("sin"), q_gain=gain("q_gain"), k_gain=gain("k_gain"))
    plan = lambda: place("plan", torch.zeros(4096, dtype=torch.uint8))
    q = lambda n: place(n, _pool(3, 4, 64))
    kv = lambda n: place(n, _pool(3, 2, 64))
    row = lambda n: place(n, _pool(5, 64))
    return {"step_plan": lambda: B.step_plan(s(), c(), plan(), stream=0),
            "kv_append": lambda: B.kv_append(q("q"), kv("k"), kv("v"), c(), s(), r(), q("q_out"), plan(), stream=0),
            "prefix_attention": lambda: B.prefix_attention(q("q"), c(), s(), 0.1, q("out"),
                                                           place("lse", torch.zeros(3, 4)), plan(), stream=0),
            "block_norm": lambda: B.block_norm(row("x"), row("f"), row("y"), row("h"), post_gain=gain("post"),
                                               pre_gain=gain("pre"), gate=row("gate"), stream=0)}


USED = {"step_plan": "pool q_start kv_len pages prefix_pages plan", "block_norm": "x f y h post pre gate",
        "kv_append": "q k v q_out pool q_start kv_len pages prefix_pages cos sin q_gain k_gain plan",
        "prefix_attention": "q out lse pool q_start kv_len pages prefix_pages plan"}


@pytest.mark.parametrize("call", USED)
def test_host_tensors_and_tensors_of_two_gpus_are_refused(no_launch, call):
    """A kernel would follow a host address, or another GPU's: an illegal access in place of an error."""
    on_gpu = lambda n, t: _elsewhere(t, 0)
    with pytest.raises(_Reached, match=call):
        _calls(on_gpu)[call]()
    with pytest.raises(TypeError):
        _calls(lambda n, t: t)[call]()
    for name in USED[call].split():
        for other in (-1, 1):
            with pytest.raises(TypeError):
                _calls(lambda n, t: _elsewhere(t, other if n == name else 0))[call]()


def test_raw_addresses_are_taken_as_they_are(no_launch):
    c, s = B.aff_kv_cache(1 << 20, 1 << 20), B.aff_step(3, 0, 1)
    with pytest.raises(_Reached, match="step_plan"):
        B.step_plan(s, c, 1 << 20, stream=0, plan_bytes=4096)


def test_a_part_of_a_wider_page_table_is_read_when_the_step_is_planned(no_launch):
    """The table is changed in place between steps, as a server's is: every plan takes it as it is then."""
    wide = _elsewhere(torch.arange(12, dtype=torch.int32).reshape(3, 4), 0)
    at = lambda t: _elsewhere(t, 0)
    s = B.step(3, 4, at(_ints(0, 1, 2, 3)), at(_ints(1, 2, 2)), wide[:, :2])
    c = B.kv_cache(at(_pool(40, 2, 16, 64)), at(_pool(40, 2, 16, 64)))
    read = s.keep[2]
    assert s.pages == read.data_ptr() and read.is_contiguous() and s.pages_stride == 2
    wide[1, 1] = 33
    with pytest.raises(_Reached):
        B.step_plan(s, c, at(torch.zeros(4096, dtype=torch.uint8)))
    assert read.tolist() == [[0, 1], [4, 33], [8, 9]]
    dense = at(torch.zeros(3, 2, dtype=torch.int32))
    assert B.step(3, 4, at(_ints(0, 1, 2, 3)), at(_ints(1, 2, 2)), dense).pages == dense.data_ptr()


def test_lengths_and_prefix_pages_are_vectors():
    """A matrix of lengths would be read as its first elements, a row of prefix pages as one page."""
    starts, pages = _ints(0, 1, 2), torch.zeros(2, 1, dtype=torch.int32)
    for kv_len, prefix in ((_ints(1, 2, 3, 4).reshape(2, 2), None), (torch.tensor(1, dtype=torch.int32), None),
                           (_ints(1, 2), _ints(0, 1).reshape(1, 2)), (_ints(1, 2), torch.tensor(0, dtype=torch.int32))):
        with pytest.raises(ValueError, match="vectors"):
            B.step(2, 4, starts, kv_len, pages, prefix, 3 if prefix is not None else 0)
