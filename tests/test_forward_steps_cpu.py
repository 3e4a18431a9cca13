"""Which layers' caches hold a step's tokens, with the library's calls replaced by records: a step that calibration
reads in part (a resumed run) reaches every layer before its sequences are used again, and a step that its caller
leaves is never read."""
import pytest

torch = pytest.importorskip("torch")

from transformer_sharding_affinity_gb300 import binding as B
from transformer_sharding_affinity_gb300 import forward as FW

D, H, G, DH, N = 8, 2, 1, 4, 3


class _Plan:
    def __init__(self, T, H, q_start, kv_len, pages, prefix_pages=None, prefix_len=0):
        self.starts, self.kv, self.pages = q_start.tolist(), kv_len.tolist(), pages.tolist()
        self.prefix = (prefix_pages.tolist() if prefix_pages is not None else [], prefix_len)


class _Recorder:
    """Stands in for the binding: notes what every layer's cache is given and what its attention reads."""
    AFF_OK = B.AFF_OK

    def __init__(self):
        self.held, self.calls, self.status = {}, [], []

    def kv_cache(self, k, v):
        self.held[len(self.held)] = set()
        return len(self.held) - 1

    def rotary(self, *a, **kw):
        return None

    step = staticmethod(_Plan)

    def step_plan_size(self, s, c):
        return 1

    def step_plan(self, s, c, plan):
        pass

    def block_norm(self, x, f, y, h=None, **kw):
        if h is not None:
            h.copy_(y)

    def _slots(self, s, b, lo, hi, page=4):
        return {(s.pages[b][j // page], j % page) for j in range(lo, hi)}

    def kv_append(self, q, k, v, c, s, r, out, plan):
        self.calls.append(c)
        for b, kv in enumerate(s.kv):
            self.held[c] |= self._slots(s, b, kv - (s.starts[b + 1] - s.starts[b]), kv)

    def prefix_attention(self, q, c, s, scale, out, lse, plan):
        out.zero_()
        for b, kv in enumerate(s.kv):
            assert self._slots(s, b, 0, kv) <= self.held[c], "reads tokens that the layer's cache does not hold"
        ids, n = s.prefix
        assert {(ids[j // 4], j % 4) for j in range(n)} <= self.held[c]

    def device_status(self, plan):
        return self.status.pop(0) if self.status else B.AFF_OK

    AffinityError, strerror = B.AffinityError, staticmethod(lambda st: str(st))


@pytest.fixture
def fwd(monkeypatch):
    monkeypatch.setattr(FW, "B", _Recorder())
    eye = lambda m, n: torch.zeros(m, n)
    layers = [dict(g_attn=torch.ones(D), gamma=torch.ones(D), Wq=eye(H * DH, D), Wk=eye(G * DH, D), Wv=eye(G * DH, D),
                   Wo=eye(D, H * DH), Wg=eye(6, D), Wu=eye(6, D), Wd=eye(D, 6)) for _ in range(N)]
    return FW.Forward(layers, H, G, DH, n_pages=32, n_pos=64, page_size=4)


def _x(n):
    return torch.ones(n, D)


@pytest.mark.parametrize("asked", [[], [0], [1], [0, 2], [2], [0, 1, 2]])
def test_a_step_read_in_part_reaches_every_layer_before_its_sequences_are_used(fwd, asked):
    prefix = fwd.new_sequence()
    fwd.run(_x(6), [prefix])
    seqs = [fwd.new_sequence() for _ in range(2)]
    inputs = fwd.layer_inputs(_x(8), seqs, [5, 3], prefix=prefix)
    for i in asked:
        assert inputs(i)["x"].shape == (8, D)
    assert [s.length for s in seqs] == [5, 3]
    fwd.run(_x(2), seqs, prefix=prefix)          # the recorder checks what it reads
    assert [s.length for s in seqs] == [6, 4]
    assert FW.B.calls == [0, 1, 2] * 3


def test_a_prefix_read_in_part_is_completed_too(fwd):
    prefix, seq = fwd.new_sequence(), fwd.new_sequence()
    fwd.layer_inputs(_x(5), [prefix])(0)
    fwd.run(_x(2), [seq], prefix=prefix)
    fwd.run(_x(1), [seq], prefix=prefix)
    assert seq.length == 3 and prefix.length == 5


def test_layers_that_have_been_passed_are_refused(fwd):
    seq = fwd.new_sequence()
    inputs = fwd.layer_inputs(_x(3), [seq])
    inputs(0)
    fwd.run(_x(1), [seq])
    with pytest.raises(ValueError, match="passed"):
        inputs(1)
    assert seq.length == 4


@pytest.mark.parametrize("layers_seen", [1, 2, 3])
def test_a_step_that_its_caller_leaves(fwd, layers_seen):
    seqs = [fwd.new_sequence(), fwd.new_sequence()]
    other = fwd.new_sequence()
    free = len(fwd.free)
    for i, a, x in fwd.blocks(_x(4), seqs):
        if i + 1 == layers_seen:
            break
    if layers_seen < N:
        for bad, prefix in (([seqs[0]], None), ([other], seqs[1])):
            with pytest.raises(ValueError, match="release"):
                fwd.run(_x(1), bad, prefix=prefix)
        for s in seqs:
            fwd.release(s)
        assert len(fwd.free) == free
    fwd.run(_x(2), seqs)
    fwd.run(_x(1), [other], prefix=seqs[0])


def test_a_step_under_way_cannot_be_built_upon(fwd):
    seq = fwd.new_sequence()
    run = fwd.blocks(_x(3), [seq])
    next(run)
    with pytest.raises(ValueError, match="release"):
        fwd.run(_x(1), [seq])
    for _ in run:
        pass
    fwd.run(_x(1), [seq])
    assert seq.length == 4


def test_a_step_that_fails_is_not_built_upon(fwd):
    seq = fwd.new_sequence()
    FW.B.status = [B.AFF_OK, B.AFF_ERR_RANGE]
    inputs = fwd.layer_inputs(_x(3), [seq])
    inputs(0)
    with pytest.raises(B.AffinityError):
        fwd.run(_x(1), [seq])
    with pytest.raises(ValueError, match="release"):
        fwd.run(_x(1), [seq])
    fwd.release(seq)
    fwd.run(_x(1), [seq])


@pytest.mark.parametrize("which", ["sequence", "prefix"])
def test_a_step_whose_pages_were_given_back_does_not_go_on(fwd, which):
    prefix, seqs = fwd.new_sequence(), [fwd.new_sequence(), fwd.new_sequence()]
    fwd.run(_x(3), [prefix])
    inputs = fwd.layer_inputs(_x(4), seqs, prefix=prefix)
    inputs(0)
    fwd.release(prefix if which == "prefix" else seqs[0])
    done = len(FW.B.calls)
    with pytest.raises(ValueError, match="released"):
        inputs(1)
    with pytest.raises(ValueError, match="release"):
        fwd.run(_x(1), [seqs[1]])
    assert len(FW.B.calls) == done
