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
