"""The forward-pass entry points without a GPU: every refusal of theirs, before any device is touched; the order of
the checks; sizes of a step's plan.  Pointers are made up where a call has to refuse before it would use them: no
call here gets as far as a launch (there may be no device, and with one the last check stands in its way)."""
import ctypes
import math
import os

import pytest

torch = pytest.importorskip("torch")

from transformer_sharding_affinity_gb300 import binding as B
from transformer_sharding_affinity_gb300 import build as BUILD

P = 1 << 20            # a 256-byte aligned pointer that nothing reads


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        BUILD.build()
    return B.load()


def _cache(**kw):
    a = dict(k=P, v=P, n_pages=10, page_stride=2 * 16 * 64, group_stride=16 * 64, token_stride=64, G=2, page_size=16,
             d_head=64, dtype=B.AFF_BF16)
    a.update(kw)
    return B.aff_kv_cache(*a.values())


def _step(**kw):
    a = dict(T=6, prefix_len=20, pages_stride=4, q_start=P, kv_len=P, pages=P, prefix_pages=P, B=3, H=4)
    a.update(kw)
    return B.aff_step(*a.values())


def _size(lib, s, c):
    n = ctypes.c_size_t(0)
    st = lib.affinity_step_plan_size(ctypes.byref(s), ctypes.byref(c), ctypes.byref(n))
    return st, n.value


SHAPES = [(dict(), dict(G=0), B.AFF_ERR_INVALID_ARG), (dict(), dict(page_size=0), B.AFF_ERR_INVALID_ARG),
          (dict(), dict(d_head=0), B.AFF_ERR_INVALID_ARG), (dict(), dict(n_pages=0), B.AFF_ERR_INVALID_ARG),
          (dict(T=0), dict(), B.AFF_ERR_INVALID_ARG), (dict(T=-3), dict(), B.AFF_ERR_INVALID_ARG),
          (dict(B=0), dict(), B.AFF_ERR_INVALID_ARG), (dict(H=0), dict(), B.AFF_ERR_INVALID_ARG),
          (dict(prefix_len=-1), dict(), B.AFF_ERR_INVALID_ARG),
          (dict(), dict(dtype=2), B.AFF_ERR_UNSUPPORTED_DTYPE), (dict(), dict(dtype=-1), B.AFF_ERR_UNSUPPORTED_DTYPE),
          (dict(H=5), dict(), B.AFF_ERR_UNSUPPORTED_SHAPE), (dict(H=4098), dict(), B.AFF_ERR_UNSUPPORTED_SHAPE),
          (dict(), dict(d_head=264, token_stride=264), B.AFF_ERR_UNSUPPORTED_SHAPE),
          (dict(), dict(d_head=60), B.AFF_ERR_UNSUPPORTED_SHAPE), (dict(), dict(page_size=12), B.AFF_ERR_UNSUPPORTED_SHAPE),
          (dict(T=1 << 29), dict(), B.AFF_ERR_UNSUPPORTED_SHAPE), (dict(B=(1 << 20) + 1), dict(), B.AFF_ERR_UNSUPPORTED_SHAPE),
          (dict(prefix_len=(1 << 30) + 1), dict(), B.AFF_ERR_UNSUPPORTED_SHAPE),
          (dict(pages_stride=1 << 27), dict(), B.AFF_ERR_UNSUPPORTED_SHAPE),
          (dict(), dict(token_stride=32), B.AFF_ERR_INVALID_ARG), (dict(), dict(page_stride=-8), B.AFF_ERR_INVALID_ARG)]


@pytest.mark.parametrize("step,cache,code", SHAPES)
def test_shapes_are_refused_by_every_call(lib, step, cache, code):
    s, c = _step(**step), _cache(**cache)
    assert _size(lib, s, c)[0] == code
    r = B.aff_rotary(P, P, None, None, 100, 1e-6, 64, 0)
    assert lib.affinity_step_plan(ctypes.byref(s), ctypes.byref(c), P, 1 << 40, None) == code
    assert lib.affinity_kv_append(P, 1024, P, 1024, P, 1024, ctypes.byref(c), ctypes.byref(s), ctypes.byref(r), P, 1024, P,
                                  1 << 40, None) == code
    assert lib.affinity_prefix_attention(P, 1024, ctypes.byref(c), ctypes.byref(s), ctypes.c_float(0.1), P, None, P, 1 << 40,
                                         None) == code


def test_null_structs(lib):
    s, c, n = _step(), _cache(), ctypes.c_size_t(7)
    for args in [(None, ctypes.byref(c), ctypes.byref(n)), (ctypes.byref(s), None, ctypes.byref(n)),
                 (ctypes.byref(s), ctypes.byref(c), None)]:
        assert lib.affinity_step_plan_size(*args) == B.AFF_ERR_INVALID_ARG
    assert lib.affinity_block_norm(None, None) == B.AFF_ERR_INVALID_ARG


def test_plan_buffers(lib):
    s, c = _step(), _cache()
    st, n = _size(lib, s, c)
    assert st == B.AFF_OK and n % 256 == 0
    for plan, size in [(None, n), (P + 128, n), (P, n - 1), (P, 0)]:
        assert lib.affinity_step_plan(ctypes.byref(s), ctypes.byref(c), plan, size, None) == B.AFF_ERR_WORKSPACE
        assert lib.affinity_prefix_attention(P, 256, ctypes.byref(c), ctypes.byref(s), ctypes.c_float(0.1), P, None, plan,
                                             size, None) == B.AFF_ERR_WORKSPACE


def test_plans_grow_with_the_step_and_hold_the_partial_rows(lib):
    _, small = _size(lib, _step(), _cache())
    _, more_tokens = _size(lib, _step(T=100), _cache())
    _, more_sequences = _size(lib, _step(B=3000), _cache())
    assert small < more_tokens and small < more_sequences
    # a prefix's rows are held twice in fp32 at most, beside a constant room for cuts
    _, decode = _size(lib, _step(T=256, B=256, H=32, prefix_len=32768), _cache(G=8, d_head=128, token_stride=128,
                                                                             group_stride=16 * 128, page_stride=8 * 16 * 128))
    assert decode < 160 << 20


def _attend(lib, q=P, q_stride=256, scale=0.1, out=P, lse=None, cache=None, step=None):
    c, s = cache or _cache(), step or _step()
    return lib.affinity_prefix_attention(q, q_stride, ctypes.byref(c), ctypes.byref(s), ctypes.c_float(scale), out, lse, P,
                                         1 << 40, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.AFF_ERR_INVALID_ARG), (dict(out=None), B.AFF_ERR_INVALID_ARG), (dict(q_stride=255), B.AFF_ERR_INVALID_ARG),
    (dict(scale=0.0), B.AFF_ERR_INVALID_ARG), (dict(scale=-1.0), B.AFF_ERR_INVALID_ARG),
    (dict(scale=math.nan), B.AFF_ERR_INVALID_ARG), (dict(scale=math.inf), B.AFF_ERR_INVALID_ARG),
    (dict(q=P + 8), B.AFF_ERR_ALIGNMENT), (dict(out=P + 2), B.AFF_ERR_ALIGNMENT), (dict(q_stride=260), B.AFF_ERR_ALIGNMENT),
    (dict(lse=P + 2), B.AFF_ERR_ALIGNMENT)])
def test_attention_arguments(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_attention_takes_heads_of_128_at_most(lib):
    c = _cache(d_head=136, token_stride=136, group_stride=16 * 136, page_stride=2 * 16 * 136)
    assert _attend(lib, q_stride=4 * 136, cache=c) == B.AFF_ERR_UNSUPPORTED_SHAPE


def _append(lib, rot=64, eps=1e-6, n_pos=100, cos=P, sin=P, gain=None, interleaved=0, q=P, k=P, v=P, out=P, qs=256, ks=128,
            vs=128, os_=256, rotary=True):
    c, s, r = _cache(), _step(), B.aff_rotary(cos, sin, gain, gain, n_pos, eps, rot, interleaved)
    return lib.affinity_kv_append(q, qs, k, ks, v, vs, ctypes.byref(c), ctypes.byref(s), ctypes.byref(r) if rotary else None,
                                  out, os_, P, 1 << 40, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.AFF_ERR_INVALID_ARG), (dict(k=None), B.AFF_ERR_INVALID_ARG), (dict(v=None), B.AFF_ERR_INVALID_ARG),
    (dict(out=None), B.AFF_ERR_INVALID_ARG), (dict(rotary=False), B.AFF_ERR_INVALID_ARG),
    (dict(qs=248), B.AFF_ERR_INVALID_ARG), (dict(ks=120), B.AFF_ERR_INVALID_ARG), (dict(vs=0), B.AFF_ERR_INVALID_ARG),
    (dict(os_=255), B.AFF_ERR_INVALID_ARG), (dict(rot=-2), B.AFF_ERR_INVALID_ARG), (dict(rot=3), B.AFF_ERR_INVALID_ARG),
    (dict(n_pos=-1), B.AFF_ERR_INVALID_ARG), (dict(cos=None), B.AFF_ERR_INVALID_ARG), (dict(sin=None), B.AFF_ERR_INVALID_ARG),
    (dict(eps=-1.0), B.AFF_ERR_INVALID_ARG), (dict(eps=math.nan), B.AFF_ERR_INVALID_ARG),
    (dict(rot=66), B.AFF_ERR_UNSUPPORTED_SHAPE), (dict(q=P + 4), B.AFF_ERR_ALIGNMENT), (dict(k=P + 8), B.AFF_ERR_ALIGNMENT),
    (dict(v=P + 1), B.AFF_ERR_ALIGNMENT), (dict(cos=P + 4), B.AFF_ERR_ALIGNMENT), (dict(gain=P + 2), B.AFF_ERR_ALIGNMENT),
    (dict(qs=260), B.AFF_ERR_ALIGNMENT), (dict(os_=257), B.AFF_ERR_ALIGNMENT)])
def test_append_arguments(lib, kw, code):
    assert _append(lib, **kw) == code


def _norm(lib, **kw):
    a = dict(x=P, f=P, gate=None, post_gain=None, pre_gain=P, y=P, h=P, T=4, D=64, x_stride=64, f_stride=64, gate_stride=0,
             y_stride=64, h_stride=64, rows_per_gate=1, scale=1.0, eps=1e-6, dtype=B.AFF_BF16)
    a.update(kw)
    s = B.aff_block_norm(*a.values())
    return lib.affinity_block_norm(ctypes.byref(s), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), B.AFF_ERR_UNSUPPORTED_DTYPE), (dict(x=None), B.AFF_ERR_INVALID_ARG), (dict(f=None), B.AFF_ERR_INVALID_ARG),
    (dict(y=None), B.AFF_ERR_INVALID_ARG), (dict(h=None), B.AFF_ERR_INVALID_ARG), (dict(pre_gain=None), B.AFF_ERR_INVALID_ARG),
    (dict(T=0), B.AFF_ERR_INVALID_ARG), (dict(D=0), B.AFF_ERR_INVALID_ARG), (dict(x_stride=63), B.AFF_ERR_INVALID_ARG),
    (dict(f_stride=0), B.AFF_ERR_INVALID_ARG), (dict(y_stride=-64), B.AFF_ERR_INVALID_ARG), (dict(h_stride=8), B.AFF_ERR_INVALID_ARG),
    (dict(gate=P), B.AFF_ERR_INVALID_ARG), (dict(gate=P, gate_stride=64, rows_per_gate=0), B.AFF_ERR_INVALID_ARG),
    (dict(eps=-1e-6), B.AFF_ERR_INVALID_ARG), (dict(eps=math.inf), B.AFF_ERR_INVALID_ARG), (dict(scale=math.nan), B.AFF_ERR_INVALID_ARG),
    (dict(D=16385, x_stride=16392, f_stride=16392, y_stride=16392, h_stride=16392), B.AFF_ERR_UNSUPPORTED_SHAPE),
    (dict(x=P + 2), B.AFF_ERR_ALIGNMENT), (dict(pre_gain=P + 4), B.AFF_ERR_ALIGNMENT)])
def test_norm_arguments(lib, kw, code):
    assert _norm(lib, **kw) == code


def test_valid_calls_need_this_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("made-up pointers")
    assert _norm(lib) == _append(lib) == _attend(lib) == B.AFF_ERR_ARCH
    s, c = _step(), _cache()
    assert lib.affinity_step_plan(ctypes.byref(s), ctypes.byref(c), P, 1 << 40, None) in (B.AFF_ERR_ARCH, B.AFF_ERR_CUDA)


# ---------------------------------------------------------------- the binding's own checks

def _pool(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def _small():
    c = B.kv_cache(_pool(4, 2, 16, 64), _pool(4, 2, 16, 64))
    s = B.step(3, 4, _ints(0, 1, 3), _ints(1, 2), torch.zeros(2, 1, dtype=torch.int32))
    return c, s


@pytest.mark.parametrize("k,v", [
    (_pool(4, 2, 16, 64), _pool(4, 2, 16, 32)), (_pool(4, 2, 64), _pool(4, 2, 64)),
    (_pool(4, 2, 16, 64), _pool(4, 16, 2, 64).transpose(1, 2)),
    (_pool(4, 2, 16, 128)[..., ::2], _pool(4, 2, 16, 128)[..., ::2])])
def test_pools_are_checked(k, v):
    with pytest.raises(ValueError):
        B.kv_cache(k, v)


def test_pools_of_two_types_or_another_type_are_refused():
    with pytest.raises((TypeError, ValueError)):
        B.kv_cache(_pool(4, 2, 16, 64), _pool(4, 2, 16, 64, dtype=torch.float32))
    with pytest.raises((TypeError, ValueError)):
        B.kv_cache(_pool(4, 2, 16, 64, dtype=torch.float16), _pool(4, 2, 16, 64, dtype=torch.float16))


@pytest.mark.parametrize("q_start,kv_len,pages", [
    (torch.zeros(3), _ints(1, 2), torch.zeros(2, 1, dtype=torch.int32)), (_ints(0, 1), _ints(1, 2), torch.zeros(2, 1, dtype=torch.int32)),
    (_ints(0, 1, 2), _ints(1, 2), torch.zeros(3, 1, dtype=torch.int32)), (_ints(0, 1, 2), _ints(1, 2), _ints(0, 0)),
    (_ints(0, 1, 2), torch.tensor([1, 2]), torch.zeros(2, 1, dtype=torch.int32))])
def test_index_arrays_are_checked(q_start, kv_len, pages):
    with pytest.raises(ValueError):
        B.step(3, 4, q_start, kv_len, pages)


def test_binding_refuses_rows_types_and_layouts(lib):
    c, s = _small()
    cos = torch.ones(8, 32)
    r = B.rotary(cos, cos)
    plan = torch.empty(B.step_plan_size(s, c), dtype=torch.uint8)
    q, k = _pool(3, 4, 64), _pool(3, 2, 64)
    with pytest.raises(ValueError):
        B.kv_append(q[:2], k, k, c, s, r, q, plan)
    with pytest.raises((TypeError, ValueError)):
        B.kv_append(q.float(), k, k, c, s, r, q, plan)
    with pytest.raises(ValueError):
        B.kv_append(q, k, k, c, s, B.rotary(cos, cos, q_gain=_pool(32)), q, plan)
    with pytest.raises(ValueError):
        B.rotary(cos, torch.ones(8, 16))
    with pytest.raises(ValueError):
        B.rotary(cos.double(), cos.double())
    with pytest.raises(ValueError):
        B.prefix_attention(q[:1], c, s, 0.1, q, None, plan)
    with pytest.raises((TypeError, ValueError)):
        B.prefix_attention(q, c, s, 0.1, q.float(), None, plan)
    with pytest.raises(ValueError):
        B.prefix_attention(q, c, s, 0.1, _pool(3, 4, 72)[..., :64], None, plan)
    with pytest.raises(ValueError):
        B.prefix_attention(q, c, s, 0.1, q, torch.zeros(3, 3), plan)
    with pytest.raises(ValueError, match="prefix"):
        B.step_plan(B.step(3, 4, _ints(0, 1, 3), _ints(1, 2), torch.zeros(2, 1, dtype=torch.int32), _ints(0), 17), c, plan)
    x = _pool(5, 64)
    with pytest.raises(ValueError):
        B.block_norm(x, x[:4], x)
    with pytest.raises(TypeError):
        B.block_norm(x, x.float(), x)
    with pytest.raises(ValueError):
        B.block_norm(x, x, x, x, pre_gain=_pool(32))
    with pytest.raises(ValueError):
        B.block_norm(x, x, x, gate=_pool(2, 64), rows_per_gate=2)
