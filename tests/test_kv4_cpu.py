"""The entry points of the 4-bit cache without a GPU: every refusal before any device is touched, the page's bytes, and
what the binding refuses.  Pointers are made up; no call here gets as far as a launch."""
import ctypes
import math
import os

import pytest

torch = pytest.importorskip("torch")

from oracle import kv4 as K
from transformer_sharding_affinity_gb300 import binding as B
from transformer_sharding_affinity_gb300 import build as BUILD

P = 1 << 20            # a 256-byte aligned pointer that nothing reads
BAD, SHAPE, TYPE, ALIGN = B.AFF_ERR_INVALID_ARG, B.AFF_ERR_UNSUPPORTED_SHAPE, B.AFF_ERR_UNSUPPORTED_DTYPE, B.AFF_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        BUILD.build()
    return B.load()


def _cache(**kw):
    a = dict(k=P, v=P, n_pages=10, page_stride=2 * 576, group_stride=576, G=2, page_size=16, d_head=64, dtype=B.AFF_BF16,
             k_scale=1.0, v_scale=0.5)
    a.update(kw)
    return B.aff_kv4_cache(*a.values())


def _step(**kw):
    a = dict(T=6, prefix_len=20, pages_stride=4, q_start=P, kv_len=P, pages=P, prefix_pages=P, B=3, H=4)
    a.update(kw)
    return B.aff_step(*a.values())


def _size(lib, s, c):
    n = ctypes.c_size_t(0)
    return lib.affinity_kv4_plan_size(ctypes.byref(s), ctypes.byref(c), ctypes.byref(n)), n.value


def _append(lib, s=None, c=None, q=P, qs=256, k=P, ks=128, v=P, vs=128, out=P, os_=256, rot=64, eps=1e-6, n_pos=100, cos=P,
            sin=P, gain=None, rotary=True, plan=P, size=1 << 40):
    r = B.aff_rotary(cos, sin, gain, gain, n_pos, eps, rot, 0)
    return lib.affinity_kv4_append(q, qs, k, ks, v, vs, ctypes.byref(c or _cache()), ctypes.byref(s or _step()),
                                   ctypes.byref(r) if rotary else None, out, os_, plan, size, None)


def _read(lib, s=None, c=None, k=P, v=P, plan=P, size=1 << 40):
    return lib.affinity_kv4_read(ctypes.byref(c or _cache()), ctypes.byref(s or _step()), k, v, plan, size, None)


def _attend(lib, s=None, c=None, q=P, q_stride=256, scale=0.1, out=P, lse=None, plan=P, size=1 << 40):
    return lib.affinity_kv4_attention(q, q_stride, ctypes.byref(c or _cache()), ctypes.byref(s or _step()),
                                      ctypes.c_float(scale), out, lse, plan, size, None)


@pytest.mark.parametrize("step,cache,code", [
    (dict(), dict(k=None), BAD), (dict(), dict(v=None), BAD), (dict(), dict(G=0), BAD), (dict(), dict(page_size=0), BAD),
    (dict(), dict(d_head=0), BAD), (dict(), dict(n_pages=0), BAD), (dict(T=0), dict(), BAD), (dict(B=0), dict(), BAD),
    (dict(H=0), dict(), BAD), (dict(prefix_len=-1), dict(), BAD), (dict(prefix_pages=None), dict(), BAD),
    (dict(), dict(dtype=2), TYPE), (dict(), dict(dtype=-1), TYPE), (dict(H=5), dict(), SHAPE),
    (dict(), dict(d_head=272), SHAPE), (dict(), dict(d_head=24), SHAPE), (dict(), dict(d_head=72), SHAPE),
    (dict(), dict(page_size=12), SHAPE), (dict(T=1 << 29), dict(), SHAPE), (dict(B=(1 << 20) + 1), dict(), SHAPE),
    (dict(pages_stride=1 << 27), dict(), SHAPE), (dict(), dict(page_stride=-16), BAD), (dict(), dict(group_stride=-16), BAD),
    (dict(), dict(page_stride=1160), ALIGN), (dict(), dict(group_stride=584), ALIGN), (dict(), dict(k=P + 8), ALIGN),
    (dict(), dict(v=P + 4), ALIGN), (dict(kv_len=P + 2), dict(), ALIGN),
    (dict(), dict(k_scale=0.0), BAD), (dict(), dict(k_scale=-1.0), BAD), (dict(), dict(v_scale=3.0), BAD),
    (dict(), dict(v_scale=math.inf), BAD), (dict(), dict(k_scale=math.nan), BAD), (dict(), dict(k_scale=2.0 ** 31), BAD),
    (dict(), dict(v_scale=2.0 ** -31), BAD), (dict(), dict(v_scale=1e-42), BAD)])
def test_steps_and_caches_are_refused_by_every_call(lib, step, cache, code):
    s, c = _step(**step), _cache(**cache)
    assert _size(lib, s, c)[0] == code
    assert lib.affinity_kv4_plan(ctypes.byref(s), ctypes.byref(c), P, 1 << 40, None) == code
    assert _append(lib, s, c, qs=4096, ks=4096, vs=4096, os_=4096) == code
    assert _read(lib, s, c) == code
    assert _attend(lib, s, c, q_stride=4096) == code


@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 30, 1.0])
def test_scales_at_the_ends(lib, scale):
    assert _size(lib, _step(), _cache(k_scale=scale, v_scale=scale))[0] == B.AFF_OK


def test_null_structs(lib):
    s, c, n = _step(), _cache(), ctypes.c_size_t(7)
    for args in [(None, ctypes.byref(c), ctypes.byref(n)), (ctypes.byref(s), None, ctypes.byref(n)),
                 (ctypes.byref(s), ctypes.byref(c), None)]:
        assert lib.affinity_kv4_plan_size(*args) == BAD
    assert lib.affinity_kv4_plan(None, None, P, 1 << 40, None) == BAD
    assert lib.affinity_kv4_read(None, ctypes.byref(s), P, P, P, 1 << 40, None) == BAD


def test_plan_buffers(lib):
    s, c = _step(), _cache()
    st, n = _size(lib, s, c)
    assert st == B.AFF_OK and n % 256 == 0
    for plan, size in [(None, n), (P + 128, n), (P, n - 1), (P, 0)]:
        assert lib.affinity_kv4_plan(ctypes.byref(s), ctypes.byref(c), plan, size, None) == B.AFF_ERR_WORKSPACE
        for call in (_append, _read, _attend):
            assert call(lib, plan=plan, size=size) == B.AFF_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(rotary=False), BAD),
    (dict(qs=248), BAD), (dict(ks=120), BAD), (dict(vs=0), BAD), (dict(os_=255), BAD), (dict(rot=-2), BAD), (dict(rot=3), BAD),
    (dict(n_pos=-1), BAD), (dict(cos=None), BAD), (dict(sin=None), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
    (dict(rot=80), SHAPE), (dict(rot=24), SHAPE), (dict(q=P + 4), ALIGN), (dict(k=P + 8), ALIGN), (dict(v=P + 1), ALIGN),
    (dict(cos=P + 4), ALIGN), (dict(gain=P + 2), ALIGN), (dict(qs=260), ALIGN), (dict(os_=257), ALIGN)])
def test_append_arguments(lib, kw, code):
    assert _append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(k=None), BAD), (dict(v=None), BAD), (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN)])
def test_read_arguments(lib, kw, code):
    assert _read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(q_stride=255), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(q=P + 8), ALIGN), (dict(out=P + 2), ALIGN),
    (dict(q_stride=260), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_attention_arguments(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_the_factor_of_the_scores_is_a_number(lib):
    for scale, k_scale in [(1e38, 2.0 ** 30), (1e-38, 2.0 ** -30)]:
        assert _attend(lib, c=_cache(k_scale=k_scale), scale=scale) == BAD


def test_attention_takes_heads_of_128_at_most(lib):
    assert _attend(lib, c=_cache(d_head=144), q_stride=4 * 144) == SHAPE


def test_page_bytes(lib):
    for page in (8, 24, 64, 136):
        for d in (16, 32, 48, 80, 128, 256):
            assert B.kv4_page_bytes(page, d) == K.page_bytes(page, d)
            assert B.kv4_page_bytes(page, d) % 16 == 0
    for page, d, code in [(0, 64, BAD), (8, 0, BAD), (12, 64, SHAPE), (8, 24, SHAPE), (8, 272, SHAPE)]:
        with pytest.raises(B.AffinityError) as e:
            B.kv4_page_bytes(page, d)
        assert e.value.status == code
    assert lib.affinity_kv4_page_bytes(8, 64, None) == BAD


def _pool(n=4, G=2, page=16, d=64, **kw):
    return torch.zeros(n, G, K.page_bytes(page, d), dtype=torch.uint8, **kw)


def test_pools_that_are_no_cache(lib):
    k = _pool()
    c = B.kv4_cache(k, _pool(), 16, 64, torch.bfloat16, 0.5, 2.0)
    assert (c.n_pages, c.G, c.page_stride, c.group_stride, c.dtype) == (4, 2, 1152, 576, B.AFF_BF16)
    pair = torch.zeros(4, 2, 2, 576, dtype=torch.uint8)           # keys and values of a page side by side
    c = B.kv4_cache(pair[:, 0], pair[:, 1], 16, 64, torch.float32)
    assert (c.page_stride, c.group_stride, c.dtype, c.k_scale) == (2304, 576, B.AFF_FP32, 1.0)
    for args in [(k, _pool(n=5), 16, 64, torch.bfloat16), (k, k.to(torch.int8), 16, 64, torch.bfloat16),
                 (k, k, 8, 64, torch.bfloat16), (k, k, 16, 128, torch.bfloat16), (k[..., ::2], k[..., ::2], 8, 64, torch.bfloat16),
                 (k.flatten(0, 1), k.flatten(0, 1), 16, 64, torch.bfloat16), (k, k.transpose(0, 1).contiguous().transpose(0, 1),
                                                                              16, 64, torch.bfloat16)]:
        with pytest.raises(ValueError):
            B.kv4_cache(*args)
    with pytest.raises(TypeError):
        B.kv4_cache(k, k, 16, 64, torch.float16)


def _host_step():
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)
    return B.step(3, 4, ints(0, 2, 3), ints(5, 9), ints(0, 1, 2, 3).view(2, 2))


def test_the_binding_checks_shapes_types_and_devices(lib):
    c, s = B.kv4_cache(_pool(), _pool(), 16, 64, torch.bfloat16), _host_step()
    one = torch.ones(16, 32)
    r = B.rotary(one, one)
    q, k, plan = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(
        1 << 20, dtype=torch.uint8)
    for args in [(q[:2], k, k, c, s, r, q, plan), (q, k[:, :1], k, c, s, r, q, plan)]:
        with pytest.raises(ValueError):
            B.kv4_append(*args)
    with pytest.raises(TypeError):
        B.kv4_append(q.float(), k, k, c, s, r, q, plan)
    for args in [(c, s, k[:2], k, plan), (c, s, k.float(), k, plan), (c, s, k, k.transpose(0, 1).contiguous().transpose(0, 1), plan)]:
        with pytest.raises(ValueError):
            B.kv4_read(*args)
    for args in [(q[:2], c, s, 1.0, q, None, plan), (q, c, s, 1.0, q, torch.zeros(3, 2), plan)]:
        with pytest.raises(ValueError):
            B.kv4_attention(*args)
    with pytest.raises(TypeError):
        B.kv4_attention(q.float(), c, s, 1.0, q, None, plan)
    for call in (lambda: B.kv4_append(q, k, k, c, s, r, q, plan), lambda: B.kv4_read(c, s, k, k.clone(), plan),
                 lambda: B.kv4_attention(q, c, s, 1.0, q, None, plan), lambda: B.step_plan(s, c, plan)):
        with pytest.raises(TypeError, match="GPU"):           # all on the host
            call()
    assert B.step_plan_size(s, c) > 0
