"""Refusals and sizes of the paged cache's C ABI and binding: no GPU, no CUDA
call.  Pointers are made up; every call here returns before a launch."""
import ctypes

import pytest
import torch

from bit_kv_cache_06_gb300 import build as kbuild
from bit_kv_cache_06_gb300 import kivi, paged


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kivi.load()


def params(**kw):
    base = dict(bits=2, group=32, residual=128, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                capacity_tokens=4096)
    base.update(kw)
    return kivi.make_params(**base)


def cache(L, p=None, **kw):
    c = kivi.kivi_paged()
    p = params() if p is None else p
    a = dict(pool=0x10000, num_pages=512, k_fp16=0x20000, v_fp16=0x30000, table=0x40000, n_tokens=0x50000,
             n_evicted=0x60004, control=0x70000)
    a.update(kw)
    st = L.kivi_paged_init(ctypes.byref(c), ctypes.byref(p), *a.values())
    return st, c


def chunk(**kw):
    x = kivi.kivi_chunk()
    a = dict(q=0x100000, k=0x200000, v=0x300000, offsets=0x400004, q_stride=1024, kv_stride=256, num_tokens=10,
             max_new=4, max_cached=0, softmax_scale=0.0, softcap=0.0, mask=0, reserved=0)
    a.update(kw)
    for k, v in a.items():
        setattr(x, k, v)
    return x


def test_structs(L):
    assert L.kivi_sizeof_paged() == ctypes.sizeof(kivi.kivi_paged) == 136
    assert L.kivi_sizeof_chunk() == ctypes.sizeof(kivi.kivi_chunk) == 80


def test_sizes(L):
    def col(**kw):
        return L.kivi_paged_columns(ctypes.byref(params(**kw)))

    assert col() == 128 and col(group=64, bits=4) == 64
    assert col(bits=3) == 0 and col(capacity_tokens=0) == 0
    assert col(capacity_tokens=1 << 31) == 0                     # token counts are 32 bits
    assert col(batch=4096, num_kv_heads=8, num_q_heads=8, capacity_tokens=1 << 21) == 0   # C P above 2^31
    assert L.kivi_paged_control_bytes(ctypes.byref(params())) == 256
    assert L.kivi_paged_control_bytes(ctypes.byref(params(batch=64))) == 512
    sizes = [L.kivi_paged_workspace_bytes(ctypes.byref(params()), n, 0) for n in (0, 1, 2, 17, 100, 1000, 5000)]
    assert sizes == sorted(sizes) and sizes[0] >= 4 * 128 * 4 and all(s % 256 == 0 for s in sizes)
    assert L.kivi_paged_workspace_bytes(ctypes.byref(params()), -1, 0) == 0
    assert L.kivi_paged_workspace_bytes(ctypes.byref(params()), 1, -1) == 0
    assert L.kivi_paged_workspace_bytes(ctypes.byref(params(bits=3)), 1, 0) == 0
    sizes = [L.kivi_paged_workspace_bytes(ctypes.byref(params()), 1000, n) for n in (1, 64, 1000, 4000, 0)]
    assert sizes == sorted(sizes)


def test_init_refuses(L):
    assert cache(L)[0] == 0
    for k in ("pool", "k_fp16", "v_fp16", "table", "n_tokens", "n_evicted", "control"):
        assert cache(L, **{k: None})[0] == kivi.KIVI_ERR_INVALID_ARG
        assert cache(L, **{k: 0x10002})[0] == kivi.KIVI_ERR_INVALID_ARG
    for k in ("pool", "k_fp16", "v_fp16"):
        assert cache(L, **{k: 0x10008})[0] == kivi.KIVI_ERR_INVALID_ARG
    assert cache(L, num_pages=0)[0] == kivi.KIVI_ERR_INVALID_ARG
    assert cache(L, num_pages=1 << 31)[0] == kivi.KIVI_ERR_INVALID_ARG
    assert cache(L, params(head_dim=64))[0] == kivi.KIVI_ERR_UNSUPPORTED
    assert cache(L, params(capacity_tokens=0))[0] == kivi.KIVI_ERR_UNSUPPORTED
    assert L.kivi_paged_init(None, None, *([None] * 1), 0, *([None] * 6)) == kivi.KIVI_ERR_INVALID_ARG


BAD = [dict(offsets=None), dict(offsets=0x400002), dict(reserved=1), dict(mask=2), dict(num_tokens=-1),
       dict(max_new=-1), dict(max_cached=-1), dict(softcap=float("nan")), dict(softmax_scale=float("inf")),
       dict(kv_stride=248), dict(kv_stride=260), dict(k=0x200008)]


def test_calls_refuse_before_they_launch(L):
    _, c = cache(L)
    ws, n = 0x800000, 1 << 40
    cc = ctypes.byref(c)

    def append(x):
        return L.kivi_paged_append(cc, x, None)

    def attention(x, out=0x900000, ws=ws, n=n):
        return L.kivi_paged_attention(cc, x, out, ws, n, None)

    def weights(x, w=0xa00004, ws=ws, n=n):
        return L.kivi_paged_weights(cc, x, w, ws, n, None)

    for call in (append, attention, weights):
        for kw in BAD:
            assert call(ctypes.byref(chunk(**kw))) == kivi.KIVI_ERR_INVALID_ARG, (call, kw)
        assert call(None) == kivi.KIVI_ERR_INVALID_ARG
        assert call(ctypes.byref(chunk(num_tokens=1 << 31))) == kivi.KIVI_ERR_UNSUPPORTED
        assert call(ctypes.byref(chunk(max_new=1 << 30))) == kivi.KIVI_ERR_UNSUPPORTED
        assert call(ctypes.byref(chunk(max_new=0))) == 0 and call(ctypes.byref(chunk(num_tokens=0))) == 0
    for call in (attention, weights):
        for kw in (dict(q=None), dict(q=0x100008), dict(q_stride=1016), dict(q_stride=1028), dict(k=None)):
            if call is weights and kw == dict(k=None):
                continue                                         # new tokens' keys are optional there
            assert call(ctypes.byref(chunk(**kw))) == kivi.KIVI_ERR_INVALID_ARG, kw
        x = ctypes.byref(chunk())
        assert call(x, None) == call(x, ws=None) == call(x, ws=0x800008) == kivi.KIVI_ERR_INVALID_ARG
        assert call(x, n=1000) == kivi.KIVI_ERR_WORKSPACE
    assert attention(ctypes.byref(chunk()), out=0x900008) == kivi.KIVI_ERR_INVALID_ARG
    assert attention(ctypes.byref(chunk(v=None))) == kivi.KIVI_ERR_INVALID_ARG
    assert weights(ctypes.byref(chunk()), w=0xa00002) == kivi.KIVI_ERR_INVALID_ARG
    assert append(ctypes.byref(chunk(v=None))) == append(ctypes.byref(chunk(k=None))) == kivi.KIVI_ERR_INVALID_ARG

    def evict(w=0xa00004, budget=4, recent=2, ws=ws, n=n):
        return L.kivi_paged_evict(cc, w, budget, recent, ws, n, None)

    for kw in (dict(w=None), dict(w=0xa00002), dict(budget=-1), dict(recent=-1), dict(ws=None), dict(ws=0x800004)):
        assert evict(**kw) == kivi.KIVI_ERR_INVALID_ARG
    assert evict(n=100) == kivi.KIVI_ERR_WORKSPACE
    c.num_pages = 0
    assert evict() == append(ctypes.byref(chunk())) == kivi.KIVI_ERR_INVALID_ARG
    assert c.kernel_launches == 0


def test_binding_checks_its_tensors(L):
    shape = kivi.CacheShape(2, 32, 64, 2, 8, 2, 128, 1024)
    with pytest.raises(ValueError, match="pages"):
        paged.KiviPagedCache(shape, 100, device="cpu")
    with pytest.raises(kivi.KiviError):
        paged.KiviPagedCache(kivi.CacheShape(2, 32, 64, 2, 8, 2, 128, 0), device="cpu")
    with pytest.raises(kivi.KiviError):
        paged.KiviPagedCache(shape, device="cpu", workspace=torch.empty(16, dtype=torch.uint8))
    c = paged.KiviPagedCache(shape, max_new=4, device="cpu")
    assert c.table.tolist()[3][:2] == [96, 97] and c.status() == 0
    bufs = [c.pool, c.k_fp16, c.v_fp16, c.table, c.n_tokens, c.n_evicted]
    for i, t in enumerate(bufs):
        for bad in (t[:-1], t.to(torch.int64) if t.dtype != torch.float16 else t.float()):
            with pytest.raises(ValueError):
                paged.KiviPagedCache(shape, 128, buffers=bufs[:i] + [bad] + bufs[i + 1:])
    q, kv = torch.zeros((6, 8, 128), dtype=torch.float16), torch.zeros((6, 2, 128), dtype=torch.float16)
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    for a in ((q.float(), kv, kv, off), (q[:, :4], kv, kv, off), (q[:5], kv, kv, off), (q, kv, kv[:5], off),
              (q, kv, None, off.long()), (q, None, kv, off), (q, kv, kv, off[:2]), (q[:, :, :64], kv, kv, off),
              (q.transpose(0, 1).contiguous().transpose(0, 1), kv, kv, off)):
        with pytest.raises(ValueError):
            c.attention(*a)
    with pytest.raises(ValueError):
        c.weights(torch.zeros((4, 31)), q, kv, off)
    with pytest.raises(ValueError):
        c.evict(torch.zeros((4, 32), dtype=torch.float64), 3)


def test_scales_and_caps_outside_fp32_are_refused(L):
    _, c = cache(L)
    cc, ws, n = ctypes.byref(c), 0x800000, 1 << 40
    for kw in (dict(softmax_scale=3e38), dict(softcap=1e-40), dict(softcap=3e38), dict(softmax_scale=1e10, softcap=1e-30)):
        x = ctypes.byref(chunk(**kw))
        assert L.kivi_paged_attention(cc, x, 0x900000, ws, n, None) == kivi.KIVI_ERR_INVALID_ARG, kw
        assert L.kivi_paged_weights(cc, x, 0xa00004, ws, n, None) == kivi.KIVI_ERR_INVALID_ARG, kw
    assert L.kivi_paged_workspace_bytes(ctypes.byref(params()), 2 ** 31 - 1, 2 ** 31 - 1) > 0
    assert c.kernel_launches == 0


def test_products_beyond_the_plan_are_unsupported(L):
    p = params(batch=1, num_q_heads=4, num_kv_heads=1, capacity_tokens=1 << 30)
    _, c = cache(L, p)
    x = chunk(max_new=1 << 20, num_tokens=1 << 20, q_stride=512, kv_stride=128)
    x.max_new = 65535 * 64 // 4
    args = ctypes.byref(c), ctypes.byref(x), 0x900000, 0x800000
    assert L.kivi_paged_attention(*args, 1000, None) == kivi.KIVI_ERR_UNSUPPORTED
    x.max_cached = 1 << 20
    assert L.kivi_paged_attention(*args, 1000, None) == kivi.KIVI_ERR_WORKSPACE
    assert L.kivi_paged_columns(ctypes.byref(params(batch=1, num_kv_heads=1, num_q_heads=1, residual=32,
                                                    capacity_tokens=(1 << 31) - 4096))) == 0
