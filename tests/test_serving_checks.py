"""Refusals of the 8-bit serving operators (CPU): every bad argument is turned
down with its documented status before anything is launched, by the C ABI and
by the binding."""
import ctypes

import pytest
import torch

from group_wise_affine_amd import qmm as Q

P = ctypes.c_void_p(0x100000)
P2 = ctypes.c_void_p(0x100002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return Q.lib()


def cache(**kw):
    a = dict(k=0x100000, v=0x100000, k_scales=0x100000, v_scales=0x100000, pages=8, heads=2, page_tokens=32,
             head_dim=128)
    a.update(kw)
    return ctypes.byref(Q._Kv8(*a.values()))


GOOD = {
    "qmm_i8_quantize": dict(x=P, ldx=64, dt=0, rows=4, K=64, codes=P, scales=P, st=None),
    "qmm_i8_t": dict(xq=P, sx=P, wq=P, sw=P, bias=None, dt=1, M=4, N=4, K=64, y=P, work=P, nb=BIG, st=None),
    "qmm_i8_linear": dict(x=P, ldx=64, wq=P, sw=P, bias=None, dt=1, M=4, N=4, K=64, y=P, work=P, nb=BIG, st=None),
    "qmm_kv8_append": dict(c=cache(), k=P, ldk=256, v=P, ldv=256, dt=0, T=3, table=P, lens=P, cu=P, S=2, W=4, st=None),
    "qmm_kv8_read": dict(c=cache(), pages=P, n=3, dt=0, k=P, v=P, st=None),
    "qmm_kv8_attention": dict(c=cache(), q=P, ldq=512, dt=0, T=3, Hq=4, table=P, lens=P, cu=P, S=2, W=4, scale=1.0,
                              out=P, lse=None, work=P, nb=BIG, st=None),
    "qmm_kv8_update": dict(c=cache(), ref=P, table=P, lens=P, parent=P, new_lens=P, S=2, W=4,
                           ref_out=ctypes.c_void_p(0x200000), table_out=ctypes.c_void_p(0x200000), short=P, work=P,
                           nb=BIG, st=None),
    "qmm_kv8_compact": dict(c=cache(), ref=P, table=P, S=2, W=4, ref_out=ctypes.c_void_p(0x200000), table_out=P,
                            remap=P, used=P, work=P, nb=BIG, st=None),
    "qmm_kv8_copy": dict(to=cache(), dst=P, source=cache(), src=P, n=2, st=None),
}


def refused(L, fn, status, **bad):
    args = dict(GOOD[fn])
    assert set(bad) <= set(args)
    args.update(bad)
    assert getattr(L, fn)(*args.values()) == status, (fn, bad, L.qmm_last_error())
    assert L.qmm_last_error().startswith(fn.encode())


def test_null_pointers(L):
    optional = {"bias", "lse", "st", "work"}
    for fn, args in GOOD.items():
        for name, v in args.items():
            if isinstance(v, ctypes.c_void_p) and name not in optional:
                refused(L, fn, Q.QMM_E_NULL, **{name: None})
        if "c" in args:
            refused(L, fn, Q.QMM_E_NULL, c=None)
            refused(L, fn, Q.QMM_E_NULL, c=cache(v_scales=0))
    refused(L, "qmm_i8_linear", Q.QMM_E_NULL, work=None, M=400)
    refused(L, "qmm_kv8_update", Q.QMM_E_NULL, work=None)
    refused(L, "qmm_kv8_compact", Q.QMM_E_NULL, work=None)
    refused(L, "qmm_kv8_copy", Q.QMM_E_NULL, source=None)


def test_dtypes(L):
    for fn, args in GOOD.items():
        if "dt" in args:
            for dt in (2, 3, -1):
                refused(L, fn, Q.QMM_E_DTYPE, dt=dt)


def test_sizes_of_the_products(L):
    for fn in ("qmm_i8_t", "qmm_i8_linear"):
        for K in (0, -16, 8, 24, 1 << 17):
            refused(L, fn, Q.QMM_E_SHAPE, K=K)
        refused(L, fn, Q.QMM_E_SHAPE, M=0)
        refused(L, fn, Q.QMM_E_SHAPE, N=-1)
        refused(L, fn, Q.QMM_E_SHAPE, M=1 << 30, N=1 << 30)
    refused(L, "qmm_i8_quantize", Q.QMM_E_SHAPE, K=40)
    refused(L, "qmm_i8_quantize", Q.QMM_E_SHAPE, rows=0)
    for fn in ("qmm_i8_quantize", "qmm_i8_linear"):
        refused(L, fn, Q.QMM_E_SHAPE, ldx=56)
        refused(L, fn, Q.QMM_E_SHAPE, ldx=68)


def test_page_shapes(L):
    for fn, args in GOOD.items():
        if "c" not in args:
            continue
        for kw in (dict(page_tokens=8), dict(page_tokens=48), dict(head_dim=96), dict(head_dim=0), dict(heads=0),
                   dict(pages=0), dict(pages=1 << 29), dict(heads=5000)):
            refused(L, fn, Q.QMM_E_SHAPE, c=cache(**kw))
        refused(L, fn, Q.QMM_E_ALIGN, c=cache(k=0x100008))
        refused(L, fn, Q.QMM_E_ALIGN, c=cache(v_scales=0x100002))
    refused(L, "qmm_kv8_copy", Q.QMM_E_SHAPE, source=cache(heads=3))
    refused(L, "qmm_kv8_copy", Q.QMM_E_SHAPE, source=cache(page_tokens=16))


def test_batches_and_strides(L):
    for fn in ("qmm_kv8_append", "qmm_kv8_attention"):
        for kw in (dict(T=0), dict(T=1 << 25), dict(S=0), dict(S=1 << 16), dict(W=0)):
            refused(L, fn, Q.QMM_E_SHAPE, **kw)
    refused(L, "qmm_kv8_append", Q.QMM_E_SHAPE, ldk=255)
    refused(L, "qmm_kv8_append", Q.QMM_E_SHAPE, ldv=260)
    refused(L, "qmm_kv8_attention", Q.QMM_E_SHAPE, ldq=504)
    refused(L, "qmm_kv8_attention", Q.QMM_E_SHAPE, T=1 << 24, Hq=512, ldq=512 * 128)
    for Hq in (1, 3, 0):
        refused(L, "qmm_kv8_attention", Q.QMM_E_SHAPE, Hq=Hq)
    refused(L, "qmm_kv8_read", Q.QMM_E_SHAPE, n=0)
    refused(L, "qmm_kv8_copy", Q.QMM_E_SHAPE, n=0)
    refused(L, "qmm_kv8_update", Q.QMM_E_SHAPE, S=0)
    refused(L, "qmm_kv8_compact", Q.QMM_E_SHAPE, W=0)


def test_alignment(L):
    for fn, names in (("qmm_i8_quantize", ("x", "codes", "scales")), ("qmm_i8_t", ("xq", "wq", "y", "sw", "work")),
                      ("qmm_i8_linear", ("x", "wq", "y", "sw", "work")), ("qmm_kv8_append", ("k", "v", "table", "lens", "cu")),
                      ("qmm_kv8_read", ("k", "v", "pages")), ("qmm_kv8_attention", ("q", "out", "table", "lens", "cu")),
                      ("qmm_kv8_update", ("ref", "table", "lens", "parent", "new_lens", "ref_out", "table_out", "short")),
                      ("qmm_kv8_compact", ("ref", "table", "ref_out", "table_out", "remap", "used")),
                      ("qmm_kv8_copy", ("dst", "src"))):
        for n in names:
            refused(L, fn, Q.QMM_E_ALIGN, **{n: P2})
    refused(L, "qmm_kv8_attention", Q.QMM_E_ALIGN, lse=P2)
    refused(L, "qmm_i8_t", Q.QMM_E_ALIGN, bias=ctypes.c_void_p(0x100001))


def test_scratch_and_aliases(L):
    refused(L, "qmm_i8_linear", Q.QMM_E_ARG, nb=100, M=400)
    need = L.qmm_i8_linear_work(400, 4, 64)
    assert need >= 65536 + 400 * 64 + 1600
    refused(L, "qmm_i8_linear", Q.QMM_E_ARG, nb=need - 1, M=400)
    refused(L, "qmm_kv8_update", Q.QMM_E_ARG, nb=L.qmm_kv8_pages_work(8) - 1)
    refused(L, "qmm_kv8_compact", Q.QMM_E_ARG, nb=0)
    refused(L, "qmm_kv8_attention", Q.QMM_E_ARG, W=4096, T=1, S=1, nb=64)
    refused(L, "qmm_kv8_update", Q.QMM_E_ARG, ref_out=P)
    refused(L, "qmm_kv8_update", Q.QMM_E_ARG, table_out=P)
    refused(L, "qmm_kv8_compact", Q.QMM_E_ARG, ref_out=P)


def test_work_sizes(L):
    assert L.qmm_i8_t_work(1, 4096, 4096) == 0
    assert L.qmm_i8_t_work(0, 1, 16) == 0
    assert L.qmm_kv8_attention_work(cache(), 1, 4, 1, 1) == 0
    assert L.qmm_kv8_attention_work(cache(heads=0), 1, 4, 1, 1) == 0
    assert L.qmm_kv8_attention_work(cache(), 1, 4, 1, 4096) > 65536


# ------------------------------------------------------------------ binding


def cpu(*shape, dt=torch.float16):
    return torch.zeros(shape, dtype=dt)


def test_binding_refuses():
    w, s = cpu(8, 64, dt=torch.int8), cpu(8, dt=torch.float32)
    c = Q.Kv8Cache(4, 2, 16, 64, device="cpu")
    tab, lens, cu = cpu(2, 3, dt=torch.int32), cpu(2, dt=torch.int32), cpu(3, dt=torch.int32)
    x3 = cpu(5, 2, 64)
    ref = cpu(4, dt=torch.int32)
    for call in (
        lambda: Q.i8_quantize(cpu(4, 4, 4)),
        lambda: Q.i8_quantize(cpu(4, 64).t()),
        lambda: Q.i8_quantize(cpu(4, 64)),                                   # not on a GPU
        lambda: Q.i8_linear(cpu(4, 64), w[:, :32], s),
        lambda: Q.i8_linear(cpu(4, 64), w, s[:4]),
        lambda: Q.i8_linear(cpu(4, 64), w, s.half()),
        lambda: Q.i8_linear(cpu(4, 64), w, s, bias=cpu(7)),
        lambda: Q.i8_linear(cpu(4, 64), w, s, bias=cpu(8, dt=torch.bfloat16)),
        lambda: Q.i8_linear(cpu(4, 64), w, s, out=cpu(4, 9)),
        lambda: Q.i8_linear(cpu(4, 64), w, s),
        lambda: Q.i8_t(cpu(4, 64, dt=torch.int8), cpu(3, dt=torch.float32), w, s),
        lambda: Q.i8_t(cpu(4, 32, dt=torch.int8), cpu(4, dt=torch.float32), w, s),
        lambda: Q.Kv8Cache.of(c.k, c.k, c.k_scales, c.v_scales),
        lambda: Q.Kv8Cache.of(c.k, c.v, c.k_scales[:2], c.v_scales),
        lambda: Q.kv8_append(c, x3, x3[:4], tab, lens, cu),
        lambda: Q.kv8_append(c, cpu(5, 3, 64), x3, tab, lens, cu),
        lambda: Q.kv8_append(c, x3, x3, tab, lens, lens),
        lambda: Q.kv8_append(c, x3, x3, tab.long(), lens, cu),
        lambda: Q.kv8_append(c, x3, x3, tab, lens, cu),
        lambda: Q.kv8_append(None, x3, x3, tab, lens, cu),
        lambda: Q.kv8_read(c, tab),
        lambda: Q.kv8_attention(c, cpu(5, 4, 32), tab, lens, cu),
        lambda: Q.kv8_attention(c, cpu(5, 4, 64), tab, lens[:1], cu),
        lambda: Q.kv8_attention(c, cpu(5, 4, 64), tab, lens, cu, out=cpu(5, 4, 32)),
        lambda: Q.kv8_attention(c, cpu(5, 4, 64), tab, lens, cu),
        lambda: Q.kv8_attention(c, cpu(5, 64, 4).transpose(1, 2), tab, lens, cu),
        lambda: Q.kv8_update(c, ref[:3], tab, lens, lens, lens),
        lambda: Q.kv8_update(c, ref, tab, lens, lens, cu),
        lambda: Q.kv8_update(c, ref, tab, lens, lens, lens),
        lambda: Q.kv8_compact(c, ref, tab[0]),
        lambda: Q.kv8_compact(c, ref, tab),
        lambda: Q.kv8_copy(c, lens, c, cu),
        lambda: Q.kv8_copy(c, lens, c, lens),
    ):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_dtypes():
    w, s = cpu(8, 64, dt=torch.int8), cpu(8, dt=torch.float32)
    with pytest.raises(Q.QmmError):
        Q.i8_linear(cpu(4, 64, dt=torch.int32), w, s)


@pytest.mark.parametrize("name", ["k", "v", "k_scales", "v_scales", "pages", "heads", "page_tokens", "head_dim"])
def test_a_cache_keeps_its_tensors(name):
    """The library holds their addresses: another tensor is another cache."""
    c = Q.Kv8Cache(4, 2, 16, 64, device="cpu")
    with pytest.raises(AttributeError):
        setattr(c, name, getattr(c, name))


@pytest.mark.parametrize("name", ["k", "v", "k_scales", "v_scales"])
@pytest.mark.parametrize("how", ["data", "resize"])
def test_a_cache_whose_memory_was_replaced_is_refused(name, how):
    tab, lens, cu = cpu(2, 3, dt=torch.int32), cpu(2, dt=torch.int32), cpu(3, dt=torch.int32)
    ref, x = cpu(4, dt=torch.int32), cpu(5, 2, 64)
    good, c = (Q.Kv8Cache(4, 2, 16, 64, device="cpu") for _ in range(2))
    keep = getattr(c, name).clone()
    if how == "data":
        getattr(c, name).data = keep
    else:
        getattr(c, name).resize_(0)
    for call in (lambda: Q.kv8_append(c, x, x, tab, lens, cu), lambda: Q.kv8_read(c, ref),
                 lambda: Q.kv8_attention(c, x, tab, lens, cu), lambda: Q.kv8_update(c, ref, tab, lens, lens, lens),
                 lambda: Q.kv8_compact(c, ref, tab), lambda: Q.kv8_copy(good, ref, c, ref),
                 lambda: Q.kv8_copy(c, ref, good, ref)):
        with pytest.raises(ValueError, match="other memory"):
            call()
