"""Refusals of the operators around the 8-bit cache (CPU): every bad argument is
turned down with its documented status before anything is launched, by the C ABI and
by the binding."""
import ctypes

import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests.test_serving_checks import BIG, P, P2, cache, cpu

P3, P4 = ctypes.c_void_p(0x200000), ctypes.c_void_p(0x300000)
ATT = dict(c=cache(), q=P, ldq=512, dt=0, T=3, Hq=4, table=P, lens=P, cu=P, S=2, W=4)
END = dict(scale=1.0, out=P, lse=None, work=P, nb=BIG, st=None)
GOOD = {
    "qmm_kv8_attention_window": dict(ATT, window=100, sinks=4, **END),
    "qmm_kv8_attention_tree": dict(ATT, parent=P, **END),
    "qmm_qk_norm_rope": dict(q=P, ldq=512, k=P4, ldk=256, dt=0, T=3, Hq=4, Hk=2, D=128, pos=P, freq=P, rot=128, inter=0,
                             wq=P, wk=P, eps=1e-6, qo=P3, ldqo=512, ko=ctypes.c_void_p(0x400000), ldko=256, st=None),
    "qmm_logprobs": dict(x=P, ld=1000, dt=2, M=3, V=1000, tokens=P, top=5, lp=P, h=P, ids=P, tl=P, work=P, nb=BIG, st=None),
}


@pytest.fixture(scope="module")
def L():
    return Q.lib()


def refused(L, fn, status, **bad):
    args = dict(GOOD[fn])
    assert set(bad) <= set(args)
    args.update(bad)
    assert getattr(L, fn)(*args.values()) == status, (fn, bad, L.qmm_last_error())
    assert L.qmm_last_error().startswith(fn.encode())


def test_null_pointers(L):
    optional = {"wq", "wk", "lse", "st", "work"}
    for fn, args in GOOD.items():
        for name, v in args.items():
            if isinstance(v, ctypes.c_void_p) and name not in optional:
                refused(L, fn, Q.QMM_E_NULL, **{name: None})
        if "c" in args:
            refused(L, fn, Q.QMM_E_NULL, c=None)
            refused(L, fn, Q.QMM_E_NULL, c=cache(k=0))
    refused(L, "qmm_logprobs", Q.QMM_E_NULL, V=200000, ld=200000, work=None)


def test_dtypes(L):
    for fn in GOOD:
        for dt in (3, -1) if fn == "qmm_logprobs" else (2, 3, -1):
            refused(L, fn, Q.QMM_E_DTYPE, dt=dt)


def test_masks(L):
    for kw in (dict(window=0), dict(window=-5), dict(sinks=-1)):
        refused(L, "qmm_kv8_attention_window", Q.QMM_E_ARG, **kw)
    for fn in ("qmm_kv8_attention_window", "qmm_kv8_attention_tree"):
        for kw in (dict(T=0), dict(T=1 << 25), dict(S=0), dict(S=1 << 16), dict(W=0), dict(Hq=1), dict(Hq=3), dict(ldq=504),
                   dict(T=1 << 24, Hq=512, ldq=512 * 128), dict(c=cache(head_dim=96)), dict(c=cache(page_tokens=8))):
            refused(L, fn, Q.QMM_E_SHAPE, **kw)
        for n in ("q", "out", "table", "lens", "cu", "lse"):
            refused(L, fn, Q.QMM_E_ALIGN, **{n: P2})
        refused(L, fn, Q.QMM_E_ARG, W=4096, T=1, S=1, nb=64, **(dict(window=1 << 40) if "window" in GOOD[fn] else {}))
    refused(L, "qmm_kv8_attention_tree", Q.QMM_E_ALIGN, parent=P2)


def test_window_work(L):
    work = lambda w, s: L.qmm_kv8_attention_window_work(cache(), 1, 4, 1, 4096, w, s)  # noqa: E731
    assert work(1000, 0) == 0                       # few tiles are not cut
    assert work(1 << 40, 0) == work(1 << 17, 5) == L.qmm_kv8_attention_work(cache(), 1, 4, 1, 4096) > 65536
    assert 65536 < work(20000, 0) and work(0, 0) == 0 and work(5, -1) == 0


def test_rotation(L):
    fn = "qmm_qk_norm_rope"
    for kw in (dict(T=0), dict(T=1 << 25), dict(Hq=0), dict(Hk=0), dict(Hq=65536, ldq=1 << 30), dict(D=0), dict(D=4), dict(D=12),
               dict(D=520), dict(rot=0), dict(rot=4), dict(rot=136), dict(rot=60), dict(ldq=504), dict(ldq=516), dict(ldk=248),
               dict(ldqo=504), dict(ldko=260), dict(T=1 << 24, Hq=200, ldq=1 << 20, ldqo=1 << 20)):
        refused(L, fn, Q.QMM_E_SHAPE, **kw)
    for n in ("q", "k", "qo", "ko", "freq", "wq", "wk", "pos"):
        refused(L, fn, Q.QMM_E_ALIGN, **{n: P2})
    for eps in (-1e-6, float("nan")):
        refused(L, fn, Q.QMM_E_ARG, eps=eps)
    for kw in (dict(qo=P, ldqo=520), dict(ko=P4, ldko=264), dict(qo=P4), dict(ko=P), dict(ko=P3)):
        refused(L, fn, Q.QMM_E_ARG, **kw)


def test_logprobs(L):
    fn = "qmm_logprobs"
    for kw in (dict(M=0), dict(M=(1 << 23) + 1), dict(V=0), dict(V=1 << 31, ld=1 << 31), dict(top=-1), dict(top=65), dict(V=3, top=5),
               dict(ld=999)):
        refused(L, fn, Q.QMM_E_SHAPE, **kw)
    for n in ("x", "tokens", "lp", "h", "ids", "tl"):
        refused(L, fn, Q.QMM_E_ALIGN, **{n: P2})
    refused(L, fn, Q.QMM_E_ALIGN, dt=0, x=ctypes.c_void_p(0x100001))
    need = L.qmm_logprobs_work(2, 3, 200000, 5)
    assert need > 65536 and L.qmm_logprobs_work(2, 3, 1000, 5) == 0
    assert L.qmm_logprobs_work(2, 3, 200000, 65) == 0 and L.qmm_logprobs_work(5, 3, 200000, 5) == 0
    refused(L, fn, Q.QMM_E_ARG, V=200000, ld=200000, nb=need - 1)
    refused(L, fn, Q.QMM_E_ALIGN, V=200000, ld=200000, work=P2)


def test_binding_refuses():
    c = Q.Kv8Cache(4, 2, 16, 64, device="cpu")
    tab, lens, cu = cpu(2, 3, dt=torch.int32), cpu(2, dt=torch.int32), cpu(3, dt=torch.int32)
    q, k, pos, f = cpu(5, 4, 64), cpu(5, 2, 64), cpu(5, dt=torch.int32), cpu(32, dt=torch.float32)
    x, t = cpu(3, 50), cpu(3, dt=torch.int32)
    for call in (
        lambda: Q.kv8_attention_window(c, q, tab, lens, cu, 5),                         # not on a GPU
        lambda: Q.kv8_attention_window(c, q, tab, lens[:1], cu, 5),
        lambda: Q.kv8_attention_window(c, cpu(5, 4, 32), tab, lens, cu, 5),
        lambda: Q.kv8_attention_window(c, q, tab, lens, cu, 5, out=cpu(5, 4, 32)),
        lambda: Q.kv8_attention_window(None, q, tab, lens, cu, 5),
        lambda: Q.kv8_attention_tree(c, q, tab, lens, cu, pos),
        lambda: Q.kv8_attention_tree(c, q, tab, lens, cu, pos[:4]),
        lambda: Q.kv8_attention_tree(c, q, tab, lens, cu, pos.long()),
        lambda: Q.kv8_attention_tree(c, q, tab, lens, cu, None),
        lambda: Q.qk_norm_rope(q, k, pos, f),
        lambda: Q.qk_norm_rope(q, k[:4], pos, f),
        lambda: Q.qk_norm_rope(q, k.bfloat16(), pos, f),
        lambda: Q.qk_norm_rope(q, k[:, :, :32], pos, f),
        lambda: Q.qk_norm_rope(q, k, pos.long(), f),
        lambda: Q.qk_norm_rope(q, k, pos[:2], f),
        lambda: Q.qk_norm_rope(q, k, pos, f.double()),
        lambda: Q.qk_norm_rope(q, k, pos, f, q_weight=cpu(32)),
        lambda: Q.qk_norm_rope(q, k, pos, f, k_weight=cpu(64, dt=torch.bfloat16)),
        lambda: Q.qk_norm_rope(q, k, pos, f, out=q),
        lambda: Q.qk_norm_rope(q, k, pos, f, out=(q, q)),
        lambda: Q.qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2), pos, f),
        lambda: Q.logprobs(x, t),
        lambda: Q.logprobs(x, t[:2]),
        lambda: Q.logprobs(x, t.long()),
        lambda: Q.logprobs(x, t, top=51),
        lambda: Q.logprobs(x, t, top=-1),
        lambda: Q.logprobs(x.t(), cpu(50, dt=torch.int32)),
        lambda: Q.logprobs(x[0], t),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: Q.logprobs(x.double(), t), lambda: Q.qk_norm_rope(q.float(), k.float(), pos, f),
                 lambda: Q.kv8_attention_tree(c, q.float(), tab, lens, cu, pos)):
        with pytest.raises(Q.QmmError):
            call()
    with pytest.raises(TypeError):
        Q.kv8_attention_window(c, q, tab, lens, cu, "wide")
