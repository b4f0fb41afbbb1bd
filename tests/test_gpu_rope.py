"""Norm and rotation of queries and keys against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from group_wise_affine_amd.devio import TORCH_DT
from tests import serving_ref as R
from tests import step_ref as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def draw(T, H, D, dt, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))).to(TORCH_DT[dt])


def freqs(rot, base=10000.0):
    return torch.tensor(base ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32)


def check(got, x, pos, freq, w, eps, inter, dt, what):
    """Tolerances, relative to the pair's magnitudes |a| + |b|: the sum of D squares
    (D / 2 + 8 roundings of 2^-24 reach the root), the reciprocal root (2^-23), three
    products (3 * 2^-24), the angle (2^-25 of a turn is 2^-22.3; for positions up to
    2^31 the 64-bit product leaves another 2^-21) with the series and its products
    (2^-22): together below D * 2^-24 + 2^-19. Then the rounding of the result."""
    want, mag = S.rotate(x.double().numpy(), pos.numpy(), freq.numpy(),
                         None if w is None else w.double().numpy(), eps, inter)
    got = got.double().cpu().numpy()
    tol = R.UNIT[dt] * np.abs(want) * (1 + 2.0 ** -7) + mag * (x.shape[2] * 2.0 ** -24 + 2.0 ** -19) + R.TINY[dt]
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, by up to {(np.abs(got - want) / tol)[bad].max()} tolerances"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 8, 2, 128, 128), (7, 3, 1, 64, 32), (5, 1, 1, 8, 8), (33, 5, 3, 80, 80),
                                           (4, 6, 2, 96, 24), (3, 2, 2, 256, 256), (3, 3, 1, 192, 64), (2, 2, 1, 512, 504),
                                           (700, 20, 4, 128, 128), (1500, 24, 8, 64, 64), (600, 17, 3, 256, 128)])
def test_norm_and_rotation(T, Hq, Hk, D, rot, inter, dt):
    q, k = draw(T, Hq, D, dt, 1), draw(T, Hk, D, dt, 2)
    wq, wk = draw(1, 1, D, dt, 3)[0, 0], draw(1, 1, D, dt, 4)[0, 0]
    pos = torch.randint(0, 200000, (T,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    f = freqs(rot)
    dev = [t.cuda() for t in (q, k, pos, f)]
    for a, b in ((wq, wk), (None, None), (wq, None), (None, wk)):
        qo, ko = Q.qk_norm_rope(*dev, *[None if w is None else w.cuda() for w in (a, b)], eps=1e-5, interleaved=inter)
        what = f"T{T} {Hq}+{Hk}x{D}/{rot} {dt} interleaved {inter} norm {a is not None}, {b is not None}"
        check(qo, q, pos, f, a, 1e-5, inter, dt, "q " + what)
        check(ko, k, pos, f, b, 1e-5, inter, dt, "k " + what)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(9000, 30, 2, 8, 8), (3000, 8, 1, 64, 64), (2403, 12, 3, 128, 64), (9001, 13, 3, 72, 72),
                                           (4000, 3, 1, 200, 200), (9000, 4, 4, 136, 136), (8000, 1, 1, 512, 512),
                                           (9000, 3, 1, 264, 16)])
def test_many_tokens(T, Hq, Hk, D, rot, inter):
    """Wavefronts that take several of a token's heads, the last ones partly."""
    q, k = draw(T, Hq, D, "bf16", 6), draw(T, Hk, D, "bf16", 7)
    w = draw(1, 1, D, "bf16", 8)[0, 0]
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(9), dtype=torch.int32)
    f = freqs(rot)
    qo, ko = Q.qk_norm_rope(*[t.cuda() for t in (q, k, pos, f)], w.cuda(), None, eps=1e-5, interleaved=inter)
    check(qo, q, pos, f, w, 1e-5, inter, "bf16", f"q T{T} {Hq}+{Hk}x{D}")
    check(ko, k, pos, f, None, 1e-5, inter, "bf16", f"k T{T} {Hq}+{Hk}x{D}")


@pytest.mark.parametrize("inter", [False, True])
def test_far_and_negative_positions(inter):
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24, 12345678, 131071, -131071], dtype=torch.int32)
    q, k = draw(len(pos), 2, 64, "f16", 10), draw(len(pos), 1, 64, "f16", 11)
    for f in (freqs(64), freqs(64, 1e6), torch.linspace(-3, 3, 32), torch.zeros(32)):
        qo, ko = Q.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), interleaved=inter)
        check(qo, q, pos, f, None, 0, inter, "f16", "q")
        check(ko, k, pos, f, None, 0, inter, "f16", "k")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
def test_rows_of_any_magnitude(dt, eps):
    """Rows whose squares leave the range of 32 bits (bf16), subnormal ones (f16)."""
    sizes = [2.0 ** p for p in ((110, 60, 1, -50, -90, -110, -120) if dt == "bf16" else (11, 5, 0, -8, -14, -18))]
    q = torch.cat([draw(1, 3, 128, "bf16", 20).double().clamp(-16, 16).mul(s).to(TORCH_DT[dt]) for s in sizes])
    k, w = q[:, :1].contiguous(), torch.ones(128, dtype=TORCH_DT[dt])
    pos, f = torch.arange(len(sizes), dtype=torch.int32), freqs(128)
    qo, ko = Q.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), w.cuda(), w.cuda(), eps=eps)
    check(qo, q, pos, f, w, eps, False, dt, f"q eps {eps}")
    check(ko, k, pos, f, w, eps, False, dt, f"k eps {eps}")


def test_zero_infinite_and_nan_rows():
    q = draw(4, 2, 64, "bf16", 30)
    q[0, 0] = 0
    q[1, 1, 5] = float("inf")
    q[2, 0, 9] = float("nan")
    w = torch.ones(64, dtype=torch.bfloat16)
    pos, f = torch.zeros(4, dtype=torch.int32), freqs(64)
    qo, _ = Q.qk_norm_rope(q.cuda(), q.cuda(), pos.cuda(), f.cuda(), w.cuda(), w.cuda())
    qo = qo.cpu()
    assert bool((qo[0, 0] == 0).all()) and bool(torch.isnan(qo[2, 0]).all())
    assert bool(torch.isnan(qo[1, 1, 5])) and bool((qo[1, 1, :5] == 0).all())   # x / inf and inf / inf
    keep = torch.ones(4, 2, dtype=torch.bool)
    keep[0, 0] = keep[1, 1] = keep[2, 0] = False
    assert bool(torch.isfinite(qo[keep]).all())


@pytest.mark.parametrize("T", [1, 6, 900])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place_slices_and_other_stream(T, inter):
    """q and k as slices of one projection: into new tensors, into slices of another
    tensor, and in place, where nothing but the two slices changes."""
    H, K, D = 12, 4, 128
    qkv = draw(T, H + 2 * K, D, "bf16", 40).cuda()
    q, k = qkv[:, :H], qkv[:, H:H + K]
    pos, f = torch.arange(T, dtype=torch.int32, device="cuda"), freqs(D).cuda()
    w = draw(1, 1, D, "bf16", 41)[0, 0].cuda()
    want = Q.qk_norm_rope(q.contiguous(), k.contiguous(), pos, f, w, w, interleaved=inter)
    got = Q.qk_norm_rope(q, k, pos, f, w, w, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    both = torch.full((T, H + K + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = Q.qk_norm_rope(q, k, pos, f, w, w, interleaved=inter, out=(both[:, :H], both[:, H:H + K]), stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(both[:, :H], want[0]) and torch.equal(both[:, H:H + K], want[1]) and bool((both[:, -1] == 7).all())
    assert got[0].data_ptr() == both.data_ptr()
    keep = qkv[:, H + K:].clone()
    Q.qk_norm_rope(q, k, pos, f, w, w, interleaved=inter, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, H + K:], keep)


def test_offsets_past_32_bits():
    """Tokens whose rows start past 2^32 bytes."""
    H, D, T, ld = 2, 64, 5, (1 << 30) + 8
    line = torch.empty(4 * ld + 4 * D, dtype=torch.bfloat16, device="cuda")
    take = lambda at: line.as_strided((T, H, D), (ld, D, 1), at)  # noqa: E731
    q, k = take(0), take(H * D)
    q.copy_(draw(T, H, D, "bf16", 50))
    k.copy_(draw(T, H, D, "bf16", 51))
    pos, f = torch.arange(T, dtype=torch.int32, device="cuda"), freqs(D).cuda()
    want = Q.qk_norm_rope(q.contiguous(), k.contiguous(), pos, f)
    got = Q.qk_norm_rope(q, k, pos, f, out=(q, k))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_replays():
    q, k = draw(3, 8, 128, "f16", 60).cuda(), draw(3, 2, 128, "f16", 61).cuda()
    pos, f, w = torch.arange(3, dtype=torch.int32, device="cuda"), freqs(128).cuda(), draw(1, 1, 128, "f16", 62)[0, 0].cuda()
    Q.qk_norm_rope(q, k, pos, f, w, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = Q.qk_norm_rope(q, k, pos, f, w, w)
    for i in range(3):
        q.copy_(draw(3, 8, 128, "f16", 70 + i))
        pos.add_(1000)
        want = Q.qk_norm_rope(q, k, pos, f, w, w)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
