"""The paged 8-bit cache on the GPU: append, read, copy and attention against
the definition (serving_ref)."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from group_wise_affine_amd.devio import TORCH_DT
from tests import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(P, H, B, D, seed):
    """A cache with codes and scales of every size in it, on both sides."""
    r = np.random.default_rng(seed)
    k = np.clip(np.rint(40 * r.standard_normal((P, H, B, D))), -127, 127).astype(np.int8)
    v = np.clip(np.rint(40 * r.standard_normal((P, H, D, B))), -127, 127).astype(np.int8)
    ks, vs = [(0.02 * np.exp(0.5 * r.standard_normal((P, H)))).astype(np.float32) for _ in range(2)]
    dev = Q.Kv8Cache.of(*[torch.from_numpy(a.copy()).cuda() for a in (k, v, ks, vs)])
    return dev, R.Cache(k, v, ks, vs)


def tables(lens, B, P, seed, W=None):
    r = np.random.default_rng(seed)
    held = [-(-n // B) for n in lens]
    order = list(r.permutation(P))
    assert sum(held) <= P
    W = W or max(held + [1])
    out = []
    for n in held:
        out.append([int(order.pop()) for _ in range(n)] + [-1] * (W - n))
    return out


def same_cache(dev, ref):
    assert np.array_equal(dev.k_scales.cpu().numpy(), ref.ks, equal_nan=True)
    assert np.array_equal(dev.v_scales.cpu().numpy(), ref.vs, equal_nan=True)
    assert np.array_equal(dev.k.cpu().numpy(), ref.k)
    assert np.array_equal(dev.v.cpu().numpy(), ref.v)


def fresh(T, H, D, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g))).to(TORCH_DT[dt])


# lens after the call and new tokens per sequence
BATCHES = [([1], [1]), ([5, 33, 0, 70], [5, 1, 0, 3]), ([16, 17, 32, 64, 65], [1, 1, 1, 1, 1]),
           ([130, 1, 64, 200], [130, 1, 64, 71]), ([48, 100], [33, 37])]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,H", [(16, 128, 2), (32, 64, 3), (64, 128, 1), (16, 256, 1), (64, 256, 2)])
@pytest.mark.parametrize("lens,new", BATCHES)
def test_append(lens, new, B, D, H, dt):
    dev, ref = make(40, H, B, D, 1)
    tab = tables(lens, B, 40, 2)
    cu = [0] + list(np.cumsum(new))
    k, v = fresh(cu[-1], H, D, dt, 3), fresh(cu[-1], H, D, dt, 4)
    Q.kv8_append(dev, k.cuda(), v.cuda(), i32(tab), i32(lens), i32(cu))
    ref.append(k.float().numpy(), v.float().numpy(), tab, lens, [int(c) for c in cu])
    same_cache(dev, ref)
    before = [t.clone() for t in (dev.k, dev.v, dev.k_scales, dev.v_scales)]
    Q.kv8_append(dev, k.cuda(), v.cuda(), i32(tab), i32(lens), i32(cu))   # again: nothing changes
    assert all(torch.equal(a, b) for a, b in zip(before, (dev.k, dev.v, dev.k_scales, dev.v_scales)))


def test_append_token_by_token_and_non_finite():
    """A page filled one token at a time, its scale rising and falling; an
    infinity makes the rest of its page and head NaN, and no other."""
    B, D, H = 16, 64, 2
    dev, ref = make(6, H, B, D, 5)
    tab = [[4, 1, 3]]
    for t in range(35):
        k, v = fresh(1, H, D, "f16", 100 + t), fresh(1, H, D, "f16", 200 + t)
        k *= (t * 7 % 5) + 0.25
        if t == 20:
            v[0, 1, 3] = float("inf")
        if t == 7:
            k[:] = 0
        Q.kv8_append(dev, k.cuda(), v.cuda(), i32(tab), i32([t + 1]), i32([0, 1]))
        ref.append(k.float().numpy(), v.float().numpy(), tab, [t + 1], [0, 1])
    same_cache(dev, ref)
    assert np.isnan(ref.vs[1, 1]) and np.isfinite(ref.vs[1, 0]) and np.isfinite(ref.vs[3, 1])


def test_append_slices_and_places_outside_the_cache():
    """k and v as slices of a fused projection; page numbers outside the cache
    get nothing, nor does a table that is too short."""
    B, D, H = 16, 64, 2
    dev, ref = make(8, H, B, D, 6)
    kv = fresh(40, 2 * H, D, "bf16", 7).cuda()
    k, v = kv[:, :H], kv[:, H:]
    tab = [[2, 99, 5]]
    Q.kv8_append(dev, k, v, i32(tab), i32([40]), i32([0, 40]))
    ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), tab, [40], [0, 40])
    same_cache(dev, ref)
    Q.kv8_append(dev, k, v, i32([[-1, -7, 8]]), i32([40]), i32([0, 40]))
    same_cache(dev, ref)
    Q.kv8_append(dev, k, v, i32([[2]]), i32([16]), i32([0, 40]))   # 16 places: the last 16 tokens
    ref.append(k[24:].float().cpu().numpy(), v[24:].float().cpu().numpy(), [[2]], [16], [0, 16])
    same_cache(dev, ref)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,H", [(16, 64, 2), (32, 128, 3), (64, 256, 1)])
def test_read(B, D, H, dt):
    dev, ref = make(9, H, B, D, 8)
    ref.ks[3, 0] = np.nan
    dev.k_scales[3, 0] = float("nan")
    pages = [3, 0, 8, 3, -1, 9]
    k, v = Q.kv8_read(dev, i32(pages), dtype=TORCH_DT[dt])
    for i, p in enumerate(pages):
        for h in range(H):
            a = ref.k[p, h].astype(np.float32) * ref.ks[p, h] if 0 <= p < 9 else np.zeros((B, D), np.float32)
            b = ref.v[p, h].T.astype(np.float32) * ref.vs[p, h] if 0 <= p < 9 else np.zeros((B, D), np.float32)
            assert torch.equal(k[i, h].cpu().nan_to_num(7.0), torch.from_numpy(a).to(TORCH_DT[dt]).nan_to_num(7.0))
            assert torch.equal(v[i, h].cpu(), torch.from_numpy(b.copy()).to(TORCH_DT[dt]))


def test_copy_between_and_within():
    a, ra = make(7, 3, 32, 128, 9)
    b, rb = make(11, 3, 32, 128, 10)
    Q.kv8_copy(b, i32([10, 0, 4, 11, 2]), a, i32([1, 6, 1, 2, -1]))
    for d, s in ((10, 1), (0, 6), (4, 1)):
        rb.k[d], rb.v[d], rb.ks[d], rb.vs[d] = ra.k[s], ra.v[s], ra.ks[s], ra.vs[s]
    same_cache(b, rb)
    Q.kv8_copy(a, i32([5]), a, i32([2]))
    ra.k[5], ra.v[5], ra.ks[5], ra.vs[5] = ra.k[2], ra.v[2], ra.ks[2], ra.vs[2]
    same_cache(a, ra)


def check_attention(got, lse, ref, q, tab, lens, cu, scale, dt, what):
    """Tolerances. Scores: fp32 sums of exact products, at most 2 D additions of
    terms whose magnitudes add up to smag, two more roundings and the
    exponential's argument (2^-24 each, in units of the largest score): e.
    Weights: exp(e) - 1, the f16 rounding (2^-11), the fp32 sums; then the
    element type's own rounding. Weights below 2^-14 of the largest round to
    2^-25 of it."""
    T, Hq, D = q.shape
    want, wlse, mag, smag = ref.attention(q.float().numpy(), tab, lens, cu, scale)
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    e = (2 * D + 8) * 2.0 ** -24 * smag
    assert np.array_equal(np.isneginf(wlse), np.isneginf(lse)), what
    fin = np.isfinite(wlse)
    n = max(lens)
    ltol = e + 2.0 ** -22 * (1 + np.abs(np.where(fin, wlse, 0))) + n * 2.0 ** -24
    assert (np.abs(np.where(fin, lse - np.where(fin, wlse, 0), 0)) <= ltol).all(), what
    top = 127 * np.nanmax(ref.vs)
    tol = (R.UNIT[dt] * np.abs(want) + (2.0 ** -11 + 2 * e + (n + 64) * 2.0 ** -24)[..., None] * mag
           + n * 2.0 ** -25 * top + R.TINY[dt]) * (1 + 2.0 ** -7)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, by up to {(np.abs(got - want) / tol).max()} tolerances"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,H,G", [(16, 128, 2, 4), (32, 64, 1, 3), (64, 128, 2, 1), (16, 256, 1, 5), (64, 64, 1, 16),
                                     (32, 128, 1, 20)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([0, 77, 64, 5, 1], [1, 1, 1, 1, 1]), ([600], [1]), ([40, 200], [3, 9]),
                                      ([130, 33, 500], [130, 1, 70])])
def test_attention(lens, new, B, D, H, G, dt):
    dev, ref = make(60, H, B, D, sum(lens))
    tab = tables(lens, B, 60, 2)
    cu = [0] + [int(c) for c in np.cumsum(new)]
    q = fresh(cu[-1], H * G, D, dt, 3)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True)
    check_attention(out, lse, ref, q, tab, lens, cu, D ** -0.5, dt, f"{lens} {new} B{B} D{D} H{H} G{G} {dt}")


@pytest.mark.parametrize("B", [16, 64])
def test_attention_long_context_is_split(B):
    """One sequence whose tiles go to many workgroups, a ragged end, and a table
    wider than the sequence."""
    n, D = 5003, 128
    dev, ref = make(-(-n // B) + 3, 1, B, D, 11)
    tab = tables([n], B, dev.pages, 12, W=-(-n // B) + 900)
    q = fresh(1, 8, D, "bf16", 13)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32([n]), i32([0, 1]), return_lse=True)
    check_attention(out, lse, ref, q, tab, [n], [0, 1], D ** -0.5, "bf16", f"split B{B}")
    for _ in range(3):   # the same bits every time
        again, l2 = Q.kv8_attention(dev, q.cuda(), i32(tab), i32([n]), i32([0, 1]), return_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new", [([2500, 100, 0, 1700], [1, 1, 1, 1]), ([3000], [40]), ([2300, 5, 2100], [33, 1, 2]),
                                      ([2100] + [9] * 70, [60] + [1] * 70)])
def test_attention_parts_are_joined(lens, new, dt):
    """Ragged batches whose longer sequences are cut into parts, for the kernels
    of both few and many query rows; more sequences than one look finds."""
    B, D, H, G = 32, 128, 1, 4
    dev, ref = make(230, H, B, D, sum(lens))
    tab = tables(lens, B, 230, 2)
    cu = [0] + [int(c) for c in np.cumsum(new)]
    q = fresh(cu[-1], H * G, D, dt, 3)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True)
    check_attention(out, lse, ref, q, tab, lens, cu, D ** -0.5, dt, f"parts {lens[:4]} {dt}")


@pytest.mark.parametrize("new", [5, 40])
def test_attention_more_new_tokens_than_tokens(new):
    """Lengths that do not hold the new tokens: the rows without a position see
    nothing, the others what is there."""
    dev, ref = make(12, 1, 16, 64, 43)
    lens, news = [3, 20], [new, 1]
    tab, cu = tables(lens, 16, 12, 44), [0, new, new + 1]
    q = fresh(new + 1, 4, 64, "f16", 45)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True)
    check_attention(out, lse, ref, q, tab, lens, cu, 64 ** -0.5, "f16", f"{news}")
    assert int(out[: new - 3].abs().max()) == 0 and bool(torch.isneginf(lse[: new - 3]).all())


def test_attention_negative_scale():
    dev, ref = make(30, 1, 16, 64, 40)
    lens, new = [130, 60], [30, 1]
    tab, cu = tables(lens, 16, 30, 41), [0, 30, 31]
    q = fresh(31, 4, 64, "bf16", 42)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True, scale=-0.2)
    check_attention(out, lse, ref, q, tab, lens, cu, -0.2, "bf16", "negative scale")


@pytest.mark.parametrize("new", [1, 40])
def test_attention_masked_places_may_hold_anything(new):
    """Places behind a sequence's end, pages that later rows alone see and
    missing pages: NaN scales there change nothing that does not see them."""
    B, D = 16, 128
    lens = [70]
    dev, ref = make(12, 1, B, D, 14)
    tab = tables(lens, B, 12, 15, W=8)
    q = fresh(new, 4, D, "f16", 16)
    args = (i32(lens), i32([0, new]))
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), *args, return_lse=True)
    spare = [p for p in range(12) if p not in tab[0][:5]]
    dev.k_scales[spare], dev.v_scales[spare] = float("nan"), float("inf")
    wide = [tab[0][:5] + spare[:3]]   # stale numbers behind the sequence's pages
    got, l2 = Q.kv8_attention(dev, q.cuda(), i32(wide), *args, return_lse=True)
    assert torch.equal(out, got) and torch.equal(lse, l2)
    last = tab[0][4]                  # tokens 64 .. 69
    dev.k_scales[last] = float("nan")
    got = Q.kv8_attention(dev, q.cuda(), i32(wide), *args)
    seen = 70 - new + torch.arange(new) >= 64
    assert torch.isnan(got[seen.cuda()]).all()
    assert torch.equal(got[~seen.cuda()], out[~seen.cuda()])
    hole = [[tab[0][0], -1, 99] + tab[0][3:]]   # missing pages are not seen
    dev, ref = make(12, 1, B, D, 14)
    got, l2 = Q.kv8_attention(dev, q.cuda(), i32(hole), *args, return_lse=True)
    check_attention(got, l2, ref, q, hole, lens, [0, new], D ** -0.5, "f16", "holes")


def test_attention_value_scales_far_apart():
    """Value scales over twelve orders of magnitude, zero among them, and large
    scores: the running maximum moves and so does the values' reference."""
    B, D = 16, 64
    dev, ref = make(30, 1, B, D, 17)
    for c, s in ((dev, torch.tensor), (ref, np.float32)):
        for p in range(30):
            x = [1e-6, 3.0, 0.0, 1e6, 1e-2][p % 5]
            (c.v_scales if c is dev else c.vs)[p, 0] = x
    lens = [470]
    tab = tables(lens, B, 30, 18)
    q = fresh(2, 4, D, "bf16", 19) * 4
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32([0, 2]), return_lse=True, scale=0.5)
    check_attention(out, lse, ref, q, tab, lens, [0, 2], 0.5, "bf16", "far apart")


def test_attention_strided_queries_and_other_stream():
    B, D, H, G = 32, 128, 2, 4
    dev, ref = make(20, H, B, D, 20)
    lens, new = [150, 40, 300], [1, 1, 1]
    tab, cu = tables(lens, B, 20, 21), [0, 1, 2, 3]
    fused = fresh(3, H * (G + 2), D, "bf16", 22).cuda()
    q = fused[:, : H * G]
    args = (i32(tab), i32(lens), i32(cu))
    want = Q.kv8_attention(dev, q.contiguous(), *args)
    assert torch.equal(want, Q.kv8_attention(dev, q, *args))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = Q.kv8_attention(dev, q, *args, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(want, out)


def test_attention_graph_replays():
    """A decoding step captured once: lengths and queries change between the
    replays, eager calls run in between."""
    B, D, H, G = 16, 128, 2, 4
    dev, ref = make(200, H, B, D, 23)
    tab = i32(tables([1500, 900], B, 200, 24))
    lens, cu = i32([1200, 7]), i32([0, 1, 2])
    q = fresh(2, H * G, D, "f16", 25).cuda()
    Q.kv8_attention(dev, q, tab, lens, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = Q.kv8_attention(dev, q, tab, lens, cu)
    for i in range(4):
        q.copy_(fresh(2, H * G, D, "f16", 30 + i))
        lens.copy_(i32([1300 + 50 * i, 10 + 200 * i]))
        want = Q.kv8_attention(dev, q, tab, lens, cu)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)


def test_offsets_past_32_bits():
    """Pages whose codes start past 2^32 bytes: append, read, attention, copy."""
    H, B, D = 8, 64, 256
    P = (1 << 32) // (H * B * D) + 600
    dev = Q.Kv8Cache(P, H, B, D)
    far = [P - 1, P - 300, 5, P - 2]
    T = 4 * B - 10
    k, v = fresh(T, H, D, "bf16", 1), fresh(T, H, D, "bf16", 2)
    Q.kv8_append(dev, k.cuda(), v.cuda(), i32([far]), i32([T]), i32([0, T]))
    small = Q.Kv8Cache(4, H, B, D)
    Q.kv8_append(small, k.cuda(), v.cuda(), i32([[0, 1, 2, 3]]), i32([T]), i32([0, T]))
    for a, b in zip(Q.kv8_read(dev, i32(far)), Q.kv8_read(small, i32([0, 1, 2, 3]))):
        assert torch.equal(a, b)
    q = fresh(3, 16, D, "bf16", 3).cuda()
    assert torch.equal(Q.kv8_attention(dev, q, i32([far]), i32([T]), i32([0, 3])),
                       Q.kv8_attention(small, q, i32([[0, 1, 2, 3]]), i32([T]), i32([0, 3])))
    Q.kv8_copy(dev, i32([P - 4]), dev, i32([P - 1]))
    assert torch.equal(dev.k[P - 4], dev.k[P - 1]) and torch.equal(dev.v[P - 4], dev.v[P - 1])


def test_attention_graph_of_two_streams():
    """Parts of a call on a side stream of a capture lie in memory that nothing
    else of the capture gets."""
    B, D, H, G = 16, 128, 2, 4
    dev, ref = make(200, H, B, D, 50)
    tab = i32(tables([1900, 900], B, 200, 51, W=400))
    lens, cu = i32([1850, 7]), i32([0, 1, 2])
    assert Q.lib().qmm_kv8_attention_work(dev._at, 2, H * G, 2, 400) > 0   # cut into parts
    q = fresh(2, H * G, D, "f16", 52).cuda()
    side, out = torch.cuda.Stream(), torch.empty(2, H * G, D, dtype=torch.float16, device="cuda")
    Q.kv8_attention(dev, q, tab, lens, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        for _ in range(3):
            Q.kv8_attention(dev, q, tab, lens, cu, out=out, stream=side)
            other = [torch.empty(1 << n, dtype=torch.uint8, device="cuda").fill_(255) for n in range(16, 25)]
        here.wait_stream(side)
    for i in range(4):
        q.copy_(fresh(2, H * G, D, "f16", 60 + i))
        lens.copy_(i32([1300 + 100 * i, 10 + 200 * i]))
        want = Q.kv8_attention(dev, q, tab, lens, cu)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)
    assert all(int(t.min()) == 255 for t in other)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [124, 118, -118, -126])
def test_attention_queries_of_any_magnitude(power, D, new):
    """bf16 queries near the ends of their range, brought back by the scale: rows
    with the largest finite and with subnormal values among them."""
    B = 16
    dev, ref = make(12, 1, B, D, 70)
    lens, cu = [new + 90], [0, new]
    tab = tables(lens, B, 12, 71)
    q = fresh(new, 2, D, "bf16", 72).float().clamp(-15, 15) * 2.0 ** power
    if power > 0:
        q[0, 0, 3] = 3.38953e38
    q = q.to(torch.bfloat16)
    scale = 2.0 ** (-4 - power)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True, scale=scale)
    check_attention(out, lse, ref, q, tab, lens, cu, scale, "bf16", f"queries of 2^{power}, D {D}, {new} new")


def test_one_token_of_a_wider_tensor():
    B, D, H, G = 16, 64, 2, 4
    a, _ = make(6, H, B, D, 80)
    b, _ = make(6, H, B, D, 80)
    line = fresh(1, 1, 800, "bf16", 81).cuda().view(-1)
    take = lambda n, at: line.as_strided((1, n, D), (n * D + 3, D, 1), at)  # noqa: E731
    k, v, q = take(H, 0), take(H, 128), take(H * G, 256)
    args = (i32([[3, 1]]), i32([20]), i32([0, 1]))
    Q.kv8_append(a, k, v, *args)
    Q.kv8_append(b, k.contiguous(), v.contiguous(), *args)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert torch.equal(Q.kv8_attention(a, q, *args), Q.kv8_attention(b, q.contiguous(), *args))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,G", [(16, 64, 4), (16, 64, 20), (32, 128, 20), (64, 256, 3), (64, 256, 20)])
@pytest.mark.parametrize("n", [2500, 5003])
def test_parts_of_every_head_size(n, B, D, G, dt):
    """Few parts and many (two kernels join them), groups of more heads than a
    workgroup takes, a second sequence that is not cut."""
    lens, cu = [n, 40], [0, 1, 2]
    held = -(-n // B)
    dev, ref = make(held + 8, 1, B, D, n)
    tab = tables(lens, B, held + 8, 2)
    q = fresh(2, G, D, dt, 3)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True)
    check_attention(out, lse, ref, q, tab, lens, cu, D ** -0.5, dt, f"{n} B{B} D{D} G{G} {dt}")


@pytest.mark.parametrize("lens,new,G", [([310], [300], 128),                      # more items than threads
                                        ([70 + i % 7 for i in range(300)], [1] * 299 + [70], 2),   # more sequences
                                        ([5, 90] * 130, [1, 3] * 129 + [1, 80], 2)])
def test_prompts_in_large_batches(lens, new, G):
    """Batches whose work items are not sorted by length."""
    B, D = 16, 64
    P = sum(-(-n // B) for n in lens) + 3
    dev, ref = make(P, 1, B, D, 90)
    tab = tables(lens, B, P, 91)
    cu = [0] + [int(c) for c in np.cumsum(new)]
    q = fresh(cu[-1], G, D, "bf16", 92)
    out, lse = Q.kv8_attention(dev, q.cuda(), i32(tab), i32(lens), i32(cu), return_lse=True)
    check_attention(out, lse, ref, q, tab, lens, cu, D ** -0.5, "bf16", f"{len(lens)} sequences, {cu[-1]} new")


@pytest.mark.parametrize("S", [64, 65, 700, 4096, 4097, 5000])
def test_many_sequences(S):
    """A sequence of an item is found in one, two or three looks at 64 boundaries:
    append and attention, some sequences without a token."""
    B, D, H = 16, 64, 1
    r = np.random.default_rng(S)
    new = [int(x) for x in r.choice([0, 1, 1, 1, 3], S)]
    new[0] = new[S - 1] = 1
    lens = [n + int(x) for n, x in zip(new, r.integers(0, 40, S))]
    P = sum(-(-n // B) for n in lens) + 1
    dev, ref = make(P, H, B, D, S)
    tab = tables(lens, B, P, 93)
    cu = [0] + [int(c) for c in np.cumsum(new)]
    T = cu[-1]
    k, v = fresh(T, H, D, "f16", 94), fresh(T, H, D, "f16", 95)
    args = (i32(tab), i32(lens), i32(cu))
    Q.kv8_append(dev, k.cuda(), v.cuda(), *args)
    ref.append(k.float().numpy(), v.float().numpy(), tab, lens, cu)
    same_cache(dev, ref)
    q = fresh(T, 2, D, "f16", 96)
    out, lse = Q.kv8_attention(dev, q.cuda(), *args, return_lse=True)
    check_attention(out, lse, ref, q, tab, lens, cu, D ** -0.5, "f16", f"{S} sequences")
