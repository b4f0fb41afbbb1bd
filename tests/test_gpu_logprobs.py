"""Log probabilities, entropy and top tokens against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests import step_ref as S

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def check(x, tokens, top, got, what):
    """Numbers and ties exactly. Sums: each term carries its exponent's roundings
    (twice 2^-24 |y|, and 2^-25 |y| of log2 e's) and the exponential's (2^-23); a lane adds
    fewer than V / 256 + 8 terms of at least four at a time, and its sums are scaled at
    most once per load (2^-22 each); joining adds 12 + 64 such steps. So with u =
    (V / 256 + 100) 2^-22 and A = 1 + sum p |x - max|: log2 S is off by u A, the entropy
    by 2 u A; a probability's own exponent by 2^-23 of it."""
    lp, h, ids, tl, mag = S.logprobs(x.double().cpu().numpy(), tokens.cpu().numpy(), top)
    g = [t.cpu().numpy().astype(np.float64) for t in got]
    assert np.array_equal(g[2].astype(int), ids), f"{what}: ids"
    u = (x.shape[1] / 256 + 100) * 2.0 ** -22 * (1 + mag)
    for name, a, b, tol in (("logprob", g[0], lp, u), ("entropy", g[1], h, 2 * u), ("top", g[3], tl, u[:, None])):
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isneginf(a), np.isneginf(b)), f"{what}: {name}"
        fin = np.isfinite(b)
        tol = tol + 2.0 ** -22 * np.abs(np.where(fin, b, 0))
        off = np.abs(np.where(fin, a, 0) - np.where(fin, b, 0))
        assert (off <= tol).all(), f"{what}: {name} off by {(off / tol).max()} tolerances"


def rows(M, V, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(M, V, generator=g)).to(DT[dt]).cuda()


def toks(M, V, seed=0):
    return torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 5), (2, 64), (5, 100), (4, 1000), (1, 2048), (3, 2049), (2, 8191), (1, 20000),
                                 (9, 4097), (300, 999), (1, 131071), (2, 70001), (1100, 257)])
def test_rows(M, V, dt):
    x, t = rows(M, V, dt, M + V), toks(M, V)
    for top in sorted({0, 1, min(5, V), min(20, V), min(64, V)}):
        check(x, t, top, Q.logprobs(x, t, top=top), f"{M}x{V} {dt} top {top}")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,V", [(2048, 300), (2100, 3001), (40, 20001), (130, 9000)])
def test_many_rows(M, V, dt):
    """Rows that fill the chip, a workgroup each, and rows in a few parts."""
    x, t = rows(M, V, dt, M + V), toks(M, V)
    x[5, V // 2:] = x[6] = -torch.inf
    x[7, 3] = float("nan")
    x[8] = 1.0
    for top in (0, 5, 64):
        check(x, t, top, Q.logprobs(x, t, top=top), f"{M}x{V} {dt} top {top}")


def test_two_streams_at_once():
    """Calls on two streams, each with parts in scratch memory of its own."""
    side = torch.cuda.Stream()
    xs, ts = [rows(3, 60000, "bf16", s) for s in (1, 2)], [toks(3, 60000, s) for s in (1, 2)]
    want = [Q.logprobs(x, t, top=20) for x, t in zip(xs, ts)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate((None, side)):
            got[i].append(Q.logprobs(xs[i], ts[i], top=20, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_rows_in_awkward_orders(V, dt):
    """Rising, falling and equal logits; most equal; two values; masked tails, heads and
    all but one; nothing allowed; zeros of both signs."""
    up = torch.linspace(-20, 20, V)
    equal, few = torch.zeros(V), torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).float()
    tail, head, one, none = up.clone(), up.clone(), torch.full((V,), -torch.inf), torch.full((V,), -torch.inf)
    tail[V // 3:] = head[:V - 7] = -torch.inf
    one[V // 2] = 3.5
    signs = torch.where(torch.arange(V) % 3 == 0, -0.0, 0.0)
    peak = torch.full((V,), -1e4)
    peak[V - 1] = 1e4
    low = torch.full((V,), float(torch.finfo(DT[dt]).min))
    x = torch.stack([up, up.flip(0), equal, few, -few, tail, head, one, none, signs, peak, low]).to(DT[dt]).cuda()
    t = toks(len(x), V, 3)
    t[7] = V // 2
    for top in (1, 20, 64):
        check(x, t, top, Q.logprobs(x, t, top=top), f"V{V} {dt} top {top}")


@pytest.mark.parametrize("V", [70, 40000])
def test_tokens_outside_and_rows_that_are_no_logits(V):
    x = rows(6, V, "f32", 5)
    x[1, V // 2] = float("nan")
    x[2, V - 1] = float("inf")
    x[3, 0] = -float("nan")
    t = torch.tensor([-1, 3, 3, 3, V, 2 ** 31 - 1], dtype=torch.int32).cuda()
    check(x, t, 9, Q.logprobs(x, t, top=9), f"V{V}")


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("V,ld", [(1001, 1003), (9000, 9001), (50001, 50001), (50001, 60000)])
def test_strides_and_alignment(V, ld, dt):
    """Rows that start anywhere, the first one too; what lies between them is not read
    as theirs."""
    M = 7
    for at in (0, 1, 5):
        line = torch.full((at + M * ld + 8,), float("nan"), dtype=DT[dt], device="cuda")
        x = line.as_strided((M, V), (ld, 1), at)
        x.copy_(rows(M, V, dt, 7 + at))
        t = toks(M, V, at)
        check(x, t, 12, Q.logprobs(x, t, top=12), f"V{V} ld{ld} at {at} {dt}")


def test_ties_across_parts_and_wavefronts():
    """Equal largest values far apart: the lowest numbers win, in order."""
    V = 131000
    x = torch.zeros(1, V, dtype=torch.bfloat16)
    at = [130999, 65536, 3, 70000, 2, 99999, 12345, 8192, 8191, 40000]
    x[0, at] = 5.0
    t = torch.tensor([3], dtype=torch.int32).cuda()
    ids = Q.logprobs(x.cuda(), t, top=14)[2][0].cpu().tolist()
    assert ids == sorted(at) + [0, 1, 4, 5]


def test_the_same_bits_every_time_and_on_another_stream():
    x, t = rows(2, 100000, "bf16", 8), toks(2, 100000)
    want = Q.logprobs(x, t, top=20)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for s in (None, st, None, st):
        got = Q.logprobs(x, t, top=20, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_replays():
    x, t = rows(3, 33000, "f16", 9), toks(3, 33000)
    assert Q.lib().qmm_logprobs_work(0, 3, 33000, 20) > 0   # parts that are joined
    Q.logprobs(x, t, top=20)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = Q.logprobs(x, t, top=20)
    for i in range(4):
        x.copy_(rows(3, 33000, "f16", 20 + i))
        t.copy_(toks(3, 33000, i))
        want = Q.logprobs(x, t, top=20)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        check(x, t, 20, out, f"replay {i}")


def test_offsets_past_32_bits():
    M, V, ld = 3, 3000, (1 << 31) + 16
    line = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    x = line.as_strided((M, V), (ld, 1), 0)
    x.copy_(rows(M, V, "bf16", 11))
    t = toks(M, V)
    assert all(torch.equal(a, b) for a, b in zip(Q.logprobs(x, t, top=7), Q.logprobs(x.contiguous(), t, top=7)))
