"""The operators of a serving step together, as a speculating decoder with a sliding
window layer uses them: int8 projection, norm and rotation, append, attention of a tree
and under a window, output projection, head, log probabilities; against the same
computed in 64 bits from the values that the 8-bit codes stand for."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests import serving_ref as R
from tests import step_ref as S
from tests.test_gpu_kv8 import i32, tables

pytestmark = pytest.mark.gpu

HIDDEN, HQ, HK, D, B, V = 256, 8, 2, 64, 16, 1000


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def f64(t):
    return t.double().cpu().numpy()


def weight(g, n, k):
    w = (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).cuda()
    return Q.i8_quantize(w)


def linear(x, w):
    """The int8 product's definition: (values, their codes' product in 64 bits)."""
    codes, sx = R.i8_quantize(x.float().cpu().numpy())
    y, _ = R.i8_t(codes, sx, w[0].cpu().numpy(), w[1].cpu().numpy())
    return y


def near(got, want, what, steps=2):
    """Each stage against its definition on the stage's own inputs: its result's
    rounding (half a step) and, for the fp32 arithmetic before it, as much again."""
    got = f64(got)
    tol = steps * 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * np.abs(want).max(axis=-1, keepdims=True)
    assert (np.abs(got - want) <= tol).all(), f"{what}: off by up to {(np.abs(got - want) / tol).max()} tolerances"


@pytest.mark.parametrize("window", [None, 24])
def test_a_step_of_drafts(window):
    """Prompts, then a step whose new tokens are trees of drafts (or, under a window, a
    chunk of tokens), verified by their log probabilities."""
    g = torch.Generator().manual_seed(5)
    qkv, out, head = weight(g, (HQ + 2 * HK) * D, HIDDEN), weight(g, HIDDEN, HQ * D), weight(g, V, HIDDEN)
    wq, wk = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) for _ in range(2)]
    freq = torch.tensor(10000.0 ** (-np.arange(0, D, 2) / D), dtype=torch.float32)
    cache, held = Q.Kv8Cache(40, HK, B, D), None
    ref = R.Cache(*[t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)])
    scale = D ** -0.5
    lens = [0, 0, 0]
    for new, parent in (([70, 33, 1], None), ([7, 1, 20], [-1, 0, 0, 1, 1, 2, 3] + [-1] + [-1] + [i // 2 for i in range(19)])):
        lens = [a + n for a, n in zip(lens, new)]
        cu = [0] + [int(c) for c in np.cumsum(new)]
        T = cu[-1]
        tab = tables([120, 64, 64], B, 40, 6) if held is None else held
        held = tab
        x = torch.randn(T, HIDDEN, generator=g).to(torch.bfloat16).cuda()
        # a draft's position is its depth, whatever its place in the cache
        if parent is None or window:
            pos = [l - n + i for l, n in zip(lens, new) for i in range(n)]
        else:
            pos = []
            for s, n in enumerate(new):
                depth = []
                for i in range(n):
                    p = parent[cu[s] + i]
                    depth.append(0 if p < 0 else depth[p] + 1)
                pos += [lens[s] - n + d for d in depth]
        args = i32(tab), i32(lens), i32(cu)
        t = Q.i8_linear(x, *qkv).view(T, HQ + 2 * HK, D)
        near(t.view(T, -1), linear(x, qkv), "projection")
        q, k, v = t[:, :HQ], t[:, HQ:HQ + HK], t[:, HQ + HK:]
        raw = t.clone()
        q, k = Q.qk_norm_rope(q, k, i32(pos), freq.cuda(), wq.cuda(), wk.cuda(), out=(q, k))
        p64, f = np.array(pos), f64(freq)
        near(q, S.rotate(f64(raw[:, :HQ]), p64, f, f64(wq), 1e-6)[0], "queries")
        near(k, S.rotate(f64(raw[:, HQ:HQ + HK]), p64, f, f64(wk), 1e-6)[0], "keys")
        assert torch.equal(t[:, HQ + HK:], raw[:, HQ + HK:])
        Q.kv8_append(cache, k, v, *args)
        ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), tab, lens, cu)
        assert np.array_equal(cache.k.cpu().numpy(), ref.k) and np.array_equal(cache.v.cpu().numpy(), ref.v)
        if window:
            a = Q.kv8_attention_window(cache, q, *args, window, 4)
            sees = S.window_sees(lens, cu, window, 4)
        elif parent is None:
            a = Q.kv8_attention(cache, q, *args)
            sees = S.window_sees(lens, cu, 10 ** 9, 0)
        else:
            a = Q.kv8_attention_tree(cache, q, *args, i32(parent))
            sees = S.tree_sees(lens, cu, parent)
        near(a, S.Masked.of(ref, sees).attention(f64(q), tab, lens, cu, scale)[0], "attention", 4)
        y = Q.i8_linear(a.view(T, HQ * D), *out)
        logits = Q.i8_linear(y, *head)
        tokens = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
        lp, h, ids, top = Q.logprobs(logits, tokens.cuda(), top=8)
        want = S.logprobs(f64(logits), tokens.numpy(), 8)
        assert np.array_equal(ids.cpu().numpy(), want[2])
        for got, w in ((lp, want[0]), (h, want[1]), (top, want[3])):
            assert (np.abs(f64(got) - w) <= 2.0 ** -14 * (1 + np.abs(w))).all()


def test_a_step_is_captured_and_replayed():
    """The whole step as one graph; its inputs change between the replays and every
    replay gives what the eager calls give on a cache of the same state."""
    g = torch.Generator().manual_seed(6)
    qkv, out, head = weight(g, (HQ + 2 * HK) * D, HIDDEN), weight(g, HIDDEN, HQ * D), weight(g, V, HIDDEN)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    freq = torch.tensor(10000.0 ** (-np.arange(0, D, 2) / D), dtype=torch.float32).cuda()
    one, two = Q.Kv8Cache(40, HK, B, D), Q.Kv8Cache(40, HK, B, D)
    tab, cu = i32(tables([300, 200], B, 40, 7)), i32([0, 5, 6])
    x, lens = torch.zeros(6, HIDDEN, dtype=torch.bfloat16, device="cuda"), i32([5, 1])
    pos, parent, tokens = i32([0] * 6), i32([-1, 0, 0, 1, 2, -1]), i32([1, 2, 3, 4, 5, 6])

    def step(cache):
        t = Q.i8_linear(x, *qkv).view(6, HQ + 2 * HK, D)
        q, k = Q.qk_norm_rope(t[:, :HQ], t[:, HQ:HQ + HK], pos, freq, w, w)
        Q.kv8_append(cache, k, t[:, HQ + HK:], tab, lens, cu)
        a = Q.kv8_attention_tree(cache, q, tab, lens, cu, parent)
        b = Q.kv8_attention_window(cache, q, tab, lens, cu, 50, 4)
        y = Q.i8_linear((a + b).view(6, HQ * D), *out)
        return (a, b, *Q.logprobs(Q.i8_linear(y, *head), tokens, top=5))

    step(two)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(one)
    for i in range(4):
        x.copy_(torch.randn(6, HIDDEN, generator=g))
        lens.copy_(i32([20 + 60 * i, 3 + 40 * i]))
        pos.copy_(i32([20 + 60 * i + d for d in (-5, -4, -4, -3, -3, 0)]))
        tokens.add_(1)
        want = step(two)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i
        assert torch.equal(one.k, two.k) and torch.equal(one.v, two.v)
