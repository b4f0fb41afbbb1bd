"""Page bookkeeping of the 8-bit cache against plain Python (serving_ref): whole
numbers, so equal."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests import serving_ref as R
from tests.test_gpu_kv8 import i32, make, same_cache, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def counts(table, P, pinned=()):
    ref = [0] * P
    for row in table:
        for p in row:
            if 0 <= p < P:
                ref[p] += 1
    for p in pinned:
        ref[p] += 1
    return ref


def run_update(dev, ref_cache, ref, table, lens, parent, new_lens):
    B = dev.page_tokens
    r, t, s = Q.kv8_update(dev, i32(ref), i32(table), i32(lens), i32(parent), i32(new_lens))
    wr, wt, ws, copies = R.update(ref, table, lens, parent, new_lens, B)
    assert s.item() == ws
    assert t.tolist() == wt
    assert r.tolist() == wr
    for a, b in copies:
        for x in (ref_cache.k, ref_cache.v, ref_cache.ks, ref_cache.vs):
            x[b] = x[a]
    same_cache(dev, ref_cache)
    return wr, wt


@pytest.mark.parametrize("case", [
    # lens, parents, new lengths
    ([40, 3, 16], [0, 1, 2], [41, 4, 17]),                 # every sequence grows by a token
    ([40, 3, 16], [0, 0, 0], [41, 41, 40]),                # all continue the first
    ([40, 33, 20], [1, 2, 0], [34, 21, 41]),               # a permutation of beams
    ([40, 33, 20], [-1, 1, -1], [0, 33, 50]),              # one dropped, one kept, one new
    ([64, 33, 20], [0, 0, 2], [20, 50, 0]),                # truncated below what a fork shares
    ([64, 5, 0], [0, 0, 7], [33, 64, 1]),
    ([0, 0], [0, 1], [1, 64]),
    ([17], [0], [3]),
])
def test_update(case):
    lens, parent, new_lens = case
    dev, ref_cache = make(40, 2, 16, 64, 1)
    table = tables(lens, 16, 40, 2, W=5)
    run_update(dev, ref_cache, counts(table, 40), table, lens, parent, new_lens)


def test_update_shared_and_pinned_pages():
    """Rows that share a prefix, a last page held by someone outside the table,
    and numbers that are no pages."""
    dev, ref_cache = make(30, 1, 16, 64, 3)
    table = [[4, 9, 7, -1], [4, 9, 12, -1], [20, 99, 3, -1], [5, -1, -1, -1]]
    lens = [40, 35, 44, 10]
    ref = counts(table, 30, pinned=[5, 29])
    for parent, new in (([0, 1, 2, 3], [41, 36, 45, 11]), ([1, 0, 0, 2], [20, 30, 48, 40]),
                        ([0, 0, 1, 3], [17, 33, 64, 64]), ([2, 9, -5, 3], [44, 5, 5, -3])):
        run_update(dev, ref_cache, ref, table, lens, parent, new)


def test_update_runs_out_of_pages():
    dev, ref_cache = make(8, 1, 16, 64, 4)
    table = [[0, 2, -1, -1], [5, 6, -1, -1]]
    ref = counts(table, 8, pinned=[1, 3])
    run_update(dev, ref_cache, ref, table, [20, 32], [0, 0], [60, 60])


@pytest.mark.parametrize("P,S,seed", [(3000, 60, 0), (20000, 300, 1), (1025, 17, 2), (300000, 40, 3)])
def test_update_many_steps(P, S, seed):
    """A random life of S slots: every step's table and counts are equal, and the
    counts are those of the table."""
    r = np.random.default_rng(seed)
    dev = Q.Kv8Cache(P, 1, 16, 64)
    W = 24
    lens = [int(x) for x in r.integers(0, 16 * W - 40, S)]
    table = tables(lens, 16, P, seed, W=W)
    ref = counts(table, P)
    for _ in range(6):
        u = r.random(S)
        parent = [s if x < 0.5 else -1 if x < 0.6 else int(r.integers(S)) for s, x in enumerate(u)]
        new = [0 if p < 0 and x < 0.5 else max(0, int((lens[p] if p >= 0 else 0) + r.integers(-30, 40)))
               for p, x in zip(parent, r.random(S))]
        new = [min(n, 16 * W) for n in new]
        a, b, c = Q.kv8_update(dev, i32(ref), i32(table), i32(lens), i32(parent), i32(new))
        ref, table, short, _ = R.update(ref, table, lens, parent, new, 16)
        assert c.item() == short and b.tolist() == table and a.tolist() == ref
        assert short == 0 and ref == counts(table, P)
        lens = new


@pytest.mark.parametrize("P,live,seed", [(1, 1, 0), (7, 0, 1), (64, 20, 2), (1024, 1000, 3), (5000, 1, 4), (5000, 2600, 5)])
def test_compact(P, live, seed):
    r = np.random.default_rng(seed)
    dev, ref_cache = make(P, 1, 16, 64, seed)
    used = [int(p) for p in r.permutation(P)[:live]]
    table = [[-1] * 9 for _ in range(5)]
    for i, p in enumerate(used[:40]):
        table[i % 5][i // 5] = p
    if live > 3:
        table[0][8] = used[1]     # a page in two rows
        table[1][8] = P + 3       # no page
    ref = counts(table, P)
    for p in used[40:]:
        ref[p] += int(r.integers(1, 4))
    out = Q.kv8_compact(dev, i32(ref), i32(table))
    wr, wt, wm, n, moves = R.compact(ref, table)
    assert out[3].item() == n
    assert out[0].tolist() == wr and out[1].tolist() == wt and out[2].tolist() == wm
    for a, b in moves:
        for x in (ref_cache.k, ref_cache.v, ref_cache.ks, ref_cache.vs):
            x[b] = x[a]
    same_cache(dev, ref_cache)


def test_a_block_of_steps_together():
    """Prompt, fork, decode, drop, compact: attention over the cache gives the
    same bits wherever the pages lie, and a fork does not disturb its parent."""
    B, D, H, G, P = 16, 64, 2, 2, 64
    dev = Q.Kv8Cache(P, H, B, D)
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    lens = i32([0, 0, 0])
    g = torch.Generator().manual_seed(1)
    new = lambda n: torch.randn(n, 2 * H, D, generator=g).half().cuda()  # noqa: E731

    def step(parent, want, tokens):
        nonlocal ref, table, lens
        want = i32(want)
        ref, table, short = Q.kv8_update(dev, ref, table, lens, i32(parent), want)
        assert short.item() == 0
        lens = want
        cu = i32([0] + list(np.cumsum(tokens)))
        kv = new(sum(tokens))
        Q.kv8_append(dev, kv[:, :H], kv[:, H:], table, lens, cu)
        return cu

    step([-1, -1, -1], [40, 21, 0], [40, 21, 0])
    q = torch.randn(3, H * G, D, generator=g).half().cuda()
    cu = step([0, 1, 0], [41, 22, 41], [1, 1, 1])
    want = Q.kv8_attention(dev, q, table, lens, cu)
    assert not torch.equal(want[0], want[2])
    k0, _ = Q.kv8_read(dev, table[0, :2].contiguous())
    k2, _ = Q.kv8_read(dev, table[2, :2].contiguous())
    assert torch.equal(k0, k2) and table[0, 2] != table[2, 2]
    # drop the middle one, pack, and look again
    ref, table, _ = Q.kv8_update(dev, ref, table, lens, i32([0, -1, 2]), i32([41, 0, 41]))
    ref, table, remap, used = Q.kv8_compact(dev, ref, table)
    n = used.item()
    assert n == 4 and int(table.max()) == n - 1 and bool((ref[:n] > 0).all()) and int(ref[n:].sum()) == 0
    got = Q.kv8_attention(dev, q, table, i32([41, 0, 41]), cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert int(got[1].abs().max()) == 0


def test_a_captured_step():
    """Bookkeeping, append and attention of a step captured together, the pages'
    scratch on a stream of its own: each replay gives what the eager calls give."""
    B, D, H, G, P, S, W = 16, 64, 2, 2, 900, 40, 16
    r = np.random.default_rng(7)
    lens0 = [int(x) for x in r.integers(1, B * W - 8, S)]
    table0 = tables(lens0, B, P, 8, W=W)
    caches = [make(P, H, B, D, 9)[0] for _ in range(2)]
    state = [dict(ref=i32(counts(table0, P)), table=i32(table0), lens=i32(lens0)) for _ in range(2)]
    parent, new, cu = i32(list(range(S))), i32([n + 1 for n in lens0]), i32(list(range(S + 1)))
    kv = torch.zeros(S, 2 * H, D, dtype=torch.float16, device="cuda")
    q = torch.zeros(S, H * G, D, dtype=torch.float16, device="cuda")
    side = torch.cuda.Stream()

    def step(c, s, on=None):
        ref, table, short = Q.kv8_update(c, s["ref"], s["table"], s["lens"], parent, new, stream=on)
        if on is not None:
            torch.cuda.current_stream().wait_stream(on)
        Q.kv8_append(c, kv[:, :H], kv[:, H:], table, new, cu)
        out = Q.kv8_attention(c, q, table, new, cu)
        return ref, table, short, out

    step(caches[1], dict(state[1]))   # (before the capture; the cache is set again below)
    caches[1].k.copy_(caches[0].k), caches[1].v.copy_(caches[0].v)
    caches[1].k_scales.copy_(caches[0].k_scales), caches[1].v_scales.copy_(caches[0].v_scales)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = step(caches[1], state[1], on=side)
    gen = torch.Generator().manual_seed(3)
    lens = lens0
    for i in range(4):
        u = r.random(S)
        par = [s if x < 0.6 else int(r.integers(S)) for s, x in enumerate(u)]
        want_lens = [min(lens[p] + 1, B * W) for p in par]
        parent.copy_(i32(par)), new.copy_(i32(want_lens))
        kv.copy_(torch.randn(S, 2 * H, D, generator=gen).half()), q.copy_(torch.randn(S, H * G, D, generator=gen).half())
        want = step(caches[0], state[0])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert want[2].item() == 0
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        for s, w in zip(state, (want, got)):
            s["ref"].copy_(w[0]), s["table"].copy_(w[1]), s["lens"].copy_(new)
        lens = want_lens
        for a, b in zip((caches[0].k, caches[0].v, caches[0].k_scales, caches[0].v_scales),
                        (caches[1].k, caches[1].v, caches[1].k_scales, caches[1].v_scales)):
            assert torch.equal(a, b)
