"""Attention over the paged 8-bit cache under a sliding window with sinks and for
trees of drafted tokens, against the definition (step_ref)."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests import step_ref as S
from tests.test_gpu_kv8 import check_attention, fresh, i32, make, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def batch(lens, new, B, D, H, G, dt, W=None, spare=5):
    P = sum(-(-n // B) for n in lens) + spare
    dev, ref = make(P, H, B, D, sum(lens))
    cu = [0] + [int(c) for c in np.cumsum(new)]
    return dev, ref, tables(lens, B, P, 2, W), cu, fresh(cu[-1], H * G, D, dt, 3)


def window(dev, ref, tab, lens, cu, q, dt, w, sinks, what, scale=None):
    out, lse = Q.kv8_attention_window(dev, q.cuda(), i32(tab), i32(lens), i32(cu), w, sinks, scale=scale, return_lse=True)
    m = S.Masked.of(ref, S.window_sees(lens, cu, w, sinks))
    check_attention(out, lse, m, q, tab, lens, cu, scale or q.shape[2] ** -0.5, dt, f"window {w}+{sinks} {what}")
    return out, lse


def tree(dev, ref, tab, lens, cu, q, dt, parent, what):
    out, lse = Q.kv8_attention_tree(dev, q.cuda(), i32(tab), i32(lens), i32(cu), i32(parent), return_lse=True)
    m = S.Masked.of(ref, S.tree_sees(lens, cu, parent))
    check_attention(out, lse, m, q, tab, lens, cu, q.shape[2] ** -0.5, dt, f"tree {what}")
    return out, lse


def grown(new, seed, roots=0.1):
    """A random tree (or several) over each sequence's new tokens."""
    r, out = np.random.default_rng(seed), []
    for n in new:
        b = max(0, n - S.TREE)
        out += [i - 1 if i < b else -1 if i == b or r.random() < roots else int(r.integers(max(b, i - 5), i)) for i in range(n)]
    return out


SHAPES = [(16, 128, 2, 4), (32, 64, 1, 3), (64, 128, 1, 1), (16, 256, 1, 5), (64, 64, 1, 16), (32, 128, 1, 20)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,H,G", SHAPES)
@pytest.mark.parametrize("lens,new", [([1], [1]), ([0, 77, 64, 5, 1], [1, 1, 1, 1, 1]), ([600], [1]), ([40, 200], [3, 9]),
                                      ([130, 33, 500], [130, 1, 70])])
def test_window(lens, new, B, D, H, G, dt):
    b = batch(lens, new, B, D, H, G, dt)
    for w, sinks in ((1, 0), (50, 3), (64, 64), (130, 0), (1 << 40, 7)):
        window(*b[:3], lens, b[3], b[4], dt, w, sinks, f"{lens} {new} B{B} D{D} H{H} G{G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("w,sinks", [(1, 1), (100, 0), (300, 4), (1500, 200), (2000, 1 << 40), (777, 65)])
@pytest.mark.parametrize("lens,new", [([5003, 40], [1, 1]), ([2500, 100, 0, 1700], [1, 1, 1, 1]), ([3000], [40]), ([2300, 5, 2100], [33, 1, 2])])
def test_window_over_long_contexts(lens, new, w, sinks, dt):
    """Tiles between the sinks and the window left out, parts of what remains joined."""
    b = batch(lens, new, 32, 128, 1, 4, dt)
    window(*b[:3], lens, b[3], b[4], dt, w, sinks, f"{lens} {new} {dt}")


def test_a_window_that_sees_everything_is_plain_attention():
    """Within the plain definition's bounds (not to the bit: the two calls may take
    other kernels, and other parts of a context)."""
    for lens, new in (([900, 30], [1, 1]), ([400, 90], [150, 20])):
        dev, ref, tab, cu, q = batch(lens, new, 16, 128, 2, 4, "bf16")
        for w, sinks in ((900, 0), (1 << 50, 0), (1, 900)):
            got = Q.kv8_attention_window(dev, q.cuda(), i32(tab), i32(lens), i32(cu), w, sinks, return_lse=True)
            check_attention(*got, ref, q, tab, lens, cu, 128 ** -0.5, "bf16", f"window {w}+{sinks}")


@pytest.mark.parametrize("new", [1, 40])
def test_window_does_not_read_what_it_does_not_see(new):
    """Pages outside the window hold NaN scales or numbers that are no page."""
    lens, B, w, sinks = [1000], 16, 100, 20
    dev, ref, tab, cu, q = batch(lens, [new], B, 128, 1, 4, "f16", spare=0)
    args = (i32(lens), i32(cu), w, sinks)
    want = Q.kv8_attention_window(dev, q.cuda(), i32(tab), *args, return_lse=True)
    first = (1000 - new - w + 1) // B   # column of the first window's first token
    out = [[p if j < 2 or j >= first else [-1, 1 << 30, p][j % 3] for j, p in enumerate(tab[0])]]
    for j in range(2, first):
        dev.k_scales[tab[0][j]] = dev.v_scales[tab[0][j]] = float("nan")
    got = Q.kv8_attention_window(dev, q.cuda(), i32(out), *args, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # pages that are missing inside the window are not seen
    hole = [[-1 if j in (0, len(tab[0]) - 3) else p for j, p in enumerate(tab[0])]]
    window(dev, ref, hole, lens, cu, q, "f16", w, sinks, "holes")


@pytest.mark.parametrize("new", [5, 40])
def test_window_more_new_tokens_than_tokens(new):
    lens, news = [3, 20], [new, 1]
    dev, ref, tab, cu, q = batch(lens, news, 16, 64, 1, 4, "f16")
    out, lse = window(dev, ref, tab, lens, cu, q, "f16", 2, 1, "short")
    assert int(out[: new - 3].abs().max()) == 0 and bool(torch.isneginf(lse[: new - 3]).all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,H,G", SHAPES)
@pytest.mark.parametrize("lens,new", [([1], [1]), ([0, 77, 64, 5, 30], [1, 7, 64, 5, 2]), ([620], [20]), ([90, 300, 33], [64, 65, 1]),
                                      ([200, 400], [200, 90])])
def test_tree(lens, new, B, D, H, G, dt):
    b = batch(lens, new, B, D, H, G, dt)
    tree(*b[:3], lens, b[3], b[4], dt, grown(new, len(new)), f"{lens} {new} B{B} D{D} H{H} G{G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lens,new", [([5003, 40], [7, 1]), ([3000], [40]), ([2300, 5, 2100], [33, 1, 64]), ([4000], [100])])
def test_tree_over_long_contexts(lens, new, dt):
    b = batch(lens, new, 32, 128, 1, 4, dt)
    tree(*b[:3], lens, b[3], b[4], dt, grown(new, 7), f"{lens} {new} {dt}")


@pytest.mark.parametrize("G", [1, 4])
def test_trees_of_every_form(G):
    """A chain, a star, separate roots, parents that are none (later tokens, the token
    itself, before the tree, any number)."""
    n = 64
    lens, new = [n + 70], [n]
    dev, ref, tab, cu, q = batch(lens, new, 16, 64, 1, G, "f16")
    for parent in ([-1] + list(range(n - 1)), [-1] + [0] * (n - 1), [-1] * n, [i // 2 - 1 for i in range(n)],
                   list(range(n)), [i + 1 for i in range(n)], [10 ** 9] * n, [-2 ** 31] * n, [63] * n):
        tree(dev, ref, tab, lens, cu, q, "f16", parent, f"{parent[:5]}")
    lens, new = [170], [90]   # 26 causal tokens, whose numbers are no parents in the tree
    dev, ref, tab, cu, q = batch(lens, new, 16, 64, 1, G, "f16")
    tree(dev, ref, tab, lens, cu, q, "f16", [3] * 90, "before the tree")


def test_a_chain_is_plain_attention():
    """Within the plain definition's bounds (not to the bit: the two calls may take
    other kernels, and other parts of a context)."""
    for lens, new in (([900, 30], [5, 1]), ([400, 90], [150, 20])):
        dev, ref, tab, cu, q = batch(lens, new, 16, 128, 2, 4, "bf16")
        chain = i32([i - 1 for n in new for i in range(n)])
        got = Q.kv8_attention_tree(dev, q.cuda(), i32(tab), i32(lens), i32(cu), chain, return_lse=True)
        check_attention(*got, ref, q, tab, lens, cu, 128 ** -0.5, "bf16", "chain")


def test_a_branch_does_not_depend_on_the_others():
    """What a token gets is what it gets alone with its ancestors: the other drafts'
    pages may hold NaN."""
    B, n = 16, 48
    lens, new = [200 + n], [n]
    dev, ref, tab, cu, q = batch(lens, new, B, 128, 1, 4, "bf16")
    parent = [-1] + list(range(15)) + [15] + list(range(16, 31)) + [15] + list(range(32, 47))   # two branches of 16
    args = (i32(tab), i32(lens), i32(cu), i32(parent))
    want = Q.kv8_attention_tree(dev, q.cuda(), *args)
    # tokens 216 .. 231 (the first branch) lie in pages 13 and 14, the second's from 232 on
    dev.k_scales[tab[0][14]] = dev.v_scales[tab[0][14]] = float("nan")   # positions 224 .. 239
    got = Q.kv8_attention_tree(dev, q.cuda(), *args)
    assert torch.equal(want[:24], got[:24]) and bool(torch.isnan(got[24:40]).all())


@pytest.mark.parametrize("new", [9, 60])
def test_tree_more_new_tokens_than_tokens(new):
    lens, news = [6, 20], [new, 3]
    dev, ref, tab, cu, q = batch(lens, news, 16, 64, 1, 4, "f16")
    tree(dev, ref, tab, lens, cu, q, "f16", grown(news, 9), "short")


@pytest.mark.parametrize("new", [1, 7, 90])
@pytest.mark.parametrize("G", [4, 40])
def test_negative_scale(new, G):
    """Few and many query rows, and groups of more heads than the draft kernel takes."""
    lens, news = [130 + new, 60], [new, 1]
    dev, ref, tab, cu, q = batch(lens, news, 16, 64, 1, G, "bf16")
    parent, args = grown(news, 4), (dev, q.cuda(), i32(tab), i32(lens), i32(cu))
    out, lse = Q.kv8_attention_tree(*args, i32(parent), scale=-0.2, return_lse=True)
    check_attention(out, lse, S.Masked.of(ref, S.tree_sees(lens, cu, parent)), q, tab, lens, cu, -0.2, "bf16", "tree")
    out, lse = Q.kv8_attention_window(*args, 50, 3, scale=-0.2, return_lse=True)
    check_attention(out, lse, S.Masked.of(ref, S.window_sees(lens, cu, 50, 3)), q, tab, lens, cu, -0.2, "bf16", "window")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [118, -118, -126])
def test_tree_queries_of_any_magnitude(power, D):
    """bf16 queries near the ends of their range, brought back by the scale."""
    lens, new = [100], [9]
    dev, ref, tab, cu, q = batch(lens, new, 16, D, 1, 2, "bf16")
    q = q.float().clamp(-15, 15) * 2.0 ** power
    if power > 0:
        q[0, 0, 3] = 3.38953e38
    q, parent, scale = q.to(torch.bfloat16), grown(new, 5), 2.0 ** (-4 - power)
    out, lse = Q.kv8_attention_tree(dev, q.cuda(), i32(tab), i32(lens), i32(cu), i32(parent), scale=scale, return_lse=True)
    check_attention(out, lse, S.Masked.of(ref, S.tree_sees(lens, cu, parent)), q, tab, lens, cu, scale, "bf16", f"2^{power}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("new", [6, 80])
def test_value_scales_far_apart(new, dt):
    """Value scales over twelve orders of magnitude, zero among them, and large scores:
    the references of the weights and of their sum move apart."""
    lens = [470 + new]
    dev, ref, tab, cu, q = batch(lens, [new], 16, 64, 1, 4, dt)
    for p in range(ref.P):
        x = [1e-6, 3.0, 0.0, 1e6 if dt == "bf16" else 30.0, 1e-2][p % 5]
        dev.v_scales[p, 0], ref.vs[p, 0] = x, x
    q, parent = (q.float() * 4).to(q.dtype), grown([new], 6)
    args = (dev, q.cuda(), i32(tab), i32(lens), i32(cu))
    out, lse = Q.kv8_attention_tree(*args, i32(parent), scale=0.5, return_lse=True)
    check_attention(out, lse, S.Masked.of(ref, S.tree_sees(lens, cu, parent)), q, tab, lens, cu, 0.5, dt, "tree")
    out, lse = Q.kv8_attention_window(*args, 200, 40, scale=0.5, return_lse=True)
    check_attention(out, lse, S.Masked.of(ref, S.window_sees(lens, cu, 200, 40)), q, tab, lens, cu, 0.5, dt, "window")


@pytest.mark.parametrize("new", [1, 9, 70])
def test_rows_behind_the_last_sequence_stay(new):
    """Tokens of the batch that no sequence owns, and outputs past a shorter one."""
    lens, news = [300 + new, 40], [new, 1]
    dev, ref, tab, cu, q = batch(lens, news, 16, 128, 2, 4, "bf16")
    more = torch.cat([q, fresh(25, 8, 128, "bf16", 8)]).cuda()
    args = (i32(tab), i32(lens), i32(cu))
    for f, m in ((Q.kv8_attention_window, (100, 5)), (Q.kv8_attention_tree, (i32(grown(news, 2) + [-1] * 25),))):
        out = torch.full_like(more, 7.0)
        f(dev, more, *args, *m, out=out)
        assert bool((out[cu[-1]:] == 7).all()) and bool(torch.isfinite(out[:cu[-1]]).all()) and not bool((out[:cu[-1]] == 7).all())


def test_strided_queries_other_stream_and_out():
    lens, new = [150, 40, 300], [4, 1, 2]
    dev, ref, tab, cu, q = batch(lens, new, 32, 128, 2, 4, "bf16")
    fused = torch.zeros(7, 12, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, :8] = q
    parent = i32(grown(new, 3))
    args = (i32(tab), i32(lens), i32(cu))
    st = torch.cuda.Stream()
    for call in (lambda x, **k: Q.kv8_attention_window(dev, x, *args, 33, 5, **k),
                 lambda x, **k: Q.kv8_attention_tree(dev, x, *args, parent, **k)):
        want = call(q.cuda())
        assert torch.equal(want, call(fused[:, :8]))
        out = torch.empty_like(want)
        st.wait_stream(torch.cuda.current_stream())
        assert call(fused[:, :8], out=out, stream=st) is not None
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(want, out)


def test_two_streams_at_once():
    """Calls on two streams, each with parts in scratch memory of its own."""
    side = torch.cuda.Stream()
    lens, new = [4000, 900], [6, 3]
    dev, ref, tab, cu, q = batch(lens, new, 32, 128, 2, 4, "bf16")
    qs = [q.cuda(), fresh(9, 8, 128, "bf16", 9).cuda()]
    parent, args = i32(grown(new, 1)), (i32(tab), i32(lens), i32(cu))

    def both(i, st):
        return (Q.kv8_attention_tree(dev, qs[i], *args, parent, stream=st),
                Q.kv8_attention_window(dev, qs[i], *args, 3000, 4, stream=st))
    want = [both(i, None) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate((None, side)):
            got[i].append(both(i, st))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


def test_graph_replays():
    """Captured once, both masks; lengths, queries and the tree change in between."""
    lens, new = [1900, 900], [6, 6]
    dev, ref, tab, cu, q = batch(lens, new, 16, 128, 2, 4, "f16", W=400)
    tab, cu, q, ln, parent = i32(tab), i32(cu), q.cuda(), i32(lens), i32(grown(new, 1))
    assert Q.lib().qmm_kv8_attention_window_work(dev._at, 12, 8, 2, 400, 1 << 20, 4) > 0   # cut into parts

    def step():
        return (Q.kv8_attention_window(dev, q, tab, ln, cu, 1 << 20, 4), Q.kv8_attention_window(dev, q, tab, ln, cu, 100, 4),
                Q.kv8_attention_tree(dev, q, tab, ln, cu, parent))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        q.copy_(fresh(12, 8, 128, "f16", 30 + i))
        ln.copy_(i32([1300 + 50 * i, 10 + 200 * i]))
        parent.copy_(i32(grown(new, 50 + i)))
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,G", [(16, 64, 4), (16, 128, 32), (32, 128, 3), (64, 64, 16)])
@pytest.mark.parametrize("lens,new", [([2600], [5]), ([5003], [9]), ([2300, 700, 1200], [4, 1, 20])])
def test_drafts_in_few_and_many_parts(lens, new, B, D, G, dt):
    """One context in up to 32 parts and several in fewer, row groups of every size and
    number, items counted by sequence and by tokens."""
    b = batch(lens, new, B, D, 1, G, dt, W=-(-max(lens) // B) + 40)
    tree(*b[:3], lens, b[3], b[4], dt, grown(new, 8), f"{lens} {new} B{B} D{D} G{G} {dt}")


@pytest.mark.parametrize("S_", [65, 700])
def test_many_sequences(S_):
    r = np.random.default_rng(S_)
    new = [int(x) for x in r.choice([0, 1, 1, 3, 6], S_)]
    new[0] = new[-1] = 2
    lens = [n + int(x) for n, x in zip(new, r.integers(0, 90, S_))]
    dev, ref, tab, cu, q = batch(lens, new, 16, 64, 1, 2, "f16")
    window(dev, ref, tab, lens, cu, q, "f16", 20, 3, f"{S_} sequences")
    tree(dev, ref, tab, lens, cu, q, "f16", grown(new, 5), f"{S_} sequences")


def test_offsets_past_32_bits():
    H, B, D = 8, 64, 256
    P = (1 << 32) // (H * B * D) + 600
    dev, small = Q.Kv8Cache(P, H, B, D), Q.Kv8Cache(4, H, B, D)
    far, near, T = [P - 1, P - 300, 5, P - 2], [0, 1, 2, 3], 4 * B - 10
    k, v = fresh(T, H, D, "bf16", 1).cuda(), fresh(T, H, D, "bf16", 2).cuda()
    for c, t in ((dev, far), (small, near)):
        Q.kv8_append(c, k, v, i32([t]), i32([T]), i32([0, T]))
    q, rest = fresh(3, 16, D, "bf16", 3).cuda(), (i32([T]), i32([0, 3]))
    for f, m in ((Q.kv8_attention_window, (100, 5)), (Q.kv8_attention_tree, (i32([-1, 0, 0]),))):
        assert torch.equal(f(dev, q, i32([far]), *rest, *m), f(small, q, i32([near]), *rest, *m))
