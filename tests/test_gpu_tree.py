"""Trees of drafted tokens on the GPU: masks, attention, accepted paths, against plain references."""
import numpy as np
import pytest

import evictref
import treeref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SCALE = 1.0 / np.sqrt(128)


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def dev(x, dtype=torch.int32):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device="cuda")


# ---- masks -------------------------------------------------------------------------------------

@pytest.mark.parametrize("S,n,padding", [(1, 1, 0), (1, 8, 0), (3, 31, 0.1), (2, 32, 0), (4, 33, 0.1),
                                         (2, 64, 0.05), (2, 65, 0), (3, 128, 0.02), (2, 129, 0),
                                         (5, 255, 0.01), (2, 256, 0), (2, 256, 1.0)])
def test_masks(S, n, padding):
    rng = np.random.default_rng(S * 1000 + n)
    parents = np.stack([treeref.random_tree(rng, n, padding) for _ in range(S)])
    if n >= 128:
        parents[0] = np.arange(n) - 1  # a chain: as deep as it gets
        parents[1] = np.where(np.arange(n) == 0, -1, 0)  # a star
    lens, first = rng.integers(0, 1000, S), rng.integers(0, 9999, S)
    W = (n + 31) // 32
    for first_pos in (first, None):
        out = [torch.full((S * n * W + 1,), 77, dtype=torch.int32, device="cuda")]
        out += [torch.full((S * n + 1,), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
        status = dev([0])
        kv().kv_nvfp4_tree_mask(dev(parents), S, n, dev(lens),
                                None if first_pos is None else dev(first), *out, status)
        mask, seqs, slots, positions = (x.cpu().numpy() for x in out)
        assert int(status.item()) == 0 and all(x[-1] == 77 for x in (mask, seqs, slots, positions))
        for s in range(S):
            words, depth = treeref.mask_words(parents[s])
            at = slice(s * n, (s + 1) * n)
            assert np.array_equal(mask[:-1].reshape(S, n, W)[s], words)
            assert (seqs[at] == s).all() and np.array_equal(slots[at], lens[s] + np.arange(n))
            assert np.array_equal(positions[at], (lens if first_pos is None else first)[s] + depth)


def test_masks_alone_and_bad_lengths():
    parents = np.array([[-1, 0, 1]] * 4, np.int32)
    mask = torch.full((4, 3, 1), 77, dtype=torch.int32, device="cuda")
    status = dev([0])
    kv().kv_nvfp4_tree_mask(dev(parents), 4, 3, dev([5, -1, 2 ** 31 - 4, 2 ** 31 - 3]), None, mask,
                            status=status)
    got = mask[:, :, 0].cpu().numpy()
    assert int(status.item()) == kv().DEV_BAD_POS
    assert got.tolist() == [[1, 3, 7], [77] * 3, [1, 3, 7], [77] * 3]


# ---- attention -----------------------------------------------------------------------------------

class Tree:
    """A cache of random rows with n nodes behind `held` tokens, queries and a mask."""

    def __init__(self, held, n, chunk, Hq, H, seed=0, mask="tree", **cache):
        rng = np.random.default_rng(seed + 100 * n + len(held))
        self.held, self.n, self.Hq, self.H, self.S = held, n, Hq, H, len(held)
        self.cache = treeref.Cache([h + n for h in held], H, seed, **cache)
        self.chunk = chunk
        self.q = treeref.random_rows(rng, (self.S * n, Hq))
        W = (n + 31) // 32
        if mask == "tree":
            rows = [treeref.ancestors(treeref.random_tree(rng, n, 0.05)) for _ in held]
            self.sees = np.array([[np.zeros(n, bool) if r is None else r for r in t] for t in rows])
        elif mask == "none":
            self.sees = np.zeros((self.S, n, n), bool)
        else:  # anything, some rows empty
            self.sees = rng.random((self.S, n, n)) < rng.choice([0, 0.1, 0.9, 1], (self.S, n, 1))
        words = np.stack([treeref.words_of(x) for x in self.sees]).view(np.uint32)
        if n % 32:  # bits behind the last node count for nothing
            words[..., -1] |= rng.integers(0, 2 ** 32, words[..., -1].shape, dtype=np.uint32) \
                << np.uint32(n % 32)
        assert words.shape == (self.S, n, W)
        self.mask = dev(words.view(np.int32))
        self.upload()

    def upload(self):
        k, c = kv(), self.cache
        self.pool = dev(c.pool, torch.uint8)
        self.table = dev(c.table)
        self.q_codes = dev(self.q[..., :64], torch.uint8)
        self.q_scales = dev(self.q[..., 64:], torch.uint8)
        self.layout = k.make_layout(self.Hq, self.H, rot_dim=0)
        size = k.kv_nvfp4_plan_workspace_bytes(self.layout, c.lens, self.n, False, self.chunk)
        self.workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        self.plan = k.kv_nvfp4_plan(self.layout, c.lens, self.n, False, self.chunk, self.workspace, size)
        rows = self.S * self.n * self.Hq * 128
        self.buffer = torch.full((rows + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.buffer[rows:] = 7
        self.out = self.buffer[:rows]
        self.status = dev([0])

    def run(self, stream=None, scale=SCALE):
        kv().kv_nvfp4_tree_attn(self.layout, self.plan, self.workspace, self.q_codes, self.q_scales,
                                self.mask, scale, self.pool, self.cache.num_pages, self.table,
                                self.table.shape[1], self.out, self.status, stream)

    def check(self, status=0, good=None):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        assert (self.buffer[self.out.numel():] == 7).all()
        got = self.out.float().cpu().numpy().astype(np.float64).reshape(self.S, self.n, self.Hq, 128)
        q = evictref.values(self.q).reshape(self.S, self.n, self.Hq, 128)
        for s in range(self.S):
            ref, tol = treeref.attend(q[s], self.cache.rows[s], self.Hq // self.H, self.sees[s], SCALE,
                                      None if good is None else good[s])
            hidden = np.isnan(ref)
            assert (np.isnan(got[s]) == hidden).all(), s
            err = np.abs(got[s] - ref)[~hidden]
            assert (err <= tol[~hidden]).all(), (s, float((err / tol[~hidden]).max()))


CASES = [
    # held, n, chunk, Hq, H: at most 8 rows per KV head and 4 heads (the decode kernel)
    ([0], 1, 64, 24, 4),
    ([0, 5, 62, 63, 64, 200, 1000], 1, 64, 24, 4),
    ([0, 57, 63, 64, 120, 700], 2, 64, 16, 4),
    ([56, 60, 63, 64, 1500], 8, 64, 3, 3),      # nodes over a page's end; odd heads
    ([0, 300, 5000], 8, 64, 1, 1),
    ([0, 300], 4, 1024, 8, 4),
    # at most 64 rows
    ([0, 97], 8, 64, 24, 4),
    ([0, 13, 63, 64, 65, 517, 2049], 8, 128, 32, 8),
    ([120, 124, 126, 127, 128, 1, 900], 9, 128, 12, 3),
    ([500, 40], 64, 128, 4, 4),
    ([0, 700, 2100], 8, 64, 8, 8),
    ([0, 63, 64, 65, 191, 192, 193], 1, 64, 20, 5),
    ([300, 40], 5, 1024, 25, 5),
    ([3000], 21, 64, 3, 1),
    # up to 128, and several tiles
    ([100, 3, 700], 16, 128, 24, 4),
    ([0, 31, 32, 33, 4000], 32, 128, 16, 4),
    ([0, 95, 96, 97], 33, 128, 8, 2),
    ([1000, 37], 64, 128, 24, 4),
    ([130, 1], 100, 192, 8, 2),
    ([0, 900], 255, 128, 6, 2),
    ([64, 1], 256, 128, 3, 1),
    ([5, 900, 3, 60, 0, 1, 2, 700, 9, 64, 30, 7], 12, 128, 8, 2),
]


@pytest.mark.parametrize("mask", ["tree", "any"])
@pytest.mark.parametrize("held,n,chunk,Hq,H", CASES)
def test_tree_attn(held, n, chunk, Hq, H, mask):
    t = Tree(held, n, chunk, Hq, H, seed=len(held), mask=mask)
    t.run()
    t.check()
    first = t.out.clone()
    t.out.fill_(float("nan"))
    t.run()  # equal inputs give equal bits, on a used workspace too
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), t.out.view(torch.int16))


@pytest.mark.parametrize("held,n,chunk,Hq,H", CASES[1:18:4] + CASES[-2:])
def test_nodes_that_see_no_node(held, n, chunk, Hq, H):
    t = Tree(held, n, chunk, Hq, H, mask="none")
    t.run()
    t.check()
    out = t.out.view(t.S, -1)
    for s, h in enumerate(held):
        assert (out[s] == 0).all() == (h == 0)


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("held,n,chunk,Hq,H", [([0, 60, 500], 2, 64, 16, 4), ([59, 3], 8, 64, 3, 3),
                                              ([0, 60, 500], 8, 128, 24, 4), ([120], 9, 64, 8, 8),
                                              ([0, 100, 700], 40, 128, 24, 4), ([90], 130, 128, 2, 1)])
def test_nan_reaches_those_that_see_it(held, n, chunk, Hq, H, which):
    t = Tree(held, n, chunk, Hq, H, mask="any", seed=3)
    rng = np.random.default_rng(n)
    for s, h in enumerate(held):
        for node in rng.choice(n, max(1, n // 6), replace=False):
            head = rng.integers(0, H)
            if which != "v":
                t.cache.rows[s][h + node, head, 64 + rng.integers(0, 8)] = rng.choice([0x7F, 0xFF])
            if which != "k":
                t.cache.rows[s][h + node, head, 136 + rng.integers(0, 8)] = rng.choice([0x7F, 0xFF])
    t.cache.write()
    t.upload()
    t.run()
    t.check()


def test_nan_alone():
    """Rows whose only visible key has a NaN score: in one segment, and in the second of two."""
    for held, n, Hq, H in (([0], 3, 2, 1), ([0], 3, 24, 4), ([0], 40, 24, 4), ([0], 200, 8, 2)):
        t = Tree(held, n, 64, Hq, H, mask="none")
        t.sees[0] = np.eye(n, dtype=bool)
        t.mask = dev(treeref.words_of(t.sees[0]))
        t.cache.rows[0][1, :, 64:72] = 0x7F
        t.cache.rows[0][n - 1, :, 64:72] = 0x7F
        t.cache.write()
        t.upload()
        t.run()
        t.check()
        assert torch.isnan(t.out.view(n, -1)[n - 1]).all()


@pytest.mark.parametrize("held,n,chunk,Hq,H", [([500, 70], 2, 64, 16, 4), ([500, 70], 9, 128, 24, 4),
                                              ([500, 70], 8, 128, 32, 8), ([300, 5], 60, 128, 8, 2)])
def test_bad_pages_are_skipped(held, n, chunk, Hq, H):
    t = Tree(held, n, chunk, Hq, H)
    bad = [(0, 1, -1), (0, (held[0] + n - 1) // 64, t.cache.num_pages), (1, 0, 2 ** 31 - 1)]
    good = [np.ones(h + n, bool) for h in held]
    for s, j, page in bad:
        t.table[s, j] = page
        good[s][64 * j:64 * (j + 1)] = False
    t.run()
    t.check(kv().DEV_BAD_PAGE, good)


def test_softmax_scale_defaults_and_unaligned_masks():
    t = Tree([200], 5, 64, 24, 4, seed=2)
    wide = torch.zeros(t.mask.numel() + 1, dtype=torch.int32, device="cuda")
    wide[1:] = t.mask.flatten()
    t.mask = wide[1:]
    t.run(scale=0.0)
    t.check()


@pytest.mark.parametrize("held,n,Hq,H", [([700, 90], 2, 16, 4), ([700, 90], 20, 24, 4)])
def test_graph_and_stream(held, n, Hq, H):
    t = Tree(held, n, 64, Hq, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    t.check()
    want = t.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.run()
        t.run()
    for _ in range(2):
        t.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.int16), t.out.view(torch.int16))


# ---- accepted paths ------------------------------------------------------------------------------

def _accept_case(rng, S, n, H, vocab, held=None, padding=0.05):
    held = rng.integers(0, 400, S).tolist() if held is None else held
    cache = treeref.Cache([h + n for h in held], H, int(rng.integers(1 << 30)))
    parents = np.stack([treeref.random_tree(rng, n, padding) for _ in range(S)])
    draft, target = rng.integers(0, vocab, (2, S, n))
    return held, cache, parents, draft, target, rng.integers(0, vocab, S)


@pytest.mark.parametrize("S,n,H,vocab", [(1, 1, 4, 1), (1, 1, 4, 2), (5, 8, 4, 2), (3, 16, 1, 1),
                                         (4, 33, 3, 2), (2, 64, 8, 1), (7, 64, 4, 3), (3, 130, 5, 1),
                                         (2, 256, 2, 1), (2, 256, 4, 2)])
def test_accept(S, n, H, vocab):
    rng = np.random.default_rng(n * 10 + vocab)
    held, cache, parents, draft, target, expected = _accept_case(rng, S, n, H, vocab)
    if n >= 64:
        parents[0] = np.arange(n) - 1  # with one token: a path of every node, none moves
        held[0] = 60  # (the cache below was made for another length: only bytes count)
        cache = treeref.Cache([h + n for h in held], H, 1)
        parents[1] = np.where(np.arange(n) < 2, -1, np.arange(n) - 1)
        parents[1, 1] = -2  # node 2 and all below hang nowhere, 0 is alone
        parents[1, 3:] = np.arange(n - 3) + 2
        parents[1, 2] = 0  # every node but 1: all rows move
    paths, tokens, want = treeref.accept(cache, parents, draft, target, expected, held)
    k = kv()
    pool, status = dev(cache.pool, torch.uint8), dev([0])
    path = torch.full((S, n), -7, dtype=torch.int32, device="cuda")
    count, nxt, lens = (torch.full((S,), -7, dtype=torch.int32, device="cuda") for _ in range(3))
    layout = k.make_layout(H, H, rot_dim=0)
    args = (S, n, dev(held), dev(cache.table), cache.table.shape[1], cache.num_pages)
    k.kv_nvfp4_tree_accept(layout, dev(parents), dev(draft), dev(target), dev(expected), *args, pool,
                           path, count, nxt, lens, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert count.tolist() == [len(p) for p in paths] and nxt.tolist() == [int(x) for x in tokens]
    assert lens.tolist() == [h + len(p) for h, p in zip(held, paths)]
    for got, p in zip(path.tolist(), paths):
        assert got == p + [-7] * (n - len(p))
    assert np.array_equal(pool.cpu().numpy(), want)
    # the same moves in another pool by the path alone, and the walk alone
    again = dev(cache.pool, torch.uint8)
    k.kv_nvfp4_tree_accept(layout, None, None, None, None, *args, again, path, count, None, None, status)
    assert np.array_equal(again.cpu().numpy(), want)
    path2, count2, nxt2 = path.clone().fill_(-7), count.clone(), nxt.clone()
    k.kv_nvfp4_tree_accept(layout, dev(parents), dev(draft), dev(target), dev(expected), S, n,
                           dev(held), None, 0, 0, None, path2, count2, nxt2, None, status)
    assert torch.equal(path, path2) and torch.equal(count, count2) and torch.equal(nxt, nxt2)
    # onto its own inputs
    own, own_next = dev(held), dev(expected)
    third = dev(cache.pool, torch.uint8)
    k.kv_nvfp4_tree_accept(layout, dev(parents), dev(draft), dev(target), own_next, S, n, own,
                           dev(cache.table), cache.table.shape[1], cache.num_pages, third, path2,
                           count2, own_next, own, status)
    assert torch.equal(own, lens) and torch.equal(own_next, nxt) and torch.equal(third, pool)
    assert int(status.item()) == 0


def test_given_paths_and_bad_sequences():
    """One good path among ones that are out of the tree, out of order, too long, or out of the table."""
    H, n = 3, 8
    held = [100, 100, 100, 100, 100, -1, 190, 100]
    rng = np.random.default_rng(0)
    cache = treeref.Cache([max(h, 0) + n for h in held], H, 5, pages_behind=0)
    assert cache.table.shape[1] == 4
    held[6] = 4 * 64 - n + 1  # the tree ends past the table
    path = np.tile(np.arange(n, dtype=np.int32), (8, 1))
    path[0, :3] = 1, 4, 7
    path[1, :3] = 1, 4, 8
    path[2, :3] = 4, 4, 5
    path[3, :3] = -1, 2, 3
    path[7, :3] = 1, 4, 7
    count = np.array([3, 3, 3, 3, n + 1, 3, 3, -1], np.int32)
    want, off = cache.pool.copy(), evictref.row_offsets(H)
    treeref.move(cache.pool, want, cache.table[0], off, [1, 4, 7], 100)
    del rng
    k = kv()
    pool, status = dev(cache.pool, torch.uint8), dev([0])
    lens = torch.full((8,), -7, dtype=torch.int32, device="cuda")
    k.kv_nvfp4_tree_accept(k.make_layout(H, H, rot_dim=0), None, None, None, None, 8, n, dev(held),
                           dev(cache.table), 4, cache.num_pages, pool, dev(path), dev(count), None, lens,
                           status)
    torch.cuda.synchronize()
    assert int(status.item()) == k.DEV_BAD_POS
    assert lens.tolist() == [103] + [-7] * 7
    assert np.array_equal(pool.cpu().numpy(), want)


def test_accept_leaves_rows_of_bad_pages():
    H, n, held = 4, 64, [40]
    cache = treeref.Cache([held[0] + n], H, 9)
    table = cache.table.copy()
    table[0, 1] = cache.num_pages + 5  # slots 64 .. 103
    path = np.full((1, n), -1, np.int32)
    path[0, :30] = np.arange(30) * 2  # rows from slots 40 .. 98 to 40 .. 69
    want, off = cache.pool.copy(), evictref.row_offsets(H)
    treeref.move(cache.pool, want, table[0], off, path[0, :30], held[0])
    k = kv()
    pool, status = dev(cache.pool, torch.uint8), dev([0])
    k.kv_nvfp4_tree_accept(k.make_layout(H, H, rot_dim=0), None, None, None, None, 1, n, dev(held),
                           dev(table), table.shape[1], cache.num_pages, pool, dev(path), dev([30]), None,
                           None, status)
    torch.cuda.synchronize()
    assert int(status.item()) == k.DEV_BAD_PAGE
    assert np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("n,Hq,H", [(2, 16, 4), (33, 16, 8)])
def test_pages_past_32_bits_of_offset(n, Hq, H):
    """The same pages at the end of a pool of more than 4 GB: the same output, the same rows moved, the
    same page copied."""
    k = kv()
    t = Tree([700, 90], n, 64, Hq, H, seed=5)
    t.run()
    t.check()
    want, few = t.out.clone(), t.cache.num_pages
    paths = dev([[0] + [0] * (n - 1), list(range(1, n)) + [0]])  # what moves: nothing, all but node 0
    count, lens = dev([1, n - 1]), dev([700, 90])
    moved = t.pool.clone().view(few, -1)
    k.kv_nvfp4_tree_accept(t.layout, None, None, None, None, 2, n, lens, t.table, t.table.shape[1], few,
                           moved, paths, count, None, None, t.status)
    far = 2 ** 32 // (9216 * H) + 100
    pool = torch.empty(far + few, 9216 * H, dtype=torch.uint8, device="cuda")
    pool[far:] = t.pool.view(few, -1)
    table = torch.where(t.table >= 0, t.table + far, t.table)
    t.out.fill_(float("nan"))
    k.kv_nvfp4_tree_attn(t.layout, t.plan, t.workspace, t.q_codes, t.q_scales, t.mask, SCALE, pool,
                         far + few, table, table.shape[1], t.out, t.status)
    assert torch.equal(t.out.view(torch.int16), want.view(torch.int16))
    k.kv_nvfp4_tree_accept(t.layout, None, None, None, None, 2, n, lens, table, table.shape[1],
                           far + few, pool, paths, count, None, None, t.status)
    assert torch.equal(pool[far:], moved) and not torch.equal(moved, t.pool.view(few, -1))
    k.kv_nvfp4_copy_pages(t.layout, pool, far + few, dev([[far, far - 1], [far + 1, 0]]), 2, t.status)
    assert torch.equal(pool[far - 1], moved[0]) and torch.equal(pool[0], moved[1])
    assert int(t.status.item()) == 0
