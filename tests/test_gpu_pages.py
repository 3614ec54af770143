"""Page accounts on the GPU against the sequential reference: any mix of forks, growing, shrinking and
copying, and the calls' corners."""
import numpy as np
import pytest

import pagesref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def dev(x, dtype=torch.int32):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device="cuda")


class Both:
    """Accounts on the GPU beside the reference's."""

    def __init__(self, S, P, N, ref=None):
        k = kv()
        self.ref = pagesref.Accounts.empty(S, P, N) if ref is None else ref
        self.work = torch.zeros(k.kv_nvfp4_pages_workspace_bytes(N) + 64, dtype=torch.uint8,
                                device="cuda")
        self.work[-64:] = 9
        self.t = [dev(x) for x in (self.ref.table, self.ref.held, self.ref.refs, self.ref.free,
                                   [self.ref.count])]
        self.pages = k.make_pages(*self.t, self.work[:-64])
        self.status, self.S = dev([0]), S
        self.copies = torch.empty(S, 2, dtype=torch.int32, device="cuda")

    def resize(self, keep, room):
        kv().kv_nvfp4_pages_resize(self.pages, dev(keep), dev(room), self.copies, self.status)
        want = self.ref.resize(keep, room)
        assert np.array_equal(self.copies.cpu().numpy(), want)
        self.same()
        return want

    def fork(self, src, dst, lens):
        kv().kv_nvfp4_pages_fork(self.pages, dev(src), dev(dst), dev(lens), len(src), self.status)
        self.ref.fork(list(src), list(dst), lens)
        self.same()

    def same(self):
        k, r = kv(), self.ref
        table, held, refs, free, count = (x.cpu().numpy() for x in self.t)
        assert np.array_equal(held, r.held)
        assert np.array_equal(table, r.table)
        assert np.array_equal(refs, r.refs)
        assert int(count[0]) == r.count and np.array_equal(free, r.free)
        bits = (k.DEV_BAD_SEQ * r.bad_seq | k.DEV_BAD_POS * r.bad_pos | k.DEV_BAD_PAGE * r.bad_page
                | k.DEV_NO_PAGE * r.no_page)
        assert int(self.status.item()) == bits
        assert (self.work[-64:] == 9).all()


def test_init():
    k = kv()
    S, P, N = 3, 70, 1000
    t = [torch.full(shape, 5, dtype=torch.int32, device="cuda") for shape in ((S, P), (S,), (N,), (N,), (1,))]
    work = torch.full((k.kv_nvfp4_pages_workspace_bytes(N),), 0xFF, dtype=torch.uint8, device="cuda")
    pages = k.make_pages(*t, work)
    k.kv_nvfp4_pages_init(pages)
    b = Both(S, P, N)
    for x, y in zip(t, b.t):
        assert torch.equal(x, y)
    copies, status = torch.empty(S, 2, dtype=torch.int32, device="cuda"), dev([0])
    k.kv_nvfp4_pages_resize(pages, dev([0] * S), dev([100, 4000, 0]), copies, status)
    b.resize([0] * S, [100, 4000, 0])
    for x, y in zip(t, b.t):
        assert torch.equal(x, y)


@pytest.mark.parametrize("S,P,N,steps,seed", [(1, 3, 5, 12, 0), (4, 6, 20, 40, 1), (7, 40, 200, 30, 2),
                                              (33, 12, 300, 30, 3), (100, 100, 4000, 15, 4),
                                              (1500, 3, 3000, 6, 5), (3, 3000, 6000, 8, 6),
                                              (8, 2500, 9000, 8, 7), (16, 3000, 50000, 6, 8),
                                              (16, 3000, 30000, 6, 9)])
def test_any_mix(S, P, N, steps, seed):
    """Random calls, some of which ask for more pages than there are."""
    rng = np.random.default_rng(seed)
    b = Both(S, P, N)
    lens = np.zeros(S, int)  # kept tokens
    for _ in range(steps):
        if S > 1 and rng.random() < 0.4:
            free = np.flatnonzero(b.ref.held == 0)
            full = np.flatnonzero(b.ref.held > 0)
            if len(free) and len(full):
                dst = rng.permutation(free)[:rng.integers(1, len(free) + 1)]
                src = rng.choice(full, len(dst))
                n = np.array([rng.integers(0, b.ref.held[a] * 64 + 1) for a in src])
                b.fork(src.tolist(), dst.tolist(), n)
                lens[dst] = n
                continue
        keep = np.where(rng.random(S) < 0.2, rng.integers(0, lens + 1), lens)
        keep = np.where(rng.random(S) < 0.15, 0, keep)
        more = rng.choice([0, 1, 16, 64, 65, 300, P * 64], S, p=[.25, .2, .2, .1, .1, .1, .05])
        room = np.minimum(keep + more * (rng.random(S) < 0.7), P * 64)
        held = b.ref.held.copy()
        b.resize(keep, room)
        done = (b.ref.held == (room + 63) // 64) & ~((held == b.ref.held) & (keep < lens))
        lens = np.where(done, np.where(rng.random(S) < 0.8, room, keep), lens)
        lens = np.minimum(lens, b.ref.held * 64)
    b.ref.check()


def test_sharing_ends_when_it_is_written():
    b = Both(4, 4, 16)
    b.resize([0] * 4, [130, 0, 0, 0])
    b.fork([0, 0, 0], [1, 2, 3], [130, 128, 64])
    want = b.resize([130, 130, 128, 64], [131, 131, 129, 65])
    # places 2 of the first two were shared by them; the others' new places are fresh without a copy
    assert (want[:2] >= 0).all() and (want[2:] == -1).all()
    b.ref.check()
    b.resize([10, 131, 129, 0], [200, 140, 129, 0])  # written again inside a shared page
    b.ref.check()


def test_no_page_leaves_a_sequence_as_it_was():
    b = Both(5, 10, 8)
    b.resize([0] * 5, [64, 128, 64, 0, 64])  # 3 left
    keep = [64, 128, 64, 0, 64]
    b.resize(keep, [64, 192, 320, 10, 0])  # 1 fits; 4 and what follows do not; the last keeps too much
    assert b.ref.held.tolist() == [1, 3, 1, 0, 1] and b.ref.no_page and b.ref.bad_pos
    assert b.ref.count == 2
    b.resize([64, 192, 64, 0, 0], [64, 192, 320, 0, 0])  # what a call frees is for the next one
    assert b.ref.held.tolist() == [1, 3, 1, 0, 0] and b.ref.count == 3
    b.resize([64, 192, 64, 0, 0], [64, 192, 256, 0, 0])
    assert b.ref.held.tolist() == [1, 3, 4, 0, 0] and b.ref.count == 0
    b.ref.check()


def test_refused_sequences_and_pages():
    b = Both(6, 4, 10)
    b.resize([0] * 6, [64, 64, 64, 128, 64, 64])
    keep = np.array([-1, 65, 64, 64, 2 ** 31 - 1, 64])
    room = np.array([10, 70, 63, 257, 2 ** 31 - 1, 64])
    b.resize(keep, room)
    assert b.ref.bad_pos and b.ref.held.tolist() == [1, 1, 1, 2, 1, 1]
    # pages outside the pool: kept, and dropped, uncounted
    for t in (b.t[0].cpu().numpy(), b.ref.table):
        t[3, 0] = 99
        t[5, 0] = -5
    b.t[0].copy_(dev(b.ref.table))
    b.resize([64, 64, 64, 1, 64, 0], [64, 64, 64, 128, 64, 0])
    assert b.ref.bad_page and b.ref.held.tolist() == [1, 1, 1, 2, 1, 0]
    b.fork([3], [5], [128])
    assert b.ref.held[5] == 2


@pytest.mark.parametrize("src,dst,lens", [
    ([0, 0], [2, 2], [64, 10]),          # the same target twice
    ([0, 2], [2, 3], [64, 64]),          # a target as a source
    ([0, 0], [0, 3], [64, 64]),          # onto itself (and a source that is a target)
    ([0], [1], [64]),                    # a target that holds pages
    ([-1, 4, 0, 0], [2, 3, 9, -2], [1, 1, 1, 1]),
    ([0, 1, 0], [2, 3, 3], [129, -1, 3]),  # longer than the source, negative, twice
    ([3], [2], [0]),                     # nothing of nothing
])
def test_refused_forks(src, dst, lens):
    b = Both(4, 4, 10)
    b.resize([0] * 4, [128, 64, 0, 0])
    b.fork(src, dst, lens)


@pytest.mark.parametrize("H,N,n", [(1, 5, 1), (4, 40, 9), (3, 700, 300), (8, 400, 200)])
def test_copy_pages(H, N, n):
    k = kv()
    rng = np.random.default_rng(n)
    pool = rng.integers(0, 256, (N, 9216 * H), dtype=np.uint8)
    order = rng.permutation(N)
    pairs = np.stack([rng.choice(order[n:], n), order[:n]], 1).astype(np.int32)
    skip = rng.random(n) < 0.3
    pairs[skip] = -1
    bad = ~skip & (rng.random(n) < 0.1)
    pairs[bad, rng.integers(0, 2)] = rng.choice([-2, -1, N, 2 ** 31 - 1])
    want = pool.copy()
    for a, b in pairs[~skip & ~bad]:
        want[b] = pool[a]
    got, status = dev(pool, torch.uint8), dev([0])
    k.kv_nvfp4_copy_pages(k.make_layout(H, H), got, N, dev(pairs), n, status)
    assert np.array_equal(got.cpu().numpy(), want)
    assert int(status.item()) == (k.DEV_BAD_PAGE if bad.any() else 0)


def test_captured_calls_follow_their_inputs():
    b = Both(3, 8, 24)
    keep, room, src, dst, n = dev([0] * 3), dev([100, 0, 0]), dev([0]), dev([1]), dev([100])
    k = kv()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        k.kv_nvfp4_pages_resize(b.pages, keep, room, b.copies, b.status)
        k.kv_nvfp4_pages_fork(b.pages, src, dst, n, 1, b.status)
    for keeps, rooms, to in (([0] * 3, [100, 0, 0], 1), ([100, 100, 0], [101, 101, 0], 2),
                             ([0, 50, 100], [300, 64, 0], 2)):
        keep.copy_(dev(keeps)), room.copy_(dev(rooms)), dst.copy_(dev([to]))
        graph.replay()
        torch.cuda.synchronize()
        b.ref.resize(keeps, rooms)
        b.ref.fork([0], [to], [100])
        b.same()


def test_most_sequences():
    """As many sequences as accounts may have: forks of half of them, and more pages asked for than
    there are."""
    S = kv().MAX_ACCOUNTED_SEQS
    b = Both(S, 3, 3 * S // 2)
    half, rest = np.arange(S // 2), np.arange(S // 2, S)
    n = np.where(half % 3 == 0, 64, 100)
    b.resize(np.zeros(S, int), np.concatenate([n, np.zeros(S // 2, int)]))
    b.fork(half.tolist(), rest.tolist(), n)
    lens = np.concatenate([n, n])
    b.resize(lens, lens + 30)
    lens = np.minimum(lens, b.ref.held * 64)
    b.resize(lens, np.minimum(lens + 90, 192))
    b.resize(np.zeros(S, int), np.zeros(S, int))
    assert b.ref.count == 3 * S // 2
    b.ref.check()


def test_captured_resize_outlives_emptied_accounts():
    k = kv()
    c = k.PagedNVFP4Cache(9, np.zeros((2, 4), np.int32), 1, 4, 2, rot_dim=0)
    c.page_accounts()
    keep, room = dev([0, 0]), dev([100, 70])
    c.resize(keep, room)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        c.resize(keep, room)
    c.page_accounts()
    room.copy_(dev([65, 10]))
    graph.replay()
    torch.cuda.synchronize()
    assert c.block_table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]]
    assert int(c.status.item()) == 0
