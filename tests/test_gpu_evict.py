"""The eviction operators on the GPU: attention with per-key weights, select, compact, the append
behind an eviction, and a run of them together, against plain 64-bit references."""
import math

import numpy as np
import pytest

import evictref
import synth
from kvrun import GpuRun, OracleRun

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _rows(o, w, s):
    """The oracle's K/V rows [n, H, 144] of sequence s."""
    a, b = o.tok_off[s], o.tok_off[s] + int(w.seq_lens[s])
    return np.concatenate([o.kc[a:b], o.ks[a:b], o.vc[a:b], o.vs[a:b]], -1)


def _queries(o, w, s):
    c = np.concatenate([o.qc, o.qs], -1)[s * w.q_len:(s + 1) * w.q_len]
    return evictref.values(c)


class Attend:
    """A workload whose new tokens are appended, with its plan and the operands of the call."""

    def __init__(self, w, chunk):
        self.w = w
        self.g = GpuRun(w)
        self.g.step(chunk_tokens=chunk)
        c = self.c = self.g.cache
        stride = c.max_pages * 64 + 3  # no multiple of anything
        gen = torch.Generator(device="cuda")
        gen.manual_seed(5)
        self.held = torch.rand(w.num_seqs, w.kv_heads, stride, generator=gen, device="cuda")
        self.weights = torch.full_like(self.held, float("nan"))
        self.out = torch.full((self.g.T, w.q_heads, 128), float("nan"), dtype=torch.bfloat16,
                              device="cuda")

    def run(self, weights_in="held"):
        win = self.held if isinstance(weights_in, str) else weights_in
        c = self.c
        need = kv().kv_nvfp4_weights_workspace_bytes(c.layout, c.plan_info)
        if c.weights_workspace is None:
            c.weights_workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        kv().kv_nvfp4_decode_attn_weights(
            c.layout, c.plan_info, c.workspace, c.weights_workspace, need, self.g.q_codes,
            self.g.q_scales, self.w.sm_scale, c.pool, c.num_pages, c.block_table, c.max_pages,
            self.out, win, self.weights, self.weights.shape[2], c.status)

    def check(self, base, good=None, status=0):
        torch.cuda.synchronize()
        assert self.g.status() == status
        w, o = self.w, OracleRun(self.w)
        out = self.out.float().cpu().numpy().astype(np.float64)
        got = self.weights.cpu().numpy().astype(np.float64)
        for s in range(w.num_seqs):
            n = int(w.seq_lens[s])
            ref, tol, ws, wtol = evictref.attend(
                _queries(o, w, s), _rows(o, w, s), w.q_heads // w.kv_heads, w.q_len, w.causal,
                w.sm_scale, None if good is None else good[s])
            err = np.abs(out[s * w.q_len:(s + 1) * w.q_len] - ref)
            assert (err <= tol).all(), (s, float((err / tol).max()))
            want = base[s, :, :n] + ws
            err = np.abs(got[s, :, :n] - want)
            # half a step of the final sum, and of the sums of up to G q_len rows
            lim = wtol + 2.0 ** -24 * want + 2.0 ** -24 * (w.q_heads // w.kv_heads * w.q_len) * ws
            assert (err <= lim + 1e-30).all(), (s, float((err / (lim + 1e-30)).max()))
            assert np.isnan(got[s, :, n:]).all()  # behind the sequence: left as it was


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


@pytest.mark.parametrize("lens,q_len,causal,chunk,Hq,Hkv", [
    ([0], 1, True, 64, 24, 4),                              # one key: its weight is the group size
    ([0, 5, 63, 64, 65, 200, 1000], 1, True, 64, 24, 4),    # page edges, split and unsplit groups
    ([0, 127, 128, 129, 700], 1, True, 1024, 24, 4),        # unsplit only
    ([10, 700], 2, False, 64, 16, 4),                       # 8 rows, not causal
    ([300, 40], 1, True, 64, 8, 1),                         # one head: a lone half pair
    ([300, 40], 2, True, 64, 9, 3),                         # odd heads
    ([0, 700, 2100], 1, True, 128, 32, 8),                  # eight KV heads: the tile kernel
    ([0, 63, 64, 65, 191, 192, 193, 255, 256, 257, 320], 1, True, 64, 20, 5),  # a lone fifth head
    ([5000, 7, 1300], 1, True, 64, 8, 8),                   # one row per head, many splits
    ([700, 90], 2, True, 128, 24, 6),                       # 8 rows per head
    ([700, 90], 2, False, 128, 24, 8),
    ([500, 0, 130], 3, True, 128, 20, 5),                   # odd heads above four, 12 rows
    ([2000, 37], 8, True, 256, 24, 4),                      # 48 rows: verify
    ([1000, 120], 8, False, 256, 24, 4),
    ([100], 11, True, 128, 24, 4),                          # 66 rows: two row tiles
    ([0, 300], 50, True, 128, 24, 4),                       # a prompt of its own; 300 rows
    ([130, 1], 200, False, 192, 8, 2),
    ([0], 300, True, 128, 3, 1),                            # causal over several key blocks
    ([5, 900, 3, 60, 0, 1, 2, 700, 9, 64, 30, 7], 1, True, 64, 8, 2),  # many, mostly short
    ([5, 900, 3, 60, 0, 1, 2, 700, 9], 9, True, 128, 8, 2),
])
def test_attend_weights(lens, q_len, causal, chunk, Hq, Hkv):
    w = synth.Workload("weights", lens, q_len=q_len, causal=causal, seed=sum(lens) + q_len,
                       q_heads=Hq, kv_heads=Hkv, chunk_tokens=chunk,
                       pool_pages=sum((c + q_len + 63) // 64 for c in lens) + 3)
    a = Attend(w, chunk)
    a.run()
    a.check(a.held.cpu().numpy().astype(np.float64))
    first, out = a.weights.clone(), a.out.clone()
    a.run()  # equal inputs give equal bits, on a used workspace too
    torch.cuda.synchronize()
    assert torch.equal(first.nan_to_num(), a.weights.nan_to_num()) and torch.equal(out, a.out)


@pytest.mark.parametrize("lens,q_len,Hq,Hkv", [([500, 20], 1, 24, 4), ([300, 40], 1, 32, 8),
                                             ([300, 40], 8, 24, 4)])
def test_attend_weights_onto_aligned_accounts(lens, q_len, Hq, Hkv):
    w = synth.Workload("aligned", lens, q_len=q_len, seed=7, q_heads=Hq, kv_heads=Hkv,
                       chunk_tokens=128)
    a = Attend(w, 128)
    a.held = a.held[..., :a.c.max_pages * 64].contiguous()
    a.weights = torch.full_like(a.held, float("nan"))
    a.run()
    a.check(a.held.cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("lens,q_len,chunk,Hq,Hkv", [
    ([600], 32, 64, 24, 4),       # 8 groups of up to 128 rows, 10 partials each
    ([1300, 5], 30, 64, 24, 4),   # 20 partials and none, padding rows in the last tile
    ([90, 700], 43, 128, 15, 5),  # 129 rows: a tile of one row
])
def test_attend_weights_merges_many_rows(lens, q_len, chunk, Hq, Hkv):
    w = synth.Workload("rows", lens, q_len=q_len, seed=q_len, q_heads=Hq, kv_heads=Hkv,
                       chunk_tokens=chunk)
    a = Attend(w, chunk)
    a.run()
    a.check(a.held.cpu().numpy().astype(np.float64))


def test_attend_weights_without_and_onto_the_accounts():
    w = synth.Workload("accounts", [70, 900], q_len=1, seed=3, chunk_tokens=64)
    a = Attend(w, 64)
    a.run(weights_in=None)
    zero = np.zeros(tuple(a.held.shape))
    a.check(zero)
    once = a.weights.cpu().numpy().astype(np.float64)
    a.run(weights_in=a.weights)  # in place: adds another time
    a.check(np.nan_to_num(once))


@pytest.mark.parametrize("q_len,Hq,Hkv", [(1, 24, 4), (8, 24, 4), (1, 32, 8)])
def test_attend_weights_of_a_bad_page_stay(q_len, Hq, Hkv):
    w = synth.Workload("bad", [500], q_len=q_len, seed=9, pool_pages=12, chunk_tokens=128,
                       q_heads=Hq, kv_heads=Hkv)
    a = Attend(w, 128)
    a.c.block_table[0, 3] = 12  # outside the pool
    a.run()
    good = np.ones(500 + q_len, bool)
    good[192:256] = False
    a.check(a.held.cpu().numpy().astype(np.float64), [good], status=kv().DEV_BAD_PAGE)


@pytest.mark.parametrize("q_len,Hq,Hkv", [(1, 24, 4), (8, 24, 4), (1, 32, 8)])
def test_attend_weights_with_no_good_page(q_len, Hq, Hkv):
    w = synth.Workload("none", [100], q_len=q_len, seed=9, pool_pages=12, chunk_tokens=128,
                       q_heads=Hq, kv_heads=Hkv)
    a = Attend(w, 128)
    a.c.block_table.fill_(-1)
    a.run()
    n = 100 + q_len
    a.check(a.held.cpu().numpy().astype(np.float64), [np.zeros(n, bool)],
            status=kv().DEV_BAD_PAGE)
    assert torch.equal(a.weights[..., :n], a.held[..., :n]) and not a.out.any()


def test_attend_weights_in_a_graph_and_on_another_stream():
    w = synth.Workload("graph", [70, 2000], q_len=1, seed=4, chunk_tokens=64)
    a = Attend(w, 64)
    a.run()
    torch.cuda.synchronize()
    first = a.weights.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            a.run()
    for _ in range(2):
        a.weights.fill_(float("nan"))
        a.out.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first.nan_to_num(), a.weights.nan_to_num())
    a.check(a.held.cpu().numpy().astype(np.float64))


# ---- select ------------------------------------------------------------------------------------

def _select(weights, lens, keep, per_head, sink, recent, n):
    k = kv()
    S, H, stride = weights.shape
    L = k.make_layout(H, H)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    index = torch.full((S, H if per_head else 1, n), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kv_nvfp4_evict_select(L, weights, stride, i32(lens), i32(keep), S, per_head, sink, recent,
                            index, n, status)
    torch.cuda.synchronize()
    return index.cpu().numpy(), int(status.item())


def _check_select(w, lens, keep, per_head, sink, recent):
    n = max(1, max(min(a, b) for a, b in zip(lens, keep))) + 1
    got, status = _select(torch.from_numpy(w).cuda(), lens, keep, per_head, sink, recent, n)
    assert status == 0
    for s, (a, b) in enumerate(zip(lens, keep)):
        for i in range(got.shape[1]):
            x = w[s, i] if per_head else evictref.head_sum(w[s])
            want = evictref.select(x, a, b, sink, recent)
            assert np.array_equal(got[s, i, :len(want)], want), (s, i)
            assert (got[s, i, len(want):] == -7).all()


@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1], [1], 0, 0), ([0, 3], [2, 0], 0, 0), ([300], [128], 4, 32), ([300], [300], 4, 32),
    ([300], [299], 0, 0), ([300], [1], 0, 0), ([300], [20], 4, 32), ([300], [36], 4, 32),
    ([300], [37], 4, 32), ([50], [20], 100, 100), ([70], [30], 0, 1 << 30),
    ([70], [30], 1 << 30, 0),
    ([5000, 1, 1023, 1025, 4097], [600, 1, 1022, 7, 2048], 3, 10),
    ([40000, 9], [5000, 4], 64, 1000), ([131072], [16384], 4, 1024),
])
def test_select(lens, keep, sink, recent, per_head):
    rng = np.random.default_rng(sum(lens) + sum(keep))
    S, H, stride = len(lens), 3, max(lens) + 5
    w = np.exp(2.5 * rng.standard_normal((S, H, stride))).astype(np.float32) * np.float32(1e-4)
    tie = rng.random(w.shape) < 0.3
    w[tie] = np.exp2(np.round(np.log2(w[tie])))
    _check_select(w, lens, keep, per_head, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "zero", "signed", "special", "neighbours", "subnormal"])
def test_select_of_hard_values(kind):
    rng = np.random.default_rng(3)
    w = np.zeros((2, 2, 3000), np.float32)
    if kind == "equal":
        w[:] = 0.125
    elif kind == "signed":
        w[:] = rng.standard_normal(w.shape)
        w[:, :, ::5] = -0.0
        w[:, :, ::7] = 0.0
    elif kind == "special":
        w[:] = rng.standard_normal(w.shape)
        w[:, :, ::3] = np.nan
        w[:, :, 1::3] = -np.inf
        w[:, :, ::50] = np.inf
    elif kind == "neighbours":  # differ in the last bits only
        w[:] = (np.float32(1.0).view(np.int32) + rng.integers(0, 9, w.shape)).astype(
            np.int32).view(np.float32)
    elif kind == "subnormal":
        w[:] = rng.integers(0, 20, w.shape).astype(np.int32).view(np.float32)
    for per_head in (True, False):
        if kind == "special" and not per_head:
            w[:, 1] = 0  # no inf - inf: the sum is the first head's
        _check_select(w, [2999, 1200], [1300, 7], per_head, 2, 9)


@pytest.mark.parametrize("H,per_head", [(1, True), (3, False)])
def test_select_of_more_slots_than_a_cluster_holds(H, per_head):
    # 16 CTAs hold 48K keys each: the rest is read again in every pass
    rng = np.random.default_rng(H)
    w = np.exp(2.5 * rng.standard_normal((1, H, 900001))).astype(np.float32)
    w[:, :, ::11] = 0.5
    for keep in (70000, 899990):
        _check_select(w, [900001], [keep], per_head, 5, 100)


@pytest.mark.parametrize("sets", [40, 700])
def test_select_of_many_sets(sets):
    rng = np.random.default_rng(sets)
    lens = [int(x) for x in rng.integers(1, 3000, sets)]
    w = rng.random((sets, 2, 3000), dtype=np.float32)
    _check_select(w, lens, [n // 3 + 1 for n in lens], True, 1, 7)


def test_select_and_compact_in_a_graph():
    # captured once, replayed on new weights and lengths
    k = kv()
    rng = np.random.default_rng(0)
    H, L = 2, k.make_layout(2, 2)
    lens, keep = [700, 300], [256, 100]
    pool, table, dst, index, weights = _compact_case(lens, keep, H, True, 5)
    dev = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
    p, t, i, w = dev(pool), dev(table), dev(index), dev(weights)
    n, m = dev(np.array(lens, np.int32)), dev(np.array(keep, np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both():
        k.kv_nvfp4_evict_select(L, w, w.shape[2], n, m, 2, True, 2, 8, i, i.shape[2], status)
        k.kv_nvfp4_evict_compact(L, i, i.shape[2], True, n, m, 2, t, t.shape[1], pool.shape[0], p,
                                 None, 0, w, w.shape[2], status)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()  # attributes are set outside the capture
        with torch.cuda.graph(graph, stream=side):
            both()
    torch.cuda.synchronize()
    for lens in ([700, 300], [650, 101], [3, 290]):
        new = rng.random(weights.shape, dtype=np.float32)
        w.copy_(torch.from_numpy(new))
        p.copy_(torch.from_numpy(pool))
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ix = np.full(index.shape, -1, np.int32)
        for s in range(2):
            for h in range(H):
                x = evictref.select(new[s, h], lens[s], keep[s], 2, 8)
                ix[s, h, :len(x)] = x
                assert np.array_equal(i[s, h, :len(x)].cpu().numpy(), x)
        want, ww = evictref.compact(pool, table, table, H, ix, lens, keep, new)
        assert np.array_equal(p.cpu().numpy(), want) and np.array_equal(w.cpu().numpy(), ww)
    assert int(status.item()) == 0


def test_select_flags_bad_sequences_and_leaves_them():
    w = torch.rand(5, 2, 100, device="cuda")
    got, status = _select(w, [101, -1, 50, 50, 50], [5, 5, -1, 21, 20], True, 0, 0, 20)
    assert status == kv().DEV_BAD_POS
    assert (got[:4] == -7).all() and (got[4] >= 0).all()


# ---- compact -----------------------------------------------------------------------------------

def _compact_case(lens, keep, H, per_head, seed, spare=2):
    rng = np.random.default_rng(seed)
    S = len(lens)
    pages = [(n + 63) // 64 for n in lens]
    more = [(min(a, b) + 63) // 64 for a, b in zip(lens, keep)]
    total = sum(pages) + sum(more) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((S, max(1, max(pages))), -1, np.int32)
    dst = np.full((S, max(1, max(more))), -1, np.int32)
    at = 0
    for s in range(S):
        table[s, :pages[s]] = order[at:at + pages[s]]
        at += pages[s]
        dst[s, :more[s]] = order[at:at + more[s]]
        at += more[s]
    n = max(1, max(min(a, b) for a, b in zip(lens, keep))) + 1
    sets = H if per_head else 1
    index = np.full((S, sets, n), -1, np.int32)
    for s, (a, b) in enumerate(zip(lens, keep)):
        for i in range(sets):
            index[s, i, :min(a, b)] = np.sort(rng.permutation(a)[:min(a, b)])
    pool = rng.integers(0, 256, (total, 9216 * H), dtype=np.uint8)
    weights = rng.random((S, H, max(lens) + 3), dtype=np.float32)
    return pool, table, dst, index, weights


def _compact(pool, table, dst, index, weights, lens, keep, H):
    k = kv()
    dev = lambda x: None if x is None else torch.from_numpy(x.copy()).cuda()  # noqa: E731
    p, t, d, i, w = map(dev, (pool, table, dst, index, weights))
    n, m = dev(np.array(lens, np.int32)), dev(np.array(keep, np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kv_nvfp4_evict_compact(k.make_layout(H, H), i, index.shape[2], index.shape[1] == H, n, m,
                             len(lens), t, table.shape[1], pool.shape[0], p, d,
                             0 if dst is None else dst.shape[1], w,
                             0 if w is None else w.shape[2], status)
    torch.cuda.synchronize()
    return p.cpu().numpy(), None if w is None else w.cpu().numpy(), int(status.item())


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,keep,H,per_head", [
    ([1], [1], 1, True), ([700], [256], 4, False), ([700], [256], 4, True), ([64], [64], 2, True),
    ([65, 0, 130], [64, 3, 129], 3, True), ([1000, 64, 63], [1, 63, 0], 5, False),
    ([3000, 900], [2990, 65], 2, True), ([9000], [5001], 1, True), ([20000], [2500], 3, False),
    ([70000], [40000], 1, True),
])
def test_compact(lens, keep, H, per_head, in_place):
    if H == 1 and not per_head:
        per_head = True
    pool, table, dst, index, weights = _compact_case(lens, keep, H, per_head, sum(lens))
    to = None if in_place else dst
    got, w, status = _compact(pool, table, to, index, weights, lens, keep, H)
    full = np.broadcast_to(index, (len(lens), H, index.shape[2]))
    want, ww = evictref.compact(pool, table, table if in_place else dst, H, full, lens, keep, weights)
    assert status == 0
    assert np.array_equal(got, want)  # every byte of the pool, moved or not
    assert np.array_equal(w, ww)
    got, w, _ = _compact(pool, table, to, index, None, lens, keep, H)
    assert w is None and np.array_equal(got, want)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,keep,H", [
    ([9000, 300], [7000, 100], 4),              # clusters of 16 for whole rows, two waves
    ([9000, 8000, 1, 7000, 64], [8990, 2000, 1, 3500, 0], 4),  # clusters of 4, many waves
    ([12000], [9000], 5),                       # halves of rows, odd heads
    ([2100] * 60, [1100] * 60, 3),              # no clusters
])
def test_compact_of_many_waves(lens, keep, H, in_place):
    pool, table, dst, index, weights = _compact_case(lens, keep, H, True, sum(keep))
    got, w, status = _compact(pool, table, None if in_place else dst, index, weights, lens, keep, H)
    want, ww = evictref.compact(pool, table, table if in_place else dst, H, index, lens, keep, weights)
    assert status == 0 and np.array_equal(got, want) and np.array_equal(w, ww)


@pytest.mark.parametrize("shape", ["dense", "first", "last", "alternate"])
def test_compact_patterns_in_place(shape):
    # few holes, none, all rows moved far, every second row: the order of reads and writes
    n, H = 20011, 2
    keep = {"dense": n - 40, "first": 9000, "last": 9000, "alternate": n // 2}[shape]
    pool, table, _, index, weights = _compact_case([n], [keep], H, True, 11)
    rng = np.random.default_rng(1)
    for h in range(H):
        index[0, h, :keep] = {
            "dense": np.sort(rng.permutation(n)[:keep]), "first": np.arange(keep),
            "last": np.arange(n - keep, n), "alternate": np.arange(keep) * 2 + h}[shape]
    got, w, status = _compact(pool, table, None, index, weights, [n], [keep], H)
    want, ww = evictref.compact(pool, table, table, H, index, [n], [keep], weights)
    assert status == 0 and np.array_equal(got, want) and np.array_equal(w, ww)


def test_compact_skips_and_flags():
    k = kv()
    lens, keep = [700, 300], [256, 100]
    pool, table, dst, index, weights = _compact_case(lens, keep, 2, True, 5)
    # a bad old page, then a bad new one: their rows are skipped, the others move
    bad = table.copy()
    bad[0, 5] = pool.shape[0]
    got, w, status = _compact(pool, bad, dst, index, weights, lens, keep, 2)
    want, ww = evictref.compact(pool, table, dst, 2, index, lens, keep, weights)
    off = evictref.row_offsets(2)
    for h in range(2):
        for j in range(256):
            if index[0, h, j] // 64 == 5:
                at = (dst[0, j // 64], off[h, j % 64])
                want[at] = pool[at]
    assert status == k.DEV_BAD_PAGE and np.array_equal(got, want) and np.array_equal(w, ww)
    # an index outside the sequence
    wrong = index.copy()
    wrong[1, 1, 7] = 300
    got, w, status = _compact(pool, table, dst, wrong, weights, lens, keep, 2)
    want, ww = evictref.compact(pool, table, dst, 2, index, lens, keep, weights)
    at = (dst[1, 0], off[1, 7])
    want[at] = pool[at]
    ww[1, 1, 7] = weights[1, 1, 7]
    assert status == k.DEV_BAD_POS and np.array_equal(got, want) and np.array_equal(w, ww)
    # bad lengths: the sequence stays, the other moves
    for n2, m2 in ((-1, 5), (300, -2), (300, 258), (64 * table.shape[1] + 1, 5)):
        got, w, status = _compact(pool, table, dst, index, weights, [700, n2], [256, m2], 2)
        want, ww = evictref.compact(pool, table, dst, 2, index, [700], [256], weights)
        assert status == k.DEV_BAD_POS and np.array_equal(got, want) and np.array_equal(w, ww)


# ---- append at a slot --------------------------------------------------------------------------

@pytest.mark.parametrize("T", [3, 400])
def test_append_slots(T):
    import oracle
    k = kv()
    rng = np.random.default_rng(T)
    H, Hq, reach = 3, 6, 9000
    c = k.PagedNVFP4Cache(40, rng.permutation(40).reshape(2, 20).astype(np.int32), reach, Hq, H)
    bits = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    q, kk, v = bits(T, Hq, 128), bits(T, H, 128), bits(T, H, 128)
    seq = (np.arange(T) % 2).astype(np.int32)
    slots = (600 + np.arange(T) // 2).astype(np.int32)
    pos = (8000 + np.arange(T) // 2).astype(np.int32)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    c.pool.fill_(0x55)
    qc, qs = c.quantized_q_buffers(T)
    c.append(kk, v, dev(seq), dev(pos), q, qc, qs, slots=dev(slots))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    table = c.rope.cpu().numpy()[:reach * 32].reshape(reach, 32)
    raw = lambda x: x.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1, 128)  # noqa: E731
    qcr, qsr = oracle.quantize_rows(raw(q), np.repeat(pos, Hq), True, table, 32)
    kc, ks = oracle.quantize_rows(raw(kk), np.repeat(pos, H), True, table, 32)
    vc, vs = oracle.quantize_rows(raw(v), None, False, None, 0)
    assert np.array_equal(qc.cpu().numpy(), qcr.reshape(-1))
    assert np.array_equal(qs.cpu().numpy(), qsr.reshape(-1))
    want = np.full((40, 9216 * H), 0x55, np.uint8)
    rows = np.concatenate([kc, ks, vc, vs], -1).reshape(T, H, 144)
    off = evictref.row_offsets(H)
    bt = c.block_table.cpu().numpy()
    for t in range(T):
        want[bt[seq[t], slots[t] // 64]][off[:, slots[t] % 64].reshape(-1)] = rows[t].reshape(-1)
    assert np.array_equal(c.pool.cpu().numpy().reshape(want.shape), want)


def test_append_slots_flags():
    k = kv()
    c = k.PagedNVFP4Cache(4, np.arange(4, dtype=np.int32).reshape(1, 4), 100, 4, 2)
    x = torch.randn(4, 2, 128, device="cuda").bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for slots, pos, bit in (((0, 256, 1, 2), (0, 1, 2, 3), k.DEV_BAD_POS),
                            ((0, -1, 1, 2), (0, 1, 2, 3), k.DEV_BAD_POS),
                            ((0, 3, 1, 2), (0, -1, 2, 3), k.DEV_BAD_POS),
                            ((0, 3, 1, 2), (0, 100, 2, 3), k.DEV_BAD_ROPE)):
        c.status.zero_()
        c.append(x, x, i32(0, 0, 0, 0), i32(*pos), slots=i32(*slots))
        torch.cuda.synchronize()
        assert int(c.status.item()) == bit


def test_the_cache_checks_its_arguments():
    k = kv()
    c = k.PagedNVFP4Cache(4, np.arange(4, dtype=np.int32).reshape(2, 2), 100, 4, 2)
    w = c.weight_accounts()
    assert tuple(w.shape) == (2, 2, 128) and not w.any()
    i32 = torch.tensor([5, 5], dtype=torch.int32, device="cuda")
    index = torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda")
    c.plan([10, 10], 1)
    out = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    qc, qs = c.quantized_q_buffers(2)
    for bad in (w.half(), w[:, :1], w.cpu(), w.transpose(0, 1)[:, :1]):
        with pytest.raises(ValueError):
            c.attend_weights(qc, qs, out, bad)
        with pytest.raises(ValueError):
            c.evict(bad, i32, i32, index)
    for bad in (out.float(), out.transpose(0, 1)):
        with pytest.raises(ValueError):
            c.attend_weights(qc, qs, bad, w)
    with pytest.raises(ValueError):
        c.attend_weights(qc, qs, out, w, weights_in=w[..., :64].contiguous())
    for lens, keep, ix in ((i32.long(), i32, index), (i32, i32[:1], index), (i32.cpu(), i32, index),
                           (i32, i32, index.long()), (i32, i32, index[0]),
                           (i32, i32, torch.zeros(2, 3, 5, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            c.evict(w, lens, keep, ix)


def test_the_cache_refuses_other_devices_and_sizes(monkeypatch):
    k = kv()
    c = k.PagedNVFP4Cache(4, np.arange(4, dtype=np.int32).reshape(2, 2), 100, 4, 2)
    w = c.weight_accounts()
    i32 = torch.tensor([5, 5], dtype=torch.int32, device="cuda")
    index = torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    qc, qs = c.quantized_q_buffers(2)
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):  # no plan yet
        c.attend_weights(qc, qs, out, w)
    c.plan([10, 10], 1)
    for bad in (out.cpu(), out[:1]):
        with pytest.raises(ValueError):
            c.attend_weights(qc, qs, bad, w)
    with pytest.raises(ValueError):
        c.evict(w, i32, i32, index.cpu())
    for slots in (i32.long(), i32[:1], i32.cpu()):
        with pytest.raises(ValueError):
            c.append(x, x, i32, i32, slots=slots)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        c.attend_weights(qc, qs, out, w)
    with pytest.raises(ValueError):
        c.evict(w, i32, i32, index)
    with pytest.raises(ValueError):
        c.append(x, x, i32, i32, slots=i32)


def test_attend_weights_grows_its_workspace_on_the_stream_it_is_given():
    k = kv()
    c = k.PagedNVFP4Cache(32, np.arange(32, dtype=np.int32).reshape(2, 16), 1100, 4, 2)
    c.pool.zero_()
    w = c.weight_accounts()
    qc, qs = c.quantized_q_buffers(2)
    qc.zero_(), qs.zero_()  # scores of 0: every key of n gets 1 / n from each of the two rows
    out = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    for n, stream in ((64, side), (1024, side.cuda_stream), (1024, None)):
        c.plan([n, n], 1)
        w.zero_()
        torch.cuda.synchronize()
        c.attend_weights(qc, qs, out, w, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(w[..., :n], torch.full_like(w[..., :n], 2.0 / n))  # powers of two: exact
        assert not w[..., n:].any() and not out.any()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("q_len,Hq,Hkv", [(1, 24, 4), (1, 16, 8), (8, 24, 4)])
def test_offsets_beyond_32_bits(q_len, Hq, Hkv):
    # the same session in a pool of 5 GB, on its last pages, with accounts 600 M slots apart, and in a
    # small one: the same bits
    k = kv()
    gen = torch.Generator(device="cuda").manual_seed(q_len + Hkv)
    many = (5 << 30) // (9216 * Hkv)
    n, stride = 170, 600_000_000
    caches = [k.PagedNVFP4Cache(pages, [table], 512, Hq, Hkv) for pages, table in
              ((many, [many - 1, 2, many - 70]), (3, [0, 1, 2]))]
    rand = lambda *d: torch.randn(*d, device="cuda", generator=gen).bfloat16()  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kk, vv, q = rand(n, Hkv, 128), rand(n, Hkv, 128), rand(n, Hq, 128)
    k2, v2 = rand(1, Hkv, 128), rand(1, Hkv, 128)
    seen = []
    for c, apart in zip(caches, (stride, 192)):
        qc, qs = c.quantized_q_buffers(n)
        c.append(kk, vv, torch.zeros(n, dtype=torch.int32, device="cuda"),
                 torch.arange(n, dtype=torch.int32, device="cuda"), q, qc, qs)
        w = torch.empty(1, Hkv, apart, device="cuda")
        w[..., :192] = 0.25
        out = torch.empty(q_len, Hq, 128, dtype=torch.bfloat16, device="cuda")
        c.plan([n], q_len, True, 64)
        c.attend_weights(qc.view(n, -1)[-q_len:], qs.view(n, -1)[-q_len:], out, w)
        index = torch.zeros(1, Hkv, 100, dtype=torch.int32, device="cuda")
        before = w[..., :192].clone()
        c.evict(w, i32([n]), i32([100]), index, 4, 20)
        c.append(k2, v2, i32([0]), i32([n]), slots=i32([100]))
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        pages = c.pool.view(c.num_pages, -1)[c.block_table[0].long()].clone()
        # bytes behind the last token were never written
        pages[2, :] = 0
        seen.append((out, before, w[..., :192].clone(), index, pages))
        c.pool = w = None
    (out, before, w, index, pages), other = seen
    assert torch.equal(out, other[0]) and torch.equal(index, other[3])
    assert torch.equal(before, other[1]) and torch.equal(w, other[2])
    assert before[..., :n].sum() > 0.25 * n * Hkv  # weight was added
    assert torch.equal(pages, other[4])


# ---- together ----------------------------------------------------------------------------------

@pytest.mark.parametrize("per_head", [True, False])
def test_a_session_evicts_and_goes_on(per_head):
    """Decode steps that account for the weights, an eviction to a budget, further steps behind it:
    outputs and accounts against the 64-bit attention over the rows that should be there."""
    H, Hq, G = 4, 24, 6
    w = synth.Workload("session", [400, 90, 1500], q_len=1, seed=21, chunk_tokens=64)
    g = GpuRun(w)
    c, S = g.cache, 3
    c.max_pos = 2048  # positions go on behind the workload's own
    c.rope = torch.empty(2048 * c.rot_dim, device="cuda")
    kv().kv_nvfp4_rope_table_init(c.rope, c.max_pos, c.rot_dim, w.theta, w.pos_scale)
    g.step(chunk_tokens=64)
    accounts = c.weight_accounts()
    out = torch.empty(S, Hq, 128, dtype=torch.bfloat16, device="cuda")
    lens = [int(x) for x in w.seq_lens]
    ref = np.zeros(tuple(accounts.shape))
    slack = np.zeros(tuple(accounts.shape))
    positions = np.array(lens)  # of the next tokens
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    keep = torch.tensor([128, 100, 300], dtype=torch.int32, device="cuda")
    q = None
    for step in range(8):
        if step:  # a new token per sequence, behind what is held
            x = [torch.randn(S, n, 128, generator=gen, device="cuda").bfloat16() for n in (Hq, H, H)]
            i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
            c.append(x[1], x[2], i32([0, 1, 2]), i32(positions.tolist()), x[0], g.q_codes,
                     g.q_scales, slots=i32(lens))
            lens = [n + 1 for n in lens]
            positions += 1
            c.plan(lens, 1, True, 64)
        c.attend_weights(g.q_codes, g.q_scales, out, accounts)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        pool = c.pool.cpu().numpy().reshape(-1, 9216 * H)
        q = np.concatenate([g.q_codes.cpu().numpy().reshape(S, 1, Hq, 64),
                            g.q_scales.cpu().numpy().reshape(S, 1, Hq, 8)], -1)
        got = accounts.cpu().numpy().astype(np.float64)
        for s in range(S):
            rows = evictref.cache_rows(pool, w.block_table, H, s, np.arange(lens[s]))
            o, tol, ws, wtol = evictref.attend(evictref.values(q[s]), rows, G, 1, True,
                                               1 / math.sqrt(128))
            assert (np.abs(out[s].float().cpu().numpy() - o[0]) <= tol[0]).all()
            ref[s, :, :lens[s]] += ws
            slack[s, :, :lens[s]] += wtol + 2.0 ** -22 * ref[s, :, :lens[s]]
        assert (np.abs(got - ref) <= slack + 1e-30).all()
        if step in (2, 5):
            kept = [min(n, int(m)) for n, m in zip(lens, keep.tolist())]
            index = torch.full((S, H if per_head else 1, 300), -1, dtype=torch.int32, device="cuda")
            before = accounts.cpu().numpy()
            c.evict(accounts, torch.tensor(lens, dtype=torch.int32, device="cuda"), keep, index,
                    sink=4, recent=16)
            torch.cuda.synchronize()
            ix = index.cpu().numpy()
            for s in range(S):
                for i in range(ix.shape[1]):
                    x = before[s, i] if per_head else evictref.head_sum(before[s])
                    assert np.array_equal(ix[s, i, :kept[s]],
                                          evictref.select(x, lens[s], kept[s], 4, 16))
            full = np.broadcast_to(ix, (S, H, 300))
            want, _ = evictref.compact(pool, w.block_table, w.block_table, H, full, lens, kept, None)
            assert np.array_equal(c.pool.cpu().numpy().reshape(want.shape), want)
            for arr in (ref, slack):
                for s in range(S):
                    for h in range(H):
                        arr[s, h, :kept[s]] = arr[s, h, full[s, h, :kept[s]]]
                        arr[s, h, kept[s]:] = 0
            lens = kept
    assert int(c.status.item()) == 0
