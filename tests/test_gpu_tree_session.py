"""Sessions that branch and draft trees, through PagedNVFP4Cache: accounts, forks, masks, appends,
attention and accepted paths together, against a plain model of the same sessions."""
import numpy as np
import pytest

import evictref
import oracle
import pagesref
import treeref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROT, MAX_POS = 32, 600


def dev(x, dtype=torch.int32):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device="cuda")


class Sessions:
    """Rows [len, H, 144] that each sequence's cache must hold, and the calls that put them there."""

    def __init__(self, S, P, N, Hq, H, seed):
        import bit_kv_cache_03_gb300 as kv
        self.S, self.Hq, self.H = S, Hq, H
        self.rng = np.random.default_rng(seed)
        self.c = kv.PagedNVFP4Cache(N, np.zeros((S, P), np.int32), MAX_POS, Hq, H, ROT)
        self.c.page_accounts()
        self.ref = pagesref.Accounts.empty(S, P, N)
        self.rope = oracle.rope_table(MAX_POS, ROT, 1e7, 1.0)
        self.rows = [np.zeros((0, H, 144), np.uint8) for _ in range(S)]

    def bf16(self, *shape):
        return torch.tensor(self.rng.standard_normal(shape), dtype=torch.bfloat16, device="cuda")

    def encode(self, x, positions):
        """Rows [T, heads, 72] of bf16 rows; positions None: V, without RoPE and rotation."""
        bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
        T, heads = bits.shape[:2]
        if positions is None:
            c, s = oracle.quantize_rows(bits.reshape(-1, 128), None, False, None, 0, 0)
        else:
            pos = np.repeat(np.asarray(positions, np.int32), heads)
            c, s = oracle.quantize_rows(bits.reshape(-1, 128), pos, True, self.rope, ROT, 0)
        return np.concatenate([c.reshape(T, heads, 64), s.reshape(T, heads, 8)], -1)

    def lens(self):
        return [len(r) for r in self.rows]

    def resize(self, keep, room):
        self.c.resize(dev(keep), dev(room))
        copies = self.ref.resize(keep, room)
        assert np.array_equal(self.c.copies.cpu().numpy(), copies)
        self.ref.check()

    def fork(self, src, dst, lens):
        self.c.fork(dev(src), dev(dst), dev(lens))
        self.ref.fork(src, dst, lens)
        for a, b, n in zip(src, dst, lens):
            self.rows[b] = self.rows[a][:n].copy()

    def prompt(self, s, n):
        """n tokens behind what sequence s has."""
        k, v = self.bf16(n, self.H, 128), self.bf16(n, self.H, 128)
        pos = len(self.rows[s]) + np.arange(n)
        self.c.append(k, v, dev(np.full(n, s)), dev(pos))
        new = np.concatenate([self.encode(k, pos), self.encode(v, None)], -1)
        self.rows[s] = np.concatenate([self.rows[s], new])

    def check(self):
        torch.cuda.synchronize()
        assert int(self.c.status.item()) == 0
        pool = self.c.pool.cpu().numpy().reshape(-1, 9216 * self.H)
        table = self.c.block_table.cpu().numpy()
        assert np.array_equal(table, self.ref.table)
        for s, rows in enumerate(self.rows):
            if len(rows):
                got = evictref.cache_rows(pool, table, self.H, s, np.arange(len(rows)))
                assert np.array_equal(got, rows), s

    def step(self, n, vocab):
        """One drafted tree of n nodes per sequence; returns the accepted counts."""
        c, S, rng = self.c, self.S, self.rng
        lens = self.lens()
        self.resize(lens, [x + n for x in lens])
        parents = np.stack([treeref.random_tree(rng, n, 0.1) for _ in range(S)])
        buffers = c.tree_buffers(n)
        c.tree_mask(dev(parents), dev(lens), buffers)
        mask, seq_ids, slots, positions = buffers
        q, k, v = (self.bf16(S * n, x, 128) for x in (self.Hq, self.H, self.H))
        q_codes, q_scales = c.quantized_q_buffers(S * n)
        c.append(k, v, seq_ids, positions, q=q, q_codes=q_codes, q_scales=q_scales, slots=slots)
        c.plan([x + n for x in lens], n, causal=False, chunk_tokens=64)
        out = torch.empty(S * n, self.Hq, 128, dtype=torch.bfloat16, device="cuda")
        c.attend_tree(q_codes, q_scales, out, mask)
        draft, target = rng.integers(0, vocab, (2, S, n))
        expected = rng.integers(0, vocab, S)
        path = torch.zeros(S, n, dtype=torch.int32, device="cuda")
        count, nxt, new = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(3))
        c.tree_accept(dev(parents), dev(draft), dev(target), dev(expected), dev(lens), path, count, nxt,
                      new)
        # the same on the plain model
        depth = np.concatenate([lens[s] + treeref.mask_words(parents[s])[1] for s in range(S)])
        nodes = np.concatenate([self.encode(k, depth), self.encode(v, None)], -1).reshape(
            S, n, self.H, 144)
        qv = evictref.values(self.encode(q, depth)).reshape(S, n, self.Hq, 128)
        got = out.float().cpu().numpy().astype(np.float64).reshape(S, n, self.Hq, 128)
        for s in range(S):
            sees = np.array([np.zeros(n, bool) if r is None else r
                             for r in treeref.ancestors(parents[s])])
            rows = np.concatenate([self.rows[s], nodes[s]])
            ref, tol = treeref.attend(qv[s], rows, self.Hq // self.H, sees, 1 / np.sqrt(128))
            assert (np.abs(got[s] - ref) <= tol).all(), s
            taken, token = treeref.walk(parents[s], draft[s], target[s], expected[s])
            assert path[s, :len(taken)].tolist() == taken and int(nxt[s]) == token
            self.rows[s] = np.concatenate([self.rows[s], nodes[s][taken]])
        assert new.tolist() == self.lens()
        self.check()
        return count.tolist()


@pytest.mark.parametrize("Hq,H,n", [(6, 2, 9), (2, 2, 3), (24, 4, 12), (10, 5, 70)])
def test_sessions(Hq, H, n):
    t = Sessions(5, 8, 40, Hq, H, seed=n)
    t.resize([0] * 5, [100, 37, 0, 0, 0])
    t.prompt(0, 100)
    t.prompt(1, 37)
    t.check()
    t.fork([0, 1, 0], [2, 3, 4], [100, 20, 64])  # whole, a part of a page, whole pages
    t.check()
    total = 0
    for _ in range(3):
        total += sum(t.step(n, 2))
    assert total > 5  # paths were taken, so that rows moved
    # one session ends, another is cut back into what it shares with others and goes on
    keep = t.lens()
    keep[0], keep[4] = 0, 30
    t.rows[0], t.rows[4] = t.rows[0][:0], t.rows[4][:30]
    t.resize(keep, keep)
    t.check()
    t.fork([4], [0], [30])
    t.step(n, 2)
    lens = t.lens()
    t.resize(lens, lens)
    t.check()
    t.resize([0] * 5, [0] * 5)
    assert t.ref.count == 40


def test_layers_share_accounts():
    """One cache's accounts, another layer's pool of as many pages under the same table: the pages that a
    resize replaces are copied in both."""
    import bit_kv_cache_03_gb300 as kv
    a = Sessions(2, 4, 12, 4, 2, seed=1)
    a.resize([0, 0], [70, 0])
    a.prompt(0, 70)
    other = torch.randint(0, 256, a.c.pool.shape, dtype=torch.uint8, device="cuda")
    before = other.clone().view(12, -1)
    a.fork([0], [1], [70])
    a.c.resize(dev([70, 70]), dev([71, 71]), copy=False)
    copies = a.ref.resize([70, 70], [71, 71])
    for pool in (a.c.pool, other):
        kv.kv_nvfp4_copy_pages(a.c.layout, pool, 12, a.c.copies, 2, a.c.status)
    a.check()
    assert (copies >= 0).all()
    for src, dst in copies:
        assert torch.equal(other.view(12, -1)[dst], before[src])


@pytest.mark.parametrize("Hq,H,n", [(8, 4, 2), (24, 4, 8), (24, 4, 40)])
def test_a_chain_of_calls_needs_no_waits(Hq, H, n):
    """The same steps with and without a wait behind every call: every kernel is launched while those
    before it run, and must not read what they have yet to write."""
    import bit_kv_cache_03_gb300 as kv
    S, P, N, steps = 6, 40, 300, 12
    rng = np.random.default_rng(n)
    held = [700, 65, 2000, 0, 129, 1500]
    parents = [dev(np.stack([treeref.random_tree(rng, n, 0.1) for _ in range(S)])) for _ in range(steps)]
    paths = [dev(np.stack([np.sort(rng.permutation(n)) for _ in range(S)])) for _ in range(steps)]
    counts = [dev(rng.integers(0, n + 1, S)) for _ in range(steps)]
    x = [[torch.tensor(rng.standard_normal((S * n, h, 128)), dtype=torch.bfloat16, device="cuda")
          for h in (Hq, H, H)] for _ in range(steps)]
    prompt = [torch.tensor(rng.standard_normal((sum(held), H, 128)), dtype=torch.bfloat16, device="cuda")
              for _ in range(2)]
    seq = dev(np.repeat(np.arange(S), held))
    pos = dev(np.concatenate([np.arange(h) for h in held]))
    lens, none, room, less = dev(held), dev([0] * S), dev([h + n for h in held]), dev(
        [h // 2 for h in held])

    def run(wait):
        def done():
            if wait:
                torch.cuda.synchronize()
        c = kv.PagedNVFP4Cache(N, np.zeros((S, P), np.int32), 4096, Hq, H, ROT)
        c.page_accounts()
        c.pool.zero_()  # pages taken anew have slots that were never written
        c.resize(none, lens)
        c.append(*prompt, seq, pos)
        c.resize(less, less)
        c.plan([h + n for h in held], n, causal=False, chunk_tokens=128)
        buffers = c.tree_buffers(n)
        mask, seq_ids, slots, positions = buffers
        q_codes, q_scales = c.quantized_q_buffers(S * n)
        outs = [torch.empty(S * n, Hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
        news = [torch.empty(S, dtype=torch.int32, device="cuda") for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            c.resize(lens if i % 3 else less, room)  # what the step before left
            done()
            c.tree_mask(parents[i], lens, buffers)
            done()
            q, k, v = x[i]
            c.append(k, v, seq_ids, positions, q=q, q_codes=q_codes, q_scales=q_scales, slots=slots)
            done()
            c.attend_tree(q_codes, q_scales, outs[i], mask)
            done()
            c.tree_accept(None, None, None, None, lens, paths[i], counts[i], None, news[i])
            done()
            if i % 3 == 2:  # pages freed and taken anew, in another order
                c.resize(less, less)
                done()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        return outs + news + [c.block_table, c.pool]

    # (rows of fresh pages are what their last holder left: the same in both runs)
    for i, (a, b) in enumerate(zip(run(True), run(False))):
        same = bool(torch.equal(a.view(torch.uint8), b.view(torch.uint8)))
        assert same, i
