"""What is left alone in a step with trees for a sequence that one of its calls refuses: its cache, and
every page that it shares."""
import numpy as np
import pytest

import treeref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def dev(x, dtype=torch.int32):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device="cuda")


def bf16(rng, *shape):
    return torch.tensor(rng.standard_normal(shape), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 3])
@pytest.mark.parametrize("by", ["length", "position"])
def test_a_refused_mask_appends_nothing(bad, by):
    """The step behind one whose buffers it uses: slots of the refused sequence that were the last
    step's nodes, accepted in the meantime, keep their rows."""
    k, rng = kv(), np.random.default_rng(0)
    S, n, Hq, H = 3, 5, 8, 4
    c = k.PagedNVFP4Cache(6, np.arange(6, dtype=np.int32).reshape(S, 2), 200, Hq, H, 32)
    c.pool.fill_(0x31)
    parents = dev(np.stack([treeref.random_tree(rng, n) for _ in range(S)]))
    buffers = c.tree_buffers(n)
    mask, seq_ids, slots, positions = buffers
    q_codes, q_scales = c.quantized_q_buffers(S * n)
    x = [bf16(rng, S * n, h, 128) for h in (Hq, H, H)]

    def step(lens, first):
        c.tree_mask(parents, dev(lens), buffers, first_pos=dev(first))
        c.append(x[1], x[2], seq_ids, positions, q=x[0], q_codes=q_codes, q_scales=q_scales, slots=slots)

    step([20, 60, 7], [20, 61, 9])
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    before, old_mask = c.pool.clone(), mask.clone()
    x = [bf16(rng, S * n, h, 128) for h in (Hq, H, H)]
    lens, first = [22, 62, 10], [30, 63, 12]
    (lens if by == "length" else first)[1] = bad
    step(lens, first)
    torch.cuda.synchronize()
    assert int(c.status.item()) == k.DEV_BAD_POS | k.DEV_BAD_SEQ
    got = c.pool.clone()
    for t in (seq_ids, slots, positions):
        t = t.view(S, n)
        assert (t[1] == -1).all() and (t[[0, 2]] >= 0).all()
    assert torch.equal(mask[1], old_mask[1])
    # the same with the other two sequences' tokens alone
    c.pool.copy_(before)
    at = torch.cat([torch.arange(n), torch.arange(2 * n, 3 * n)]).cuda()
    c.append(x[1][at], x[2][at], seq_ids[at], positions[at], slots=slots[at])
    assert torch.equal(got, c.pool)
    assert torch.equal(got.view(3, 2, -1)[1], before.view(3, 2, -1)[1])
    assert not torch.equal(got, before)


def test_a_refused_tree_has_no_accepted_nodes():
    """The count of a tree that is not walked is 0, not the last step's, which a further layer's call
    would move rows by."""
    import evictref
    k, rng = kv(), np.random.default_rng(1)
    S, n, H = 4, 6, 2
    held = [50, 60, 70, 10]
    cache = treeref.Cache([h + n for h in held], H, 7)
    P = cache.table.shape[1]
    lens = np.array([50, -1, P * 64 - n + 1, 10], np.int32)
    parents = np.tile(np.array([-1, -1, 1, 2, 3, 4], np.int32), (S, 1))
    ones = np.ones((S, n), np.int32)
    ones[:, 0] = 2  # not the awaited token: the path is 1, 2, 3, 4, 5
    path = dev(np.tile(np.array([1, 2, 4, 0, 0, 0]), (S, 1)))
    count, nxt, new = dev([3] * S), dev([-7] * S), dev([-7] * S)
    layout, status = k.make_layout(H, H, rot_dim=0), dev([0])
    args = (S, n, dev(lens), dev(cache.table), P, cache.num_pages)
    pool, other = dev(cache.pool, torch.uint8), dev(cache.pool, torch.uint8)
    k.kv_nvfp4_tree_accept(layout, dev(parents), dev(ones), dev(ones), dev([1] * S), *args, pool, path,
                           count, nxt, new, status)
    assert int(status.item()) == k.DEV_BAD_POS
    assert count.tolist() == [5, 0, 0, 5]
    assert nxt.tolist() == [1, -7, -7, 1] and new.tolist() == [55, -7, -7, 15]
    assert path[1:3].tolist() == [[1, 2, 4, 0, 0, 0]] * 2
    want, off = cache.pool.copy(), evictref.row_offsets(H)
    for s in (0, 3):
        treeref.move(cache.pool, want, cache.table[s], off, [1, 2, 3, 4, 5], held[s])
    # a further layer, with lengths that name the sequences' tokens again
    again = (S, n, dev(held), *args[3:])
    k.kv_nvfp4_tree_accept(layout, None, None, None, None, *again, other, path, count, None, None, status)
    for got in (pool, other):
        assert np.array_equal(got.cpu().numpy(), want)


def _served(ref, keep, room):
    """keep, or -1 for a sequence that a resize of these accounts must refuse, from the header's words."""
    S, P = ref.table.shape
    out, demand = [], 0
    for s in range(S):
        k, r, h = int(keep[s]), int(room[s]), int(ref.held[s])
        need = (r + 63) // 64
        if k < 0 or r < k or need > P or (k + 63) // 64 > h:
            out.append(-1)
            continue
        fresh = max(0, need - h) + sum(ref.refs[ref.table[s, j]] > 1 for j in range(k // 64, min(h, need)))
        demand += fresh
        out.append(k if fresh == 0 or demand <= ref.count else -1)
    return out


@pytest.mark.parametrize("S,P,N", [(5, 20, 40), (40, 20, 300), (16, 300, 3000), (16, 300, 1500),
                                   (16, 3000, 60000), (2000, 3, 3000)])
def test_a_resize_says_whom_it_refused(S, P, N):
    from test_gpu_pages import Both
    k, rng = kv(), np.random.default_rng(S + P)
    b = Both(S, P, N)
    kept = torch.full((S + 1,), 77, dtype=torch.int32, device="cuda")
    refused = 0
    for step in range(6):
        keep = np.where(rng.random(S) < 0.5, b.ref.held * 64, rng.integers(0, b.ref.held * 64 + 1))
        room = np.minimum(keep + rng.integers(0, P * 64, S) * (rng.random(S) < 0.6), P * 64)
        odd = rng.random(S) < 0.1
        keep[odd], room[odd] = rng.choice([-1, 2 ** 31 - 1, 5]), rng.choice([-5, 4, P * 64 + 1])
        if step % 2:  # sequences that share, some of them to be written
            free, full = np.flatnonzero(b.ref.held == 0), np.flatnonzero(b.ref.held > 0)
            if len(free) and len(full):
                b.fork(rng.choice(full, len(free)).tolist(), free.tolist(), np.full(len(free), 64))
                keep[free], room[free] = rng.integers(0, 65, len(free)), 100
        want = _served(b.ref, keep, room)
        k.kv_nvfp4_pages_resize(b.pages, dev(keep), dev(room), b.copies, b.status, kept=kept[:S])
        b.ref.resize(keep, room)
        b.same()
        assert kept.tolist() == want + [77]
        refused += sum(w < 0 <= x for w, x in zip(want, keep))
        if step == 3:  # room again
            b.resize(np.zeros(S, int), np.where(np.arange(S) % 2, 0, 64))
    assert refused and (b.ref.no_page or S * P < 2 * N)  # (pages enough, for some of the cases)


@pytest.mark.parametrize("Hq,H,n", [(8, 4, 2), (24, 4, 9), (10, 5, 70)])
@pytest.mark.parametrize("resized", [True, False], ids=["refused", "not asked"])
def test_shared_pages_outlive_an_exhausted_pool(Hq, H, n, resized):
    """A sequence and its forks at 70 and at 100 of its 100 tokens, with too few free pages for all of
    their trees (or no resize at all): the step's other calls leave the pages that several hold as they
    are, in a further layer too, and the served sequence's tree is the only one to be accepted."""
    import evictref
    from test_gpu_tree_session import Sessions
    k = kv()
    # room for the parent's own copy of the shared page and its tree, none for the others
    t = Sessions(3, 8, 2 + 1 + (100 + n + 63) // 64 - 2, Hq, H, seed=n)
    c, S = t.c, 3
    t.resize([0, 0, 0], [100, 0, 0])
    t.prompt(0, 100)
    t.fork([0, 0], [1, 2], [70, 100])
    t.check()
    layer = k.PagedNVFP4Cache(c.num_pages, np.zeros((3, 8), np.int32), 600, Hq, H, 32)
    layer.block_table = c.block_table
    layer.pool.copy_(c.pool)
    lens = [100, 70, 100]
    if resized:
        c.resize(dev(lens), dev([x + n for x in lens]), copy=False)
        for pool in (c.pool, layer.pool):
            k.kv_nvfp4_copy_pages(c.layout, pool, c.num_pages, c.copies, S, c.status)
        assert c.kept.tolist() == [100, -1, -1] and int(c.status.item()) == k.DEV_NO_PAGE
    served = [0] if resized else []
    c.status.zero_()
    before = [x.pool.clone() for x in (c, layer)]
    parents = dev(np.tile(np.arange(n) - 1, (S, 1)))
    buffers = c.tree_buffers(n)
    mask, seq_ids, slots, positions = buffers
    for x in (seq_ids, slots, positions):
        x.zero_()  # what a step before may have left
    c.tree_mask(parents, dev(lens), buffers)
    assert seq_ids.view(S, n)[:, 0].tolist() == [s if s in served else -1 for s in range(S)]
    q, kk, v = (t.bf16(S * n, h, 128) for h in (Hq, H, H))
    q_codes, q_scales = c.quantized_q_buffers(S * n)
    for x in (c, layer):
        x.append(kk, v, seq_ids, positions, q=q, q_codes=q_codes, q_scales=q_scales, slots=slots)
    c.plan([x + n for x in lens], n, causal=False, chunk_tokens=64)
    out = torch.empty(S * n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    c.attend_tree(q_codes, q_scales, out, mask)
    tokens = dev(np.ones((S, n)))
    path, count, nxt, new = dev(np.zeros((S, n))), dev([n] * S), dev([9] * S), dev([9] * S)
    c.tree_accept(parents, tokens, tokens, dev([1] * S), dev(lens), path, count, nxt, new)
    layer.tree_accept(None, None, None, None, dev(lens), path, count, None)
    torch.cuda.synchronize()
    assert count.tolist() == [n if s in served else 0 for s in range(S)]
    assert nxt.tolist() == [1] * S
    assert new.tolist() == [x + (n if s in served else 0) for s, x in enumerate(lens)]
    want = k.DEV_SHARED_PAGE | k.DEV_BAD_SEQ | k.DEV_BAD_POS
    # (a refused sequence without room: attention misses pages of its plan)
    assert int(c.status.item()) & ~k.DEV_BAD_PAGE == want
    table = c.block_table.cpu().numpy()
    for x, old in zip((c, layer), before):
        pool = x.pool.cpu().numpy().reshape(-1, 9216 * H)
        old = old.cpu().numpy().reshape(-1, 9216 * H)
        for s in range(S):
            at = np.arange(lens[s])
            assert np.array_equal(evictref.cache_rows(pool, table, H, s, at),
                                  evictref.cache_rows(old, table, H, s, at)), s
        own = table[served][table[served] >= 0]
        others = np.setdiff1d(np.arange(len(pool)), own)
        assert np.array_equal(pool[others], old[others])
        assert (not np.array_equal(pool, old)) == bool(served)
    # plain tokens, at the position and at a slot
    before = c.pool.clone()
    c.status.zero_()
    ids, pos = dev([1, 2]), dev([70, 100])
    c.append(kk[:2], v[:2], ids, pos)
    c.append(kk[:2], v[:2], ids, dev([71, 101]), slots=pos)
    layer.pages = c.pages
    layer.append(kk[:2], v[:2], ids, pos)
    torch.cuda.synchronize()
    assert int(c.status.item()) == k.DEV_SHARED_PAGE and torch.equal(c.pool, before)
    assert int(layer.status.item()) & k.DEV_SHARED_PAGE
    if not served:
        return
    # one of the two holders ends: the other's page is its own
    c.resize(dev([100 + n, 0, 100]), dev([100 + n, 0, 100]))
    c.resize(dev([100 + n, 0, 100]), dev([100 + n, 0, 101]))
    assert c.kept.tolist() == [100 + n, 0, 100]
    c.status.zero_()
    c.append(kk[1:2], v[1:2], dev([2]), dev([100]))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0 and not torch.equal(c.pool, before)


@pytest.mark.parametrize("T", [1, 700])
def test_appends_beside_refused_rows(T):
    """Rows of the same call into pages of their own: as written without accounts, by both append
    kernels (few rows, many)."""
    k, rng = kv(), np.random.default_rng(T)
    Hq, H, S = 24, 4, 3
    c = k.PagedNVFP4Cache(40, np.zeros((S, 12), np.int32), 1000, Hq, H, 32)
    c.page_accounts()
    c.pool.fill_(0x22)
    c.resize(dev([0] * S), dev([64 * 12, 64 * 12, 0]))
    c.fork(dev([0]), dev([2]), dev([64 * 3]))
    seq = dev(np.sort(rng.integers(0, S, T)) if T > 1 else [1])
    pos = dev(np.concatenate([np.arange((seq == s).sum().item()) for s in range(S)]))
    q, kk, v = (bf16(rng, T, h, 128) for h in (Hq, H, H))
    codes, scales = c.quantized_q_buffers(T)
    c.append(kk, v, seq, pos, q=q, q_codes=codes, q_scales=scales)
    bad = (seq != 1) & (pos < 192)  # the shared pages
    missing = (seq == 2) & (pos >= 192)
    want = k.PagedNVFP4Cache(40, c.block_table.cpu().numpy(), 1000, Hq, H, 32)
    want.pool.fill_(0x22)
    codes2, scales2 = want.quantized_q_buffers(T)
    good = ~bad
    want.append(kk[good], v[good], seq[good], pos[good])
    all_q = k.PagedNVFP4Cache(40, c.block_table.cpu().numpy(), 1000, Hq, H, 32)
    all_q.append(kk, v, seq, pos, q=q, q_codes=codes2, q_scales=scales2)
    torch.cuda.synchronize()
    assert torch.equal(c.pool, want.pool)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)
    assert int(c.status.item()) == (k.DEV_SHARED_PAGE * bool(bad.any())
                                    | k.DEV_BAD_PAGE * bool(missing.any()))


@pytest.mark.parametrize("Hq,H,q_len", [(24, 4, 1), (8, 4, 3), (3, 3, 1)])
def test_a_decode_step_beside_a_refused_sequence(Hq, H, q_len):
    """The fused step of forked sequences that got no page of their own: the shared page stays, the other
    sequences' rows and outputs are those of a step without it."""
    k, rng = kv(), np.random.default_rng(Hq)
    S, P, lens = 4, 4, [100, 100, 100, 30]
    c = k.PagedNVFP4Cache(4, np.zeros((S, P), np.int32), 300, Hq, H, 32)
    c.page_accounts()
    c.pool.copy_(torch.tensor(rng.integers(0x20, 0x40, c.pool.numel(), dtype=np.uint8)))
    c.resize(dev([0] * S), dev([100, 0, 0, 30]))
    c.fork(dev([0, 0]), dev([1, 2]), dev([100, 100]))
    c.resize(dev(lens), dev([x + q_len for x in lens]))
    assert c.kept.tolist() == [100, -1, -1, 30]
    c.status.zero_()
    before, table = c.pool.clone(), c.block_table.clone()
    q, kk, v = (bf16(rng, S * q_len, h, 128) for h in (Hq, H, H))
    c.plan([x + q_len for x in lens], q_len, chunk_tokens=64)
    out = torch.empty(S * q_len, Hq, 128, device="cuda")
    c.decode_step(q, kk, v, out)
    torch.cuda.synchronize()
    assert int(c.status.item()) == k.DEV_SHARED_PAGE
    # the same without the refused ones
    at = torch.cat([torch.arange(q_len), torch.arange(3 * q_len, 4 * q_len)]).cuda()
    want = k.PagedNVFP4Cache(4, table[[0, 3]].cpu().numpy(), 300, Hq, H, 32)
    want.pool.copy_(before)
    want.plan([lens[0] + q_len, lens[3] + q_len], q_len, chunk_tokens=64)
    out2 = torch.empty(2 * q_len, Hq, 128, device="cuda")
    want.decode_step(q[at], kk[at], v[at], out2)
    torch.cuda.synchronize()
    assert int(want.status.item()) == 0
    assert torch.equal(c.pool, want.pool) and not torch.equal(c.pool, before)
    # (another plan may split a sequence elsewhere: P is rounded to f16 about another maximum, half a
    # step of 2^-11 on either side, and |V| is at most 6 times a scale of 1.875)
    assert torch.allclose(out[at], out2, rtol=0, atol=2.0 ** -10 * 11.25 + 2.0 ** -12)
    # one of them ends, the other is served: as without accounts (the ended one has no pages)
    c.resize(dev([100, 0, 100, 30]), dev([100, 0, 100, 30]))
    lens = [100 + q_len, 64, 100 + q_len, 30 + q_len]
    c.resize(dev([100, 0, 100, 30]), dev([100 + q_len, 0, 100 + q_len, 30 + q_len]))
    assert c.kept.tolist() == [100, 0, 100, 30]
    c.status.zero_()
    c.plan(lens, q_len, chunk_tokens=64)
    want = k.PagedNVFP4Cache(4, c.block_table.cpu().numpy(), 300, Hq, H, 32)
    want.pool.copy_(c.pool)
    want.plan(lens, q_len, chunk_tokens=64)
    out.zero_()
    out3 = torch.zeros_like(out)
    c.decode_step(q, kk, v, out)
    want.decode_step(q, kk, v, out3)
    torch.cuda.synchronize()
    assert int(c.status.item()) == int(want.status.item()) == k.DEV_BAD_PAGE
    assert torch.equal(c.pool, want.pool) and torch.equal(out, out3)
