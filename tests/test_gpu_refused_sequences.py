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
