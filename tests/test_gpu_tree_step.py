"""A whole step with drafted trees: behind an eviction, where a token's slot is not its position, and
captured as one graph."""
import numpy as np
import pytest

import evictref
import treeref
from test_gpu_tree_session import Sessions, dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,H,n,per_head", [(8, 4, 2, True), (24, 4, 9, False), (10, 5, 40, True)])
def test_a_tree_behind_an_eviction(Hq, H, n, per_head):
    import bit_kv_cache_03_gb300 as kv
    lens, keep = [200, 70, 130], [90, 70, 63]
    S = len(lens)
    t = Sessions(S, 6, 18, Hq, H, seed=n)
    t.resize([0] * S, [x + 64 for x in lens])
    for s, x in enumerate(lens):
        t.prompt(s, x)
    c, rng = t.c, t.rng
    weights = c.weight_accounts()
    weights.copy_(torch.tensor(rng.random(weights.shape), dtype=torch.float32))
    index = torch.zeros(S, H if per_head else 1, 100, dtype=torch.int32, device="cuda")
    c.evict(weights, dev(lens), dev(keep), index, sink=4, recent=8)
    pool = lambda: c.pool.cpu().numpy().reshape(-1, 9216 * H)  # noqa: E731
    table = c.block_table.cpu().numpy()
    old = [evictref.cache_rows(pool(), table, H, s, np.arange(m)) for s, m in enumerate(keep)]
    for s, m in enumerate(keep):  # the kept rows, of each head's own slots
        for h in range(H):
            assert np.array_equal(old[s][:, h], t.rows[s][index[s, h if per_head else 0, :m].cpu(), h])

    parents = np.stack([treeref.random_tree(rng, n, 0.1) for _ in range(S)])
    buffers = c.tree_buffers(n)
    mask, seq_ids, slots, positions = buffers
    c.tree_mask(dev(parents), dev(keep), buffers, first_pos=dev(lens))
    q, k, v = (t.bf16(S * n, x, 128) for x in (Hq, H, H))
    q_codes, q_scales = c.quantized_q_buffers(S * n)
    c.append(k, v, seq_ids, positions, q=q, q_codes=q_codes, q_scales=q_scales, slots=slots)
    c.plan([m + n for m in keep], n, causal=False, chunk_tokens=64)
    out = torch.empty(S * n, Hq, 128, dtype=torch.bfloat16, device="cuda")
    c.attend_tree(q_codes, q_scales, out, mask)
    draft, target = rng.integers(0, 2, (2, S, n))
    expected = rng.integers(0, 2, S)
    path = torch.zeros(S, n, dtype=torch.int32, device="cuda")
    count, nxt, new = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(3))
    c.tree_accept(dev(parents), dev(draft), dev(target), dev(expected), dev(keep), path, count, nxt, new)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    depth = np.concatenate([lens[s] + treeref.mask_words(parents[s])[1] for s in range(S)])
    nodes = np.concatenate([t.encode(k, depth), t.encode(v, None)], -1).reshape(S, n, H, 144)
    qv = evictref.values(t.encode(q, depth)).reshape(S, n, Hq, 128)
    got = out.float().cpu().numpy().astype(np.float64).reshape(S, n, Hq, 128)
    for s in range(S):
        sees = np.array([np.zeros(n, bool) if r is None else r for r in treeref.ancestors(parents[s])])
        ref, tol = treeref.attend(qv[s], np.concatenate([old[s], nodes[s]]), Hq // H, sees,
                                  1 / np.sqrt(128))
        assert (np.abs(got[s] - ref) <= tol).all(), s
        taken, token = treeref.walk(parents[s], draft[s], target[s], expected[s])
        assert path[s, :len(taken)].tolist() == taken and int(nxt[s]) == token
        assert int(new[s]) == keep[s] + len(taken)
        rows = evictref.cache_rows(pool(), table, H, s, np.arange(int(new[s])))
        assert np.array_equal(rows, np.concatenate([old[s], nodes[s][taken]]))


@pytest.mark.parametrize("Hq,H,n", [(8, 4, 2), (24, 4, 9), (24, 4, 40), (16, 8, 5)])
def test_a_step_as_one_graph(Hq, H, n):
    """Room, masks, append, attention and the accepted path captured together and replayed on new
    inputs, at the lengths of its plan: every output and the cache as from the same calls one by one."""
    import bit_kv_cache_03_gb300 as kv
    held, steps = [150, 64, 0, 700], 4
    S, P, N = len(held), 16, 60
    rng = np.random.default_rng(n)
    prompt = [torch.tensor(rng.standard_normal((sum(held), H, 128)), dtype=torch.bfloat16, device="cuda")
              for _ in range(2)]
    seq = dev(np.repeat(np.arange(S), held))
    pos = dev(np.concatenate([np.arange(h) for h in held]))
    inputs = []
    for _ in range(steps):
        draft, target = rng.integers(0, 2, (2, S, n))
        inputs.append([dev(np.stack([treeref.random_tree(rng, n, 0.1) for _ in range(S)])), dev(draft),
                       dev(target), dev(rng.integers(0, 2, S))]
                      + [torch.tensor(rng.standard_normal((S * n, h, 128)), dtype=torch.bfloat16,
                                      device="cuda") for h in (Hq, H, H)])

    def run(captured):
        c = kv.PagedNVFP4Cache(N, np.zeros((S, P), np.int32), 2000, Hq, H, 32)
        c.page_accounts()
        c.pool.zero_()
        lens, room = dev(held), dev([h + n for h in held])
        c.resize(dev([0] * S), lens)
        c.append(*prompt, seq, pos)
        c.plan([h + n for h in held], n, causal=False, chunk_tokens=64)
        buffers = c.tree_buffers(n)
        mask, seq_ids, slots, positions = buffers
        q_codes, q_scales = c.quantized_q_buffers(S * n)
        x = [torch.empty_like(a) for a in inputs[0]]
        parents, draft, target, expected, q, k, v = x
        out = torch.empty(S * n, Hq, 128, dtype=torch.bfloat16, device="cuda")
        path = torch.full((S, n), -1, dtype=torch.int32, device="cuda")
        count, nxt, new = (dev([0] * S) for _ in range(3))

        def step():
            c.resize(lens, room)
            c.tree_mask(parents, lens, buffers)
            c.append(k, v, seq_ids, positions, q=q, q_codes=q_codes, q_scales=q_scales, slots=slots)
            c.attend_tree(q_codes, q_scales, out, mask)
            c.tree_accept(parents, draft, target, expected, lens, path, count, nxt, new)
            c.resize(new, new)
            c.resize(lens, lens)

        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
                step()
        results = []
        for a in inputs:
            for to, value in zip(x, a):
                to.copy_(value)
            path.fill_(-1)
            graph.replay() if captured else step()
            results += [y.clone() for y in (out, path, count, nxt, new, c.block_table, c.pool, mask,
                                            c.kept)]
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        return results

    for i, (a, b) in enumerate(zip(run(False), run(True))):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
