"""Corners of the eviction calls' contract: which protected slots a small budget keeps, and what the
calls write outside their own buffers' contents."""
import numpy as np
import pytest

import evictref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


@pytest.mark.parametrize("lens,keep,sink,recent,want", [
    ([6], [2], 0, 4, [2, 3]),       # the newest two of the last four go, whatever their weights
    ([6], [3], 1, 4, [0, 2, 3]),
    ([6], [5], 1, 4, [0, 2, 3, 4, 5]),
    ([6], [1], 9, 9, [0]),
    ([2000], [512], 4, 1024, [0, 1, 2, 3, *range(976, 1484)]),
])
@pytest.mark.parametrize("per_head", [True, False])
def test_protected_slots_rank_by_slot_alone(lens, keep, sink, recent, want, per_head):
    k = kv()
    w = np.zeros((1, 2, max(lens)), np.float32)
    w[..., :] = np.resize([1, 9, 2, 8, 3, 7], max(lens)) + np.arange(max(lens))  # later ones weigh more
    index = torch.full((1, 2 if per_head else 1, keep[0]), -7, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kv_nvfp4_evict_select(k.make_layout(2, 2), torch.from_numpy(w).cuda(), w.shape[2], dev(lens),
                            dev(keep), 1, per_head, sink, recent, index, keep[0], status)
    assert int(status.item()) == 0
    for row in index[0].cpu().numpy():
        assert row.tolist() == want
        assert row.tolist() == evictref.select(w[0, 0], lens[0], keep[0], sink, recent).tolist()


@pytest.mark.parametrize("lens,q_len,chunk,Hq,Hkv", [
    ([5, 64, 1500], 1, 64, 24, 4),     # at most 8 rows: stored scores
    ([300, 40], 2, 64, 9, 3),
    ([63, 2100], 1, 128, 32, 8),       # more than four KV heads
    ([700, 90], 2, 128, 40, 5),
    ([2000, 37], 8, 256, 24, 4),       # the weight pass
    ([900, 64], 60, 128, 8, 2),
    ([1, 300], 9, 128, 8, 8),
])
def test_the_workspaces_old_bytes_do_not_matter_and_nothing_is_written_behind_them(lens, q_len, chunk,
                                                                                  Hq, Hkv):
    import synth
    from kvrun import GpuRun
    k = kv()
    w = synth.Workload("poison", lens, q_len=q_len, seed=11, q_heads=Hq, kv_heads=Hkv,
                       chunk_tokens=chunk)
    g = GpuRun(w)
    g.step(chunk_tokens=chunk)
    c = g.cache
    need, plan = k.kv_nvfp4_weights_workspace_bytes(c.layout, c.plan_info), c.plan_info
    guard, size = 8192, plan.workspace_bytes
    first = torch.empty(size + guard, dtype=torch.uint8, device="cuda")
    second = torch.empty(need + guard, dtype=torch.uint8, device="cuda")
    seen = []
    for byte in (0, 0xFF, 0x7F, 0x3C):  # zeros, NaN, large and ordinary values
        first.fill_(byte), second.fill_(byte)
        first[:plan.off_partials] = c.workspace[:plan.off_partials]
        out = torch.zeros(g.T, Hq, 128, dtype=torch.bfloat16, device="cuda")
        acc = torch.full((len(lens), Hkv, c.max_pages * 64), 0.25, device="cuda")
        k.kv_nvfp4_decode_attn_weights(
            c.layout, plan, first, second, need, g.q_codes, g.q_scales, w.sm_scale, c.pool,
            c.num_pages, c.block_table, c.max_pages, out, acc, acc, acc.shape[2], c.status)
        torch.cuda.synchronize()
        assert (first[size:] == byte).all() and (second[need:] == byte).all()
        assert torch.equal(first[:plan.off_partials], c.workspace[:plan.off_partials])
        seen.append((out, acc))
    assert g.status() == 0
    for out, acc in seen[1:]:
        assert torch.equal(out.view(torch.int16), seen[0][0].view(torch.int16))
        assert torch.equal(acc.view(torch.int32), seen[0][1].view(torch.int32))
