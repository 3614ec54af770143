"""The eviction entry points' sizes and refusals, before any CUDA call, and the references that
the GPU tests compare with (CPU)."""
import ctypes

import numpy as np
import pytest

import evictref
import oracle


@pytest.fixture(scope="module")
def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def _plan(kv, Hq, Hkv, lens, q_len, chunk=64, ctas=8):
    L = kv.make_layout(Hq, Hkv)
    return L, kv.kv_nvfp4_plan_host(L, lens, q_len, True, chunk, ctas)[0]


@pytest.mark.parametrize("Hq,Hkv,lens,q_len", [(24, 4, [100, 900], 1), (24, 4, [5000], 8),
                                              (32, 8, [70, 3000], 1), (3, 3, [64], 64)])
def test_weights_workspace_holds_statistics_and_row_sums(kv, Hq, Hkv, lens, q_len):
    L, info = _plan(kv, Hq, Hkv, lens, q_len)
    need = kv.kv_nvfp4_weights_workspace_bytes(L, info)
    rows = len(lens) * q_len * Hq
    assert need >= 8 * rows
    if Hq // Hkv * q_len > 8 or Hkv > 4:
        assert need >= 8 * rows + 512 * info.num_partials


def test_weights_workspace_refuses_a_foreign_plan(kv):
    L, info = _plan(kv, 24, 4, [100], 1)
    for other in (kv.make_layout(24, 8), kv.make_layout(48, 4)):
        with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
            kv.kv_nvfp4_weights_workspace_bytes(other, info)
    n = ctypes.c_size_t()
    f = kv.lib().kv_nvfp4_weights_workspace_bytes
    assert f(ctypes.byref(L), None, ctypes.byref(n)) == -1
    assert f(ctypes.byref(L), ctypes.byref(info), None) == -1


A = 1 << 20  # a 16-byte aligned address that is never read


@pytest.mark.parametrize("change", [
    dict(workspace=0), dict(weights_workspace=0), dict(q_codes=0), dict(q_scales=0), dict(pool=0),
    dict(block_table=0), dict(out=0), dict(weights_out=0), dict(num_pages=0), dict(max_pages=0),
    dict(max_pages=1), dict(weights_stride=99), dict(out=A + 8), dict(pool=A + 1),
    dict(weights_workspace=A + 4), dict(weights_out=A + 2), dict(weights_in=A + 1),
])
def test_attend_weights_refuses(kv, change):
    L, info = _plan(kv, 24, 4, [100], 1)
    a = dict(layout=L, plan=info, workspace=A, weights_workspace=A, ww_bytes=1 << 20, q_codes=A,
             q_scales=A, sm_scale=0.0, pool=A, num_pages=4, block_table=A, max_pages=2, out=A,
             weights_in=None, weights_out=A, weights_stride=128, status=None, stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_decode_attn_weights(**a)


def test_attend_weights_refuses_a_small_workspace(kv):
    L, info = _plan(kv, 24, 4, [100], 1)
    need = kv.kv_nvfp4_weights_workspace_bytes(L, info)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-3\)"):
        kv.kv_nvfp4_decode_attn_weights(L, info, A, A, need - 1, A, A, 0.0, A, 4, A, 2, A, None, A,
                                        128, None, 0)


@pytest.mark.parametrize("change", [
    dict(weights=0), dict(seq_lens=0), dict(keep=0), dict(index=0), dict(weights_stride=0),
    dict(index_stride=0), dict(sink=-1), dict(recent=-1), dict(num_seqs=-1),
    dict(weights=A + 2), dict(index=A + 1), dict(keep=A + 3),
])
def test_select_refuses(kv, change):
    a = dict(layout=kv.make_layout(24, 4), weights=A, weights_stride=64, seq_lens=A, keep=A,
             num_seqs=1, per_head=True, sink=0, recent=0, index=A, index_stride=8, status=None,
             stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_evict_select(**a)


@pytest.mark.parametrize("change", [
    dict(index=0), dict(seq_lens=0), dict(keep=0), dict(block_table=0), dict(pool=0),
    dict(pool=A + 8), dict(index_stride=0), dict(max_pages=0), dict(num_pages=0),
    dict(num_seqs=-1), dict(dst_max_pages=2), dict(dst_block_table=A), dict(weights=A),
    dict(index=A + 2), dict(weights=A + 2, weights_stride=64),
])
def test_compact_refuses(kv, change):
    a = dict(layout=kv.make_layout(24, 4), index=A, index_stride=8, per_head=True, seq_lens=A,
             keep=A, num_seqs=1, block_table=A, max_pages=2, num_pages=4, pool=A, status=None,
             stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_evict_compact(**a)


def test_append_slots_refuses(kv):
    L = kv.make_layout(24, 4)
    good = [L, None, A, A, A, A, A, 1, A, 64, A, 1, 1, 4, A]
    for at, bad in ((4, 0), (5, 0), (6, 0), (7, -1), (14, A + 8), (9, 0)):
        a = list(good)
        a[at] = bad
        with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
            kv.kv_nvfp4_append_slots(*a, stream=0)


def test_no_sequences_and_no_tokens_do_nothing(kv):
    L = kv.make_layout(24, 4)
    kv.kv_nvfp4_evict_select(L, 0, 0, 0, 0, 0, True, 0, 0, 0, 0, stream=0)
    kv.kv_nvfp4_evict_compact(L, 0, 0, True, 0, 0, 0, 0, 0, 0, 0, stream=0)
    kv.kv_nvfp4_append_slots(L, None, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 1, 1, 0, stream=0)


# ---- the references themselves -------------------------------------------------------------

def test_row_offsets_cover_a_page_once_and_match_the_oracle():
    for H in (1, 2, 3, 4):
        off = evictref.row_offsets(H)
        assert np.array_equal(np.sort(off.reshape(-1)), np.arange(9216 * H))
        rng = np.random.default_rng(H)
        pool = rng.integers(0, 256, (3, 9216 * H), dtype=np.uint8)
        table = np.array([[2, 0]], np.int32)
        kc, ks, vc, vs, bad = oracle.paged_gather(pool.reshape(-1), 3, H, table, 0, 0, 128)
        rows = evictref.cache_rows(pool, table, H, 0, np.arange(128))
        assert bad == 0 and np.array_equal(rows, np.concatenate([kc, ks, vc, vs], -1))


def test_reference_select_orders_protected_then_weight_then_slot():
    w = np.array([0, 5, np.nan, 5, -np.inf, 1, -0.0, 7], np.float32)
    assert evictref.select(w, 8, 3, 0, 0).tolist() == [1, 3, 7]
    assert evictref.select(w, 8, 2, 0, 0).tolist() == [1, 7]
    assert evictref.select(w, 8, 5, 0, 0).tolist() == [0, 1, 3, 5, 7]  # 0 before -0 by slot
    assert evictref.select(w, 8, 7, 0, 0).tolist() == [0, 1, 3, 4, 5, 6, 7]  # NaN last
    assert evictref.select(w, 8, 4, 1, 2).tolist() == [0, 1, 6, 7]
    assert evictref.select(w, 8, 2, 1, 2).tolist() == [0, 6]
    assert evictref.select(w, 5, 9, 0, 0).tolist() == [0, 1, 2, 3, 4]
