"""The tree and page entry points' refusals before any CUDA call, and the references that the GPU tests
compare with (CPU)."""
import ctypes

import numpy as np
import pytest

import pagesref
import treeref

A = 1 << 20  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def _plan(kv, Hq=24, Hkv=4, lens=(100,), q_len=8, causal=False):
    L = kv.make_layout(Hq, Hkv)
    return L, kv.kv_nvfp4_plan_host(L, list(lens), q_len, causal, 64, 8)[0]


@pytest.mark.parametrize("change", [
    dict(parents=0), dict(lens=0), dict(mask=0), dict(n=0), dict(n=257), dict(num_seqs=-1),
    dict(seq_ids=0), dict(slots=0), dict(positions=0), dict(seq_ids=0, slots=0),
    dict(parents=A + 2), dict(mask=A + 1), dict(first_pos=A + 3), dict(slots=A + 2),
])
def test_tree_mask_refuses(kv, change):
    a = dict(parents=A, num_seqs=1, n=8, lens=A, first_pos=A, mask=A, seq_ids=A, slots=A, positions=A,
             status=None, stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_tree_mask(**a)


@pytest.mark.parametrize("change", [
    dict(workspace=0), dict(q_codes=0), dict(q_scales=0), dict(mask=0), dict(pool=0),
    dict(block_table=0), dict(out=0), dict(num_pages=0), dict(max_pages=0), dict(max_pages=1),
    dict(out=A + 8), dict(pool=A + 1), dict(mask=A + 2), dict(workspace=A + 8),
])
def test_tree_attn_refuses(kv, change):
    L, info = _plan(kv)
    a = dict(layout=L, plan=info, workspace=A, q_codes=A, q_scales=A, mask=A, sm_scale=0.0, pool=A,
             num_pages=4, block_table=A, max_pages=2, out=A, status=None, stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_tree_attn(**a)


@pytest.mark.parametrize("plan", [
    dict(causal=True), dict(q_len=257, lens=(300,)), dict(Hq=32, Hkv=8),
])
def test_tree_attn_refuses_a_foreign_plan(kv, plan):
    _, info = _plan(kv, **plan)
    L = kv.make_layout(24, 4)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_tree_attn(L, info, A, A, A, A, 0.0, A, 4, A, 9, A, None, 0)


@pytest.mark.parametrize("change", [
    dict(parents=0), dict(draft=0), dict(target=0), dict(expected=0), dict(next_token=0),
    dict(lens=0), dict(path=0), dict(count=0), dict(n=0), dict(n=257), dict(num_seqs=-1),
    dict(block_table=0), dict(max_pages=0), dict(num_pages=0), dict(pool=0), dict(pool=A + 8),
    dict(path=A + 2), dict(new_lens=A + 1), dict(draft=A + 2),
    dict(parents=0, draft=0, target=0, expected=0),                     # next, but no tree
    dict(parents=0, draft=0, target=0, expected=0, next_token=0, pool=0, block_table=0, max_pages=0,
         num_pages=0),                                                  # nothing to do
])
def test_tree_accept_refuses(kv, change):
    a = dict(layout=kv.make_layout(24, 4), parents=A, draft=A, target=A, expected=A, num_seqs=1, n=8,
             lens=A, block_table=A, max_pages=2, num_pages=4, pool=A, path=A, count=A, next_token=A,
             new_lens=A, status=None, stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_tree_accept(**a)


def _pages(kv, **change):
    a = dict(block_table=A, held=A, refs=A, free_list=A, free_count=A, workspace=A, num_seqs=2,
             max_pages=4, num_pages=8)
    a.update(change)
    return kv.Pages(*a.values())


@pytest.mark.parametrize("change", [
    *[{name: bad} for name in ("block_table", "held", "refs", "free_list", "free_count")
      for bad in (0, A + 2)],
    dict(workspace=0), dict(workspace=A + 4), dict(num_seqs=0), dict(num_seqs=8193),
    dict(max_pages=0), dict(num_pages=0), dict(num_seqs=8192, max_pages=1 << 18),
])
def test_accounts_are_checked(kv, change):
    p = _pages(kv, **change)
    for call in (lambda: kv.kv_nvfp4_pages_init(p, stream=0),
                 lambda: kv.kv_nvfp4_pages_fork(p, A, A, A, 1, None, 0),
                 lambda: kv.kv_nvfp4_pages_resize(p, A, A, A, None, 0)):
        with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
            call()


def test_page_calls_refuse(kv):
    p, L = _pages(kv), kv.make_layout(24, 4)
    for args in ((0, A, A, 1), (A, 0, A, 1), (A, A, 0, 1), (A + 2, A, A, 1), (A, A, A, -1),
                 (A, A, A, 3)):
        with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
            kv.kv_nvfp4_pages_fork(p, *args, None, 0)
    for args in ((0, A, A), (A, 0, A), (A, A, 0), (A, A + 1, A), (A, A, A + 2)):
        with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
            kv.kv_nvfp4_pages_resize(p, *args, None, 0)
    for args in ((0, 4, A, 1), (A, 0, A, 1), (A, 4, 0, 1), (A, 4, A, -1), (A + 8, 4, A, 1),
                 (A, 4, A + 2, 1)):
        with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
            kv.kv_nvfp4_copy_pages(L, *args, None, 0)
    assert kv.lib().kv_nvfp4_pages_init(None, None) == -1
    assert kv.lib().kv_nvfp4_pages_workspace_bytes(-1) == 0


def test_nothing_to_do(kv):
    L = kv.make_layout(24, 4)
    kv.kv_nvfp4_tree_mask(0, 0, 8, 0, 0, 0, stream=0)
    kv.kv_nvfp4_tree_accept(L, 0, 0, 0, 0, 0, 8, 0, 0, 0, 0, 0, 0, 0, 0, stream=0)
    kv.kv_nvfp4_pages_fork(_pages(kv), 0, 0, 0, 0, stream=0)
    kv.kv_nvfp4_copy_pages(L, 0, 0, 0, 0, stream=0)


def test_accounts_are_taken_from_int32_tensors(kv):
    torch = pytest.importorskip("torch")
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    good = dict(block_table=i32(2, 4), held=i32(2), refs=i32(8), free_list=i32(8), free_count=i32(1),
                workspace=torch.zeros(kv.kv_nvfp4_pages_workspace_bytes(8), dtype=torch.uint8))
    p = kv.make_pages(**good)
    assert (p.num_seqs, p.max_pages, p.num_pages) == (2, 4, 8)
    assert p.refs == good["refs"].data_ptr()
    for change in (dict(held=i32(3)), dict(refs=torch.zeros(8)), dict(free_list=i32(16)[::2]),
                   dict(free_count=i32(2)), dict(workspace=good["workspace"][1:]),
                   dict(block_table=torch.zeros(2, 4, dtype=torch.int64)),
                   dict(held=i32(2).to("meta"))):
        with pytest.raises(ValueError, match="accounts"):
            kv.make_pages(**{**good, **change})


# ---- the references themselves -------------------------------------------------------------

def test_reference_masks_and_walks():
    #        0         4     padding 5, and 6 below it
    #      1   2       |
    #      |
    #      3
    parents = np.array([-1, 0, 0, 1, -1, 9, 5], np.int32)
    words, depth = treeref.mask_words(parents)
    assert words[:, 0].tolist() == [1, 3, 5, 11, 16, 0, 0]
    assert depth.tolist() == [0, 1, 1, 2, 0, 0, 0]
    draft = [7, 8, 8, 9, 7, 7, 7]
    assert treeref.walk(parents, draft, [8, 9, 1, 5, 1, 1, 1], 7) == ([0, 1, 3], 5)
    assert treeref.walk(parents, draft, [8, 1, 9, 5, 1, 1, 1], 7) == ([0, 1], 1)  # the lower sibling
    assert treeref.walk(parents, draft, [8] * 7, 3) == ([], 3)
    sees = np.array([[r is not None and r[j] for j in range(7)] for r in treeref.ancestors(parents)])
    assert np.array_equal(treeref.words_of(sees), words)


def test_reference_accounts():
    a = pagesref.Accounts.empty(3, 4, 6)
    assert (a.resize([0, 0, 0], [130, 0, 64]) == -1).all()
    a.check()
    assert a.table.tolist() == [[0, 1, 2, -1], [-1] * 4, [3, -1, -1, -1]] and a.count == 2
    a.fork([0], [1], [100])
    a.check()
    assert a.table[1].tolist() == [0, 1, -1, -1] and a.refs.tolist() == [2, 2, 1, 1, 0, 0]
    # both write behind token 100: page 1 is shared, so each gets a page, and page 1 falls free
    copies = a.resize([100, 100, 64], [101, 101, 64])
    a.check()
    assert copies.tolist() == [[1, 4], [1, 5], [-1, -1]]
    assert a.table[:2, :2].tolist() == [[0, 4], [0, 5]] and a.free[:a.count].tolist() == [2, 1]
    a.resize([101, 101, 64], [101, 256, 128])  # two pages more, and one: two are free
    a.check()
    assert a.no_page and a.held.tolist() == [2, 4, 1] and a.table[1].tolist() == [0, 5, 1, 2]
    a.resize([0, 256, 64], [0, 256, 64])
    a.check()
    assert a.free[:a.count].tolist() == [4] and a.refs[0] == 1
