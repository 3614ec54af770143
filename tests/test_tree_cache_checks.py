"""What PagedNVFP4Cache refuses of trees and page accounts before any launch, with the launches replaced
by a record (CPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def calls(monkeypatch):
    """The library calls that come through, in the place of launches; memory on the CPU."""
    import contextlib

    import bit_kv_cache_03_gb300.cache as cache
    seen = []
    for name in ("kv_nvfp4_tree_mask", "kv_nvfp4_tree_attn", "kv_nvfp4_tree_accept",
                 "kv_nvfp4_pages_init", "kv_nvfp4_pages_fork", "kv_nvfp4_pages_resize",
                 "kv_nvfp4_copy_pages"):
        monkeypatch.setattr(cache, name, lambda *a, name=name: seen.append(name))
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_check_current", lambda self: None)
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_hold_captured", lambda self, stream: None)
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_on", staticmethod(lambda s: contextlib.nullcontext()))
    return seen


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _cache(num_seqs=2):
    import bit_kv_cache_03_gb300 as kv
    return kv.PagedNVFP4Cache(2 * num_seqs, np.full((num_seqs, 2), -1, np.int32), 1, 4, 2, rot_dim=0,
                              device="cpu")


def test_tree_mask(calls):
    c = _cache()
    b = c.tree_buffers(33)
    assert [tuple(x.shape) for x in b] == [(2, 33, 2), (66,), (66,), (66,)]
    c.tree_mask(i32(2, 33), i32(2), b)
    c.tree_mask(i32(2, 33), i32(2), b, first_pos=i32(2))
    assert calls == ["kv_nvfp4_tree_mask"] * 2
    good = dict(parents=i32(2, 33), lens=i32(2), buffers=b, first_pos=i32(2))
    for change in (dict(parents=i32(3, 33)), dict(parents=i32(66)), dict(parents=i32(2, 32)),
                   dict(parents=i32(2, 257)), dict(parents=i32(2, 33).long()),
                   dict(parents=i32(33, 2).T), dict(lens=i32(3)), dict(lens=i32(2).to("meta")),
                   dict(first_pos=i32(1)), dict(buffers=c.tree_buffers(32)),
                   dict(buffers=(b[0], b[1], b[2].long(), b[3]))):
        with pytest.raises(ValueError):
            c.tree_mask(**{**good, **change})
    for n in (0, 257):
        with pytest.raises(ValueError):
            c.tree_buffers(n)
    assert len(calls) == 2


def test_attend_tree(calls):
    import bit_kv_cache_03_gb300 as kv
    c = _cache()
    q, s = c.quantized_q_buffers(2 * 3)
    out = torch.empty(6, 4, 128, dtype=torch.bfloat16)
    mask = c.tree_buffers(3)[0]
    with pytest.raises(ValueError, match="plan"):
        c.attend_tree(q, s, out, mask)
    for causal, lens in ((True, [10, 10]), (False, [10, 10, 10])):
        c.plan_info = kv.kv_nvfp4_plan_host(c.layout, lens, 3, causal, 64, 8)[0]
        with pytest.raises(ValueError, match="plan"):
            c.attend_tree(q, s, out, mask)
    c.plan_info = kv.kv_nvfp4_plan_host(c.layout, [10, 10], 3, False, 64, 8)[0]
    c.workspace = torch.empty(1, dtype=torch.uint8)
    c.attend_tree(q, s, out, mask)
    assert calls == ["kv_nvfp4_tree_attn"]
    for a in ((q[:-1], s, out, mask), (q, s[:-1], out, mask), (q, s, out[:-1], mask),
              (q, s, out.float(), mask), (q, s, out, mask[:1]), (q, s, out, mask.long()),
              (q, s, out.to("meta"), mask)):
        with pytest.raises(ValueError):
            c.attend_tree(*a)
    assert len(calls) == 1


def test_tree_accept(calls):
    c = _cache()
    good = dict(parents=i32(2, 5), draft=i32(2, 5), target=i32(2, 5), expected=i32(2), lens=i32(2),
                path=i32(2, 5), count=i32(2), next_token=i32(2), new_lens=i32(2))
    c.tree_accept(**good)
    c.tree_accept(None, None, None, None, i32(2), i32(2, 5), i32(2), None)
    assert calls == ["kv_nvfp4_tree_accept"] * 2
    for change in (dict(parents=i32(2, 4)), dict(draft=i32(5)), dict(target=i32(2, 5).long()),
                   dict(expected=i32(3)), dict(lens=None), dict(path=i32(10)), dict(path=i32(1, 5)),
                   dict(count=None), dict(next_token=i32(1)), dict(new_lens=i32(2).to("meta"))):
        with pytest.raises(ValueError):
            c.tree_accept(**{**good, **change})
    assert len(calls) == 2


def test_accounts(calls):
    c = _cache(3)
    with pytest.raises(ValueError, match="accounts"):
        c.resize(i32(3), i32(3))
    with pytest.raises(ValueError, match="accounts"):
        c.fork(i32(1), i32(1), i32(1))
    p = c.page_accounts()
    assert (p.num_seqs, p.max_pages, p.num_pages) == (3, 2, 6)
    assert p.block_table == c.block_table.data_ptr()
    c.resize(i32(3), i32(3))
    c.resize(i32(3), i32(3), copy=False)
    c.fork(i32(2), i32(2), i32(2))
    assert calls == ["kv_nvfp4_pages_init", "kv_nvfp4_pages_resize", "kv_nvfp4_copy_pages",
                     "kv_nvfp4_pages_resize", "kv_nvfp4_pages_fork"]
    for a in ((i32(2), i32(3)), (i32(3), i32(3).long()), (i32(3), i32(6)[::2])):
        with pytest.raises(ValueError):
            c.resize(*a)
    for a in ((i32(1), i32(2), i32(2)), (i32(2), i32(2), i32(2).long()), (i32(4), i32(4), i32(4))):
        with pytest.raises(ValueError):
            c.fork(*a)
    assert len(calls) == 5


def test_accounts_are_emptied_in_place(calls):
    c = _cache(3)
    p, copies = c.page_accounts(), c.copies
    assert c.page_accounts() is p and c.copies is copies  # what a captured resize works on
    assert calls == ["kv_nvfp4_pages_init"] * 2


def test_accounts_are_of_the_table_in_use(calls):
    a, b = _cache(3), _cache(3)
    p = a.page_accounts()
    b.block_table = a.block_table  # another layer's pool under the same table
    a.resize(i32(3), i32(3))
    a.block_table = b.block_table.clone()
    for call in (lambda: a.resize(i32(3), i32(3)), lambda: a.fork(i32(1), i32(1), i32(1))):
        with pytest.raises(ValueError, match="block table"):
            call()
    assert a.page_accounts() is not p and a.pages.block_table == a.block_table.data_ptr()
