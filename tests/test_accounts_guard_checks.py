"""Calls that are given the page accounts: what they refuse before any CUDA call, and which calls of
PagedNVFP4Cache hand its accounts on (CPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
A = 1 << 20  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def _pages(kv, **change):
    a = dict(block_table=A, held=A, refs=A, free_list=A, free_count=A, workspace=A, num_seqs=2,
             max_pages=4, num_pages=8)
    a.update(change)
    return kv.Pages(*a.values())


@pytest.mark.parametrize("change", [dict(refs=0), dict(block_table=A + 2), dict(num_seqs=1),
                                    dict(num_pages=0)])
def test_foreign_accounts_are_refused(kv, change):
    p, L = _pages(kv, **change), kv.make_layout(24, 4)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_tree_mask(A, 2, 8, A, None, A, A, A, A, None, 0, pages=p)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_tree_accept(L, A, A, A, A, 2, 8, A, A, 4, 8, A, A, A, A, A, None, 0, pages=p)


@pytest.mark.parametrize("change", [
    dict(pages="bad"), dict(k=0), dict(v=0), dict(seq_ids=0), dict(positions=0), dict(pool=0),
    dict(k=A + 2), dict(v=A + 8), dict(pool=A + 8), dict(T=-1), dict(q=A), dict(rope_table=0),
    dict(rope_max_pos=0),
])
def test_pages_append_refuses(kv, change):
    a = dict(layout=kv.make_layout(24, 4), pages=_pages(kv), q=None, k=A, v=A, seq_ids=A, slots=None,
             positions=A, T=3, rope_table=A, rope_max_pos=10, pool=A, status=None, stream=0)
    a.update(change)
    if a["pages"] == "bad":
        a["pages"] = _pages(kv, refs=0)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_pages_append(**a)


def test_pages_append_of_nothing(kv):
    kv.kv_nvfp4_pages_append(kv.make_layout(24, 4), _pages(kv), None, 0, 0, 0, 0, 0, 0, 0, 0, 0, stream=0)


@pytest.mark.parametrize("change", [
    dict(refs=0), dict(workspace=0), dict(q=0), dict(k=0), dict(v=0), dict(pool=0), dict(out=0),
    dict(rope=0), dict(rope_max_pos=0), dict(max_pages=1), dict(num_seqs=1), dict(q_codes_out=A),
    dict(out=A + 8), dict(heads=(32, 8)), dict(q_len=2),
])
def test_pages_decode_step_refuses(kv, change):
    change = dict(change)
    pages = _pages(kv, **{x: change.pop(x) for x in ("refs", "max_pages", "num_seqs") if x in change})
    L = kv.make_layout(*change.pop("heads", (24, 4)))
    plan = kv.kv_nvfp4_plan_host(L, [100, 70], change.pop("q_len", 1), True, 64, 8)[0]
    a = dict(layout=L, pages=pages, plan=plan, workspace=A, q=A, k=A, v=A, rope=A, rope_max_pos=200,
             pool=A, q_codes_out=None, q_scales_out=None, sm_scale=0.0, out=A, status=None, stream=0)
    a.update(change)
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_pages_decode_step(**a)


@pytest.mark.parametrize("kept", [A + 2, A, A + 64])
def test_resize_refuses_a_result_that_is_unaligned_or_an_input(kv, kept):
    with pytest.raises(kv.KVNVFP4Error, match=r"\(-1\)"):
        kv.kv_nvfp4_pages_resize(_pages(kv), A, A + 64, A + 128, None, 0, kept=kept)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_the_cache_hands_its_accounts_on(kv, monkeypatch):
    import contextlib

    import bit_kv_cache_03_gb300.cache as cache
    seen = []
    for name in ("append", "append_slots", "pages_append", "tree_mask", "tree_accept", "pages_init",
                 "pages_resize", "copy_pages", "decode_step", "pages_decode_step"):
        monkeypatch.setattr(cache, "kv_nvfp4_" + name, lambda *a, name=name: seen.append((name, a)))
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_check_current", lambda self: None)
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_hold_captured", lambda self, stream: None)
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_on", staticmethod(lambda s: contextlib.nullcontext()))

    def make(pages=6):
        return kv.PagedNVFP4Cache(pages, np.full((3, 2), -1, np.int32), 1, 4, 2, rot_dim=0, device="cpu")

    def calls(c):
        del seen[:]
        k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
        c.append(k, k, i32(3), i32(3))
        c.append(k, k, i32(3), i32(3), slots=i32(3))
        c.tree_mask(i32(3, 5), i32(3), c.tree_buffers(5))
        c.tree_accept(None, None, None, None, i32(3), i32(3, 5), i32(3), None)
        c.decode_step(k, k, k, k)
        return [name for name, _ in seen], [any(x is c.pages for x in a) for _, a in seen]

    without = ["append", "append_slots", "tree_mask", "tree_accept", "decode_step"]
    c, layer = make(), make()
    assert calls(c)[0] == without
    c.page_accounts()
    with_accounts = (["pages_append"] * 2 + ["tree_mask", "tree_accept", "pages_decode_step"], [True] * 5)
    assert calls(c) == with_accounts
    del seen[:]
    c.resize(i32(3), i32(3))
    assert seen[0][0] == "pages_resize" and seen[0][1][-1] is c.kept and c.kept.tolist() == [0] * 3
    layer.block_table = c.block_table  # a further layer without the accounts, and with them
    assert calls(layer)[0] == without
    layer.pages = c.pages
    assert calls(layer) == with_accounts
    c.block_table = c.block_table.clone()  # no longer the accounts' table
    assert calls(c)[0][0] == "append" and not any(calls(c)[1])
    fewer = make(5)
    fewer.block_table, fewer.pages = layer.block_table, layer.pages
    with pytest.raises(ValueError, match="accounts"):
        calls(fewer)
