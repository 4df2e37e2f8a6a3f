"""The C-ABI of include/df11_search.h: exported symbols, the binding's names and
what the host-side checks refuse.  No GPU work is started here; the pointers
handed in are never followed."""
import ctypes
import os
import re

import pytest

import huffman_decode_block_amd as hdb
from conftest import ROOT
from test_step_abi import BAD_CACHES, cache

P = 1 << 20  # an aligned address that only the host-side checks see
BAD, SMALL = hdb.DF11_E_INVALID_ARG, hdb.DF11_E_BUFFER_TOO_SMALL


def test_every_declared_symbol_is_exported_and_bound():
    src = open(os.path.join(ROOT, "include", "df11_search.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(df11_[a-z0-9_]+)\s*\(", src)))
    lib = ctypes.CDLL(hdb.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
        assert callable(getattr(hdb, n)), n
        assert n in hdb.__all__, n
    assert sorted(hdb.SEARCH_EXPORTS) == names


def tree(**change):
    a = dict(q=P, q_batch_stride=8192, q_node_stride=1024, q_head_stride=128, mask=P, mask_batch_stride=5, mask_node_stride=1,
             counts=None, starts=None, starts_batch_stride=0, starts_node_stride=0, batch=2, nodes=5, q_heads=8, scale=1.0)
    a.update(change)
    return hdb.search.df11_tree(**a)


def attend(c=None, t=None, table=P, ts=4, width=4, lens=P, out=P, lse=P, ws=None, size=0):
    return hdb.lib().df11_paged_tree_attention(ctypes.byref(c or cache()), ctypes.byref(t or tree()), table, ts, width, lens, out, lse,
                                               ws, size, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_refusals(change, status):
    assert attend(cache(**change)) == status


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=P + 1), dict(mask=P + 4), dict(counts=P + 2), dict(starts=P + 1), dict(q_heads=0), dict(q_heads=12),
    dict(q_heads=1 << 21), dict(nodes=(1 << 20) + 1), dict(batch=(1 << 24) + 1), dict(nodes=65), dict(q_batch_stride=1 << 41),
    dict(q_node_stride=1 << 48), dict(q_head_stride=1 << 46), dict(mask_batch_stride=1 << 41), dict(mask_node_stride=0),
    dict(starts=P, starts_batch_stride=1 << 41), dict(starts=P, starts_node_stride=1 << 48), dict(nodes=1 << 20, q_node_stride=1 << 30, mask=None),
    dict(batch=1 << 15, q_batch_stride=1 << 33), dict(batch=1 << 20, q_heads=128, mask=None), dict(batch=1 << 24, q_heads=8, nodes=1, mask=None),
    dict(batch=1 << 10, nodes=1 << 19, mask=None, q_batch_stride=0, q_node_stride=0),
])
def test_tree_refusals(change):
    assert attend(t=tree(**change), ws=P, size=1 << 62) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(table=None), BAD), (dict(table=P + 2), BAD), (dict(lens=None), BAD), (dict(lens=P + 1), BAD), (dict(out=None), BAD),
    (dict(out=P + 8), BAD), (dict(lse=P + 2), BAD), (dict(width=0), BAD), (dict(ts=3), BAD), (dict(width=1 << 26, ts=1 << 26), BAD),
    (dict(ts=1 << 41), BAD), (dict(width=4096, ts=4096), SMALL), (dict(width=4096, ts=4096, ws=P + 4, size=1 << 40), BAD),
    (dict(width=4096, ts=4096, ws=None, size=1 << 40), BAD),
])
def test_tree_call_refusals(change, status):
    assert attend(**change) == status


def test_null_structures():
    L, c = hdb.lib(), cache()
    assert L.df11_paged_tree_attention(None, ctypes.byref(tree()), P, 4, 4, P, P, P, None, 0, None) == BAD
    assert L.df11_paged_tree_attention(ctypes.byref(c), None, P, 4, 4, P, P, P, None, 0, None) == BAD
    assert L.df11_paged_copy(None, 1, 0, 0, P, P, P, 1, None) == BAD
    assert L.df11_paged_compact(None, 1, 0, 0, P, 1, P, P, 4, 4, P, 1, None) == BAD


def test_empty_calls_need_no_pointers():
    L, c = hdb.lib(), ctypes.byref(cache())
    for t in (tree(batch=0, q=None, mask=None), tree(nodes=0, q=None, mask=None)):
        assert L.df11_paged_tree_attention(c, ctypes.byref(t), None, 4, 4, None, None, None, None, 0, None) == hdb.DF11_OK
    assert L.df11_paged_copy(c, 1, 0, 0, None, None, None, 0, None) == hdb.DF11_OK
    assert L.df11_paged_compact(c, 1, 0, 0, None, 3, None, None, 4, 4, None, 0, None) == hdb.DF11_OK
    assert L.df11_paged_compact(c, 1, 0, 0, None, 0, None, None, 4, 4, None, 3, None) == hdb.DF11_OK
    assert L.df11_beam_select(None, 0, 0, 4, 100, 400, 100, None, None, 4, 0, None, None, None, None, 0, None) == hdb.DF11_OK


PAGES = [(change, status) for change, status in BAD_CACHES if change != dict(dtype=hdb.DF11_CACHE_E4M3)]  # scales are not looked at


@pytest.mark.parametrize("change,status", PAGES + [
    (dict(n_pages=1 << 30, k_page_stride=1 << 18), BAD), (dict(kv_heads=1 << 16, v_head_stride=1 << 32), BAD)])
def test_pages_refusals(change, status):
    c = ctypes.byref(cache(**change))
    assert hdb.lib().df11_paged_copy(c, 1, 0, 0, P, P, P, 1, None) == status
    assert hdb.lib().df11_paged_compact(c, 1, 0, 0, P, 1, P, P, 4, 4, P, 1, None) == status


@pytest.mark.parametrize("change", [
    dict(layers=0), dict(layers=65536), dict(kl=4), dict(vl=12), dict(kl=1 << 41), dict(layers=65535, vl=1 << 33), dict(src=None), dict(dst=None),
    dict(src=P + 1), dict(dst=P + 2), dict(rows=P + 3), dict(n=1 << 31), dict(n=(1 << 31) - 1), dict(layers=60000, n=60000),
])
def test_copy_refusals(change):
    a = dict(layers=2, kl=1 << 20, vl=1 << 20, src=P, dst=P, rows=P, n=3)
    a.update(change)
    assert hdb.lib().df11_paged_copy(ctypes.byref(cache()), a["layers"], a["kl"], a["vl"], a["src"], a["dst"], a["rows"], a["n"], None) == BAD


@pytest.mark.parametrize("change", [
    dict(layers=0), dict(kl=4), dict(path=None), dict(path=P + 2), dict(accepted=None), dict(accepted=P + 1), dict(table=None), dict(table=P + 1),
    dict(lens=None), dict(lens=P + 2), dict(depth=1025), dict(width=0), dict(ts=3), dict(width=1 << 28, ts=1 << 28), dict(ts=1 << 41),
    dict(batch=1 << 31), dict(batch=1 << 30, ts=1 << 18), dict(batch=1 << 30, layers=4, kl=0, vl=0),
])
def test_compact_refusals(change):
    a = dict(layers=2, kl=1 << 20, vl=1 << 20, path=P, depth=3, accepted=P, table=P, ts=4, width=4, lens=P, batch=2)
    a.update(change)
    assert hdb.lib().df11_paged_compact(ctypes.byref(cache()), a["layers"], a["kl"], a["vl"], a["path"], a["depth"], a["accepted"], a["table"],
                                        a["ts"], a["width"], a["lens"], a["batch"], None) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(parents=P + 1), BAD), (dict(batch=4097), BAD), (dict(table=None), BAD), (dict(table=P + 2), BAD), (dict(ts=3), BAD), (dict(ts=(1 << 32) + 1), BAD),
    (dict(width=0), BAD), (dict(width=1 << 25, ts=1 << 25), BAD), (dict(width=1 << 22, ts=1 << 22, page=1024), BAD), (dict(page=0), BAD),
    (dict(page=12), BAD), (dict(page=4), BAD), (dict(page=2048), BAD), (dict(lens=None), BAD), (dict(lens=P + 1), BAD), (dict(refs=None), BAD),
    (dict(refs=P + 2), BAD), (dict(pool=0), BAD), (dict(pool=1 << 31), BAD), (dict(room=(1 << 30) + 1), BAD), (dict(src=None), BAD), (dict(dst=P + 1), BAD),
    (dict(rows=None), BAD), (dict(missing=None), BAD), (dict(missing=P + 2), BAD), (dict(ws=None), BAD), (dict(ws=P + 8), BAD), (dict(size=8), SMALL),
    (dict(batch=4096, width=1 << 20, ts=1 << 20, room=1 << 30), BAD),
])
def test_fork_refusals(change, status):
    a = dict(parents=P, batch=3, table=P, ts=4, width=4, page=16, lens=P, refs=P, pool=100, room=1, src=P, dst=P, rows=P, missing=P, ws=P, size=1 << 40)
    a.update(change)
    got = hdb.lib().df11_paged_fork(a["parents"], a["batch"], a["table"], a["ts"], a["width"], a["page"], a["lens"], a["refs"], a["pool"], a["room"],
                                    a["src"], a["dst"], a["rows"], a["missing"], a["ws"], a["size"], None)
    assert got == status


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), BAD), (dict(logits=P + 1), BAD), (dict(dtype=1, logits=P + 2), BAD), (dict(dtype=2), hdb.DF11_E_UNSUPPORTED), (dict(k=0), BAD),
    (dict(k=65), BAD), (dict(beams=0), BAD), (dict(beams=1025), BAD), (dict(vocab=0), BAD), (dict(vocab=1 << 29), BAD), (dict(batch=1 << 22), BAD),
    (dict(bs=1 << 41), BAD), (dict(batch=1 << 10, bs=1 << 39), BAD), (dict(scores=None), BAD), (dict(scores=P + 2), BAD), (dict(best=None), BAD),
    (dict(parents=P + 1), BAD), (dict(tokens=None), BAD), (dict(ws=None), BAD), (dict(ws=P + 8), BAD), (dict(size=64), SMALL),
    (dict(batch=1 << 16, vocab=(1 << 29) - 1), BAD),
])
def test_beam_refusals(change, status):
    a = dict(logits=P, dtype=0, batch=2, beams=4, vocab=1000, bs=4000, ns=1000, scores=P, k=8, best=P, parents=P, tokens=P, ws=P, size=1 << 40)
    a.update(change)
    got = hdb.lib().df11_beam_select(a["logits"], a["dtype"], a["batch"], a["beams"], a["vocab"], a["bs"], a["ns"], a["scores"], None, a["k"], 0,
                                     a["best"], a["parents"], a["tokens"], a["ws"], a["size"], None)
    assert got == status


def test_workspace_sizes():
    need = hdb.df11_paged_tree_attention_workspace_bytes
    assert need(2, 5, 8, 8, 128, 16, 4) == 0
    assert need(1, 5, 32, 8, 128, 16, 4096) >= 2 * 5 * 32 * 130 * 4
    for refused in ((1, 5, 33, 8, 128, 16, 4096), (1, 5, 32, 8, 96, 16, 4096), (1, 5, 32, 8, 128, 17, 4096), (1, 1 << 21, 32, 8, 128, 16, 4096),
                    (1 << 24, 5, 32, 8, 128, 16, 4096), (1, 5, 32, 8, 128, 16, 0)):
        assert need(*refused) == 0
    assert hdb.df11_paged_fork_workspace_bytes(4, 100, 16, 1000, 1) >= 4 * 2 * 4
    assert hdb.df11_paged_fork_workspace_bytes(4, 100, 16, 1000, 1 << 20) >= 4 * 100 * 2 * 4
    assert hdb.df11_paged_fork_workspace_bytes(4, 100, 17, 1000, 1) == hdb.df11_paged_fork_workspace_bytes(0, 100, 16, 1000, 1) == 0
    assert hdb.df11_beam_select_workspace_bytes(2, 4, 1000, 8) >= 2 * 4 * (2 + 16) * 4
    assert hdb.df11_beam_select_workspace_bytes(2, 4, 1000, 65) == hdb.df11_beam_select_workspace_bytes(0, 4, 1000, 8) == 0


@pytest.mark.parametrize("batch", [0, 1, 2, 3, 63, 64, 65, 1 << 24])
def test_empty_trees_need_no_workspace(batch):
    """Without nodes nothing is cut, however wide the table is."""
    need = hdb.df11_paged_tree_attention_workspace_bytes
    for width in (4, 16, 17, 64, 4096, (1 << 26) - 1):
        assert need(batch, 0, 32, 8, 128, 16, width) == need(0, batch % 64, 32, 8, 128, 16, width) == 0
        assert need(batch, 0, 8, 1, 64, 16, width) == need(batch, 0, 16, 8, 256, 16, width) == 0


@pytest.mark.parametrize("batch,nodes,q_heads,dim", [(2, 1 << 20, 1 << 20, 128), (64, 1 << 20, 1 << 19, 128), (3, 1 << 19, 1 << 20, 256),
                                                     (1, 1 << 20, 1 << 20, 64), (1 << 24, 1 << 20, 1 << 20, 64)])
def test_more_rows_than_a_launch_holds(batch, nodes, q_heads, dim):
    """Sizes in their limits one by one whose tiles pass 32 bits."""
    c, t = cache(kv_heads=1, head_dim=dim), tree(batch=batch, nodes=nodes, q_heads=q_heads, mask=None, q_batch_stride=0, q_node_stride=0)
    for width in (1, 4, 64, 4096):
        assert hdb.df11_paged_tree_attention_workspace_bytes(batch, nodes, q_heads, 1, dim, 16, width) == 0
        assert attend(c, t, ts=width, width=width, ws=P, size=1 << 62) == BAD


def test_host_tensors_are_refused():
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        hdb.df11_paged_tree_attention(torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16), pages, pages, i.view(2, 1), i)
    with pytest.raises(TypeError):
        hdb.df11_paged_copy(i, i, pages, pages)
    with pytest.raises(TypeError):
        hdb.df11_paged_compact(i.view(2, 1), i, i.view(2, 1), i, pages, pages)
    with pytest.raises(TypeError):
        hdb.df11_paged_fork(i, i.view(2, 1), i, i, 16)
    with pytest.raises(TypeError):
        hdb.df11_beam_select(torch.zeros(1, 2, 5), torch.zeros(1, 2), 2)


def test_inline_assembly_does_not_set_m0():
    """m0 cannot be named as changed (the compiler keeps it for itself): what reads it takes it as an operand."""
    csrc = os.path.join(os.path.dirname(hdb.LIB_PATH), "csrc")
    readers = 0
    for name in sorted(os.listdir(csrc)):
        src = open(os.path.join(csrc, name)).read()
        for text in re.findall(r"\basm\b[^;(]*\((.*?)\);", src, flags=re.S):
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split("::")[0]))
            assert not re.search(r"\bm0\b", code), (name, text)
            if "_load_lds_" in code:
                readers += 1
                assert '"{m0}"' in text, (name, text)
    assert readers == 2


def test_no_kernel_of_these_keeps_registers_in_memory():
    """The compiler may store a vector register before the lanes that a loop left behind are on again, so that they
    read back what was there before: seen where a kernel of these had more values than registers."""
    built = open(hdb.LIB_PATH, "rb").read()
    seen = set()
    for m in re.finditer(rb"(_ZN12_GLOBAL__N_1\d+((?:tree|beam|fork)_\w+?_kernel|copy_kernel|compact_kernel)\w*)\.kd", built):
        count = re.compile(rb"\.vgpr_spill_count(.)", re.S).search(built, m.end())
        if count is None or count.start() - m.end() > 400:
            continue  # a name elsewhere than in the kernel's description
        seen.add(m.group(2).decode())
        assert count.group(1) == b"\0", m.group(1)
    assert {"tree_few_kernel", "tree_many_kernel", "tree_join_kernel", "beam_part_kernel", "beam_choose_kernel", "fork_plan_kernel",
            "fork_table_kernel", "copy_kernel", "compact_kernel"} <= seen


def test_no_kernel_of_the_library_keeps_registers_in_memory():
    built = open(hdb.LIB_PATH, "rb").read()
    seen = set()
    for m in re.finditer(rb"(_ZN12_GLOBAL__N_1\w+)\.kd", built):
        count = re.compile(rb"\.vgpr_spill_count(.)", re.S).search(built, m.end())
        if count is None or count.start() - m.end() > 400:
            continue  # a name elsewhere than in the kernel's description
        seen.add(m.group(1))
        assert count.group(1) == b"\0", m.group(1)
    for name in (b"tile_kernel", b"token_kernel", b"attend_kernel", b"df11_decode_kernel", b"run_pack_kernel", b"tree_few_kernel", b"beam_part_kernel"):
        assert any(name in s for s in seen), name
    assert len(seen) > 90
