"""The host side of the served step (pages, adapters' indices): no GPU needed,
the device's part is replaced by records of what it was given."""
from collections import namedtuple

import pytest
import torch

from weight_only_quantized_dequant_gb300 import layer, serving

Batch = namedtuple("Batch", "cu_q kv_len page_table")


@pytest.fixture
def table(monkeypatch):
    monkeypatch.setattr(layer, "SeqBatch", Batch)
    return lambda *a: serving.PageTable(*a)


def state(t):
    return ({i: list(p) for i, p in t.pages.items()}, dict(t.lens), list(t.free))


def whole(t, n_pages):
    """Every page is free or held once."""
    held = [p for ps in t.pages.values() for p in ps]
    return sorted(held + t.free) == list(range(n_pages))


@pytest.mark.parametrize("new", [{8: 16}, {7: 1, 8: 16}, {9: 1, 8: 16}, {8: 40}, {9: 0, 8: 49},
                                 {7: 9}, {9: -1}])
def test_a_refused_step_changes_nothing(table, new):
    t = table(4, 16, 3)
    t.step({7: 40, 8: 1}, "cpu")  # three pages and one: the pool is full
    before = state(t)
    for _ in range(2):
        with pytest.raises((RuntimeError, ValueError)):
            t.step(new, "cpu")
        assert state(t) == before


def test_a_refused_step_can_be_tried_again(table):
    t = table(4, 16, 3)
    t.step({7: 40, 8: 1}, "cpu")
    page = t.pages[8][0]
    with pytest.raises(RuntimeError):
        t.step({8: 16}, "cpu")
    t.release(7)
    b = t.step({8: 16}, "cpu")
    assert b.cu_q.tolist() == [0, 16] and b.kv_len.tolist() == [17]
    assert b.page_table[0, 0] == page and b.page_table[0, 1] == t.pages[8][1]
    assert len(t.pages[8]) == 2 and whole(t, 4)


def test_a_step_that_cannot_be_sent_changes_nothing(table, monkeypatch):
    def broken(*_):
        raise MemoryError("no device memory")
    t = table(4, 16, 3)
    t.step({7: 10}, "cpu")
    before = state(t)
    monkeypatch.setattr(layer, "SeqBatch", broken)
    with pytest.raises(MemoryError):
        t.step({7: 10, 8: 5}, "cpu")
    assert state(t) == before


def test_pages_are_handed_out_in_order(table):
    t = table(6, 8, 4)
    b = t.step({1: 9, 2: 0, 3: 8}, "cpu")
    assert b.page_table.dtype == torch.int32
    assert b.page_table.tolist() == [[0, 1, 0, 0], [0, 0, 0, 0], [2, 0, 0, 0]]
    assert b.cu_q.tolist() == [0, 9, 9, 17] and b.kv_len.tolist() == [9, 0, 8]
    b = t.step({3: 1, 1: 7, 2: 1}, "cpu")
    assert b.page_table.tolist() == [[2, 3, 0, 0], [0, 1, 0, 0], [4, 0, 0, 0]]
    t.release(1)
    t.release("never seen")
    assert 1 not in t.lens and whole(t, 6)


@pytest.mark.parametrize("index,want", [(None, []), ("rows", ["q", "v"])])
def test_a_step_without_an_index_has_no_adapters(monkeypatch, index, want):
    calls = []
    monkeypatch.setattr(layer, "lora", lambda x, y, ad, i, out: calls.append((ad, i, out is y)))
    lay = object.__new__(serving.ServedLayer)
    lay.adapters = {"q": "q", "v": "v"}
    lay.products = lambda names, x: [n + x for n in names]
    assert lay._linear(("q", "k", "v"), "x", index) == ["qx", "kx", "vx"]
    assert calls == [(n, index, True) for n in want]
