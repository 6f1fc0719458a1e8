"""The cache's bookkeeping when a copy of pages is refused."""
import pytest
import torch

from bit_quantized_gemm_qmm_b200 import kv
from test_kv_plan_cpu import book  # noqa: F401 - a fixture


def test_refused_copies_change_nothing(book, monkeypatch):  # noqa: F811
    """A fork, a cut and an accept whose page copies are refused leave pages, lengths and the pool."""
    c, s = book
    a = s.add()
    k = torch.zeros(7, 1, 64)
    s.step([a], k, k, k, [7])  # pages of 4: one full, one partly filled
    b = s.fork(a)              # shares the first
    s.step([b], k[:6], k[:6], k[:6], [6])
    d = s.fork(b)              # shares three
    before = {x: (s.length(x), s.pages(x)) for x in (a, b, d)}, s.free_pages()

    def refuse(*args, **kwargs):
        raise ValueError("refused")

    with monkeypatch.context() as m:
        m.setattr(kv, "kv_copy_pages", refuse)
        for call in (lambda: s.fork(a), lambda: s.truncate(b, 2), lambda: s.accept([b], [[0, 2]])):
            with pytest.raises(ValueError, match="refused"):
                call()
            assert ({x: (s.length(x), s.pages(x)) for x in (a, b, d)}, s.free_pages()) == before
    e = s.fork(a)
    s.accept([b], [[0, 2]])
    for x in (a, b, d, e):
        s.free(x)
    assert s.free_pages() == c.pages
