"""A Score's descriptor follows its attributes: what is assigned after construction is what the next
call passes (CPU: the descriptor alone, whose pointers nothing reads)."""
import pytest

from paged_kv_cache_238_gb300 import binding as B

torch = pytest.importorskip("torch")


def fields(score):
    d = score._desc
    return d.softcap, d.window, d.alibi_slopes, d.key_start, d.prefix_len


def test_assigned_arguments_reach_the_descriptor():
    a, b, c = (torch.ones(4) for _ in range(3))
    score = B.Score()
    assert fields(score) == (0.0, 0, None, None, None)
    score.softcap, score.window = 30.0, 77
    score.alibi_slopes, score.key_start, score.prefix_len = a, b, c
    assert fields(score) == (30.0, 77, a.data_ptr(), b.data_ptr(), c.data_ptr())
    assert (score.softcap, score.window) == (30.0, 77) and score.alibi_slopes is a and score.key_start is b
    score.key_start = c
    score.prefix_len = None
    score.window = 0
    assert fields(score) == (30.0, 0, a.data_ptr(), c.data_ptr(), None)
    assert score.prefix_len is None and score.key_start is c


def test_construction_and_assignment_agree():
    a, b, c = (torch.ones(4) for _ in range(3))
    whole = B.Score(softcap=20, alibi_slopes=a, window=5, key_start=b, prefix_len=c)
    parts = B.Score(softcap=1.0, alibi_slopes=b, window=9, key_start=a)
    parts.softcap, parts.alibi_slopes, parts.window, parts.key_start, parts.prefix_len = 20, a, 5, b, c
    assert fields(whole) == fields(parts)


def test_misspelt_arguments_are_refused():
    with pytest.raises(AttributeError):
        B.Score().windows = 3
