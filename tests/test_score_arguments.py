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


def test_causal_prefix_argument():
    score = B.Score()
    assert score.prefix_causal is False and score._desc.prefix_causal == 0
    score.prefix_causal = True
    assert score.prefix_causal is True and score._desc.prefix_causal == 1
    assert B.Score(prefix_causal=True)._desc.prefix_causal == 1


@pytest.mark.parametrize("value", [-1, 2, 1 << 30])
def test_calls_refuse_other_values_of_the_causal_flag(value):
    from test_scored_abi import FAKE
    desc = B.ScoreDesc(prefix_causal=value)
    lib = B.load()
    assert lib.pa_decode_scored(FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 2, 64, 8, 2, 128, 16, 16, 0.1, desc, B.PA_BF16, FAKE,
                                1 << 30, None) == B.PA_ERR_INVALID_ARG
    assert lib.pa_prefill_scored(FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, 2, 16, 64, 8, 2, 128, 16, 16, 0.1, desc,
                                 B.PA_BF16, FAKE, 1 << 30, None) == B.PA_ERR_INVALID_ARG


def test_copies_are_apart():
    """A copied Score that is changed leaves the first one as it was."""
    import copy
    a, b = torch.ones(4), torch.zeros(4)
    first = B.Score(softcap=20.0, alibi_slopes=a, window=5, prefix_causal=True)
    for second in (copy.copy(first), copy.deepcopy(first)):
        assert (second.softcap, second.window, second.prefix_causal) == (20.0, 5, True)
        assert torch.equal(second.alibi_slopes, a)
        second.window, second.softcap, second.alibi_slopes, second.prefix_causal = 9, 0.0, b, False
        assert fields(first) == (20.0, 5, a.data_ptr(), None, None) and first._desc.prefix_causal == 1
    assert copy.copy(first).alibi_slopes is a
