"""Blocks given back behind a window and pools that grow and shrink: the library's block manager
against the reference model, extended here with the two operations. CPU only."""
import os
import random
import shutil

import pytest

from oracle import block_pool as BP
from paged_kv_cache_238_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    os.path.join(ROOT, "paged_kv_cache_238_gb300", "libpa.so")), reason="needs nvcc to build libpa")


def test_release_behind_frees_whole_blocks_only():
    bm = B.BlockManager(32, enable_caching=False)
    bm.add_request(1, list(range(100)))            # 7 blocks
    ids = bm.block_ids(1)
    free = bm.num_free()
    assert bm.release_behind(1, 15) == 0           # block 0 still holds position 15
    assert bm.release_behind(1, 50, keep=1) == 2   # blocks 1 and 2; block 0 is kept
    assert bm.block_ids(1) == [ids[0], 0, 0] + ids[3:]
    assert bm.num_free() == free + 2
    assert bm.release_behind(1, 50, keep=1) == 0   # once
    assert bm.free_queue()[:2] == [ids[1], ids[2]]  # tail first: the lower position is reused first
    with pytest.raises(B.PaError):
        bm.slot_mapping(1, 40, 10)
    assert bm.slot_mapping(1, 48, 3) == [ids[3] * 16 + i for i in range(3)]
    for first, keep in ((101, 0), (-1, 0), (10, -1)):
        with pytest.raises(B.PaError) as e:
            bm.release_behind(1, first, keep)
        assert e.value.status == B.PA_ERR_INVALID_ARG
    with pytest.raises(B.PaError):
        bm.release_behind(2, 0)
    bm.fork(1, 2)
    assert bm.release_behind(2, 64) == 2 and bm.num_free() == free + 2  # shared with 1: stay held
    bm.free_request(1)
    bm.free_request(2)
    assert bm.num_free() == 31 and 0 not in bm.free_queue()


def test_released_blocks_can_still_be_hit_and_commit_skips_them():
    bm = B.BlockManager(32)
    toks = list(range(70))
    bm.add_request(1, toks)
    bm.commit(1, 48)
    assert bm.release_behind(1, 48) == 3
    bm.commit(1, 70)                               # hashes block 3, never the null block
    assert bm.block_info(0)[1] is None
    assert bm.add_request(2, toks) == 64           # all four full blocks are found
    bm.append_tokens(1, [1] * 30)
    assert len(bm.block_ids(1)) == 7


def test_append_after_everything_was_released():
    bm = B.BlockManager(16, enable_caching=False)
    bm.add_request(1, list(range(32)))
    assert bm.release_behind(1, 32) == 2
    bm.fork(1, 2)
    bm.append_tokens(1, [7])
    bm.append_tokens(2, [8])
    assert bm.block_ids(1)[:2] == [0, 0] and bm.block_ids(1)[2] != bm.block_ids(2)[2]


def _content(bm, ref_content, rid):
    return [ref_content.get(b) for b in bm.block_ids(rid)]


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("caching", [True, False])
def test_random_traffic_with_resizes(seed, caching):
    """Blocks carry a token-content stand-in that moves with them; after every operation each
    request's blocks still hold its own content, reference counts and the free queue agree with
    the requests, and prefix hits stay right."""
    rng = random.Random(100 + seed)
    bm = B.BlockManager(40, enable_caching=caching)
    nb, reqs, content, nxt = 40, {}, {}, 1

    def write(rid):  # the request's K/V: every block that holds its tokens gets them
        for i, b in enumerate(bm.block_ids(rid)):
            if b:
                content[b] = tuple(reqs[rid][i * 16:(i + 1) * 16])

    def check():
        counts = {}
        for rid, toks in reqs.items():
            for i, b in enumerate(bm.block_ids(rid)):
                assert 0 <= b < nb
                if b:
                    counts[b] = counts.get(b, 0) + 1
                    full = tuple(toks[i * 16:(i + 1) * 16])
                    assert content[b][:len(full)] == full, (rid, i, b)
        q = bm.free_queue()
        assert len(q) == len(set(q)) == bm.num_free()
        assert sorted(q + list(counts)) == list(range(1, nb))
        for b in range(1, nb):
            assert bm.block_info(b)[0] == counts.get(b, 0)

    for _ in range(250):
        op = rng.random()
        live = sorted(reqs)
        try:
            if op < 0.3 or not live:
                toks = [rng.randrange(3) for _ in range(rng.randrange(1, 70))]
                bm.add_request(nxt, toks)
                reqs[nxt] = toks
                write(nxt)
                bm.commit(nxt, len(toks))
                nxt += 1
            elif op < 0.5:
                rid = rng.choice(live)
                toks = [rng.randrange(3) for _ in range(rng.randrange(1, 20))]
                bm.append_tokens(rid, toks)
                for s, d in bm.take_copies():
                    content[d] = content[s]
                reqs[rid] = reqs[rid] + toks
                write(rid)
            elif op < 0.6:
                rid = rng.choice(live)
                bm.fork(rid, nxt)
                reqs[nxt] = list(reqs[rid])
                nxt += 1
            elif op < 0.72:
                rid = rng.choice(live)
                bm.release_behind(rid, rng.randrange(0, len(reqs[rid]) + 1), rng.randrange(0, 40))
            elif op < 0.85:
                rid = rng.choice(live)
                bm.free_request(rid)
                del reqs[rid]
            else:
                want = rng.randrange(2, 70)
                before = {rid: bm.block_ids(rid) for rid in live}
                try:
                    moves = bm.resize(want)
                except B.PaError as e:
                    assert e.status == B.PA_ERR_NO_SPACE
                    assert before == {rid: bm.block_ids(rid) for rid in live}
                    held = {b for ids in before.values() for b in ids if b}
                    assert len(held) > want - 1
                    continue
                src, dst = [s for s, _ in moves], [d for _, d in moves]
                assert src == sorted(set(src)) and dst == sorted(set(dst))
                assert not moves or (dst[-1] < src[0] and src[0] >= want and dst[0] >= 1)
                new = {d: content[s] for s, d in moves}
                content.update(new)
                for b in [b for b in content if b >= want]:
                    del content[b]
                to = dict(moves)
                for rid in live:
                    assert bm.block_ids(rid) == [to.get(b, b) for b in before[rid]]
                nb = want
        except B.PaError as e:
            assert e.status == B.PA_ERR_NO_SPACE
        check()


def test_resize_keeps_hashes_with_their_content():
    bm = B.BlockManager(20)
    bm.add_request(9, list(range(1000, 1160)))     # blocks 1..10
    toks = list(range(64))
    bm.add_request(1, toks)                        # blocks 11..14
    bm.commit(1, 64)
    bm.free_request(9)
    h = [bm.block_info(b)[1] for b in bm.block_ids(1)]
    moves = bm.resize(8)
    assert [s for s, _ in moves] == [11, 12, 13, 14]
    assert [bm.block_info(b)[1] for b in bm.block_ids(1)] == h and all(h)
    assert bm.add_request(2, toks + [1]) == 64 and bm.block_ids(2)[:4] == bm.block_ids(1)
    assert bm.resize(30) == [] and bm.num_free() == 29 - 5
    bm.add_request(3, list(range(5000, 5000 + 24 * 16)))
    assert bm.num_free() == 0


def test_resize_refusals_change_nothing():
    bm = B.BlockManager(20, enable_caching=False)
    bm.add_request(1, list(range(100)))            # 7 blocks
    state = (bm.block_ids(1), bm.free_queue())
    for n, status in ((7, B.PA_ERR_NO_SPACE), (1, B.PA_ERR_INVALID_ARG), (0, B.PA_ERR_INVALID_ARG),
                      (-5, B.PA_ERR_INVALID_ARG)):
        with pytest.raises(B.PaError) as e:
            bm.resize(n)
        assert e.value.status == status
        assert (bm.block_ids(1), bm.free_queue()) == state
    bm.fork(1, 2)
    bm.append_tokens(2, [5])                       # a copy-on-write pair waits
    with pytest.raises(B.PaError) as e:
        bm.resize(40)
    assert e.value.status == B.PA_ERR_INVALID_ARG
    bm.take_copies()
    assert bm.resize(40) == []


def test_reference_model_agrees_after_a_resize_back():
    """Growing and shrinking over free blocks only leaves ordinary traffic as the reference model has it."""
    ref = BP.BlockPool(24, enable_caching=True, seed="s", block_size=16)
    bm = B.BlockManager(24, hash_seed="s")
    assert bm.resize(50) == [] and bm.resize(24) == []
    for rid in range(1, 4):
        toks = list(range(rid, rid + 60))
        assert ref.add_request(rid, toks, b"") == bm.add_request(rid, toks)
        ref.commit(rid, 60)
        bm.commit(rid, 60)
    assert bm.free_queue() == ref.queue
    assert all(bm.block_ids(r) == ref.block_ids(r) for r in (1, 2, 3))
