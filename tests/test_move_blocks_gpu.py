"""pa_move_blocks on the GPU against indexing in numpy: bit-exact copies in every pool, block tables
rewritten, everything else left as it was."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_238_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_errors(clear=True)
    yield
    assert B.pa_get_device_errors(clear=True) == 0, "a kernel raised a device error"


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).cpu().numpy()


def expected(pools, pairs, tokens):
    want = []
    for p in pools:
        old = bits(p)
        new = old.copy()
        for i, (s, d) in enumerate(pairs):
            n = old.shape[2] if tokens is None else min(max(tokens[i], 0), old.shape[2])
            new[d, :, :n] = old[s, :, :n]
        want.append(new)
    return want


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("H,BS,D,dtype,n_pools", [
    (1, 16, 64, torch.bfloat16, 1), (8, 16, 128, torch.bfloat16, 2), (3, 32, 64, torch.float32, 5),
    (2, 128, 128, torch.bfloat16, 7), (1, 16, 8, torch.bfloat16, 3), (5, 64, 4, torch.float32, 2),
    (2, 16, 128, torch.bfloat16, 300)])
@pytest.mark.parametrize("partial", [False, True])
def test_copies(H, BS, D, dtype, n_pools, partial):
    g = torch.Generator(device="cuda").manual_seed(3)
    NB = 23
    pools = [torch.randn(NB, H, BS, D, generator=g, device="cuda").to(dtype) for _ in range(n_pools)]
    pools[0][5] = float("nan")  # a copy is bitwise
    pairs = [(5, 6), (5, 7), (1, 22), (9, 9), (0, 3), (21, 2)]
    tokens = [1, BS, BS - 1, 4, 0, BS + 50] if partial else None
    want = expected(pools, pairs, tokens)
    B.pa_move_blocks(pools, i32(pairs), tokens=None if tokens is None else i32(tokens))
    for p, w in zip(pools, want):
        assert np.array_equal(bits(p), w)


def test_table_rewrite():
    rng = np.random.default_rng(4)
    NB, BS, S, MB = 4000, 32, 70, 41
    pools = [torch.randn(NB, 1, BS, 64, device="cuda").to(torch.bfloat16) for _ in range(2)]
    src = np.sort(rng.choice(np.arange(2000, NB), 1500, replace=False))
    dst = np.sort(rng.choice(np.arange(1, 2000), 1500, replace=False))
    pairs = np.stack([src, dst], axis=1).tolist()
    table = rng.integers(-3, NB + 5, (S, MB)).astype(np.int32)  # rubbish behind a row's length is not read as ids
    lens = np.array([[0, 1, BS, BS + 1, MB * BS, MB * BS + 99, -4][i % 7] for i in range(S)], dtype=np.int32)
    want = table.copy()
    to = dict(pairs)
    for s in range(S):
        for i in range(min(MB, max(0, -(-int(lens[s]) // BS)))):
            want[s, i] = to.get(int(table[s, i]), table[s, i])
    want_pools = expected(pools, pairs, None)
    t = torch.from_numpy(table).cuda()
    B.pa_move_blocks(B.PoolList(pools), i32(pairs), block_table=t, seq_lens=torch.from_numpy(lens).cuda())
    assert np.array_equal(t.cpu().numpy(), want)
    for p, w in zip(pools, want_pools):
        assert np.array_equal(bits(p), w)


def test_more_pools_than_one_launch_takes_rewrites_the_table_once():
    pools = [torch.randn(8, 1, 16, 64, device="cuda").to(torch.bfloat16) for _ in range(520)]
    want = expected(pools, [(6, 1), (7, 6 - 4)], None)
    t = i32([[6, 7, 3], [7, 0, 6]])
    B.pa_move_blocks(pools, i32([(6, 1), (7, 2)]), block_table=t, seq_lens=i32([48, 32]))
    assert t.tolist() == [[1, 2, 3], [2, 0, 6]]
    for p, w in zip(pools, want):
        assert np.array_equal(bits(p), w)


def test_bad_pairs_are_caught():
    pools = [torch.randn(8, 1, 16, 64, device="cuda").to(torch.bfloat16)]
    before = bits(pools[0])
    B.pa_move_blocks(pools, i32([(8, 1), (-1, 2), (3, 99), (4, -7)]))
    assert B.pa_get_device_errors(clear=True) == B.PA_DEVERR_BLOCK_RANGE
    assert np.array_equal(bits(pools[0]), before)
    B.pa_move_blocks(pools, i32([(6, 1), (5, 2)]), block_table=i32([[6]]), seq_lens=i32([16]))
    assert B.pa_get_device_errors(clear=True) == B.PA_DEVERR_PAIR_ORDER


def test_in_a_graph_and_on_another_stream():
    pools = [torch.randn(16, 2, 16, 128, device="cuda").to(torch.bfloat16) for _ in range(4)]
    lst, pairs = B.PoolList(pools), i32([(9, 1), (12, 4)])
    want = expected(pools, [(9, 1), (12, 4)], None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.pa_move_blocks(lst, pairs)
    g.replay()
    for p, w in zip(pools, want):
        assert np.array_equal(bits(p), w)
    pairs.copy_(i32([(1, 2), (4, 3)]))
    want = expected(pools, [(1, 2), (4, 3)], None)
    g.replay()
    for p, w in zip(pools, want):
        assert np.array_equal(bits(p), w)


def test_offsets_past_32_bits():
    NB = (1 << 31) // (16 * 128) + 40
    pool = torch.zeros(NB, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    pool[NB - 1] = 3.0
    pool[2] = 5.0
    B.pa_move_blocks([pool], i32([(NB - 1, 1), (2, NB - 2)]))
    assert (pool[1] == 3).all() and (pool[NB - 2] == 5).all()


@pytest.mark.parametrize("H,BS,D,dtype", [(1, 16, 8, torch.bfloat16), (1, 16, 64, torch.bfloat16), (3, 16, 64, torch.bfloat16),
                                          (2, 32, 128, torch.float32)])
@pytest.mark.parametrize("partial", [False, True])
def test_many_small_blocks(H, BS, D, dtype, partial):
    """Several pairs to a CTA: more pairs than one CTA takes, the last group not full, ids that are equal or out of range."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n = 333
    NB = 2 * n + 5
    pools = [torch.randn(NB, H, BS, D, generator=g, device="cuda").to(dtype) for _ in range(3)]
    order = np.random.default_rng(5).permutation(NB)
    pairs = [(int(order[i]), int(order[n + i])) for i in range(n)]
    pairs[7] = (pairs[7][0], pairs[7][0])
    tokens = [(5 * i) % (BS + 3) - 1 for i in range(n)] if partial else None
    want = expected(pools, pairs, tokens)
    B.pa_move_blocks(pools, i32(pairs), tokens=None if tokens is None else i32(tokens))
    for p, w in zip(pools, want):
        assert np.array_equal(bits(p), w)
    before = [p.clone() for p in pools]
    bad = [(0, NB)] * 200 + [(-1, 3)] * 100 + [(2, 4)]
    B.pa_move_blocks(pools, i32(bad))
    assert B.pa_get_device_errors(clear=True) == B.PA_DEVERR_BLOCK_RANGE
    for p, b in zip(pools, before):
        b[4] = b[2]
        assert torch.equal(p, b)


@pytest.mark.parametrize("H", [1, 8])
def test_tables_without_pools(H):
    table, lens = i32([[3, 5, 9, 0], [5, 3, 2, 9]]), i32([40, 64])
    pairs = i32([(3, 1), (9, 4)])
    status = B.load().pa_move_blocks(None, 0, H, 128, 16, 16, B.PA_BF16, pairs.data_ptr(), 2, None, table.data_ptr(), 4,
                                     lens.data_ptr(), 2, None)
    assert status == B.PA_OK
    torch.cuda.synchronize()
    assert table.tolist() == [[1, 5, 4, 0], [5, 1, 2, 4]]
