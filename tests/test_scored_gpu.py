"""Scored attention (capped, distance-biased and masked scores) on the GPU against its fp64
definition, with the tolerance derived in scored_reference.py. Cells of keys that no row sees, and
the null block, hold NaN."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_238_gb300 import binding as B  # noqa: E402

from helpers import to_dev, to_f64  # noqa: E402
from scored_reference import Case, alibi  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_errors(clear=True)
    yield
    assert B.pa_get_device_errors(clear=True) == 0, "a kernel raised a device error"


class OnDevice:
    def __init__(self, c: Case, extra_rows=0):
        self.c = c
        self.q = to_dev(c.q)
        self.k, self.v = to_dev(c.k_cache), to_dev(c.v_cache)
        self.table, self.lens, self.qsl = to_dev(c.table), to_dev(c.lens), to_dev(c.qsl)
        opt = lambda a: None if a is None else to_dev(a)  # noqa: E731
        self.score = B.Score(softcap=c.cap, alibi_slopes=opt(c.slopes), window=c.window, key_start=opt(c.key_start),
                             prefix_len=opt(c.prefix))
        self.out = torch.full_like(self.q, float("nan"))
        self.max_len = int(c.lens.max())
        S = len(c.lens)
        if c.decode:
            n = B.pa_decode_scored_workspace_size(S, c.H_q, c.H_kv, c.D, self.max_len, self.q.dtype)
        else:
            n = B.pa_prefill_scored_workspace_size(S, int(c.chunks.max()), c.H_q, c.H_kv, c.D, self.max_len, self.q.dtype)
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None

    def run(self, stream=None):
        c = self.c
        if c.decode:
            B.pa_decode_scored(self.out, self.q, self.k, self.v, self.table, self.lens, self.max_len, c.scale,
                               self.score, self.ws, stream)
        else:
            B.pa_prefill_scored(self.out, self.q, self.k, self.v, self.table, self.lens, self.qsl,
                                int(c.chunks.max()), self.max_len, c.scale, self.score, self.ws, stream)
        return self.out


def check(c: Case, what=""):
    d = OnDevice(c)
    got = to_f64(d.run())
    ref, tol = c.reference()
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} values are not finite"
    bad = np.abs(got - ref) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - ref) - tol), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; worst at {i}: got {got[i]} ref {ref[i]} "
                             f"tolerance {tol[i]}")
    return d


DECODE_LENS = [1, 0, 15, 16, 17, 128, 129, 300, 777, 33]


def decode_scores(kind, lens, H_q):
    """Score arguments of a named kind for a decode batch."""
    lens = np.asarray(lens)
    if kind == "plain":
        return {}
    if kind == "cap":
        return dict(cap=20.0, sharp=6.0)
    if kind == "distance":
        return dict(slopes=alibi(H_q))
    if kind == "window":
        return dict(window=37)
    if kind == "window 1":
        return dict(window=1)
    if kind == "window prefix":
        return dict(window=50, prefix=[(7 * i) % 90 for i in range(len(lens))])
    if kind == "documents":  # starts inside, at the last key, behind the sequence (no key), negative
        return dict(key_start=[[L // 2, L - 1, L, 0, -5, max(0, L - 40)][i % 6] for i, L in enumerate(lens)])
    return dict(cap=15.0, sharp=4.0, slopes=alibi(H_q), window=70, prefix=[(11 * i) % 60 for i in range(len(lens))],
                key_start=[[0, 3, max(0, L - 20), L + 2][i % 4] for i, L in enumerate(lens)])


KINDS = ["plain", "cap", "distance", "window", "window 1", "window prefix", "documents", "all"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H_q,H_kv,D,BS,dtype", [
    (8, 2, 128, 16, "bf16"), (4, 4, 64, 32, "bf16"), (6, 2, 128, 64, "bf16"), (16, 1, 64, 128, "bf16"),
    (24, 1, 128, 16, "bf16"), (4, 2, 64, 16, "f32"), (5, 1, 128, 32, "f32")])
def test_decode_scores(kind, H_q, H_kv, D, BS, dtype):
    c = Case(11, DECODE_LENS, H_q, H_kv, D, BS, dtype, **decode_scores(kind, DECODE_LENS, H_q))
    check(c, f"{kind} {H_q}/{H_kv} D{D} BS{BS} {dtype}")


@pytest.mark.parametrize("H_q,H_kv,dtype", [(1, 1, "bf16"), (2, 2, "bf16"), (7, 7, "bf16"), (10, 2, "bf16"),
                                            (36, 4, "bf16"), (71, 1, "bf16"), (71, 1, "f32")])
def test_decode_head_layouts(H_q, H_kv, dtype):
    lens = [5, 190, 64]
    check(Case(12, lens, H_q, H_kv, 64, 16, dtype, **decode_scores("all", lens, H_q)))


@pytest.mark.parametrize("kind", ["cap", "window prefix", "documents"])
def test_decode_one_long_sequence_is_split(kind):
    lens = [6007]
    check(Case(13, lens, 8, 2, 128, 16, "bf16", **decode_scores(kind, lens, 8)))
    check(Case(13, lens, 2, 1, 64, 32, "f32", **decode_scores(kind, lens, 2)))


def test_decode_many_short_sequences():
    lens = [(i * 7) % 40 for i in range(1500)]
    check(Case(14, lens, 4, 1, 64, 16, "bf16", **decode_scores("all", lens, 4)))


CHUNKS = [(1, 1), (40, 7), (129, 129), (16, 16), (300, 45), (0, 0), (257, 128), (17, 1)]  # (keys, rows)


def chunk_scores(kind, H_q, pairs=CHUNKS):
    lens = [L for L, _ in pairs]
    pos = [p for L, C in pairs for p in range(L - C, L)]
    n = len(pairs)
    if kind == "plain":
        return {}
    if kind == "cap":
        return dict(cap=20.0, sharp=6.0)
    if kind == "distance":
        return dict(slopes=alibi(H_q))
    if kind == "window":
        return dict(window=37)
    if kind == "window 1":
        return dict(window=1)
    if kind == "prefix":  # rows before the prefix's end see keys behind themselves
        return dict(prefix=[[0, 30, 200, 5, 280, 0, 140, 400][i % 8] for i in range(n)])
    if kind == "window prefix":
        return dict(window=50, prefix=[(37 * i) % 150 for i in range(n)])
    if kind == "documents":  # documents of 23 tokens; every 11th row sees nothing
        return dict(key_start=[p + 1 if i % 11 == 10 else p // 23 * 23 for i, p in enumerate(pos)])
    return dict(cap=15.0, sharp=4.0, slopes=alibi(H_q), window=70, prefix=[(29 * i) % 120 for i in range(n)],
                key_start=[max(lens) if i % 13 == 12 else p // 90 * 90 for i, p in enumerate(pos)])


CHUNK_KINDS = ["plain", "cap", "distance", "window", "window 1", "prefix", "window prefix", "documents", "all"]


@pytest.mark.parametrize("kind", CHUNK_KINDS)
@pytest.mark.parametrize("H_q,H_kv,D,BS,dtype", [
    (8, 2, 128, 16, "bf16"), (4, 4, 64, 32, "bf16"), (6, 2, 128, 64, "bf16"), (16, 1, 64, 128, "bf16"),
    (24, 1, 128, 16, "bf16"), (4, 2, 64, 16, "f32"), (5, 1, 128, 32, "f32")])
def test_prefill_scores(kind, H_q, H_kv, D, BS, dtype):
    lens, chunks = zip(*CHUNKS)
    c = Case(21, lens, H_q, H_kv, D, BS, dtype, chunks=chunks, **chunk_scores(kind, H_q))
    check(c, f"{kind} {H_q}/{H_kv} D{D} BS{BS} {dtype}")


@pytest.mark.parametrize("H_q,H_kv,dtype", [(1, 1, "bf16"), (14, 2, "bf16"), (71, 1, "bf16"), (160, 1, "bf16"),
                                            (71, 1, "f32")])
def test_prefill_head_layouts(H_q, H_kv, dtype):
    pairs = [(70, 9), (150, 20)]
    lens, chunks = zip(*pairs)
    check(Case(22, lens, H_q, H_kv, 64, 16, dtype, chunks=chunks, **chunk_scores("all", H_q, pairs)))


@pytest.mark.parametrize("kind", ["cap", "window prefix", "documents", "distance"])
def test_prefill_long_context(kind):
    pairs = [(2311, 333), (1500, 700)]
    lens, chunks = zip(*pairs)
    check(Case(23, lens, 4, 1, 128, 16, "bf16", chunks=chunks, **chunk_scores(kind, 4, pairs)))
    check(Case(23, lens, 4, 2, 64, 64, "bf16", chunks=chunks, **chunk_scores(kind, 4, pairs)))


@pytest.mark.parametrize("kind", ["cap", "window prefix"])
def test_prefill_few_rows_on_a_long_context(kind):
    pairs = [(9001, 3), (4100, 5)]
    lens, chunks = zip(*pairs)
    check(Case(24, lens, 8, 2, 128, 16, "bf16", chunks=chunks, **chunk_scores(kind, 8, pairs)))
    check(Case(24, lens, 2, 2, 64, 16, "f32", chunks=chunks, **chunk_scores(kind, 2, pairs)))


def test_prefill_leaves_other_rows_alone():
    """Rows behind the last sequence of query_start_loc keep what they held."""
    c = Case(25, [40, 90], 8, 2, 128, 16, chunks=[7, 30], cap=20.0)
    d = OnDevice(c)
    T = d.q.shape[0]
    d.q = torch.cat([d.q, torch.zeros(9, 8, 128, dtype=d.q.dtype, device="cuda")])
    d.out = torch.full_like(d.q, 7.0)
    got = to_f64(d.run())
    ref, tol = c.reference()
    assert (np.abs(got[:T] - ref) <= tol).all()
    assert (got[T:] == 7.0).all()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_every_time_on_any_stream_and_in_a_graph(decode, dtype):
    lens = [500, 33, 1203]
    chunks = None if decode else [100, 33, 5]
    pairs = list(zip(lens, [1] * 3 if decode else chunks))
    c = Case(31, lens, 8, 2, 128, 16, dtype, chunks=chunks, **chunk_scores("all", 8, pairs))
    d = OnDevice(c)
    first = d.run().clone()
    for _ in range(3):
        d.out.fill_(float("nan"))
        assert torch.equal(d.run(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d.out.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(d.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.run()
    for _ in range(3):
        d.out.fill_(float("nan"))
        g.replay()
        assert torch.equal(d.out, first)
    # another batch through the same graph: new queries, new lengths in place
    d.q.copy_(d.q.flip(0))
    g.replay()
    again = d.out.clone()
    assert torch.equal(d.run(), again)


def test_two_graphs_share_a_workspace_one_after_the_other():
    a = OnDevice(Case(32, [900, 20], 8, 2, 128, 16, cap=20.0))
    b = OnDevice(Case(33, [1000], 8, 2, 128, 16, window=300))
    ws = torch.zeros(max(x.ws.numel() if x.ws is not None else 16 for x in (a, b)), dtype=torch.uint8, device="cuda")
    a.ws = b.ws = ws
    want = [x.run().clone() for x in (a, b)]
    graphs = []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
    for x, w in zip((a, b), want):
        assert torch.equal(x.out, w)


def test_no_score_equals_the_plain_calls_definition():
    """Without a descriptor the scored calls compute plain causal attention."""
    c = Case(34, [65, 300], 8, 2, 128, 16)
    d = OnDevice(c)
    d.score = None
    ref, tol = c.reference()
    assert (np.abs(to_f64(d.run()) - ref) <= tol).all()


def test_bad_tables_and_lengths_raise_device_errors():
    """Block ids and lengths out of range are caught by the kernels' own checks: nothing is read
    through them and the error word says so."""
    c = Case(35, [100, 40], 8, 2, 128, 16)
    d = OnDevice(c)
    d.table[1, 0] = 10 ** 6
    d.run()
    assert B.pa_get_device_errors(clear=True) & B.PA_DEVERR_BLOCK_RANGE
    d = OnDevice(c)
    d.lens[0] = 10 ** 6
    d.run()
    assert B.pa_get_device_errors(clear=True) & B.PA_DEVERR_LEN_RANGE
    c = Case(36, [100, 40], 8, 2, 128, 16, chunks=[20, 40])
    d = OnDevice(c)
    d.lens[1] = 39  # a chunk longer than its sequence
    out = to_f64(d.run())
    assert B.pa_get_device_errors(clear=True) & B.PA_DEVERR_LEN_RANGE
    ref, tol = c.reference()
    assert (np.abs(out[:20] - ref[:20]) <= tol[:20]).all(), "the other sequence's rows are right all the same"
    d = OnDevice(c)
    d.table[0, 2] = -3
    d.run()
    assert B.pa_get_device_errors(clear=True) & B.PA_DEVERR_BLOCK_RANGE


def test_offsets_past_32_bits():
    """Pages whose element offsets in the pool pass 2^31 are addressed in 64 bits."""
    c = Case(37, [200, 77], 8, 2, 128, 16, cap=20.0)
    d = OnDevice(c)
    NB = c.k_cache.shape[0]
    far = (1 << 31) // (2 * 16 * 128) + 1000  # blocks until 2^31 elements, and more
    big_k = torch.empty((far + NB, 2, 16, 128), dtype=d.k.dtype, device="cuda")
    big_v = torch.empty_like(big_k)
    big_k[:NB], big_v[:NB] = float("nan"), float("nan")
    big_k[far:], big_v[far:] = d.k, d.v
    d.k, d.v = big_k, big_v
    d.table = d.table + far
    ref, tol = c.reference()
    assert (np.abs(to_f64(d.run()) - ref) <= tol).all()
    c2 = Case(38, [200, 77], 8, 2, 128, 16, cap=20.0, chunks=[60, 77])
    e = OnDevice(c2)
    NB = c2.k_cache.shape[0]
    big_k[far:far + NB], big_v[far:far + NB] = e.k[:big_k.shape[0] - far], e.v[:big_k.shape[0] - far]
    e.k, e.v, e.table = big_k, big_v, e.table + far
    ref, tol = c2.reference()
    assert (np.abs(to_f64(e.run()) - ref) <= tol).all()


# ------------------------------------------------------------------- a run of them, as in use

def test_windowed_generation_gives_pages_back_and_shrinks_the_pool():
    """A request under a sliding window, step by step: prefill in chunks, decode, pages behind the
    window given back, the pool shrunk while it runs (pages moved in two layers, the table
    rewritten), and every output against the definition on the request's whole history."""
    rng = np.random.default_rng(5)
    H_q, H_kv, D, BS, window, keep = 8, 2, 128, 16, 60, 10
    layers, NB = 2, 64
    bm = B.BlockManager(NB, enable_caching=False)
    pools = [torch.full((NB, H_kv, BS, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2 * layers)]
    hog = list(range(40 * BS))
    bm.add_request(99, hog)                      # pushes the request's blocks to high ids
    total = 230
    prompt = 150
    bm.add_request(1, list(range(prompt)))
    bm.free_request(99)
    hist = [torch.randn(total, 2, H_kv, D, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
            for i in range(layers)]
    W_TABLE = 40
    table = torch.zeros(1, W_TABLE, dtype=torch.int32, device="cuda")
    prefix = torch.tensor([keep], dtype=torch.int32, device="cuda")
    score = B.Score(softcap=25.0, window=window, prefix_len=prefix)
    scale = D ** -0.5
    ws = torch.zeros(max(16, B.pa_decode_scored_workspace_size(1, H_q, H_kv, D, W_TABLE * BS, torch.bfloat16),
                         B.pa_prefill_scored_workspace_size(1, 50, H_q, H_kv, D, W_TABLE * BS, torch.bfloat16)),
                     dtype=torch.uint8, device="cuda")

    def put_table():
        table.copy_(torch.tensor([bm.block_ids(1, W_TABLE)], dtype=torch.int32))

    def reference(layer, q, first):
        c = Case.__new__(Case)
        L, C = first + q.shape[0], q.shape[0]
        c.H_q, c.H_kv, c.D, c.dtype, c.cap, c.window, c.scale = H_q, H_kv, D, "bf16", 25.0, window, scale
        c.slopes, c.lens, c.chunks, c.qsl = None, [L], [C], [0, C]
        from helpers import to_host_bits
        from scored_reference import keys_seen
        c.q = to_host_bits(q)
        c.keys, c.vals = [to_f64(hist[layer][:L, 0].contiguous())], [to_f64(hist[layer][:L, 1].contiguous())]
        c.seen = [np.stack([keys_seen(L, p, 0, min(keep, L), window) for p in range(first, L)])]
        return c.reference()

    def step(first, n):
        put_table()
        slots = torch.tensor(bm.slot_mapping(1, first, n), dtype=torch.int64, device="cuda")
        lens = torch.tensor([first + n], dtype=torch.int32, device="cuda")
        for layer in range(layers):
            k, v = pools[2 * layer], pools[2 * layer + 1]
            new = hist[layer][first:first + n]
            B.pa_reshape_and_cache(new[:, 0].contiguous(), new[:, 1].contiguous(), k, v, slots)
            q = torch.from_numpy(rng.standard_normal((n, H_q, D), dtype=np.float32) * 3).to(torch.bfloat16).cuda()
            out = torch.empty_like(q)
            if n == 1:
                B.pa_decode_scored(out, q, k, v, table, lens, first + n, scale, score, ws)
            else:
                qsl = torch.tensor([0, n], dtype=torch.int32, device="cuda")
                B.pa_prefill_scored(out, q, k, v, table, lens, qsl, n, first + n, scale, score, ws)
            ref, tol = reference(layer, q, first)
            assert (np.abs(to_f64(out) - ref) <= tol).all(), (first, n, layer)

    for first in range(0, prompt, 50):
        step(first, 50)
        bm.release_behind(1, max(0, first + 50 - window + 1), keep)
    at = prompt
    for i in range(total - prompt):
        bm.append_tokens(1, [at])
        step(at, 1)
        at += 1
        bm.release_behind(1, max(0, at - window + 1), keep)
        if i == 30:  # shrink under the running request: one launch for both layers and the table
            put_table()
            moves = bm.resize(12)
            assert moves
            pairs = torch.tensor(moves, dtype=torch.int32, device="cuda")
            lens = torch.tensor([at], dtype=torch.int32, device="cuda")
            B.pa_move_blocks(pools, pairs, block_table=table, seq_lens=lens)
            used = -(-at // BS)
            assert table[0, :used].tolist() == bm.block_ids(1, used)
            pools = [p[:12].clone() for p in pools]
    held = [b for b in bm.block_ids(1) if b]
    assert len(held) <= 1 + window // BS + 2 and max(held) < 12
    bm.close()


SPLIT_CHUNKS = [(4099, 3), (2600, 70), (130, 5), (0, 0), (700, 1), (257, 257)]


@pytest.mark.parametrize("kind", CHUNK_KINDS)
@pytest.mark.parametrize("H_q,H_kv,D,BS,dtype", [(8, 2, 128, 16, "bf16"), (3, 1, 64, 128, "bf16"), (2, 1, 64, 16, "f32")])
def test_prefill_key_lists_split_among_ctas(kind, H_q, H_kv, D, BS, dtype):
    """Few rows on long contexts: the keys of a row group go to several CTAs, of sequences that are
    long enough; short ones, and those without rows, lie between them."""
    lens, chunks = zip(*SPLIT_CHUNKS)
    c = Case(26, lens, H_q, H_kv, D, BS, dtype, chunks=chunks, **chunk_scores(kind, H_q, SPLIT_CHUNKS))
    d = check(c, kind)
    first = d.out.clone()
    for _ in range(3):  # the workspace needs nothing between calls; results do not depend on who ends last
        d.out.fill_(float("nan"))
        assert torch.equal(d.run(), first)


def test_prefill_split_workspace_serves_other_shapes():
    """One workspace, sized for the largest: calls that split, that do not and whose sequences lost their rows."""
    shapes = [[(3000, 2), (2500, 2)], [(40, 40)], [(2500, 2), (0, 0)], [(900, 100)], [(3000, 1)]]
    cases = [Case(27 + i, [L for L, _ in p], 4, 2, 64, 16, "bf16", chunks=[C for _, C in p], cap=30.0)
             for i, p in enumerate(shapes)]
    n = B.pa_prefill_scored_workspace_size(2, 100, 4, 2, 64, 3000, torch.bfloat16)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for c in cases + cases[::-1]:
        d = OnDevice(c)
        assert d.ws is None or d.ws.numel() <= n
        d.ws = ws
        ref, tol = c.reference()
        assert (np.abs(to_f64(d.run()) - ref) <= tol).all()
    dec = OnDevice(Case(33, [1500, 3], 4, 2, 64, 16, "bf16"))  # the counters at its start are as they were
    dec.ws[:65536].copy_(ws[:65536])
    ref, tol = dec.c.reference()
    assert (np.abs(to_f64(dec.run()) - ref) <= tol).all()


def test_prefill_split_is_captured_and_replayed():
    c = Case(34, [2100, 3500], 8, 2, 128, 16, "bf16", chunks=[4, 9], slopes=alibi(8))
    d = OnDevice(c)
    d.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run()
    ref, tol = c.reference()
    for _ in range(3):
        d.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert (np.abs(to_f64(d.out) - ref) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_split_refuses_a_small_workspace(dtype):
    c = Case(35, [3000], 4, 1, 64, 16, dtype, chunks=[2])
    d = OnDevice(c)
    assert d.ws is not None
    for ws in (None, d.ws[:-16], d.ws[8:]):
        d.ws = ws
        with pytest.raises(B.PaError):
            d.run()


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (6, 1, 64)])
@pytest.mark.parametrize("cap,slope", [(51.0, 1.0), (51.0, -0.02), (20.0, 30.0), (3.0, 0.01), (60.0, None), (60.0, 0.5),
                                       (300.0, -0.01)])
def test_prefill_caps_with_and_without_a_bias(H_q, H_kv, D, cap, slope):
    """Caps on both sides of the fixed reference's limit; slopes from none over steep to negative (the bias
    then grows with the distance); rows that see only keys far behind or before them."""
    pairs = [(300, 200), (150, 150), (700, 5), (64, 64)]
    lens, chunks = zip(*pairs)
    pos = [p for L, C in pairs for p in range(L - C, L)]
    slopes = None if slope is None else [slope * 2.0 ** -(h % 5) for h in range(H_q)]
    common = dict(cap=cap, sharp=8.0, slopes=slopes)
    check(Case(41, lens, H_q, H_kv, D, 16, "bf16", chunks=chunks, **common))
    # every third row sees the prefix alone (from inside it, before it or behind it), some of them nothing
    start = [p + 1 if i % 3 == 0 else 0 for i, p in enumerate(pos)]
    check(Case(42, lens, H_q, H_kv, D, 16, "bf16", chunks=chunks, key_start=start, prefix=[250, 40, 100, 64], **common))


def test_decode_one_kv_head_on_a_long_context():
    """A segment that all CTAs could share goes to a limited number of them."""
    check(Case(43, [9001], 8, 1, 128, 16, "bf16", cap=20.0))
    check(Case(44, [5000, 40], 4, 1, 64, 64, "bf16", window=3000))


@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(8, 1, 64, "f32"), (3, 1, 128, "f32"), (130, 1, 64, "bf16")])
def test_general_path_in_many_partitions(H_q, H_kv, D, dtype):
    """One sequence, few rows, fp32 (and a group that the tensor cores do not take): as many partitions as there are."""
    check(Case(45, [40011], H_q, H_kv, D, 16, dtype))
    if H_q < 100:
        check(Case(46, [40011], H_q, H_kv, D, 16, dtype, chunks=[1], prefix=[100], window=30000))
        check(Case(47, [9000, 50], H_q, H_kv, D, 16, dtype, chunks=[2, 50], cap=10.0))


WIDE_CHUNKS = {  # name: (keys, rows), H_q, H_kv: what a CTA of the bf16 kernel takes
    "two tiles": ([(900, 300), (805, 200), (20, 20)], 40, 40),
    "one tile of a short chunk": ([(1 + 41 * i % 700, 1 + i % 40 if 1 + 41 * i % 700 > 40 else 1) for i in range(40)], 8, 4),
    "one tile of short contexts": ([(190, 190), (130, 2), (64, 64), (129, 100), (1, 1), (0, 0)], 12, 4),
}


@pytest.mark.parametrize("kind", CHUNK_KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(WIDE_CHUNKS))
def test_prefill_tiles_of_a_cta(name, D, kind):
    pairs, H_q, H_kv = WIDE_CHUNKS[name]
    lens, chunks = zip(*pairs)
    check(Case(48, lens, H_q, H_kv, D, 32, "bf16", chunks=chunks, **chunk_scores(kind, H_q, pairs)), f"{name} {kind}")


@pytest.mark.parametrize("sharp", [0.0, 1.0])
@pytest.mark.parametrize("cap", [1e-6, 1e-30, 1e-38])
def test_tiny_caps(cap, sharp):
    """Caps so small that the scale over them overflows: every score is 0 or the cap, also where q.k is 0."""
    for slopes in (None, alibi(4)):
        check(Case(49, [300, 40], 4, 2, 64, 16, "bf16", chunks=[150, 40], cap=cap, sharp=sharp, slopes=slopes))
        check(Case(49, [300, 40], 4, 2, 128, 16, "bf16", cap=cap, sharp=sharp, slopes=slopes))
        check(Case(49, [300, 40], 4, 2, 64, 16, "f32", chunks=[15, 4], cap=cap, sharp=sharp, slopes=slopes))
