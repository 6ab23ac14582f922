"""Attention over 4-bit pools against the fp64 definition, with the tolerance derived in fp4_reference.py."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import fp4_reference as R  # noqa: E402
from helpers import to_dev, to_f64  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_errors_left():
    B.pa_get_device_errors()
    yield
    assert B.pa_get_device_errors() == 0


class Device:
    def __init__(self, c, max_len=None, max_chunk=None):
        self.c, self.q = c, to_dev(c.q)
        self.k, self.v = (to_dev(p) for p in c.pools)
        self.table, self.lens, self.qsl = to_dev(c.table), to_dev(c.lens), to_dev(c.qsl)
        self.out = torch.full_like(self.q, 7.0)
        S = len(c.lens)
        self.max_len = max(1, int(c.lens.max(initial=0))) if max_len is None else max_len
        self.max_chunk = int(c.chunks.max(initial=0)) if max_chunk is None else max_chunk
        if c.decode:
            n = B.pa_decode_fp4_workspace_size(S, c.H_q, c.H_kv, c.D, self.max_len, self.q.dtype)
        else:
            n = B.pa_prefill_fp4_workspace_size(S, self.max_chunk, c.H_q, c.H_kv, c.D, self.max_len, self.q.dtype)
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None

    def run(self, out=None, ws=None, stream=None):
        c, out = self.c, self.out if out is None else out
        kw = dict(k_scale=c.k_scale, v_scale=c.v_scale, stream=stream)
        ws = self.ws if ws is None else ws
        if c.decode:
            B.pa_decode_fp4(out, self.q, self.k, self.v, self.table, self.lens, self.max_len, c.scale, ws, **kw)
        else:
            B.pa_prefill_fp4(out, self.q, self.k, self.v, self.table, self.lens, self.qsl, self.max_chunk, self.max_len,
                             c.scale, ws, **kw)

    def got(self):
        torch.cuda.synchronize()
        return to_f64(self.out)


def check(c, **kw):
    d = Device(c, **kw)
    d.run()
    got = d.got()
    ref, tol = c.reference()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)):.2f} x"
    return d


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H_q,H_kv,D,BS", [(4, 4, 64, 16), (8, 2, 128, 16), (6, 2, 64, 32), (5, 1, 128, 64), (16, 2, 64, 128),
                                           (7, 1, 64, 16), (16, 1, 128, 16), (12, 1, 64, 16), (40, 2, 128, 32)])
def test_decode_edges(dtype, H_q, H_kv, D, BS):
    check(R.Case(1, EDGES, H_q, H_kv, D, BS, dtype, k_scale=0.25, v_scale=2.0 ** -5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H_q,H_kv,D", [([1], 8, 8, 64), ([0, 0, 0], 4, 2, 64), ([3000], 8, 1, 128), ([5000, 3, 0, 800], 8, 2, 128),
                                             ([9000], 32, 1, 64), (list(range(1, 200)), 2, 2, 64)])
def test_decode_lengths(dtype, lens, H_q, H_kv, D):
    check(R.Case(2, lens, H_q, H_kv, D, 16, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sharp", [0.0, 1e-30, 1e-6, 30.0, 3e4])
def test_decode_magnitudes_of_q(dtype, sharp):
    """Queries far from 1, which fp16 does not hold as they are; one row of zeros."""
    c = R.Case(3, [300, 17, 40], 8, 2, 128, 16, dtype, sharp=sharp)
    c.q[1, 3] = 0
    if sharp == 1e-6:  # elements of one row 2^-60 to 1 apart
        w = np.float32(2.0) ** -np.arange(0, 64, 0.5, dtype=np.float32)
        c.q[0, 0] = R.W.f32_to_bf16_bits(w) if dtype == "bf16" else w
    check(c)


def test_decode_scales_of_a_pool_at_the_ends():
    """Scales of 448 and of 2^-9 in one pool: values from 2^-10 to 2688."""
    c = R.Case(4, [200, 33], 8, 2, 128, 16)
    for p, i in zip(c.pools, range(2)):
        pages = p.reshape(p.shape[0], 2, 1, 9 * 128)[..., 8 * 128:]
        pick = np.random.default_rng(i).random(pages.shape)
        pages[pick < 0.1] = 1
        if i == 1:
            pages[pick > 0.9] = 126
        c.values[i] = R.from_pool(p, 1.0)
    check(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks,lens,H_q,H_kv,D,BS", [
    ([1, 5, 0, 33, 2], [1, 64, 20, 33, 300], 8, 2, 128, 16),
    ([17, 128, 129, 1], [17, 128, 400, 1000], 4, 4, 64, 32),
    ([64, 40], [64, 650], 8, 1, 128, 128),
    ([100, 7], [230, 7], 12, 4, 64, 16),
    ([33], [33], 5, 1, 128, 64),
    ([20, 3], [150, 9], 16, 1, 64, 16),
    ([9], [4000], 16, 2, 128, 16),
    ([0, 0], [30, 0], 4, 2, 64, 16)])
def test_prefill_edges(dtype, chunks, lens, H_q, H_kv, D, BS):
    check(R.Case(5, lens, H_q, H_kv, D, BS, dtype, chunks=chunks, k_scale=4.0, v_scale=0.5))


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (16, 16, 64), (6, 2, 64), (10, 2, 128), (8, 1, 128)])
def test_prefill_tiles(H_q, H_kv, D):
    check(R.Case(6, [300, 700, 257, 520], H_q, H_kv, D, 16, "bf16", chunks=[300, 256, 1, 391], v_scale=2.0 ** -6))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks", [None, [150, 40, 3]])
def test_rows_that_are_no_numbers(dtype, chunks):
    """NaN and infinities in one row of q reach that row's outputs alone."""
    c = R.Case(14, [300, 40, 17], 8, 2, 128, 16, dtype, chunks=chunks)
    ref, tol = c.reference()
    bad = {(0, 1): np.nan, (len(c.q) - 1, 6): np.inf}
    for (r, h), x in bad.items():
        c.q[r, h, 5] = R.W.f32_to_bf16_bits(np.float32([x]))[0] if dtype == "bf16" else x
    d = Device(c)
    d.run()
    got = d.got()
    keep = np.ones(got.shape[:2], dtype=bool)
    for rh in bad:
        keep[rh] = False
    assert np.isnan(got[0, 1]).all()
    assert (np.abs(got - ref) <= tol)[keep].all()


def test_pools_do_not_reach_calls_of_another_type():
    c = R.Case(15, [20], 4, 2, 64, 16)
    d = Device(c)
    with pytest.raises(TypeError):
        B.pa_decode(d.out, d.q, d.k, d.v, d.table, d.lens, 20, 0.1, d.ws)
    with pytest.raises(TypeError):
        B.pa_reshape_and_cache(d.q[:, :2].contiguous(), d.q[:, :2].contiguous(), d.k, d.v, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        B.pa_decode_scored(d.out, d.q, d.k, d.v, d.table, d.lens, 20, 0.1, None, d.ws)
    wide = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        B.pa_decode_fp4(d.out, d.q, wide, wide, d.table, d.lens, 20, 0.1, d.ws)


def test_prefill_magnitudes_of_q():
    for sharp in (0.0, 1e-30, 30.0):
        c = R.Case(7, [200, 40], 4, 2, 128, 16, "bf16", chunks=[150, 40], sharp=sharp)
        check(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_larger_than_the_batch(dtype):
    check(R.Case(8, [40, 0, 7], 8, 2, 64, 16, dtype), max_len=48)
    c = R.Case(8, [40, 0, 7], 8, 2, 64, 16, dtype, chunks=[20, 0, 7])
    check(c, max_len=48, max_chunk=41)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_blocks_and_lengths(dtype):
    c = R.Case(9, [100, 40, 90], 8, 2, 128, 16, dtype)
    ref, tol = c.reference()
    d = Device(c)
    d.table[1, 1] = 1 << 20  # outside the pool: not read
    d.run()
    assert B.pa_get_device_errors() == B.PA_DEVERR_BLOCK_RANGE
    got = d.got()
    for s in (0, 2):
        assert (np.abs(got[s] - ref[s]) <= tol[s]).all()
    d = Device(c)
    d.lens[1] = 1000
    d.run()
    assert B.pa_get_device_errors() & B.PA_DEVERR_LEN_RANGE
    got = d.got()
    for s in (0, 2):
        assert (np.abs(got[s] - ref[s]) <= tol[s]).all()
    c = R.Case(9, [100, 40, 90], 8, 2, 128, 16, dtype, chunks=[10, 40, 20])
    ref, tol = c.reference()
    d = Device(c)
    d.lens[1] = 30  # a chunk longer than its sequence: left as it was
    d.run()
    assert B.pa_get_device_errors() == B.PA_DEVERR_LEN_RANGE
    got = d.got()
    assert (got[10:50] == 7.0).all()
    assert (np.abs(got - ref) <= tol)[np.r_[0:10, 50:70]].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks", [None, [1, 30, 300, 16]])
def test_workspace_serves_call_after_call(dtype, chunks):
    """Calls of different shapes on one workspace, again and again, in a captured graph too; equal bits each time."""
    c = R.Case(10, [4000, 30, 700, 16], 8, 2, 128, 16, dtype, chunks=chunks)
    e = R.Case(11, [900, 2100], 4, 4, 64, 32, dtype, chunks=None if chunks is None else [3, 2])
    d, f = Device(c), Device(e)
    n = max(x.ws.numel() if x.ws is not None else 0 for x in (d, f))
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    first = {}
    for i in range(3):
        for x in (d, f):
            x.out.fill_(7.0)
            x.run(ws=ws)
            got = x.got()
            ref, tol = x.c.reference() if i == 0 else (None, None)
            if i == 0:
                assert (np.abs(got - ref) <= tol).all()
                first[x] = got
            assert (got == first[x]).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run(ws=ws)
        f.run(ws=ws)
        d.run(ws=ws)
    for _ in range(3):
        d.out.fill_(7.0)
        f.out.fill_(7.0)
        graph.replay()
        assert (d.got() == first[d]).all() and (f.got() == first[f]).all()


def test_threads_with_a_stream_and_workspace_each():
    cases = [R.Case(20 + i, [600 + 100 * i, 5, 0, 33], 8, 2, 128, 16, "bf16", chunks=None if i % 2 else [100, 5, 0, 7])
             for i in range(4)]
    devs = [Device(c) for c in cases]
    refs = [c.reference() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(d, ref):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                d.run(stream=s)
            s.synchronize()
            got = to_f64(d.out)
            if not (np.abs(got - ref[0]) <= ref[1]).all():
                bad.append("outside")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=x) for x in zip(devs, refs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """A pool of more than 4 GiB whose used blocks lie at its end."""
    c = R.Case(30, [70, 33], 8, 8, 128, 128, dtype)
    p = R.Case(30, [70, 33], 8, 8, 128, 128, dtype, chunks=[20, 33])
    per = 8 * 128 * 72
    NB = (5 << 30) // per
    for x in (c, p):
        d = Device(x)
        shift = NB - x.pools[0].shape[0]
        big = []
        for pool in (d.k, d.v):
            b = torch.empty(NB, 8, 128, 72, dtype=torch.uint8, device="cuda")
            b[shift:] = pool
            big.append(b)
        d.k, d.v = big
        d.table += shift
        d.run()
        got = d.got()
        ref, tol = x.reference()
        assert (np.abs(got - ref) <= tol).all()
        rows = [torch.empty(3, 8, 128, dtype=torch.float32, device="cuda") for _ in range(2)]
        ids = x.table[0, 0]
        slots = (shift + int(ids)) * 128 + torch.arange(3, device="cuda")
        B.pa_gather_fp4(*rows, *big, slots)
        assert (to_f64(rows[1]) == x.values[1][ids, :, :3].transpose(1, 0, 2)).all()
        del big, d


def test_refused_tensors():
    c = R.Case(12, [20, 5], 8, 2, 64, 16)
    d = Device(c)
    ok = dict(out=d.out, q=d.q, k_cache=d.k, v_cache=d.v, block_table=d.table, seq_lens=d.lens, max_seq_len=20, scale=0.1,
              workspace=d.ws)
    for bad in (dict(out=d.out.float()), dict(out=d.out[:1]), dict(q=d.q.transpose(0, 1)), dict(q=d.q.half()),
                dict(k_cache=d.k.to(torch.bfloat16)), dict(v_cache=d.v[:2]), dict(k_cache=d.k[..., :18]), dict(block_table=d.table.long()),
                dict(block_table=d.table[:1]), dict(seq_lens=d.lens.long()), dict(seq_lens=d.lens.cpu())):
        with pytest.raises((ValueError, TypeError)):
            B.pa_decode_fp4(**{**ok, **bad})
    with pytest.raises(ValueError):
        B.pa_decode_fp4(**{**ok, "q": torch.cat([d.q, d.q]), "out": torch.cat([d.out, d.out])})
    with pytest.raises(B.PaError):
        B.pa_decode_fp4(**ok, k_scale=0.3)
    if d.ws is not None:
        with pytest.raises(B.PaError):
            B.pa_decode_fp4(**{**ok, "workspace": d.ws[:16]})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_request_from_prompt_to_tokens(dtype, interleaved):
    """Prompts in two chunks, decode steps, a fork and a compaction, as a serving loop makes them."""
    H_q, H, D, BS, S, ks, vs = 8, 2, 64, 16, 2, 0.5, 0.25
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(0)
    cs = np.concatenate([np.cos(a := np.arange(256)[:, None] * 10000.0 ** (-np.arange(0, D, 2) / D)), np.sin(a)], axis=1).astype(np.float32)
    dcs = to_dev(cs)
    bm = B.BlockManager(40, block_size=BS, enable_caching=False)
    pools = [torch.full(B.fp4_pool_shape(40, H, BS, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    lens, hist = [0] * S, [[[], []] for _ in range(S)]  # per request: k and v rows as the pool holds them
    prompts = [[37, 30], [21, 50]]
    for s in range(S):
        bm.add_request(s, list(range(sum(prompts[s]))))

    def new(counts):
        T = sum(counts)
        qkv = torch.from_numpy(rng.standard_normal((T, H_q + 2 * H, D)).astype(np.float32)).cuda().to(dt)
        q, k, v = qkv.split([H_q, H, H], dim=1)
        pos, slots = [], []
        for s, n in enumerate(counts):
            pos += range(lens[s], lens[s] + n)
            slots += bm.slot_mapping(s, lens[s], n)
        q_out = torch.empty(T, H_q, D, dtype=dt, device="cuda")
        B.pa_rotate_and_cache(q_out, q, k, v, torch.tensor(pos, device="cuda"), dcs, *pools,
                              torch.tensor(slots, device="cuda"), interleaved=interleaved, k_scale=ks, v_scale=vs)
        kr = R.rounded(R.rotate(to_f64(k.contiguous()), cs[pos].astype(np.float64), interleaved)[0], dtype)
        at = 0
        for s, n in enumerate(counts):
            for j, (x, f) in enumerate(((kr, ks), (to_f64(v.contiguous()), vs))):
                c, sc = R.quantise(x[at:at + n], f)
                hist[s][j].append(R.GRID[c & 7] * np.where(c & 8, -1, 1) * np.repeat(R.e4m3_values(sc), 16, axis=-1) * f)
            lens[s] += n
            at += n
        return q_out

    def expect(q_out, counts, out):
        c = R.Case(0, lens, H_q, H, D, BS, dtype, chunks=counts, k_scale=ks, v_scale=vs)
        c.q = q_out.cpu().numpy() if dtype == "f32" else q_out.view(torch.int16).cpu().numpy().view(np.uint16)
        c.keys = lambda s: [np.concatenate(h, axis=0).transpose(1, 0, 2) for h in hist[s]]
        ref, tol = c.reference()
        assert (np.abs(to_f64(out) - ref) <= tol).all()

    def table():
        rows = [bm.block_ids(s) for s in range(S)]
        w = max(map(len, rows))
        return torch.tensor([r + [0] * (w - len(r)) for r in rows], dtype=torch.int32, device="cuda")

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for step in range(2):
        counts = [prompts[s][step] for s in range(S)]
        q = new(counts)
        out = torch.empty_like(q)
        n = B.pa_prefill_fp4_workspace_size(S, max(counts), H_q, H, D, max(lens), dt)
        B.pa_prefill_fp4(out, q, *pools, table(), i32(lens), i32([0, counts[0], sum(counts)]), max(counts), max(lens), D ** -0.5,
                         torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None, k_scale=ks, v_scale=vs)
        expect(q, counts, out)
    ws = torch.zeros(max(16, B.pa_decode_fp4_workspace_size(4, H_q, H, D, 256, dt)), dtype=torch.uint8, device="cuda")

    def decode_step():
        for s in range(S):
            bm.append_tokens(s, [7])
        pairs = bm.take_copies()
        if pairs:
            B.pa_move_blocks(pools, i32(pairs))
        q = new([1] * S)
        out = torch.empty_like(q)
        B.pa_decode_fp4(out, q, *pools, table(), i32(lens), max(lens), D ** -0.5, ws, k_scale=ks, v_scale=vs)
        expect(q, [1] * S, out)

    for _ in range(3):
        decode_step()
    bm.fork(0, 2)  # shares request 0's blocks; the partly filled last one is copied at the next token
    S = 3
    lens.append(lens[0])
    hist.append([list(h) for h in hist[0]])
    for _ in range(2):
        decode_step()
    moves = bm.resize(26)
    if moves:
        B.pa_move_blocks(pools, i32(moves))
    pools = [p[:26].contiguous() for p in pools]
    for _ in range(2):
        decode_step()
    rows = [torch.empty(lens[0], H, D, dtype=dt, device="cuda") for _ in range(2)]
    B.pa_gather_fp4(*rows, *pools, torch.tensor(bm.slot_mapping(0, 0, lens[0]), device="cuda"), k_scale=ks, v_scale=vs)
    for r, h in zip(rows, hist[0]):
        assert (to_f64(r) == np.concatenate(h, axis=0)).all()


def test_move_of_whole_blocks():
    rng = np.random.default_rng(1)
    host = [rng.integers(0, 256, B.fp4_pool_shape(12, 1, 16, 64)).astype(np.uint8) for _ in range(3)]
    pools = [to_dev(h) for h in host]
    pairs = [(7, 2), (9, 1), (11, 3)]
    table = torch.tensor([[7, 4, 11], [9, 7, 7]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([48, 20], dtype=torch.int32, device="cuda")
    B.pa_move_blocks(B.PoolList(pools), torch.tensor(pairs, dtype=torch.int32, device="cuda"), block_table=table, seq_lens=lens)
    for h, p in zip(host, pools):
        for a, b in pairs:
            h[b] = h[a]
        assert (p.cpu().numpy() == h).all()
    assert table.tolist() == [[2, 4, 3], [1, 2, 7]]
    with pytest.raises(B.PaError):
        B.pa_move_blocks(pools, torch.tensor(pairs, dtype=torch.int32, device="cuda"),
                         tokens=torch.ones(3, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [0.0, -1.0, 1e-38])
@pytest.mark.parametrize("chunks", [None, [40, 3]])
def test_other_scales(dtype, factor, chunks):
    """Scales of zero (uniform weights), below zero, and so small that they vanish."""
    c = R.Case(13, [77, 9], 8, 2, 64, 16, dtype, chunks=chunks)
    c.scale *= factor
    d = Device(c)
    d.run()
    ref, tol = c.reference()
    assert (np.abs(d.got() - ref) <= np.abs(tol)).all()


@pytest.mark.parametrize("chunks", [None, [150, 40, 3]])
@pytest.mark.parametrize("sharp,factor", [(1e-30, 1.0), (1e-6, 1.0), (30.0, 1.0), (3e36, 1e-36), (3e-38, 1e30)])
def test_fp32_queries_of_any_size(chunks, sharp, factor):
    """fp32 queries whose halves need the whole range of their row's power of two; elements of one row 2^-32 to 1 apart."""
    c = R.Case(17, [300, 40, 17], 8, 2, 128, 16, "f32", chunks=chunks, sharp=sharp)
    c.scale *= factor
    c.q[1, 3] = 0
    c.q[0, 0] = np.float32(2.0) ** -np.arange(0, 64, 0.5, dtype=np.float32) * np.float32(sharp)
    check(c)


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (16, 16, 64), (6, 2, 64), (10, 2, 128), (96, 1, 64)])
def test_prefill_tiles_of_fp32_queries(H_q, H_kv, D):
    check(R.Case(18, [300, 700, 257, 520], H_q, H_kv, D, 16, "f32", chunks=[300, 256, 1, 391], v_scale=2.0 ** -6))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_heads_than_a_tile_has_rows(dtype):
    check(R.Case(15, [40, 17, 0, 300], 130, 1, 64, 16, dtype))
    check(R.Case(15, [40, 17, 0, 300], 130, 1, 64, 16, dtype, chunks=[9, 17, 0, 5]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunks", [None, [20, 0, 150]])
def test_the_largest_bound(dtype, chunks):
    """A table of 2^24 - 1 blocks a sequence, of which a few are used: more units than a launch counts."""
    c = R.Case(16, [40, 0, 300], 16, 16, 64, 128, dtype, chunks=chunks)
    d = Device(c, max_len=(2 ** 24 - 1) * 128)
    wide = torch.zeros(3, 2 ** 24 - 1, dtype=torch.int32, device="cuda")
    wide[:, :d.table.shape[1]] = d.table
    d.table = wide
    d.run()
    ref, tol = c.reference()
    assert (np.abs(d.got() - ref) <= tol).all()


@pytest.mark.parametrize("lens,chunks", [([8000] * 24, None), ([6000, 8000], [100, 60])])
def test_fp32_sums_over_many_keys(lens, chunks):
    """Sums that are rounded, not cut off, have errors that do not add up: of a sum over n / 16 pages the root mean square
    of (n / 16) roundings, each within u and 0.58 u in the mean, 7.8e-7 for 8000 keys if all partial sums were as large
    as the result; 2e-7 from scores, 5e-8 from the halves. Sums cut off towards zero are off by n / 16 u, 3e-5."""
    c = R.Case(19, lens, 8, 8, 64, 16, "f32", chunks=chunks)
    d = Device(c)
    d.run()
    ref, _ = c.reference()
    assert np.linalg.norm(d.got() - ref) <= 1.05e-6 * np.linalg.norm(ref)
