"""Scored attention at its edges on the GPU, against the fp64 definition and the tolerance of
scored_reference.py (or a tighter one, derived beside its test)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from paged_kv_cache_238_gb300 import workloads as W  # noqa: E402

from helpers import to_f64  # noqa: E402
from scored_reference import Case, U, alibi  # noqa: E402
from test_scored_gpu import OnDevice, check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    B.pa_get_device_errors(clear=True)
    yield
    assert B.pa_get_device_errors(clear=True) == 0, "a kernel raised a device error"


FORMS = {  # a name for each arithmetic of the scores
    "plain": {}, "cap": dict(cap=20.0, sharp=6.0), "distance": dict(slopes=alibi(2)),
    "cap distance": dict(cap=20.0, sharp=6.0, slopes=alibi(2)), "large cap": dict(cap=100.0, sharp=6.0)}


def repeats(c, what, times=20):
    """Right, and the same bits every time."""
    d = check(c, what)
    first = d.out.clone()
    for _ in range(times):
        d.out.fill_(float("nan"))
        assert torch.equal(d.run(), first), what


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D", [64, 128])
def test_query_tiles_without_keys(D, form):
    """A query tile of 128 rows that uses no key tile of its CTA: its rows see nothing (documents that begin
    behind them), or it belongs to a run of keys that only the other query tile of the CTA sees. 2 heads
    with a kv head each: a query tile is 128 tokens."""
    kw = FORMS[form]
    L, C = 700, 256
    for empty in (range(0, 128), range(128, 256), range(0, 256)):
        start = [L if r in empty else 0 for r in range(C)]
        repeats(Case(61, [L], 2, 2, D, 16, "bf16", chunks=[C], key_start=start, **kw), f"{form} {empty}")
    # 256 rows from position 3840 under a window of 600: key tiles 25 to 31 in runs of three, three and one
    # (rows 3840 to 3967 see nothing of the last); a window of 900 gives other runs
    for window in (600, 900, 130):
        repeats(Case(62, [4096], 2, 2, D, 16, "bf16", chunks=[C], window=window, **kw), f"{form} window {window}")


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("H_q,H_kv,D", [(2, 2, 64), (2, 2, 128), (8, 1, 128)])
def test_ends_of_split_runs(H_q, H_kv, D, form):
    """Key lists cut into runs of two and more key tiles at every offset of the first visible key: nothing past a
    run's end is multiplied, and the next run's tiles are not lost."""
    kw = dict(FORMS[form])
    if "slopes" in kw:
        kw["slopes"] = alibi(H_q)
    for L, C, window in ((640, 5, 0), (641, 130, 0), (1279, 16, 0), (3000, 40, 1111), (2047, 129, 1500)):
        repeats(Case(63, [L, 300], H_q, H_kv, D, 32, "bf16", chunks=[C, 3], window=window, **kw),
                f"{form} {L} {C} {window}", times=3)


@pytest.mark.parametrize("decode", [True, False])
def test_score_assigned_between_calls(decode):
    """A serving loop's Score: key_start and prefix_len of the step, a window, a cap assigned after it was made, and
    tensors whose storage changes, against a Score made for each call."""
    lens, chunks = [300, 90, 17], None if decode else [60, 90, 5]
    rows = 3 if decode else sum(chunks)
    gen = torch.Generator().manual_seed(5)
    d = OnDevice(Case(64, lens, 4, 2, 64, 16, "bf16", chunks=chunks, prefix=[300, 90, 17], free_invisible=False))
    i32 = lambda hi, n: torch.randint(0, hi, (n,), generator=gen, dtype=torch.int32).cuda()  # noqa: E731
    kept = B.Score()
    for step in range(6):
        args = dict(softcap=[0.0, 20.0, 100.0][step % 3], window=[0, 40, 7][step % 3], key_start=i32(60, rows),
                    prefix_len=i32(90, 3) if step != 4 else None,
                    alibi_slopes=torch.rand(4, generator=gen).cuda() if step % 2 else None)
        d.score = B.Score(**args)
        want = d.run().clone()
        for name, value in args.items():
            setattr(kept, name, value)
        if step == 5:  # other storage under the same tensors
            for t in (kept.key_start, kept.prefix_len, kept.alibi_slopes):
                fresh = t.clone()
                old = t.data
                t.data = fresh
                old.fill_(0)
        d.score = kept
        d.out.fill_(float("nan"))
        assert torch.equal(d.run(), want), step


def outputs(c, score_error):
    """(out, tolerance) from fp64, where score_error(z) bounds the error of a row's visible scores z
    (capped, before the bias) and bias: the tolerance of scored_reference.py with that bound in place of its dz."""
    G = c.H_q // c.H_kv
    q = W.as_f64(c.q)
    out, tol = np.zeros((len(q), c.H_q, c.D)), np.zeros((len(q), c.H_q, c.D))
    half = 2.0 ** -8 if c.dtype == "bf16" else U
    for s, seen in enumerate(c.seen):
        L, C = int(c.lens[s]), int(c.chunks[s])
        for h in range(c.H_q):
            K, V = c.keys[s][:, h // G], c.vals[s][:, h // G]
            for r in range(C):
                vis = np.flatnonzero(seen[r])
                if len(vis) == 0:
                    continue
                row = q[c.qsl[s] + r, h]
                z = K[vis] @ row * c.scale
                mag = (np.abs(K[vis]) @ np.abs(row)).max() * c.scale
                if c.cap:
                    z = c.cap * np.tanh(z / c.cap)
                bias = 0.0 if c.slopes is None else float(c.slopes[h]) * np.abs(L - C + r - vis)
                dz = score_error(mag, z, bias)
                z = z - bias
                w = np.exp(z - z.max())
                w /= w.sum()
                o, A = w @ V[vis], w @ np.abs(V[vis])
                rel = 2 * (dz + 2.0 ** -21) * (1 + dz) + 2 * (len(vis) + 16) * U + (2.0 ** -8 if c.dtype == "bf16" else 0.0)
                out[c.qsl[s] + r, h] = o
                tol[c.qsl[s] + r, h] = rel * A + half * (np.abs(o) + rel * A)
    return out, tol


def within(c, score_error, what):
    got = to_f64(OnDevice(c).run())
    ref, tol = outputs(c, score_error)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.nanmax(np.abs(got - ref) - tol)}"


def one_product(c, amplitude):
    """Queries with one element: scores are exact products of a power of two and a bf16 (or fp32) number."""
    q = np.zeros(W.as_f64(c.q).shape, dtype=np.float32)
    q[..., 3] = amplitude
    c.q = W.f32_to_bf16_bits(q) if c.dtype == "bf16" else q
    return c


@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "bf16"), (4, 2, 128, "f32")])
@pytest.mark.parametrize("form", ["product", "negative product", "slope", "product and slope"])
def test_scores_of_many_thousands(H_q, H_kv, D, dtype, form):
    """Scores up to 10^5 either way, where 8 bits do not resolve what separates two weights. The dot products are
    exact, so a score is off by its later roundings alone: dz = 8 u max(|z|, |bias|) (below 0.1 here)."""
    error = lambda mag, z, bias: 8 * U * max(np.abs(z).max(), np.abs(bias).max())  # noqa: E731
    size = {"product": 2.0 ** 18, "negative product": -2.0 ** 17, "slope": 1.0, "product and slope": 2.0 ** 14}[form]
    slopes = [-30.0 * 2.0 ** -(h % 3) for h in range(H_q)] if "slope" in form else None
    for lens, chunks in (([300, 64, 1], [100, 64, 1]), ([2500, 130], [40, 130]), ([1500, 900, 33], None)):
        c = Case(65, lens, H_q, H_kv, D, 16, dtype, chunks=chunks, slopes=slopes)
        within(one_product(c, size), error, f"{form} {lens}")


# A capped score may be off by 2^-20 of itself (not of the cap) besides the dot product and the later roundings.
CAP_ERROR = {
    "drawn": lambda D: lambda mag, z, bias: ((D + 16) * U * mag + 8 * U * max(np.abs(z).max(), np.abs(bias).max())
                                             + 2.0 ** -20 * np.abs(z).max()),
    "exact": lambda D: lambda mag, z, bias: (8 * U * max(np.abs(z).max(), np.abs(bias).max())
                                             + 2.0 ** -20 * np.abs(z).max())}


def small_cap_error(cap):
    """bf16 prefill takes caps up to 256 by forms of the tanh whose error is 2^-20 of the cap: 2^-12 at most, an
    eighth of what rounding the weights to bf16 may move."""
    return 2.0 ** -20 * cap if cap <= 256 else 0.0


@pytest.mark.parametrize("cap", [60.0, 256.0, 300.0, 1e4, 1e6, 1e9, 1e30, 2.5e38, 2.99e38])
@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "bf16"), (4, 2, 128, "f32")])
def test_large_caps(H_q, H_kv, D, dtype, cap):
    """Caps far above the scores leave them as they are, up to the largest cap that the calls take."""
    for slopes in (None, [0.5 * 2.0 ** -(h % 4) for h in range(H_q)]):
        for lens, chunks in (([300, 64, 1], [100, 64, 1]), ([1500, 40], [30, 40]), ([700, 300, 33, 1], None)):
            c = Case(66, lens, H_q, H_kv, D, 16, dtype, chunks=chunks, cap=cap, slopes=slopes, sharp=4.0)
            within(c, lambda *z: CAP_ERROR["drawn"](D)(*z) + small_cap_error(cap), f"cap {cap} {lens}")


@pytest.mark.parametrize("cap,amplitude", [(40.0, 2.0 ** 8), (100.0, 2.0 ** 9), (256.0, 2.0 ** 11), (300.0, 2.0 ** 11),
                                           (1e4, 2.0 ** 16), (1e6, 2.0 ** 22)])
@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "bf16"), (4, 2, 128, "f32")])
def test_scores_around_a_cap(H_q, H_kv, D, dtype, cap, amplitude):
    """Scores from none over the place where one form of the tanh gives way to the other to several caps."""
    error = CAP_ERROR["exact"](D)
    bound = lambda mag, z, bias: error(mag, z, bias) + small_cap_error(cap)  # noqa: E731
    for lens, chunks in (([300, 64, 1], [100, 64, 1]), ([1500, 40], [30, 40]), ([700, 300, 33, 1], None)):
        c = one_product(Case(67, lens, H_q, H_kv, D, 16, dtype, chunks=chunks, cap=cap), amplitude)
        within(c, bound, f"cap {cap} {lens}")


INT_MAX, INT_MIN = 2 ** 31 - 1, -2 ** 31


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "bf16"), (64, "f32")])
def test_arguments_at_the_ends_of_their_range(D, dtype, form):
    """A window, a prefix and document starts near 2^31 mean all keys, or none."""
    for lens, chunks in (([300, 64, 1, 200], [200, 64, 1, 9]), ([2500, 130], [3, 130]), ([700, 300, 33, 1], None)):
        rows = len(lens) if chunks is None else sum(chunks)
        make = lambda **kw: OnDevice(Case(68, lens, 2, 2, D, 16, dtype, chunks=chunks, free_invisible=False,  # noqa: E731
                                          **FORMS[form], **kw))
        want = make().run().clone()
        for window in (INT_MAX, INT_MAX - 1, INT_MAX - 200, max(lens)):
            assert torch.equal(make(window=window).run(), want), window
        for none in (0, -1, INT_MIN):
            assert torch.equal(make(prefix=[none] * len(lens)).run(), want), none
            assert torch.equal(make(key_start=[none] * rows).run(), want), none
        whole = make(prefix=lens).run().clone()
        for every in (INT_MAX, INT_MAX - 1, max(lens)):
            assert torch.equal(make(prefix=[every] * len(lens)).run(), whole), every
            assert torch.equal(make(prefix=[every] * len(lens), window=INT_MAX).run(), whole), every
        for start in (INT_MAX, INT_MAX - 1, max(lens)):
            d = make(key_start=[start if r % 3 == 1 else 0 for r in range(rows)], prefix=lens, window=INT_MAX)
            got = d.run()
            assert torch.equal(got[1::3], torch.zeros_like(got[1::3])), start
            # The other rows by the definition: their last bits may depend on the empty rows beside them, as
            # the CUDA-core kernel takes new references for all rows of a warp when one row's maximum grows.
            ref, tol = d.c.reference()
            assert (np.abs(to_f64(got) - ref) <= tol).all(), start


def causal(c):
    """The case under a causal prefix: rows see no key behind themselves; cells and pages that no row then sees
    hold NaN and the null block."""
    nan = np.float32(np.nan) if c.dtype == "f32" else np.uint16(0x7fc0)
    for s, (L, C) in enumerate(zip(c.lens.tolist(), c.chunks.tolist())):
        j, seen = np.arange(L), np.zeros((C, L), dtype=bool)
        for r in range(C):
            p = L - C + r
            start = 0 if c.key_start is None else int(c.key_start[c.qsl[s] + r])
            seen[r] = (j <= p) & (j >= start) & ((j < int(c.prefix[s])) | (c.window == 0) | (j > p - c.window))
        assert not (seen & ~c.seen[s]).any()
        c.seen[s] = seen
        any_row = seen.any(axis=0)
        for b in range(-(-L // c.BS)):
            page, mine = c.table[s, b], any_row[b * c.BS:(b + 1) * c.BS]
            if not mine.any():
                c.table[s, b] = 0
            for o in np.flatnonzero(~mine):
                c.k_cache[page, :, o] = nan
                c.v_cache[page, :, o] = nan
    return c


CAUSAL_CHUNKS = {
    "chunks": ([(129, 129), (300, 300), (257, 128), (40, 7), (16, 16), (1, 1), (0, 0), (700, 256)],
               [30, 200, 180, 38, 16, 1, 5, 600]),
    "few rows on long contexts": ([(4099, 3), (2600, 70), (700, 1), (257, 257)], [4098, 2570, 100, 40]),
    "one tile of short contexts": ([(190, 190), (130, 2), (64, 64)], [100, 129, 4])}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("H_q,H_kv,D,BS,dtype", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 64, "bf16"), (4, 2, 64, 16, "f32")])
@pytest.mark.parametrize("name", list(CAUSAL_CHUNKS))
def test_first_tokens_of_a_causal_model_stay_visible(name, H_q, H_kv, D, BS, dtype, form):
    """prefix_causal: rows inside the prefix see what is before them, rows behind it the prefix and their window."""
    pairs, prefix = CAUSAL_CHUNKS[name]
    lens, chunks = zip(*pairs)
    kw = dict(FORMS[form])
    if "slopes" in kw:
        kw["slopes"] = alibi(H_q)
    pos = [p for L, C in pairs for p in range(L - C, L)]
    documents = [p + 1 if i % 17 == 16 else p // 90 * 90 for i, p in enumerate(pos)]
    for window, starts in ((0, None), (50, None), (1, None), (50, documents), (0, documents)):
        c = causal(Case(69, lens, H_q, H_kv, D, BS, dtype, chunks=chunks, prefix=prefix, window=window, key_start=starts, **kw))
        d = OnDevice(c)
        d.score.prefix_causal = True
        ref, tol = c.reference()
        got = to_f64(d.run())
        assert (np.abs(got - ref) <= tol).all(), (window, starts is None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_causal_prefix_prefill_agrees_with_decode_step_by_step(dtype):
    """Each row of a prompt's prefill is what decode gives for the sequence that ends there, first tokens of the
    prompt included (within both calls' tolerances)."""
    L, window, sinks = 120, 24, 5
    c = causal(Case(70, [L], 4, 2, 64, 16, dtype, chunks=[L], cap=20.0, prefix=[sinks], window=window))
    d = OnDevice(c)
    d.score.prefix_causal = True
    rows = to_f64(d.run())
    ref, tol = c.reference()
    for p in (0, 1, sinks - 1, sinks, sinks + 1, window, L - 1):
        q, out = d.q[p:p + 1].contiguous(), torch.empty_like(d.q[:1])
        n = B.pa_decode_scored_workspace_size(1, 4, 2, 64, p + 1, q.dtype)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
        B.pa_decode_scored(out, q, d.k, d.v, d.table, torch.tensor([p + 1], dtype=torch.int32, device="cuda"), p + 1, c.scale,
                           d.score, ws)
        assert (np.abs(to_f64(out)[0] - rows[p]) <= 2 * tol[p]).all(), p


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("H_q,H_kv,dtype", [(4, 2, "f32"), (130, 1, "bf16")])
def test_offsets_past_32_bits_on_the_cuda_cores(H_q, H_kv, dtype, decode):
    """fp32, and groups that the tensor cores do not take: K and V are read through element offsets, which pass
    2^32 here. (bf16 decode takes any group on the tensor cores: there the pool's rows are coordinates.)"""
    D, BS = 128, 16
    c = Case(71, [200, 77], H_q, H_kv, D, BS, dtype, chunks=None if decode else [6, 77], cap=20.0)
    d = OnDevice(c)
    NB, per_block = c.k_cache.shape[0], H_kv * BS * D
    far = (1 << 32) // per_block + 1000
    assert far + NB < 1 << 25
    pools = []
    for small in (d.k, d.v):
        big = torch.empty((far + NB, H_kv, BS, D), dtype=small.dtype, device="cuda")
        big[:NB] = float("nan")      # where a 32-bit offset would land
        big[far - (1 << 32) // per_block:][:NB] = float("nan")
        big[far:] = small
        pools.append(big)
    d.k, d.v = pools
    d.table = d.table + far
    ref, tol = c.reference()
    assert (np.abs(to_f64(d.run()) - ref) <= tol).all()


@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(8, 2, 128, "bf16"), (4, 2, 64, "bf16"), (4, 2, 128, "f32")])
@pytest.mark.parametrize("form", ["plain", "cap", "distance", "cap distance", "large cap", "larger cap"])
@pytest.mark.parametrize("decode", [True, False])
def test_infinite_and_nan_scores(H_q, H_kv, D, dtype, form, decode):
    """Visible keys with an infinite or NaN score. A cap takes infinite scores to its ends; without one a row that
    sees +inf, as one that sees NaN, is NaN, and -inf weighs nothing. Other rows are not touched."""
    kw = dict(cap=1000.0) if form == "larger cap" else dict(FORMS[form], sharp=1.0)
    if "slopes" in kw:
        kw["slopes"] = alibi(H_q)
    lens, chunks = [400, 200, 300], None if decode else [150, 200, 3]
    for value in (np.inf, -np.inf, np.nan):
        c = one_product(Case(72, lens, H_q, H_kv, D, 16, dtype, chunks=chunks, **kw), 4.0)
        d = OnDevice(c)
        for s, j in ((0, 299), (1, 60)):  # sequence 2 has none
            d.k[c.table[s, j // 16], :, j % 16, 3] = float(value)
            c.keys[s] = c.keys[s].copy()
            c.keys[s][j, :, 3] = value
        capped = c.cap > 0
        got = to_f64(d.run())
        bad = np.zeros(got.shape[0], dtype=bool)
        if np.isnan(value) or (value > 0 and not capped):
            for s, j in ((0, 299), (1, 60)):
                bad[c.qsl[s]:c.qsl[s + 1]] = c.seen[s][:, j]
        assert bad.any() == (np.isnan(value) or (value > 0 and not capped))
        assert np.isnan(got[bad]).all(), (form, value)
        # the others by the definition; what they may be off does not depend on the infinite score, which is exact
        # after the cap (its dz is that of a score of the cap's size)
        error = lambda mag, z, bias: (8 * U * max(np.abs(z[np.isfinite(z)]).max(), np.abs(bias).max())  # noqa: E731
                                      + (D + 16) * U * (mag if np.isfinite(mag) else 4.0 * 8.0) + 2.0 ** -20 * c.cap)
        with np.errstate(invalid="ignore", over="ignore"):
            ref, tol = outputs(zero_times_infinity(c), error)
        assert (np.abs(got - ref) <= tol)[~bad].all(), (form, value)


def zero_times_infinity(c):
    """The case with queries of one element cut down to it, so that fp64 forms no 0 x inf either."""
    k = [keys[..., 3:4] for keys in c.keys]
    cut = Case.__new__(Case)
    cut.__dict__.update(c.__dict__)
    cut.keys = k
    q = W.as_f64(c.q)[..., 3:4]
    cut.q = q.astype(np.float32) if c.dtype == "f32" else W.f32_to_bf16_bits(q.astype(np.float32))
    return cut


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_threads_with_a_stream_and_a_workspace_each(dtype, decode):
    """Calls of several threads at once, each with its stream and workspace, equal the same calls alone."""
    import threading
    calls, want = [], []
    for i, lens in enumerate(([2000, 33], [700, 700], [3001], [50] * 20)):
        chunks = None if decode else [min(9, L) for L in lens]
        calls.append(OnDevice(Case(73 + i, lens, 4, 2, 64, 16, dtype, chunks=chunks, cap=[0.0, 20.0, 100.0, 400.0][i])))
        want.append(calls[-1].run().clone())
    torch.cuda.synchronize()
    failed = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(25):
                calls[i].out.fill_(float("nan"))
                calls[i].run()
                stream.synchronize()
                if not torch.equal(calls[i].out, want[i]):
                    failed.append(i)
                    return

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_tensors_that_are_not_contiguous_or_elsewhere_are_refused():
    c = Case(77, [300, 40], 4, 2, 64, 16, "bf16", cap=20.0, slopes=alibi(4), prefix=[3, 4], key_start=[0, 1])
    wide = lambda t: torch.stack([t, t], dim=-1)[..., 0]  # noqa: E731
    for name in ("out", "q", "k", "v", "table", "lens"):
        for change in (wide, lambda t: t.cpu()):
            d = OnDevice(c)
            setattr(d, name, change(getattr(d, name)))
            with pytest.raises(ValueError):
                d.run()
    for name in ("alibi_slopes", "prefix_len", "key_start"):
        for change in (wide, lambda t: t.cpu(), lambda t: t[:1]):
            d = OnDevice(c)
            setattr(d.score, name, change(getattr(d.score, name)))
            with pytest.raises(ValueError):
                d.run()
        d = OnDevice(c)
        setattr(d.score, name, getattr(d.score, name).double())
        with pytest.raises(TypeError):
            d.run()
    d = OnDevice(c)
    for ws in (d.ws[::2], d.ws.cpu()):
        d.ws = ws
        with pytest.raises(ValueError):
            d.run()


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_row_that_sees_one_key_is_its_value(form, H_q, H_kv, D):
    """One visible key has weight 1 whatever its score: the output is its V, bit for bit (the two roundings of a
    quotient p v / p in fp32 are far below half a step of bf16)."""
    kw = dict(FORMS[form])
    if "slopes" in kw:
        kw["slopes"] = alibi(H_q)
    for lens, chunks in (([1, 190, 64, 17], [1, 190, 9, 17]), ([1200, 300, 1], [200, 300, 1]), ([3000], [4]),
                         ([1, 1500, 33, 777], None)):
        c = Case(78, lens, H_q, H_kv, D, 16, "bf16", chunks=chunks, window=1, **kw)
        got = to_f64(OnDevice(c).run())
        for s, (L, C) in enumerate(zip(lens, chunks or [1] * len(lens))):
            for r in range(C):
                v = c.vals[s][L - C + r]  # [H_kv, D]
                assert np.array_equal(got[c.qsl[s] + r], np.repeat(v, H_q // H_kv, axis=0)), (form, L, r)


@pytest.mark.parametrize("H_q,H_kv,D", [(32, 2, 64), (32, 4, 128)])
@pytest.mark.parametrize("cap", [5.0, 30.0, 51.0])
def test_rows_of_two_and_three_keys(cap, H_q, H_kv, D):
    """Few weights of one size, where an error of the sums does not average out against those of P V."""
    for seed in range(6):
        for window in (2, 3):
            check(Case(90 + seed, [189, 8, 17, 77, 13], H_q, H_kv, D, 16, "bf16", chunks=[149, 8, 7, 47, 1], window=window,
                       cap=cap), f"{cap} {window} {seed}")
