"""Rotation into the cache and reads of 4-bit pools against the fp64 definitions of fp4_reference.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import fp4_reference as R  # noqa: E402
from helpers import to_dev, to_f64, to_host_bits  # noqa: E402
from paged_kv_cache_238_gb300 import binding as B  # noqa: E402
from paged_kv_cache_238_gb300 import workloads as W  # noqa: E402

pytestmark = pytest.mark.gpu
LONGEST = 500


@pytest.fixture(autouse=True)
def no_errors_left():
    B.pa_get_device_errors()
    yield
    assert B.pa_get_device_errors() == 0


def typed(x, dtype):
    return W.f32_to_bf16_bits(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)


def table(rot, seed=1):
    rate = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    angle = np.arange(LONGEST)[:, None] * 37.7 * rate  # far positions among them
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


class New:
    """Tokens with their slots, and pools that hold something already."""

    def __init__(self, T, Hq, H, D, rot, BS, dtype, fp4, seed=0, packed=True, ks=1.0, vs=1.0, pad=()):
        rng = np.random.default_rng(seed)
        self.T, self.Hq, self.H, self.D, self.BS, self.dtype, self.fp4, self.ks, self.vs = T, Hq, H, D, BS, dtype, fp4, ks, vs
        qkv = rng.standard_normal((T, Hq + 2 * H, D))
        qkv[:, Hq:Hq + H] *= ks
        qkv[:, Hq + H:] *= vs
        self.bits = typed(qkv, dtype)
        self.x = W.as_f64(self.bits)
        self.cs = table(rot)
        self.pos = rng.integers(0, LONGEST, T)
        self.NB = 2 + -(-T // BS)
        self.slots = BS + rng.permutation((self.NB - 1) * BS)[:T]
        for t in pad:
            self.slots[t] = -1 - t
        old = [rng.standard_normal((self.NB, H, BS, D)) * f for f in (ks, vs)]
        self.old = [R.to_pool(o, f) if fp4 else typed(o, dtype) for o, f in zip(old, (ks, vs))]
        d = to_dev(self.bits)
        self.q, self.k, self.v = d.split([Hq, H, H], dim=1)
        if not packed:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.pools = [to_dev(o) for o in self.old]
        self.q_out = torch.full((T, Hq, D), 7.0, dtype=self.q.dtype, device="cuda")

    def run(self, interleaved, **kw):
        a = dict(q_out=self.q_out, q=self.q, k=self.k, v=self.v, positions=to_dev(self.pos), cos_sin=to_dev(self.cs),
                 k_cache=self.pools[0], v_cache=self.pools[1], slot_mapping=to_dev(self.slots), interleaved=interleaved)
        if self.fp4:
            a.update(k_scale=self.ks, v_scale=self.vs)
        a.update(kw)
        B.pa_rotate_and_cache(**a)
        torch.cuda.synchronize()

    def check(self, interleaved, skipped=()):
        """q_out and the pools; `skipped`: tokens that had to be left out."""
        Hq, H, BS = self.Hq, self.H, self.BS
        done = np.array([t not in skipped for t in range(self.T)])
        q, qm = R.rotate(self.x[:, :Hq], self.cs[self.pos % LONGEST].astype(np.float64), interleaved)
        k, km = R.rotate(self.x[:, Hq:Hq + H], self.cs[self.pos % LONGEST].astype(np.float64), interleaved)
        got = to_f64(self.q_out)
        assert (np.abs(got - q) <= R.rotate_tolerance(q, qm, self.dtype))[done].all()
        assert (got[~done] == 7.0).all()
        wrote = done & (self.slots >= 0)
        blk, at = self.slots[wrote] // BS, self.slots[wrote] % BS
        for pool, old, rows, mag, f in ((self.pools[0], self.old[0], k, km, self.ks),
                                        (self.pools[1], self.old[1], self.x[:, Hq + H:], None, self.vs)):
            if self.fp4:  # every byte of the pool
                want = old.copy()
                codes, scales = R.quantise(R.rounded(rows[wrote], self.dtype), f)
                pages = want.reshape(self.NB, H, BS // 16, 9 * self.D)
                want_s = pages[..., 8 * self.D:].reshape(self.NB, H, BS, -1).copy()
                want_s[blk, :, at] = scales
                pages[..., 8 * self.D:] = want_s.reshape(pages[..., 8 * self.D:].shape)
                c = pages[..., :8 * self.D].reshape(self.NB, H, BS, -1).copy()
                c[blk, :, at] = codes[..., 0::2] | codes[..., 1::2] << 4
                pages[..., :8 * self.D] = c.reshape(pages[..., :8 * self.D].shape)
                assert (pool.cpu().numpy() == want).all()
                continue
            bits = to_host_bits(pool)
            new = np.zeros((self.NB, BS), dtype=bool)
            new[blk, at] = True
            kept = ~new[:, None].repeat(H, axis=1)
            assert (bits[kept] == old[kept]).all()
            got = W.as_f64(bits)[blk, :, at]
            if mag is None:
                assert (got == rows[wrote]).all()
            else:
                assert (np.abs(got - rows[wrote]) <= R.rotate_tolerance(rows[wrote], mag[wrote], self.dtype)).all()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,rot,BS,packed", [
    (1, 1, 1, 64, 64, 16, True), (5, 6, 2, 64, 16, 32, True), (67, 12, 4, 64, 48, 16, False),
    (33, 8, 8, 128, 128, 128, True), (40, 5, 1, 128, 96, 64, True), (700, 32, 8, 128, 128, 16, True),
    (1500, 16, 16, 64, 32, 64, False)])
def test_rotate_and_cache(fp4, dtype, interleaved, T, Hq, H, D, rot, BS, packed):
    n = New(T, Hq, H, D, rot, BS, dtype, fp4, seed=T, packed=packed, ks=0.25, vs=2.0 ** -5, pad=(2, 3) if T > 4 else ())
    n.run(interleaved)
    n.check(interleaved)


@pytest.mark.parametrize("fp4", [False, True])
def test_tokens_that_are_left_out(fp4):
    n = New(40, 4, 2, 64, 64, 16, "bf16", fp4, pad=(5,))
    n.pos[[3, 17]] = [-1, LONGEST]
    n.run(False)
    assert B.pa_get_device_errors() == B.PA_DEVERR_POSITION
    n.check(False, skipped=(3, 17))
    # a slot past the pool: q is rotated, nothing is written
    n = New(40, 4, 2, 64, 64, 16, "bf16", fp4)
    n.slots[[7, 8]] = [n.NB * 16, 2 ** 40]
    n.run(False)
    assert B.pa_get_device_errors() == B.PA_DEVERR_SLOT_RANGE
    n.slots[[7, 8]] = -1
    n.check(False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_q_in_place_and_absent(interleaved):
    n = New(50, 8, 2, 128, 64, 16, "bf16", False)
    want, mag = R.rotate(n.x[:, :8], n.cs[n.pos].astype(np.float64), interleaved)
    n.run(interleaved, q_out=n.q)  # a view of the packed projection
    assert (np.abs(to_f64(n.q) - want) <= R.rotate_tolerance(want, mag, "bf16")).all()
    n.q_out = n.q.contiguous()
    n.check(interleaved)
    n = New(50, 8, 2, 128, 64, 16, "bf16", True)
    n.run(interleaved, q=None, q_out=None)
    n.q_out = to_dev(typed(R.rotate(n.x[:, :8], n.cs[n.pos].astype(np.float64), interleaved)[0], "bf16"))
    n.check(interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("factor", [1.0, 2.0 ** -24, 2.0 ** 24])
def test_borders_of_the_codes(dtype, factor):
    """Values on every border between codes and between scales, and next to it; the ends of the range."""
    H, D, BS, T = 2, 64, 16, 508
    groups = np.zeros((T * H * D // 16, 16))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    s = R.e4m3_values(np.arange(127, dtype=np.uint8))
    mids = (s[:-1] + s[1:]) / 2
    near = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    for g in range(len(groups)):
        kind, i = g % 4, g // 4
        if kind < 2:  # borders of codes under scale i
            sc = s[1 + i % 126]
            y = np.concatenate([ties, -ties, [6.0], [0.1]]) * sc
            groups[g] = y if kind == 0 else y * (1 + near * np.where(np.arange(16) % 2, 1, -1))
            groups[g, 14] = 6 * sc
        else:  # borders of scales: the largest magnitude is 6 times a midpoint, or next to it
            m = 6 * mids[i % 126]
            groups[g] = np.linspace(-1, 1, 16) * m * 0.99
            groups[g, i % 16] = m * (1 if kind == 2 else 1 + near * (1 if i % 2 else -1))
    groups[:6] = [[0.0] * 16, [2.0 ** -12] * 16, [2689.0] * 16, [1e6] * 16, [-3e4] * 8 + [1.0] * 8, [2.0 ** -10 * 6] * 16]
    n = New(T, 1, H, D, 64, BS, dtype, True, ks=factor, vs=factor)
    n.cs = np.concatenate([np.ones((LONGEST, 32)), np.zeros((LONGEST, 32))], axis=1).astype(np.float32)  # no turn
    bits = typed(groups.reshape(T, H, D) * factor, dtype)
    n.k = n.v = to_dev(bits)
    n.x[:, 1:1 + H] = n.x[:, 1 + H:] = W.as_f64(bits)
    n.run(False)
    n.check(False)


def test_numbers_without_a_code():
    n = New(4, 1, 1, 64, 64, 16, "bf16", True)
    n.cs = np.concatenate([np.ones((LONGEST, 32)), np.zeros((LONGEST, 32))], axis=1).astype(np.float32)
    x = n.x[:, 2:].copy()
    x[0, 0, 3] = np.inf
    x[1, 0, 20] = -np.inf
    x[2, 0, 40] = np.nan
    n.v = to_dev(typed(x, "bf16"))
    n.run(False)
    out = [torch.empty(4, 1, 64, dtype=torch.float32, device="cuda") for _ in range(2)]
    B.pa_gather_fp4(*out, *n.pools, to_dev(n.slots))
    got = out[1].cpu().numpy()
    assert np.isfinite(got).all()
    assert got[0, 0, 3] == 2688.0 and got[1, 0, 20] == -2688.0
    y = x[2, 0, 32:48].copy()
    y[8] = 0.0  # the NaN takes no part in its group's scale
    codes, scales = R.quantise(y[None])
    want = R.GRID[codes & 7] * np.where(codes & 8, -1, 1) * R.e4m3_values(scales)[..., None][0]
    keep = np.arange(16) != 8
    assert (got[2, 0, 32:48][keep] == want[0][keep]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_turns_that_are_infinite(dtype, interleaved):
    """An infinity turned is two infinities (its angle's sine and cosine are not zero), and so is a turn past the type's
    range: stored as the largest code under the largest scale. Other groups are as ever."""
    n = New(3, 1, 1, 64, 64, 16, dtype, True)
    n.pos[:] = 1
    i = 9  # a pair whose angle is neither small nor near a multiple of 90 degrees
    angle = np.float32(0.7)
    n.cs[1, i], n.cs[1, 32 + i] = np.cos(angle), np.sin(angle)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, 32 + i)
    x = n.x[:, 1:2].copy()
    x[0, 0, lo] = np.inf
    x[1, 0, hi] = -np.inf
    x[2, 0, [lo, hi]] = 3e38
    n.bits[:, 1:2] = typed(x, dtype)
    n.k = to_dev(n.bits[:, 1:2].copy())
    n.run(interleaved)
    out = [torch.empty(3, 1, 64, dtype=torch.float32, device="cuda") for _ in range(2)]
    B.pa_gather_fp4(*out, *n.pools, to_dev(n.slots))
    got = out[0].cpu().numpy()[:, 0]
    assert np.isfinite(got).all()
    assert (got[0, [lo, hi]] == 2688.0).all()
    assert (got[1, [lo, hi]] == [2688.0, -2688.0]).all()
    assert got[2, hi] == 2688.0  # 3e38 (cos + sin)
    k, _ = R.rotate(n.x[:, 1:2], n.cs[n.pos].astype(np.float64), interleaved)
    codes, scales = R.quantise(R.rounded(k, dtype))
    want = R.GRID[codes & 7] * np.where(codes & 8, -1, 1) * np.repeat(R.e4m3_values(scales), 16, axis=-1)
    same = ~np.isin(np.arange(64) // 16, [lo // 16, hi // 16])
    assert (got[:, same] == want[:, 0][:, same]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,D,BS", [(1, 64, 16), (3, 128, 32), (8, 128, 128)])
def test_gather(dtype, H, D, BS):
    rng = np.random.default_rng(3)
    NB, f = 5, (0.25, 4.0)
    pools = [R.to_pool(rng.standard_normal((NB, H, BS, D)) * x, x) for x in f]
    slots = rng.integers(0, NB * BS, 77)
    slots[[0, 5, 76]] = [-1, slots[4], NB * BS - 1]
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    out = [torch.full((77, H, D), 9.0, dtype=t, device="cuda") for _ in range(2)]
    B.pa_gather_fp4(*out, to_dev(pools[0]), to_dev(pools[1]), to_dev(slots), k_scale=f[0], v_scale=f[1])
    for o, p, x in zip(out, pools, f):
        want = R.from_pool(p, x).transpose(0, 2, 1, 3).reshape(NB * BS, H, D)[slots]
        want[0] = 0.0
        assert (to_f64(o) == want).all()
    slots[3] = NB * BS
    B.pa_gather_fp4(*out, to_dev(pools[0]), to_dev(pools[1]), to_dev(slots), k_scale=f[0], v_scale=f[1])
    assert B.pa_get_device_errors() == B.PA_DEVERR_SLOT_RANGE
    assert (to_f64(out[0])[3] == 0.0).all()


def test_nothing_to_do():
    n = New(2, 4, 2, 64, 64, 16, "bf16", True)
    z = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    zq, zi = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    B.pa_rotate_and_cache(zq, zq, z, z, zi, to_dev(n.cs), *n.pools, zi)
    B.pa_gather_fp4(z, z, *n.pools, zi)
    assert (n.pools[0].cpu().numpy() == n.old[0]).all()


def test_refused_tensors():
    n = New(6, 4, 2, 64, 64, 16, "bf16", True)
    ok = dict(q_out=n.q_out, q=n.q, k=n.k, v=n.v, positions=to_dev(n.pos), cos_sin=to_dev(n.cs), k_cache=n.pools[0],
              v_cache=n.pools[1], slot_mapping=to_dev(n.slots))
    for bad in (dict(q=n.q.float()), dict(q_out=n.q_out[:, :2]), dict(q=n.q.transpose(1, 2)), dict(v=n.v[:, :1]),
                dict(v=n.v[:3]), dict(k=n.k[..., ::2]), dict(positions=to_dev(n.pos).int()), dict(cos_sin=to_dev(n.cs).half()),
                dict(cos_sin=to_dev(n.cs)[:, ::2]), dict(k_cache=n.pools[0][:, :1]), dict(v_cache=n.pools[1][:1]),
                dict(k_cache=n.pools[0].to(torch.bfloat16)), dict(slot_mapping=to_dev(n.slots)[:3]), dict(v=n.v.cpu()),
                dict(cos_sin=to_dev(n.cs).cpu())):
        with pytest.raises((ValueError, TypeError)):
            B.pa_rotate_and_cache(**{**ok, **bad})
    with pytest.raises(B.PaError):  # heads not apart by whole 16-byte chunks
        B.pa_rotate_and_cache(**{**ok, "k": torch.zeros(6 * 132, dtype=torch.bfloat16, device="cuda").as_strided((6, 2, 64), (132, 64, 1))})
    assert (n.pools[0].cpu().numpy() == n.old[0]).all()


def test_captured_and_on_another_stream():
    n = New(64, 8, 2, 128, 128, 16, "bf16", True)
    args = (n.q_out, n.q, n.k, n.v, to_dev(n.pos), to_dev(n.cs), *n.pools, to_dev(n.slots))
    rows = [torch.empty(64, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.pa_rotate_and_cache(*args, stream=s)
    s.synchronize()
    n.check(False)
    for p, o in zip(n.pools, n.old):
        p.copy_(to_dev(o))
    n.q_out.fill_(7.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.pa_rotate_and_cache(*args)
        B.pa_gather_fp4(*rows, *n.pools, args[-1])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    n.check(False)
    codes, scales = R.quantise(n.x[:, 10:])
    want = R.GRID[codes & 7] * np.where(codes & 8, -1, 1) * np.repeat(R.e4m3_values(scales), 16, axis=-1)
    assert (to_f64(rows[1]) == want).all()
