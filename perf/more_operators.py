"""Cases and plain forms of the operators around the 4-bit paged KV pool, for measuring them.

  rotate    new tokens' q and k rotated by their positions, k and v written into the paged pool
            in their own type (bf16 or fp32)
  quantise  the same into a pool held in 4 bits, and the pool's rows read back as values
  decode    one query row per sequence over the pages of a 4-bit pool
  prefill   a chunk of new query rows per sequence over the pages of a 4-bit pool

The 4-bit pool: 16 consecutive dims of a token's head row share a scale s in e4m3, the largest
magnitude / 6; each value is a code in e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) times s
times the pool's own factor, a power of two. A page of 16 tokens of a kv head is 16 rows of codes
(two a byte, the even dim in the low half), then 16 rows of scales. K is rounded to the call's type
between rotation and quantisation.

`own` False: `run` computes them from elementary torch operations. `own` True: `run` calls the
library's entry points. Lengths come from the case alone, their order, the pages and all values from
the seed.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_NEG = float("-inf")
_PAGE = 16   # tokens of a page
_GROUP = 16  # dims that share a scale


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step of a serving batch: one new token per sequence, where latency counts
        _rotate("rotate step", tokens=64, seqs=64, hq=32, hkv=8, dim=128, rot=128, block=16),
        # the new tokens of a mixed step: prompt chunks and decode tokens, padding among them
        _rotate("rotate prompt", tokens=8448, seqs=16, hq=32, hkv=8, dim=128, rot=128, block=16, pad=16),
        # fp32 small model, interleaved pairs, half of the dims rotated, ragged
        _rotate("rotate f32 partial", tokens=1003, seqs=5, hq=12, hkv=4, dim=64, rot=32, block=32, dtype="f32",
                interleaved=True, pad=3),
        # the same step and prompt into a 4-bit pool
        _rotate("quantise step", tokens=64, seqs=64, hq=32, hkv=8, dim=128, rot=128, block=16, fp4=True),
        _rotate("quantise prompt", tokens=8448, seqs=16, hq=32, hkv=8, dim=128, rot=128, block=64, pad=16, fp4=True,
                vs=0.03125),
        # a few interactive users: the smallest decode step
        _decode("decode few", seqs=4, lo=17, hi=700, hq=32, hkv=8, dim=128, block=16),
        # a serving batch of ragged contexts
        _decode("decode batch", seqs=64, lo=500, hi=16384, hq=32, hkv=8, dim=128, block=64, vs=0.03125),
        # one kv head per q head, head_dim 64, short to middling contexts
        _decode("decode mha", seqs=96, lo=16, hi=2048, hq=16, hkv=16, dim=64, block=32),
        # few long contexts, eight q heads per kv head: the work is split along the keys
        _decode("decode long", seqs=8, lo=20000, hi=32768, hq=64, hkv=8, dim=128, block=16),
        # fp32 queries, three q heads per kv head, ragged from one token up
        _decode("decode f32", seqs=24, lo=1, hi=777, hq=12, hkv=4, dim=64, block=16, dtype="f32"),
        # the prefill half of a mixed step: 16 chunks of 512 tokens on up to 4096 earlier ones
        _prefill("prefill chunks", seqs=16, clo=512, chi=512, plo=0, phi=4096, hq=32, hkv=8, dim=128, block=16),
        # one kv head per q head, head_dim 64, ragged chunks
        _prefill("prefill mha ragged", seqs=8, clo=100, chi=1000, plo=0, phi=1500, hq=16, hkv=16, dim=64, block=32,
                 vs=0.03125),
    ]


def _rotate(name, tokens, seqs, hq, hkv, dim, rot, block, dtype="bf16", interleaved=False, pad=0, fp4=False, ks=1.0,
            vs=1.0, packed=True):
    return dict(name=name, kind="quantise" if fp4 else "rotate", tokens=tokens, seqs=seqs, hq=hq, hkv=hkv, dim=dim,
                rot=rot, block=block, dtype=dtype, interleaved=interleaved, pad=pad, ks=ks, vs=vs, packed=packed)


def _decode(name, seqs, lo, hi, hq, hkv, dim, block, dtype="bf16", ks=1.0, vs=1.0):
    return dict(name=name, kind="decode", seqs=seqs, lo=lo, hi=hi, hq=hq, hkv=hkv, dim=dim, block=block, dtype=dtype,
                ks=ks, vs=vs)


def _prefill(name, seqs, clo, chi, plo, phi, hq, hkv, dim, block, dtype="bf16", ks=1.0, vs=1.0):
    return dict(name=name, kind="prefill", seqs=seqs, clo=clo, chi=chi, plo=plo, phi=phi, hq=hq, hkv=hkv, dim=dim,
                block=block, dtype=dtype, ks=ks, vs=vs)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "rotate", "quantise"])
    hkv, dim, block = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    group = min(rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16]), 64 // hkv)
    shape = dict(kind=kind, hq=hkv * group, hkv=hkv, dim=dim, block=block, dtype="f32" if rng.random() < 0.2 else "bf16",
                 ks=rng.choice([1.0, 1.0, 0.25, 4.0]), vs=rng.choice([1.0, 0.25, 0.03125]))
    if kind in ("rotate", "quantise"):
        tokens = min(_log_int(rng, 1, 16384), 30_000_000 // (hkv * (group + 2) * dim))
        return dict(shape, tokens=tokens, seqs=min(tokens, _log_int(rng, 1, 200)),
                    rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.4,
                    pad=rng.choice([0, 0, tokens // 50]), packed=rng.random() < 0.7)
    if kind == "decode":
        seqs = _log_int(rng, 1, 200)
        hi = max(2, min(_log_int(rng, 8, 40000), 250_000_000 // (seqs * hkv * dim)))
        return dict(shape, seqs=seqs, lo=max(1, int(hi * rng.choice([0.01, 0.1, 0.5, 1.0]))), hi=hi)
    seqs = _log_int(rng, 1, 16)
    phi = _log_int(rng, 1, 10000)
    chi = max(1, min(_log_int(rng, 1, 2048), int(0.6e9 / (seqs * hkv * group * (phi + 600)))))
    if shape["dtype"] == "f32":
        chi = min(chi, 300)
    return dict(shape, seqs=seqs, clo=max(1, int(chi * rng.choice([0.05, 0.3, 1.0]))), chi=chi,
                plo=rng.choice([0, phi // 2, phi]), phi=phi)


# ------------------------------------------------------------------------- what a case means

def _spread(lo, hi, n):
    """n whole numbers from lo to hi, spread over their logarithm."""
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return [int(round(math.exp(a + (b - a) * (i / (n - 1) if n > 1 else 1.0)) - 1.0)) for i in range(n)]


def _even(lo, hi, n):
    """n whole numbers from lo to hi at equal steps."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _rows(case):
    """(keys, query rows) of each sequence, before the seed orders them."""
    n = case["seqs"]
    if case["kind"] == "decode":
        return [(L, 1) for L in _spread(case["lo"], case["hi"], n)]
    chunks, priors = _spread(case["clo"], case["chi"], n), _even(case["plo"], case["phi"], n)
    random.Random(n).shuffle(priors)
    return [(p + c, c) for p, c in zip(priors, chunks)]


def _pool_blocks(case):
    """Blocks of a rotate case's pool: the null block, the new tokens' and a few held ones."""
    need = -(-case["tokens"] // case["block"])
    return 1 + need + case["seqs"] // 8 + 2


def work(case):
    size, D, H = (4 if case["dtype"] == "f32" else 2), case["dim"], case["hkv"]
    if case["kind"] in ("rotate", "quantise"):
        T, kept = case["tokens"], case["tokens"] - case["pad"]
        moved = 2 * T * case["hq"] * D * size + T * (case["rot"] * 4 + 16) + 2 * kept * H * D * size
        flops = 3 * T * case["rot"] * (case["hq"] + H)
        if case["kind"] == "rotate":
            return {"bytes": moved + 2 * kept * H * D * size, "flops": flops}
        slots, row = _pool_blocks(case) * case["block"], D * 9 // 16
        # codes written; then all of the pool read, and written as values
        return {"bytes": moved + 2 * kept * H * row + 2 * slots * H * (row + D * size), "flops": flops}
    rows = _rows(case)
    seen = sum(C * (L - C) + C * (C + 1) // 2 for L, C in rows)
    keys, queries = sum(L for L, _ in rows), sum(C for _, C in rows)
    return {"bytes": 2 * keys * H * (D * 9 // 16) + 2 * queries * case["hq"] * D * size, "flops": 4 * seen * case["hq"] * D}


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_rotate(case, g, seed) if case["kind"] in ("rotate", "quantise") else _prepare_attend(case, g, seed)


def _prepare_rotate(case, g, seed):
    dt, T, D, BS = _DTYPES[case["dtype"]], case["tokens"], case["dim"], case["block"]
    Hq, H, R, NB, n = case["hq"], case["hkv"], case["rot"], _pool_blocks(case), case["seqs"]
    longest = 32768
    # angles in 64 bits, the table in 32: what a program makes once for its longest context
    rate = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * rate
    cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    # each sequence's tokens continue it from a position of its own
    host = torch.Generator().manual_seed(seed)
    counts = [T // n + (i < T % n) for i in range(n)]
    starts = torch.randint(0, longest - max(counts), (n,), generator=host).tolist()
    positions = torch.cat([torch.arange(s, s + c) for s, c in zip(starts, counts)]).cuda()
    padded = torch.randperm(T, generator=host)[:case["pad"]]
    slots = BS + torch.randperm((NB - 1) * BS, generator=host)[:T]
    slots[padded] = -1
    keep = torch.nonzero(slots >= 0).flatten().cuda()
    amp = torch.cat([torch.ones(Hq), torch.full((H,), case["ks"]), torch.full((H,), case["vs"])]).cuda()
    qkv = (torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda") * amp[:, None]).to(dt)
    q, k, v = qkv.split([Hq, H, H], dim=1)  # views of the packed projection
    if not case["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    s = dict(case=case, q=q, k=k, v=v, positions=positions, cos_sin=cos_sin, slots=slots.cuda(), keep=keep,
             kept_slots=slots.cuda()[keep], q_out=torch.empty(T, Hq, D, dtype=dt, device="cuda"))
    shape = (NB, H, BS, D)
    held = [torch.randn(shape, generator=g, device="cuda") * f for f in (case["ks"], case["vs"])]
    if case["kind"] == "rotate":
        s["k_cache"], s["v_cache"] = held[0].to(dt), held[1].to(dt)
        return s
    s["k_cache"], s["v_cache"] = _pool4(held[0], case["ks"]), _pool4(held[1], case["vs"])
    s["all_slots"] = torch.arange(NB * BS, device="cuda")
    s["k_rows"], s["v_rows"] = (torch.empty(NB * BS, H, D, dtype=dt, device="cuda") for _ in range(2))
    return s


def _prepare_attend(case, g, seed):
    order = torch.randperm(case["seqs"], generator=torch.Generator().manual_seed(seed)).tolist()
    every = _rows(case)
    rows = [every[i] for i in order]
    H, D, BS, dt = case["hkv"], case["dim"], case["block"], _DTYPES[case["dtype"]]
    lens, chunks = [L for L, _ in rows], [C for _, C in rows]
    blocks = [-(-L // BS) for L in lens]
    held = torch.arange(max(blocks))[None, :] < torch.tensor(blocks)[:, None]
    total = sum(blocks)
    NB = 1 + total + total // 16
    held = held.cuda()
    table = torch.zeros(held.shape, dtype=torch.int32, device="cuda")
    table[held] = 1 + torch.randperm(NB - 1, generator=g, device="cuda", dtype=torch.int32)[:total]
    pools = []
    for factor in (case["ks"], case["vs"]):
        pool = torch.empty(NB, H, BS, D * 9 // 16, dtype=torch.uint8, device="cuda")
        step = max(1, 64_000_000 // (H * BS * D))
        for b in range(0, NB, step):
            n = min(step, NB - b)
            pool[b:b + n] = _pool4(torch.randn(n, H, BS, D, generator=g, device="cuda") * factor, factor)
        pools.append(pool)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = [0]
    for C in chunks:
        starts.append(starts[-1] + C)
    q = torch.randn(starts[-1], case["hq"], D, generator=g, device="cuda").to(dt)
    s = dict(case=case, scale=1.0 / math.sqrt(D), table=table, lens=i32(lens), qsl=i32(starts), k=pools[0], v=pools[1], q=q,
             out=torch.empty_like(q), max_len=max(lens), max_chunk=max(chunks))
    if own:
        from paged_kv_cache_238_gb300 import binding as pa
        if case["kind"] == "decode":
            n = pa.pa_decode_fp4_workspace_size(case["seqs"], case["hq"], H, D, s["max_len"], dt)
        else:
            n = pa.pa_prefill_fp4_workspace_size(case["seqs"], s["max_chunk"], case["hq"], H, D, s["max_len"], dt)
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    return s


# ------------------------------------------------------------------- the 4-bit pool, plain form

def _codes(x, factor):
    """x [..., D] -> (codes 0..15 [..., D], scales as e4m3 bytes [..., D / 16]); in 64 bits: values lie
    next to the borders between codes."""
    y = (x.double() / factor).unflatten(-1, (-1, _GROUP))
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    a = y.abs() / s.double().clamp(min=2.0 ** -20)[..., None]
    # ties go to the even code
    code = torch.zeros_like(a, dtype=torch.uint8)
    code += (a > 0.25)
    code += (a >= 0.75)
    code += (a > 1.25)
    code += (a >= 1.75)
    code += (a > 2.5)
    code += (a >= 3.5)
    code += (a > 5.0)
    code = torch.where(s.float()[..., None] > 0, code + 8 * (y < 0).to(torch.uint8), 0)
    return code.flatten(-2), s.view(torch.uint8)


def _packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _parts(pool):
    """Views of a pool [..., BS, 9 D / 16]: codes [..., BS / 16, 16, D / 2] and scales [..., BS / 16, 16, D / 16]."""
    row = pool.shape[-1]
    pages = pool.view(*pool.shape[:-2], pool.shape[-2] // _PAGE, _PAGE * row)
    codes, scales = pages.split([_PAGE * row * 8 // 9, _PAGE * row // 9], dim=-1)
    return codes.unflatten(-1, (_PAGE, -1)), scales.unflatten(-1, (_PAGE, -1))


def _pool4(x, factor):
    """x [NB, H, BS, D] as a 4-bit pool."""
    NB, H, BS, D = x.shape
    pool = torch.empty(NB, H, BS, D * 9 // 16, dtype=torch.uint8, device=x.device)
    codes, scales = _parts(pool)
    c, s = _codes(x, factor)
    codes.copy_(_packed(c).view(codes.shape))
    scales.copy_(s.view(scales.shape))
    return pool


def _values(pool, factor):
    """The values of a pool [..., BS, 9 D / 16], fp32 [..., BS, D]."""
    packed, scales = _parts(pool)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=pool.device)
    codes = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2)
    x = grid[codes.int()].unflatten(-1, (-1, _GROUP)) * (scales.contiguous().view(torch.float8_e4m3fn).float() * factor)[..., None]
    return x.flatten(-2).flatten(-3, -2)


# -------------------------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    if kind in ("rotate", "quantise"):
        return _plain_rotate(state)
    return _plain_decode(state) if kind == "decode" else _plain_prefill(state)


def _own(s, kind):
    from paged_kv_cache_238_gb300 import binding as pa
    case = s["case"]
    if kind == "rotate":
        pa.pa_rotate_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"],
                               s["slots"], interleaved=case["interleaved"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if kind == "quantise":
        pa.pa_rotate_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"], s["v_cache"],
                               s["slots"], interleaved=case["interleaved"], k_scale=case["ks"], v_scale=case["vs"])
        pa.pa_gather_fp4(s["k_rows"], s["v_rows"], s["k_cache"], s["v_cache"], s["all_slots"], k_scale=case["ks"],
                         v_scale=case["vs"])
        return [s["q_out"], s["k_rows"], s["v_rows"]]
    if kind == "decode":
        pa.pa_decode_fp4(s["out"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["max_len"], s["scale"], s["workspace"],
                         k_scale=case["ks"], v_scale=case["vs"])
    else:
        pa.pa_prefill_fp4(s["out"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["qsl"], s["max_chunk"], s["max_len"],
                          s["scale"], s["workspace"], k_scale=case["ks"], v_scale=case["vs"])
    return s["out"]


def _rotated(x, cs, interleaved):
    """x [T, H, D] with its first R dims rotated; cs [T, R]: cosines, sines."""
    R = cs.shape[1]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _plain_rotate(s):
    case = s["case"]
    dt, BS, D = s["q"].dtype, case["block"], case["dim"]
    cs = s["cos_sin"][s["positions"]]
    q_out = _rotated(s["q"].float(), cs, case["interleaved"]).to(dt)
    block, at = s["kept_slots"] // BS, s["kept_slots"] % BS
    if case["kind"] == "rotate":
        k = _rotated(s["k"].float(), cs, case["interleaved"]).to(dt)
        s["k_cache"][block, :, at] = k[s["keep"]]
        s["v_cache"][block, :, at] = s["v"][s["keep"]]
        return [q_out, s["k_cache"], s["v_cache"]]
    # in 64 bits: a value next to a border goes to the same code on every way to compute it
    k = _rotated(s["k"].double(), cs.double(), case["interleaved"]).to(dt)
    outs = [q_out]
    for x, pool, factor in ((k, s["k_cache"], case["ks"]), (s["v"], s["v_cache"], case["vs"])):
        codes, scales = _parts(pool)
        c, sc = _codes(x[s["keep"]], factor)
        codes[block, :, at // _PAGE, at % _PAGE] = _packed(c)
        scales[block, :, at // _PAGE, at % _PAGE] = sc
        outs.append(_values(pool, factor).transpose(1, 2).reshape(-1, case["hkv"], D).to(dt))
    return outs


def _attend(s, q, pos, valid):
    """q [S, H_kv, G, C, D] at positions pos [S, C], valid [S, C]. Returns [S, H_kv, G, C, D] in fp32."""
    case = s["case"]
    S, H, G, C, D = q.shape
    at = s["table"].long()
    k, v = (_values(p[at], f).permute(0, 2, 1, 3, 4).reshape(S, H, -1, D)
            for p, f in ((s["k"], case["ks"]), (s["v"], case["vs"])))
    N = k.shape[2]
    x = torch.matmul(q.reshape(S, H, G * C, D), k.transpose(2, 3)).view(S, H, G, C, N) * s["scale"]
    seen = (torch.arange(N, device=q.device) <= pos[:, :, None]) & valid[:, :, None]
    x = torch.where(seen[:, None, None], x, _NEG)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == _NEG, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, H, G * C, N), v).view(S, H, G, C, D)
    return torch.where(total > 0, o / total, 0.0)


def _plain_decode(s):
    case = s["case"]
    S, D = case["seqs"], case["dim"]
    pos = (s["lens"].long() - 1)[:, None]
    o = _attend(s, s["q"].float().view(S, case["hkv"], -1, 1, D), pos, pos >= 0)
    return o.reshape(S, case["hq"], D).to(s["q"].dtype)


def _plain_prefill(s):
    case = s["case"]
    S, D, C = case["seqs"], case["dim"], s["max_chunk"]
    first, chunk = s["qsl"][:-1].long(), (s["qsl"][1:] - s["qsl"][:-1]).long()
    t = torch.arange(C, device=s["q"].device)
    valid = t < chunk[:, None]
    pos = s["lens"].long()[:, None] - chunk[:, None] + t
    q = s["q"].float()[torch.where(valid, first[:, None] + t, 0)]
    o = _attend(s, q.view(S, C, case["hkv"], -1, D).permute(0, 2, 3, 1, 4).contiguous(), pos, valid)
    # row r of the packed output: its sequence, and its place in the chunk
    r = torch.arange(s["q"].shape[0], device=t.device)
    seq = torch.searchsorted(s["qsl"].long(), r, right=True) - 1
    return o.permute(0, 3, 1, 2, 4).reshape(S, C, case["hq"], D)[seq, r - first[seq]].to(s["q"].dtype)


# --------------------------------------------------------------------- the definition, in fp64

def _e4m3(x):
    """The nearest number of 4 exponent and 3 mantissa bits, ties to even, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3.0)
    return torch.clamp(torch.round(x / step) * step, max=448.0)


def _e2m1(a):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to even; a >= 0."""
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.clamp(torch.round(a / step) * step, max=6.0)


def _held(x, factor):
    """What a 4-bit pool holds of x [..., D], fp64."""
    groups = (x.double() / factor).reshape(*x.shape[:-1], -1, _GROUP)
    scale = _e4m3(groups.abs().max(dim=-1, keepdim=True).values / 6.0)
    got = torch.where(scale > 0, _e2m1(groups.abs() / torch.where(scale > 0, scale, 1.0)) * scale, 0.0)
    return (torch.copysign(got, groups) * factor).reshape(x.shape)


def _turned(x, angles, R, interleaved):
    """x rotated as complex numbers; angles [T, R] holds cosines and sines."""
    z = torch.complex(angles[:, :R // 2], angles[:, R // 2:])[:, None]
    out = x.clone()
    if interleaved:
        w = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous()) * z
        out[..., :R] = torch.view_as_real(w).reshape(*x.shape[:-1], R)
    else:
        w = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
        out[..., :R // 2], out[..., R // 2:R] = w.real, w.imag
    return out


def _unpacked(pages, D, factor):
    """Bytes [n, 9 D] of pages -> values [16 n, D], fp64."""
    codes = pages[:, :8 * D].reshape(-1, D // 2).long()
    byte = pages[:, 8 * D:].reshape(-1, D // 16).long()
    e, m = byte >> 3, (byte & 7).double()
    scale = torch.where(e > 0, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0), m * 2.0 ** -9) * factor
    nib = torch.empty(codes.shape[0], D, dtype=torch.long, device=pages.device)
    nib[:, 0::2], nib[:, 1::2] = codes % 16, codes // 16
    e, m = (nib % 8) // 2, (nib % 2).double()
    mag = torch.where(e > 0, (1.0 + m / 2.0) * torch.exp2(e.double() - 1.0), m * 0.5)
    return torch.where(nib >= 8, -mag, mag) * scale.repeat_interleave(16, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    D, BS, H = case["dim"], case["block"], case["hkv"]
    if case["kind"] in ("rotate", "quantise"):
        angles = s["cos_sin"][s["positions"]].double()
        q = _turned(s["q"].double(), angles, case["rot"], case["interleaved"])
        k, v = _turned(s["k"].double(), angles, case["rot"], case["interleaved"]), s["v"].double()
        if case["kind"] == "rotate":
            pools = [s["k_cache"].double(), s["v_cache"].double()]
        else:
            k, v = _held(k.to(s["k"].dtype), case["ks"]), _held(v, case["vs"])
            pools = [torch.stack([_unpacked(x.reshape(-1, 9 * D), D, f)]).reshape(-1, H, BS, D)
                     for x, f in ((s["k_cache"], case["ks"]), (s["v_cache"], case["vs"]))]
        for pool, rows in zip(pools, (k, v)):
            pool[s["kept_slots"] // BS, :, s["kept_slots"] % BS] = rows[s["keep"]]
        return [q] + (pools if case["kind"] == "rotate" else [p.permute(0, 2, 1, 3).reshape(-1, H, D) for p in pools])
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G = case["hq"] // H
    for i, n in enumerate(s["lens"].tolist()):
        r0, r1 = s["qsl"][i].item(), s["qsl"][i + 1].item()
        ids = s["table"][i, : -(-n // BS)].long()
        K, V = (_unpacked(p[ids].transpose(0, 1).reshape(-1, 9 * D), D, f).reshape(H, -1, D)[:, :n]
                for p, f in ((s["k"], case["ks"]), (s["v"], case["vs"])))
        for b0 in range(r0, r1, 512):
            b1 = min(r1, b0 + 512)
            last = torch.arange(n - (r1 - b0), n - (r1 - b1), device="cuda")[:, None]
            hidden = torch.arange(n, device="cuda")[None, :] > last
            for h in range(case["hq"]):
                z = (s["q"][b0:b1, h].double() @ K[h // G].T) * s["scale"]
                z[hidden] = _NEG
                out[b0:b1, h] = torch.softmax(z, dim=1) @ V[h // G]
    return out
