"""Cases and plain forms of the scored-attention and page-move operators, for measuring them.

Three operators over the paged KV pool:

  decode   one query row per sequence over its pages, with scores that are capped by a tanh,
           biased by distance, or masked (sliding window, visible prefix, document start)
  prefill  a chunk of new query rows per sequence over its pages, with the same scores
  move     copies of pages in every layer's pools (forked tails, compaction), with the block
           tables rewritten to follow them

`own` False: `run` computes them from elementary torch operations in fp32. `own` True: `run`
calls the library's entry points. Lengths come from the case alone (spread over its range),
their order, the physical pages and all values from the seed.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_NEG = float("-inf")


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a few interactive users: the smallest decode step, where latency counts
        _decode("decode few capped", seqs=4, lo=17, hi=700, hq=32, hkv=8, dim=128, block=16, cap=50.0, sharp=5.0),
        # a serving batch with a sliding window whose first tokens stay visible; pages behind
        # the window have been given back to the pool
        _decode("decode batch window", seqs=64, lo=500, hi=16384, hq=32, hkv=8, dim=128, block=64, window=4096,
                prefix=64),
        # distance bias, one kv head per q head, head_dim 64, short to middling contexts
        _decode("decode mha distance", seqs=96, lo=16, hi=2048, hq=16, hkv=16, dim=64, block=32, alibi=True),
        # few long contexts: the work has to be split along the keys
        _decode("decode long capped", seqs=8, lo=20000, hi=32768, hq=64, hkv=8, dim=128, block=16, cap=30.0,
                sharp=4.0),
        # fp32, three q heads per kv head, ragged from one token up, packed documents
        _decode("decode f32 documents", seqs=24, lo=1, hi=777, hq=12, hkv=4, dim=64, block=16, dtype="f32",
                alibi=True, docs=True),
        # the mixed step's prefill half (16 chunks of 512 tokens on up to 4096) with capped scores
        _prefill("prefill chunks capped", seqs=16, clo=512, chi=512, plo=0, phi=4096, hq=32, hkv=8, dim=128, block=16,
                 cap=50.0, sharp=5.0),
        # long prompts under a sliding window: chunks of 2048 tokens far into the prompt
        _prefill("prefill long window", seqs=2, clo=2048, chi=2048, plo=14000, phi=16384, hq=32, hkv=8, dim=128,
                 block=64, window=4096, cap=30.0, sharp=4.0),
        # distance bias, one kv head per q head, head_dim 64, ragged chunks
        _prefill("prefill mha distance", seqs=8, clo=100, chi=1000, plo=0, phi=1500, hq=16, hkv=16, dim=64, block=16,
                 alibi=True),
        # prompts whose first tokens see one another, packed documents behind them, an odd group
        _prefill("prefill prefix documents", seqs=12, clo=64, chi=700, plo=0, phi=40, hq=24, hkv=8, dim=128, block=32,
                 prefix=200, docs=True),
        # fp32 check run of a small model: short ragged chunks under a window
        _prefill("prefill f32 window", seqs=4, clo=17, chi=96, plo=0, phi=900, hq=8, hkv=2, dim=64, block=16,
                 dtype="f32", window=256, cap=20.0, sharp=3.0),
        # parallel sampling: the partly filled last pages of forked requests, in every layer
        _move("move forked tails", pools=64, pairs=6, blocks=256, hkv=8, dim=128, block=128, partial=True),
        # shrinking a pool: held pages move below the new end and the block tables follow
        _move("move compaction", pools=64, pairs=960, blocks=2048, hkv=8, dim=128, block=16, seqs=64, row=256),
    ]


def _decode(name, seqs, lo, hi, hq, hkv, dim, block, dtype="bf16", cap=0.0, sharp=1.0, alibi=False, window=0, prefix=0,
            docs=False):
    return dict(name=name, kind="decode", seqs=seqs, lo=lo, hi=hi, hq=hq, hkv=hkv, dim=dim, block=block, dtype=dtype,
                cap=cap, sharp=sharp, alibi=alibi, window=window, prefix=prefix, docs=docs)


def _prefill(name, seqs, clo, chi, plo, phi, hq, hkv, dim, block, dtype="bf16", cap=0.0, sharp=1.0, alibi=False,
             window=0, prefix=0, docs=False):
    return dict(name=name, kind="prefill", seqs=seqs, clo=clo, chi=chi, plo=plo, phi=phi, hq=hq, hkv=hkv, dim=dim,
                block=block, dtype=dtype, cap=cap, sharp=sharp, alibi=alibi, window=window, prefix=prefix, docs=docs)


def _move(name, pools, pairs, blocks, hkv, dim, block, dtype="bf16", partial=False, seqs=0, row=0):
    return dict(name=name, kind="move", pools=pools, pairs=pairs, blocks=blocks, hkv=hkv, dim=dim, block=block,
                dtype=dtype, partial=partial, seqs=seqs, row=row)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _scores(rng):
    """One of the score forms, or two together."""
    cap = rng.choice([0.0, 0.0, 20.0, 30.0, 50.0])
    return dict(cap=cap, sharp=rng.uniform(2.0, 5.0) if cap else 1.0, alibi=rng.random() < 0.35,
                window=_log_int(rng, 16, 6000) if rng.random() < 0.5 else 0,
                prefix=rng.randint(1, 300) if rng.random() < 0.3 else 0, docs=rng.random() < 0.3)


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "move"])
    hkv, dim, block = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    group = rng.choice([1, 1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if kind == "move":
        pairs = _log_int(rng, 1, 600)
        blocks = 2 * pairs + rng.randint(4, 900)
        # fewer bytes than the compaction case
        page = hkv * dim * block * (4 if dtype == "f32" else 2)
        pools = max(1, min(2 * rng.randint(1, 40), 60 * 2048 * 8 * 128 * 16 * 2 // (blocks * page)))
        with_tables = rng.random() < 0.5
        return dict(kind="move", pools=pools, pairs=pairs, blocks=blocks, hkv=hkv, dim=dim, block=block, dtype=dtype,
                    partial=not with_tables and rng.random() < 0.5, seqs=rng.randint(1, 100) if with_tables else 0,
                    row=rng.randint(1, 300) if with_tables else 0)
    if hkv * group > 64:
        group = 64 // hkv
    if kind == "decode":
        seqs = _log_int(rng, 1, 200)
        hi = max(2, min(_log_int(rng, 8, 40000), 500_000_000 // (seqs * hkv * dim)))
        return dict(kind="decode", seqs=seqs, lo=max(1, int(hi * rng.choice([0.01, 0.1, 0.5, 1.0]))), hi=hi,
                    hq=hkv * group, hkv=hkv, dim=dim, block=block, dtype=dtype, **_scores(rng))
    seqs = _log_int(rng, 1, 16)
    phi = _log_int(rng, 1, 10000)
    chi = max(1, min(_log_int(rng, 1, 2048), int(0.6e9 / (seqs * hkv * group * (phi + 600)))))
    if dtype == "f32":
        chi = min(chi, 300)
    return dict(kind="prefill", seqs=seqs, clo=max(1, int(chi * rng.choice([0.05, 0.3, 1.0]))), chi=chi,
                plo=rng.choice([0, phi // 2, phi]), phi=phi, hq=hkv * group, hkv=hkv, dim=dim, block=block,
                dtype=dtype, **_scores(rng))


# ------------------------------------------------------------------------- what a case means

def _spread(lo, hi, n):
    """n whole numbers from lo to hi, spread over their logarithm."""
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return [int(round(math.exp(a + (b - a) * (i / (n - 1) if n > 1 else 1.0)) - 1.0)) for i in range(n)]


def _even(lo, hi, n):
    """n whole numbers from lo to hi at equal steps."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _rows(case):
    """Per sequence of the case, before the seed orders them: (keys, query rows, visible prefix,
    first position of each query row's document)."""
    n = case["seqs"]
    if case["kind"] == "decode":
        lens, chunks = _spread(case["lo"], case["hi"], n), [1] * n
    else:
        chunks = _spread(case["clo"], case["chi"], n)
        priors = _even(case["plo"], case["phi"], n)
        random.Random(n).shuffle(priors)
        lens = [p + c for p, c in zip(priors, chunks)]
    got = []
    for i, (L, C) in enumerate(zip(lens, chunks)):
        prefix = min(L, max(1, case["prefix"] * (i + 1) // n)) if case["prefix"] else 0
        # documents of uneven length follow the prefix; a row sees its own document's keys
        # (rows inside the prefix belong to a document that starts at 0)
        starts = [0] * C
        if case["docs"]:
            step = max(5, L // 4 + 3 * i % 7)
            starts = [((p - prefix) // step * step + prefix if p >= prefix else 0) for p in range(L - C, L)]
            if case["kind"] == "prefill" and C > 8:  # a padding row: its document starts behind it
                starts[-1] = L
        got.append((L, C, prefix, starts))
    return got


def _spans(case, L, prefix, p, start):
    """Keys that a query at position p sees: [start, prefix) and [b, p + 1), as two spans without
    a common key."""
    b = max(start, p + 1 - case["window"] if case["window"] else 0)
    a1 = min(prefix, L)
    first = (start, max(start, a1))
    second = (max(b, first[1]) if first[1] > first[0] else b, p + 1)
    return first, (second[0], max(second))


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["kind"] == "move":
        tokens = _move_tokens(case)
        moved = sum(tokens) * case["pools"] * case["hkv"] * case["dim"] * size
        return {"bytes": 2 * moved + 8 * case["pairs"] + 8 * case["seqs"] * case["row"], "flops": 0}
    seen = kept = rows = 0
    for L, C, prefix, starts in _rows(case):
        lo = [L, L]
        end = 0
        for r in range(C):
            (a0, a1), (b0, b1) = _spans(case, L, prefix, L - C + r, starts[r])
            seen += a1 - a0 + b1 - b0
            if a1 > a0:
                lo[0], end = min(lo[0], a0), max(end, a1)
            if b1 > b0:
                lo[1] = min(lo[1], b0)
        kept += max(0, end - lo[0]) + max(0, L - max(lo[1], end))
        rows += C
    return {"bytes": size * case["dim"] * (2 * rows * case["hq"] + 2 * kept * case["hkv"]),
            "flops": 4 * seen * case["hq"] * case["dim"]}


def _move_tokens(case):
    """Tokens copied per page: whole pages, or the filled part of each forked request's last one."""
    if not case["partial"]:
        return [case["block"]] * case["pairs"]
    return [1 + (i * 37 + 11) % case["block"] for i in range(case["pairs"])]


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["kind"] == "move":
        return _prepare_move(case, g)
    order = torch.randperm(case["seqs"], generator=torch.Generator().manual_seed(seed)).tolist()
    every = _rows(case)
    rows = [every[i] for i in order]
    H, D, BS, dt = case["hkv"], case["dim"], case["block"], _DTYPES[case["dtype"]]
    width = max(1, max(-(-L // BS) for L, _, _, _ in rows))
    # pages that no row of a sequence can see are not held: the table names page 0 there
    held = torch.zeros(len(rows), width, dtype=torch.bool)
    for s, (L, C, prefix, starts) in enumerate(rows):
        for r in {0, C - 1} | ({i for i in range(C) if starts[i] != starts[i - 1]} if case["docs"] else set()):
            for lo, hi in _spans(case, L, prefix, L - C + r, starts[r]):
                if hi > lo:
                    held[s, lo // BS:-(-hi // BS)] = True
        if case["kind"] == "prefill":  # the rows between the first and the last
            first = _spans(case, L, prefix, L - C, starts[0])[1][0]
            held[s, min(first, L - C) // BS:-(-L // BS)] = True
    n_held = int(held.sum())
    num_blocks = 1 + n_held + n_held // 16
    held = held.cuda()
    table = torch.zeros(held.shape, dtype=torch.int32, device="cuda")
    table[held] = 1 + torch.randperm(num_blocks - 1, generator=g, device="cuda", dtype=torch.int32)[:n_held]
    pool = (num_blocks, H, BS, D)
    T = sum(C for _, C, _, _ in rows)
    starts = [0]
    for _, C, _, _ in rows:
        starts.append(starts[-1] + C)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(
        case=case, scale=1.0 / math.sqrt(D), table=table, lens=i32([L for L, _, _, _ in rows]),
        k=torch.randn(pool, generator=g, device="cuda", dtype=dt), v=torch.randn(pool, generator=g, device="cuda", dtype=dt),
        q=(torch.randn(T, case["hq"], D, generator=g, device="cuda") * case["sharp"]).to(dt),
        qsl=i32(starts), max_len=max(L for L, _, _, _ in rows), max_chunk=max(C for _, C, _, _ in rows),
        slopes=torch.tensor([2.0 ** (-8.0 * (h + 1) / case["hq"]) for h in range(case["hq"])], device="cuda")
        if case["alibi"] else None,
        key_start=i32([x for _, _, _, st in rows for x in st]) if case["docs"] else None,
        prefix=i32([p for _, _, p, _ in rows]) if case["prefix"] else None)
    s["out"] = torch.empty_like(s["q"])
    if own:
        from paged_kv_cache_238_gb300 import binding as pa
        s["score"] = pa.Score(softcap=case["cap"], alibi_slopes=s["slopes"], window=case["window"],
                              key_start=s["key_start"], prefix_len=s["prefix"])
        if case["kind"] == "decode":
            n = pa.pa_decode_scored_workspace_size(case["seqs"], case["hq"], H, D, s["max_len"], dt)
        else:
            n = pa.pa_prefill_scored_workspace_size(case["seqs"], s["max_chunk"], case["hq"], H, D, s["max_len"], dt)
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda") if n else None
    return s


def _prepare_move(case, g):
    dt, n, NB = _DTYPES[case["dtype"]], case["pairs"], case["blocks"]
    pools = torch.randn((case["pools"], NB, case["hkv"], case["block"], case["dim"]), generator=g, device="cuda", dtype=dt)
    if case["seqs"]:  # compaction: ascending pages from the upper half to free ones of the lower
        cut = NB // 2
        src = cut + torch.randperm(NB - cut, generator=g, device="cuda")[:n].sort().values
        dst = 1 + torch.randperm(cut - 1, generator=g, device="cuda")[:n].sort().values
    else:  # forks: several children may copy one parent's page
        ids = 1 + torch.randperm(NB - 1, generator=g, device="cuda")
        parents = max(1, n // 3)
        src, dst = ids[:parents].repeat(-(-n // parents))[:n], ids[parents:parents + n]
    n = min(src.numel(), dst.numel())
    s = dict(case=case, pools=pools, pairs=torch.stack([src[:n], dst[:n]], dim=1).to(torch.int32).contiguous(),
             tokens=torch.tensor(_move_tokens(case)[:n], dtype=torch.int32, device="cuda") if case["partial"] else None,
             table=None, lens=None)
    if case["seqs"]:
        s["table"] = torch.randint(1, NB, (case["seqs"], case["row"]), generator=g, device="cuda", dtype=torch.int32)
        s["lens"] = torch.tensor(_spread(1, case["row"] * case["block"], case["seqs"]), dtype=torch.int32, device="cuda")
    if own:
        from paged_kv_cache_238_gb300 import binding as pa
        s["list"] = pa.PoolList(list(pools.unbind(0)))
    return s


# -------------------------------------------------------------------------------- one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    if kind == "move":
        return _plain_move(state)
    return _plain_decode(state) if kind == "decode" else _plain_prefill(state)


def _own(s, kind):
    from paged_kv_cache_238_gb300 import binding as pa
    if kind == "decode":
        pa.pa_decode_scored(s["out"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["max_len"], s["scale"],
                            s["score"], s["workspace"])
        return s["out"]
    if kind == "prefill":
        pa.pa_prefill_scored(s["out"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["qsl"], s["max_chunk"],
                             s["max_len"], s["scale"], s["score"], s["workspace"])
        return s["out"]
    pa.pa_move_blocks(s["list"], s["pairs"], tokens=s["tokens"], block_table=s["table"], seq_lens=s["lens"])
    return [s["pools"], s["table"]]


def _gathered(s):
    """Keys and values of every sequence in logical order, fp32: [S, H_kv, keys, D]."""
    case = s["case"]
    S, W = s["table"].shape
    at = s["table"].long()
    return [p[at].float().permute(0, 2, 1, 3, 4).reshape(S, case["hkv"], W * case["block"], case["dim"])
            for p in (s["k"], s["v"])]


def _attend(s, q, pos, key_start, prefix, valid):
    """q [S, H_kv, G, C, D] at positions pos [S, C]; key_start [S, C] or None, prefix [S] or None;
    valid [S, C]. Returns [S, H_kv, G, C, D] in fp32."""
    case = s["case"]
    k, v = _gathered(s)
    S, H, G, C, D = q.shape
    N = k.shape[2]
    x = torch.matmul(q.reshape(S, H, G * C, D), k.transpose(2, 3)).view(S, H, G, C, N) * s["scale"]
    if case["cap"]:
        x = case["cap"] * torch.tanh(x / case["cap"])
    j = torch.arange(N, device=q.device)
    if s["slopes"] is not None:
        away = (pos[:, :, None] - j).abs().float()[:, None, None]
        x = x - s["slopes"].view(1, H, G, 1, 1) * away
    near = j <= pos[:, :, None]
    if case["window"]:
        near = near & (j > pos[:, :, None] - case["window"])
    if prefix is not None:
        near = near | (j < prefix[:, None, None])
    if key_start is not None:
        near = near & (j >= key_start[:, :, None])
    near = near & (j < s["lens"][:, None, None]) & valid[:, :, None]
    x = torch.where(near[:, None, None], x, _NEG)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == _NEG, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, H, G * C, N), v).view(S, H, G, C, D)
    return torch.where(total > 0, o / total, 0.0)


def _plain_decode(s):
    case = s["case"]
    S, D = case["seqs"], case["dim"]
    q = s["q"].float().view(S, case["hkv"], -1, 1, D)
    pos = (s["lens"].long() - 1)[:, None]
    start = s["key_start"].long()[:, None] if s["key_start"] is not None else None
    o = _attend(s, q, pos, start, s["prefix"], pos >= 0)
    return o.reshape(S, case["hq"], D).to(s["q"].dtype)


def _plain_prefill(s):
    case = s["case"]
    S, D, C = case["seqs"], case["dim"], s["max_chunk"]
    first, chunk = s["qsl"][:-1].long(), (s["qsl"][1:] - s["qsl"][:-1]).long()
    t = torch.arange(C, device=s["q"].device)
    valid = t < chunk[:, None]
    row = torch.where(valid, first[:, None] + t, 0)
    pos = s["lens"].long()[:, None] - chunk[:, None] + t
    q = s["q"].float()[row].view(S, C, case["hkv"], -1, D).permute(0, 2, 3, 1, 4).contiguous()
    start = s["key_start"].long()[row] if s["key_start"] is not None else None
    o = _attend(s, q, pos, start, s["prefix"], valid)
    return o.permute(0, 3, 1, 2, 4).reshape(S, C, case["hq"], D)[valid].to(s["q"].dtype)


def _plain_move(s):
    src, dst = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    if s["tokens"] is None:
        s["pools"][:, dst] = s["pools"][:, src]
    else:
        keep = torch.arange(s["case"]["block"], device=src.device) < s["tokens"][:, None]
        s["pools"][:, dst] = torch.where(keep[:, None, :, None], s["pools"][:, src], s["pools"][:, dst])
    if s["table"] is not None:
        to = torch.arange(s["case"]["blocks"], device=src.device, dtype=torch.int32)
        to[src] = s["pairs"][:, 1]
        used = torch.arange(s["table"].shape[1], device=src.device) * s["case"]["block"] < s["lens"][:, None]
        s["table"].copy_(torch.where(used, to[s["table"].long()], s["table"]))
    return [s["pools"], s["table"]]


# --------------------------------------------------------------------- the definition, in fp64

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "move":
        pools, table = s["pools"].double(), s["table"]
        for i, (a, b) in enumerate(s["pairs"].tolist()):
            n = int(s["tokens"][i]) if s["tokens"] is not None else case["block"]
            pools[:, b, :, :n] = s["pools"][:, a, :, :n].double()
        if table is not None:
            to = dict(s["pairs"].tolist())
            rows = table.tolist()
            for r, n in zip(rows, s["lens"].tolist()):
                for i in range(-(-n // case["block"])):
                    r[i] = to.get(r[i], r[i])
            table = torch.tensor(rows, dtype=torch.int32, device="cuda")
        return [pools, table]
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G, BS = case["hq"] // case["hkv"], case["block"]
    for i, n in enumerate(s["lens"].tolist()):
        r0, r1 = s["qsl"][i].item(), s["qsl"][i + 1].item()
        pages = s["table"][i, : -(-n // BS)].long()
        K, V = (p[pages].transpose(0, 1).reshape(case["hkv"], -1, case["dim"])[:, :n].double() for p in (s["k"], s["v"]))
        P = s["prefix"][i].item() if s["prefix"] is not None else 0
        for b0 in range(r0, r1, 512):
            b1 = min(r1, b0 + 512)
            at = torch.arange(n - (r1 - b0), n - (r1 - b1), device="cuda").double()[:, None]
            key = torch.arange(n, device="cuda").double()[None, :]
            hidden = key > at
            if case["window"]:
                hidden |= at - key >= case["window"]
            hidden &= key >= P
            if s["key_start"] is not None:
                hidden |= key < s["key_start"][b0:b1, None].double()
            for h in range(case["hq"]):
                z = (s["q"][b0:b1, h].double() @ K[h // G].T) * s["scale"]
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if s["slopes"] is not None:
                    z -= s["slopes"][h].double() * (at - key).abs()
                z[hidden] = _NEG
                w = torch.nan_to_num(torch.softmax(z, dim=1), nan=0.0)
                out[b0:b1, h] = w @ V[h // G]
    return out
