"""Cases of the cache-eviction operators: attention that accumulates each key's weight, the choice of
the tokens to keep, the compaction of the paged cache, and the append behind an eviction.

`run` computes an operator in its plain form (elementary torch operations, fp32 and wider) or, with
`own` set, through the library's entry points, on what `prepare` made from a seed. `exact` gives the
outputs from the operators' definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
D = 128          # head dim
PAGE = 64        # token slots per page
ROT = 32         # rotary dims of the append cases
THETA = 1e7
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # E2M1 magnitudes by code


# ---- cases -------------------------------------------------------------------------------------

def _lens(case):
    return [int(x) for x in str(case["lens"]).split(",")]


def _keeps(case):
    return [int(x) for x in str(case["keep"]).split(",")]


def listed():
    return [
        # the first tokens of one short chat: latency counts
        {"name": "attend one short sequence", "op": "attend", "lens": "97", "q_len": 1, "causal": True,
         "q_heads": 24, "kv_heads": 4},
        # the benchmark's decode shape: four long sequences, one new token each
        {"name": "attend decode 4 x 131072", "op": "attend", "lens": ",".join(["131072"] * 4),
         "q_len": 1, "causal": True, "q_heads": 24, "kv_heads": 4},
        # a batch of sessions of mixed age on a model with eight KV heads
        {"name": "attend ragged, 8 KV heads", "op": "attend",
         "lens": "13,517,2049,4100,8191,11000,20011,32769", "q_len": 1, "causal": True,
         "q_heads": 32, "kv_heads": 8},
        # speculative verify: 8 drafted tokens over 100K cached ones
        {"name": "attend verify 4 x 100000", "op": "attend", "lens": ",".join(["100000"] * 4),
         "q_len": 8, "causal": True, "q_heads": 24, "kv_heads": 4},
        # the last 64 tokens of a prompt observed over the whole prompt, to evict right after it
        {"name": "attend window 64 of 2 x 32768", "op": "attend", "lens": "32768,32768", "q_len": 64,
         "causal": True, "q_heads": 24, "kv_heads": 4},
        # a small budget in a short chat, every KV head on its own
        {"name": "select 128 of 300", "op": "select", "lens": "300", "keep": "128",
         "kv_heads": 4, "per_head": True, "sink": 4, "recent": 32},
        # long sessions cut to an eighth, every KV head on its own
        {"name": "select 4 x 16384 of 131072", "op": "select", "lens": ",".join(["131072"] * 4),
         "keep": ",".join(["16384"] * 4), "kv_heads": 4, "per_head": True, "sink": 4, "recent": 1024},
        # the longest context the position scaling covers, one set of tokens for all heads
        {"name": "select 65536 of 600000", "op": "select", "lens": "600000", "keep": "65536",
         "kv_heads": 4, "per_head": False, "sink": 64, "recent": 8192},
        # a short chat compacted, one set of tokens for all heads
        {"name": "compact 256 of 700", "op": "compact", "lens": "700", "keep": "256", "kv_heads": 4,
         "per_head": False},
        # the long sessions' caches compacted, every KV head on its own
        {"name": "compact 4 x 16384 of 131072", "op": "compact",
         "lens": ",".join(["131072"] * 4), "keep": ",".join(["16384"] * 4), "kv_heads": 4,
         "per_head": True},
        # one new token for each of four evicted sessions
        {"name": "append 4 tokens", "op": "append", "tokens": "1,1,1,1", "held": "16384,16384,4096,777",
         "q_heads": 24, "kv_heads": 4},
        # a new 8192-token message behind an evicted history
        {"name": "append 8192 tokens", "op": "append", "tokens": "8192", "held": "16384",
         "q_heads": 24, "kv_heads": 4},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "select", "compact", "append"])
    q_heads, kv_heads = rng.choice([(24, 4), (24, 4), (32, 8), (16, 2), (8, 8), (12, 3), (20, 5)])
    if op == "attend":
        n = rng.randint(1, 8)
        q_len = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 64)])
        # at most the tokens of the largest listed cases, and their (row, key) pairs
        most = min(400000 // n, 2 * 32768 * 24 * 64 // (q_len * q_heads * n), 400000 * 4 // kv_heads // n)
        lens = [max(q_len, _log_int(rng, 1, max(q_len + 1, most))) for _ in range(n)]
        return {"op": op, "lens": ",".join(map(str, lens)), "q_len": q_len,
                "causal": rng.random() < 0.8, "q_heads": q_heads, "kv_heads": kv_heads}
    if op == "append":
        n = rng.randint(1, 4)
        return {"op": op, "tokens": ",".join(str(_log_int(rng, 1, 8192 // n // max(1, kv_heads // 4)))
                                             for _ in range(n)),
                "held": ",".join(str(rng.randint(0, 20000)) for _ in range(n)),
                "q_heads": q_heads, "kv_heads": kv_heads}
    n = rng.randint(1, 6)
    most = 4 * 131072 * 4 // kv_heads // n
    lens = [_log_int(rng, 1, most) for _ in range(n)]
    keep = [max(1, int(x * rng.uniform(0.02, 0.125)) if rng.random() < 0.9 else x + rng.randint(-3, 5))
            for x in lens]
    if op == "compact":  # no more kept rows than the listed case has
        keep = [min(k, 16384 * 4 * 4 // kv_heads // n) for k in keep]
    case = {"op": op, "lens": ",".join(map(str, lens)), "keep": ",".join(map(str, keep)),
            "kv_heads": kv_heads, "per_head": rng.random() < 0.6}
    if op == "select":  # the first sequence has tokens to choose from; a shorter one may have none
        lens[0] = max(lens[0], rng.randint(1000, 2000))
        keep[0] = max(keep[0], 100)
        case |= {"lens": ",".join(map(str, lens)), "keep": ",".join(map(str, keep)),
                 "sink": rng.choice([0, 4, rng.randint(1, 32)]),
                 "recent": rng.choice([0, 32, rng.randint(1, max(32, keep[0] // 2))])}
    return case


def work(case):
    """Bytes and operations one pass cannot do without."""
    op, H = case["op"], case.get("kv_heads")
    if op == "attend":
        lens, q, hq = _lens(case), case["q_len"], case["q_heads"]
        t = sum(lens)
        pairs = sum(n * q - (q * (q - 1) // 2 if case["causal"] else 0) for n in lens) * hq
        rows = len(lens) * q * hq
        return {"bytes": t * H * (144 + 8) + rows * (72 + 2 * D), "flops": 4 * D * pairs}
    if op == "select":
        lens, keep = _lens(case), _keeps(case)
        sets = H if case["per_head"] else 1
        kept = sum(min(a, b) for a, b in zip(lens, keep))
        return {"bytes": 4 * H * sum(lens) + 4 * sets * kept, "flops": sum(lens) * H}
    if op == "compact":
        lens, keep = _lens(case), _keeps(case)
        kept = sum(min(a, b) for a, b in zip(lens, keep) if b < a)
        cut = sum(a - min(a, b) for a, b in zip(lens, keep))
        sets = H if case["per_head"] else 1
        return {"bytes": kept * H * (144 + 144 + 8) + 4 * sets * kept + 4 * H * cut + 64, "flops": 0}
    rows = sum(int(x) for x in str(case["tokens"]).split(",")) * (case["q_heads"] + 2 * H)
    return {"bytes": rows * (256 + 72), "flops": rows * D * (14 + 2)}


# ---- the cache's formats -----------------------------------------------------------------------

def _encode(x):
    """NVFP4 of fp32 rows [..., 128]: (codes [..., 64], scales [..., 8]) as uint8."""
    b = x.reshape(*x.shape[:-1], 8, 16)
    amax = b.abs().amax(-1)
    scales = (amax / torch.full_like(amax, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = scales.float()[..., None].expand_as(b)
    q = torch.where(sf == 0, torch.zeros_like(b), b / sf)
    a = q.abs()
    # the E2M1 code of |q|, ties to the even code: steps of 0.5 below 2, of 1 below 4, of 2 above
    code = torch.where(a < 2, torch.round(a * 2),
                       torch.where(a < 4, torch.round(a) + 2, torch.round(a * 0.5) + 4)).clamp(max=7)
    code = code.to(torch.uint8) | (torch.signbit(q) & (sf != 0)).to(torch.uint8) << 3
    code = code.reshape(*x.shape[:-1], 64, 2)
    return code[..., 0] | code[..., 1] << 4, scales.view(torch.uint8)


def _pack_pages(kc, ks, vc, vs):
    """Page blocks [pages, 9216 H] of one sequence from codes and scales [H, pages * 64, 64 | 8]."""
    H, T, _ = kc.shape
    p, e = T // PAGE, H // 2 * 2
    k = kc.view(H, p, 8, 8, 4, 16).permute(1, 0, 2, 4, 3, 5).reshape(p, H * 4096)
    pair = ks[:e].reshape(e // 2, 2, p, 2, 32, 2, 4).permute(2, 0, 5, 4, 1, 3, 6).reshape(p, e * 512)
    lone = ks[e:].reshape(H - e, p, 2, 32, 2, 4).permute(1, 0, 4, 3, 2, 5).reshape(p, (H - e) * 512)
    v = vc.view(H, p, PAGE * 64).transpose(0, 1).reshape(p, H * 4096)
    s = vs.view(H, p, PAGE * 8).transpose(0, 1).reshape(p, H * 512)
    return torch.cat([k, pair, lone, v, s], 1)


def _unpack_pages(pages, H):
    """Codes and scales [S, H, P * 64, 64 | 8] of K and V from page blocks [S, P, 9216 H]."""
    S, P, _ = pages.shape
    e, T = H // 2 * 2, P * PAGE
    k, pair, lone, v, s = pages.split([H * 4096, e * 512, (H - e) * 512, H * 4096, H * 512], 2)
    kc = k.reshape(S, P, H, 8, 4, 8, 16).permute(0, 2, 1, 3, 5, 4, 6).reshape(S, H, T, 64)
    ks = torch.cat([
        pair.reshape(S, P, e // 2, 2, 32, 2, 2, 4).permute(0, 2, 5, 1, 6, 4, 3, 7).reshape(S, e, T, 8),
        lone.reshape(S, P, H - e, 2, 32, 2, 4).permute(0, 2, 1, 5, 4, 3, 6).reshape(S, H - e, T, 8)], 1)
    vc = v.reshape(S, P, H, PAGE, 64).transpose(1, 2).reshape(S, H, T, 64)
    vs = s.reshape(S, P, H, PAGE, 8).transpose(1, 2).reshape(S, H, T, 8)
    return kc, ks, vc, vs


def _decode(codes, scales):
    """fp32 values [..., 128] of NVFP4 rows."""
    grid = torch.tensor(GRID + [-x for x in GRID], device=codes.device)
    byte = torch.arange(256, device=codes.device)
    both = torch.stack([grid[byte & 15], grid[byte >> 4]], 1)
    x = both[codes.int()].reshape(*codes.shape[:-1], 8, 16)
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).reshape(*codes.shape[:-1], D)


def _row_bytes(H):
    """Byte offsets [H, 64, 144] in a page block: K codes, K scales, V codes, V scales of each slot."""
    h = torch.arange(H, device=DEV)[:, None, None]
    k = torch.arange(PAGE, device=DEV)[None, :, None]
    j = torch.arange(64, device=DEV)[None, None, :]
    b = torch.arange(8, device=DEV)[None, None, :]
    kc = h * 4096 + k // 8 * 512 + j // 16 * 128 + k % 8 * 16 + j % 16
    two = 4096 * H + h // 2 * 1024 + b // 4 * 512 + k % 32 * 16 + h % 2 * 8 + k // 32 * 4 + b % 4
    one = 4096 * H + h // 2 * 1024 + b // 4 * 256 + k % 32 * 8 + k // 32 * 4 + b % 4
    ks = torch.where(h // 2 * 2 + 1 < H, two, one)
    vc = 4608 * H + h * 4096 + k * 64 + j
    vs = 8704 * H + h * 512 + k * 8 + b
    return torch.cat([kc, ks, vc, vs], 2)


# ---- inputs ------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _block_table(lens, g, spare=3):
    """Pages of the sequences scattered over a pool: (table [S, P] int32, pages in the pool)."""
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=g, device=DEV).int()
    table = torch.zeros(len(lens), max(1, max(pages)), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += n
    return table, total


def _prepare_attend(case, g):
    lens, q_len, Hq, H = _lens(case), case["q_len"], case["q_heads"], case["kv_heads"]
    S = len(lens)
    table, total = _block_table(lens, g)
    pool = torch.zeros(total, 9216 * H, dtype=torch.uint8, device=DEV)
    queries = []
    for s, n in enumerate(lens):
        # most keys are noise to the queries; a few (and the first ones) lie along the direction
        # that the head looks for, and gather most of the weight
        p = (n + PAGE - 1) // PAGE
        look = torch.randn(H, 1, D, generator=g, device=DEV)
        heavy = (torch.rand(H, p * PAGE, 1, generator=g, device=DEV) < 0.01).float()
        heavy[:, :4] = 1
        k = torch.randn(H, p * PAGE, D, generator=g, device=DEV) + 0.5 * heavy * look
        kc, ks = _encode(k)
        vc, vs = _encode(torch.randn(H, p * PAGE, D, generator=g, device=DEV))
        pool[table[s, :p].long()] = _pack_pages(kc, ks, vc, vs)
        q = 1.3 * torch.randn(q_len, H, Hq // H, D, generator=g, device=DEV) + 0.6 * look
        queries.append(q.reshape(q_len, Hq, D))
    q_codes, q_scales = _encode(torch.cat(queries))
    slots = table.shape[1] * PAGE
    # what earlier steps left: spread over many powers of ten, about as much as one pass adds
    held = torch.exp(2.5 * torch.randn(S, H, slots, generator=g, device=DEV)) * 1e-6
    return {"pool": pool, "table": table, "q_codes": q_codes, "q_scales": q_scales,
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "held": held,
            "weights": torch.zeros(S, H, slots, device=DEV),
            "out": torch.zeros(S * q_len, Hq, D, dtype=torch.bfloat16, device=DEV)}


def _prepare_select(case, g):
    lens, keep, H = _lens(case), _keeps(case), case["kv_heads"]
    S, slots = len(lens), (max(lens) + PAGE - 1) // PAGE * PAGE
    # accumulated weights spread over many powers of ten; some tie
    w = torch.exp(2.5 * torch.randn(S, H, slots, generator=g, device=DEV)) * 1e-4
    tied = torch.rand(S, H, slots, generator=g, device=DEV) < 0.05
    w = torch.where(tied, torch.exp2(torch.round(torch.log2(w))), w)
    most = max(min(a, b) for a, b in zip(lens, keep))
    sets = H if case["per_head"] else 1
    return {"weights": w, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "keep": torch.tensor(keep, dtype=torch.int32, device=DEV),
            "index": torch.full((S, sets, most), -1, dtype=torch.int32, device=DEV)}


def _prepare_compact(case, g):
    lens, keep, H = _lens(case), _keeps(case), case["kv_heads"]
    S, sets = len(lens), H if case["per_head"] else 1
    table, total = _block_table(lens, g)
    pool = torch.randint(0, 256, (total, 9216 * H), generator=g, device=DEV, dtype=torch.uint8)
    most = max(min(a, b) for a, b in zip(lens, keep))
    index = torch.full((S, sets, most), -1, dtype=torch.int32, device=DEV)
    for s, (n, m) in enumerate(zip(lens, keep)):
        m = min(n, m)
        luck = torch.rand(sets, n, generator=g, device=DEV)
        luck[:, :min(4, m)] = 2  # the first tokens stay, and the last ones
        luck[:, max(4, n - m // 8):] = 2
        index[s, :, :m] = luck.topk(m, 1).indices.sort(1).values.int()
    slots = table.shape[1] * PAGE
    return {"pool": pool, "table": table, "index": index,
            "weights": torch.rand(S, H, slots, generator=g, device=DEV),
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "keep": torch.tensor(keep, dtype=torch.int32, device=DEV),
            "row_bytes": _row_bytes(H)}


def _prepare_append(case, g):
    tokens = [int(x) for x in str(case["tokens"]).split(",")]
    held = [int(x) for x in str(case["held"]).split(",")]
    Hq, H = case["q_heads"], case["kv_heads"]
    table, total = _block_table([a + b for a, b in zip(held, tokens)], g)
    pool = torch.zeros(total, 9216 * H, dtype=torch.uint8, device=DEV)
    loud = torch.ones(D, device=DEV)
    loud[[3, 77, 101, 120]] = 12  # outlier channels of Q and K
    T = sum(tokens)
    q = (torch.randn(T, Hq, D, generator=g, device=DEV) * loud).bfloat16()
    k = (torch.randn(T, H, D, generator=g, device=DEV) * loud).bfloat16()
    v = torch.randn(T, H, D, generator=g, device=DEV).bfloat16()
    seqs, slots, positions = [], [], []
    for s, (n, h) in enumerate(zip(tokens, held)):
        seqs += [s] * n
        slots += range(h, h + n)
        positions += range(4 * h, 4 * h + n)  # three of four earlier tokens were evicted
    reach = max(positions) + 1
    angle = (torch.arange(reach, device=DEV).double()[:, None]
             * THETA ** (-2.0 * torch.arange(ROT // 2, device=DEV).double() / ROT))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"pool": pool, "table": table, "q": q, "k": k, "v": v, "seqs": i32(seqs),
            "slots": i32(slots), "positions": i32(positions),
            "rope": torch.cat([angle.cos(), angle.sin()], 1).float(),
            "q_codes": torch.empty(T, Hq, 64, dtype=torch.uint8, device=DEV),
            "q_scales": torch.empty(T, Hq, 8, dtype=torch.uint8, device=DEV),
            "row_bytes": _row_bytes(H)}


def prepare(case, seed):
    make = {"attend": _prepare_attend, "select": _prepare_select, "compact": _prepare_compact,
            "append": _prepare_append}[case["op"]]
    state = make(case, _generator(seed))
    state["case"] = case
    if own:  # the library's handles that a serving program keeps: layout, status word, the step's plan
        import bit_kv_cache_03_gb300 as kv
        H = case["kv_heads"]
        state["kv"] = kv
        state["layout"] = kv.make_layout(case.get("q_heads", H), H, D, PAGE,
                                         ROT if case["op"] == "append" else 0)
        state["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if case["op"] == "attend":
            L, lens, q_len, causal = state["layout"], _lens(case), case["q_len"], case["causal"]
            chunk = PAGE if case["q_heads"] // H * q_len <= 8 and H <= 4 else 2 * PAGE
            size = kv.kv_nvfp4_plan_workspace_bytes(L, lens, q_len, causal, chunk)
            state["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
            state["plan"] = kv.kv_nvfp4_plan(L, lens, q_len, causal, chunk, state["workspace"], size)
            size = kv.kv_nvfp4_weights_workspace_bytes(L, state["plan"])
            state["account"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return state


# ---- one pass ----------------------------------------------------------------------------------

def _own(s):
    kv, case = s["kv"], s["case"]
    if case["op"] == "attend":
        kv.kv_nvfp4_decode_attn_weights(
            s["layout"], s["plan"], s["workspace"], s["account"], s["account"].numel(),
            s["q_codes"], s["q_scales"], 1.0 / math.sqrt(D), s["pool"], s["pool"].shape[0],
            s["table"], s["table"].shape[1], s["out"], s["held"], s["weights"],
            s["weights"].shape[2], s["status"])
        return {"out": s["out"], "weights": s["weights"]}
    if case["op"] == "select":
        kv.kv_nvfp4_evict_select(
            s["layout"], s["weights"], s["weights"].shape[2], s["lens"], s["keep"],
            s["lens"].shape[0], case["per_head"], case["sink"], case["recent"], s["index"],
            s["index"].shape[2], s["status"])
        return {"index": s["index"]}
    if case["op"] == "compact":
        kv.kv_nvfp4_evict_compact(
            s["layout"], s["index"], s["index"].shape[2], case["per_head"], s["lens"], s["keep"],
            s["lens"].shape[0], s["table"], s["table"].shape[1], s["pool"].shape[0], s["pool"],
            None, 0, s["weights"], s["weights"].shape[2], s["status"])
        return {"pool": s["pool"], "weights": s["weights"]}
    kv.kv_nvfp4_append_slots(
        s["layout"], s["q"], s["k"], s["v"], s["seqs"], s["slots"], s["positions"],
        s["seqs"].shape[0], s["rope"], s["rope"].shape[0], s["table"], s["table"].shape[0],
        s["table"].shape[1], s["pool"].shape[0], s["pool"], s["q_codes"], s["q_scales"], s["status"])
    return {"pool": s["pool"], "q_codes": s["q_codes"], "q_scales": s["q_scales"]}


def _plain_attend(s):
    case = s["case"]
    H, Hq, q_len = case["kv_heads"], case["q_heads"], case["q_len"]
    S, P = s["table"].shape
    R, T = Hq // H * q_len, P * PAGE
    kc, ks, vc, vs = _unpack_pages(s["pool"][s["table"].long()], H)
    q = _decode(s["q_codes"], s["q_scales"])
    q = q.view(S, q_len, H, Hq // H, D).transpose(1, 2).reshape(S, H, R, D)
    scores = q @ _decode(kc, ks).transpose(2, 3) * (1.0 / math.sqrt(D))
    lens = s["lens"].long()
    token = torch.arange(R, device=DEV) // (Hq // H)
    sees = lens[:, None] - q_len + 1 + token if case["causal"] else lens[:, None].expand(S, R)
    slot = torch.arange(T, device=DEV)
    scores = scores.masked_fill(slot >= sees[:, None, :, None], -math.inf)
    p = torch.exp(scores - scores.amax(3, keepdim=True))
    p = p / p.sum(3, keepdim=True)
    out = (p @ _decode(vc, vs)).view(S, H, q_len, Hq // H, D).transpose(1, 2).reshape(S * q_len, Hq, D)
    weights = torch.where(slot < lens[:, None, None], s["held"] + p.sum(2), s["weights"])
    return {"out": out.bfloat16(), "weights": weights}


def _plain_select(s):
    case, w = s["case"], s["weights"]
    if not case["per_head"]:
        w = sum(w.unbind(1))[:, None]  # head after head, in fp32
    T, lens = w.shape[2], s["lens"].long()[:, None, None]
    bits = (w + 0.0).view(torch.int32)  # -0 counts as 0
    rank = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()  # ascending with the value
    rank = torch.where(torch.isnan(w), -2 ** 31, rank)
    slot = torch.arange(T, device=DEV)
    rank = torch.where((slot < case["sink"]) | (slot >= lens - case["recent"]), 2 ** 32, rank)
    rank = torch.where(slot < lens, rank, -2 ** 40)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices
    kept = torch.minimum(s["lens"], s["keep"]).long()[:, None, None]
    first = order[..., :s["index"].shape[2]]
    at = torch.arange(first.shape[2], device=DEV)
    index = torch.sort(torch.where(at < kept, first, T), dim=2).values
    return {"index": torch.where(at < kept, index, -1).int()}


def _plain_compact(s):
    case, index = s["case"], s["index"].long()
    S, H, T = s["weights"].shape
    index = index.expand(S, H, index.shape[2])
    kept = torch.minimum(s["lens"], s["keep"]).long()[:, None, None]
    at = torch.arange(index.shape[2], device=DEV)
    seq, head, row = torch.nonzero(at < kept.expand(S, H, 1), as_tuple=True)
    old = index[seq, head, row]
    flat, block = s["pool"].view(-1), s["pool"].shape[1]
    table, bytes_of = s["table"].long(), s["row_bytes"]
    src = (table[seq, old // PAGE] * block)[:, None] + bytes_of[head, old % PAGE]
    dst = (table[seq, row // PAGE] * block)[:, None] + bytes_of[head, row % PAGE]
    flat[dst] = flat[src]
    w = s["weights"]
    moved = w[seq, head, old]
    slot = torch.arange(T, device=DEV)
    w.masked_fill_((slot >= kept) & (slot < s["lens"].long()[:, None, None]), 0)
    w[seq, head, row] = moved
    return {"pool": s["pool"], "weights": w}


def _turn_and_rotate(x, rope):
    """RoPE on the first dims and the normalised Hadamard rotation, each step rounded to fp32."""
    half = ROT // 2
    a, b, c, d = x[..., :half], x[..., half:ROT], rope[:, None, :half], rope[:, None, half:]
    x = torch.cat([a * c - b * d, b * c + a * d, x[..., ROT:]], -1)
    for step in (1, 2, 4, 8, 16, 32, 64):
        y = x.reshape(*x.shape[:-1], D // (2 * step), 2, step)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
    return x * torch.tensor(2.0 ** -3.5, device=DEV)


def _plain_append(s):
    rope = s["rope"][s["positions"].long()]
    q_codes, q_scales = _encode(_turn_and_rotate(s["q"].float(), rope))
    k = _encode(_turn_and_rotate(s["k"].float(), rope))
    rows = torch.cat([*k, *_encode(s["v"].float())], -1)  # [T, H, 144]
    slot = s["slots"].long()
    page = s["table"].long()[s["seqs"].long(), slot // PAGE]
    block = s["pool"].shape[1]
    dst = (page * block)[:, None, None] + s["row_bytes"][:, slot % PAGE].transpose(0, 1)
    s["pool"].view(-1)[dst] = rows
    return {"pool": s["pool"], "q_codes": q_codes, "q_scales": q_scales}


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "select": _plain_select, "compact": _plain_compact,
            "append": _plain_append}[state["case"]["op"]](state)


# ---- in 64 bits --------------------------------------------------------------------------------

def _value64(codes, scales):
    """Values of NVFP4 rows from the formats' definitions: sign, two exponent bits and one fraction
    bit (E2M1, bias 1), times four exponent bits and three fraction bits (E4M3, bias 7)."""
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D).double()
    sign = 1 - 2 * torch.floor(nib / 8)
    e, f = torch.floor(nib / 2) % 4, nib % 2
    x = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e - 1))
    sc = scales.double()
    e, f = torch.floor(sc / 8) % 16, sc % 8
    y = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7))
    return sign * x * y.repeat_interleave(16, -1)


def exact(case, seed):
    if case["op"] in ("select", "append"):  # indices and codes: no value but their own
        return None
    s = prepare(case, seed)
    if case["op"] == "compact":  # moved bytes have none either; the weights move as they are
        weights = s["weights"].double()
        for b, (n, m) in enumerate(zip(_lens(case), _keeps(case))):
            m = min(n, m)
            for h in range(case["kv_heads"]):
                kept = s["index"][b, h if case["per_head"] else 0, :m].long()
                weights[b, h, :n] = torch.cat([weights[b, h, kept], weights.new_zeros(n - m)])
        return {"pool": None, "weights": weights}
    H, Hq, q_len, lens = case["kv_heads"], case["q_heads"], case["q_len"], _lens(case)
    G, offsets = Hq // H, _row_bytes(H)
    out = torch.zeros(len(lens) * q_len, Hq, D, dtype=torch.float64, device=DEV)
    weights = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        place = s["table"][b].long()[t // PAGE] * (9216 * H)
        for h in range(H):
            row = s["pool"].view(-1)[place[:, None] + offsets[h, t % PAGE]]
            k, v = _value64(row[:, :64], row[:, 64:72]), _value64(row[:, 72:136], row[:, 136:])
            total = s["held"][b, h, :n].double()
            for i in range(q_len):
                mine = (b * q_len + i, slice(h * G, h * G + G))
                q = _value64(s["q_codes"][mine], s["q_scales"][mine])
                end = n - q_len + i + 1 if case["causal"] else n
                p = torch.softmax(q @ k[:end].T / math.sqrt(D), 1)
                out[mine] = p @ v[:end]
                total[:end] += p.sum(0)
            weights[b, h, :n] = total
    return {"out": out, "weights": weights}
