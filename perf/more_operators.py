"""Cases of speculative decoding with a drafted tree, and of the pages of sessions that branch: the
tree's masks, its attention over the paged cache, the accepted path, and forking, reserving, copying
and freeing pages.

`run` computes an operator in its plain form (elementary torch operations, fp32 and wider) or, with
`own` set, through the library's entry points, on what `prepare` made from a seed. `exact` gives the
attention's output from its definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
D = 128          # head dim
PAGE = 64        # token slots per page
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # E2M1 magnitudes by code
VOCAB = 32000    # of the drafted tokens


# ---- cases -------------------------------------------------------------------------------------

def _ints(text):
    return [int(x) for x in str(text).split(",")]


def listed():
    return [
        # a short chat with a small tree of drafts: latency counts
        {"name": "attend tree of 8 over 97", "op": "attend", "held": "97", "nodes": 8,
         "q_heads": 24, "kv_heads": 4},
        # a batch of sessions of mixed age on a model with eight KV heads, two of them new
        {"name": "attend trees of 8, ragged, 8 KV heads", "op": "attend",
         "held": "0,13,517,2049,4100,8191,20011,32769", "nodes": 8, "q_heads": 32, "kv_heads": 8},
        # four long sessions, trees of the size that drafters build
        {"name": "attend trees of 32 over 4 x 100000", "op": "attend",
         "held": ",".join(["100000"] * 4), "nodes": 32, "q_heads": 24, "kv_heads": 4},
        # the benchmark's four long sessions with wide trees
        {"name": "attend trees of 64 over 4 x 131072", "op": "attend",
         "held": ",".join(["131072"] * 4), "nodes": 64, "q_heads": 24, "kv_heads": 4},
        # one session's draft, a few nodes
        {"name": "mask of one tree of 8", "op": "mask", "sessions": 1, "nodes": 8},
        # a full server with the largest trees
        {"name": "masks of 128 trees of 256", "op": "mask", "sessions": 128, "nodes": 256},
        # one session's verified tree
        {"name": "accept from one tree of 16", "op": "accept", "sessions": 1, "nodes": 16,
         "most": 1000, "kv_heads": 4},
        # a full server's verified trees
        {"name": "accept from 64 trees of 64", "op": "accept", "sessions": 64, "nodes": 64,
         "most": 4000, "kv_heads": 8},
        # every step of four long sessions: room for the tree, and what it left given back
        {"name": "reserve 16 slots for 4 sessions", "op": "pages", "kind": "reserve", "sessions": 4,
         "most": 131072, "tokens": 16},
        # the same on a full server
        {"name": "reserve 64 slots for 256 sessions", "op": "pages", "kind": "reserve",
         "sessions": 256, "most": 32768, "tokens": 64},
        # parallel answers to one long prompt: shared pages, the last one copied for each
        {"name": "branch 100037 tokens into 9", "op": "pages", "kind": "branch", "sessions": 1,
         "held": 100037, "children": 8, "tokens": 100, "kv_heads": 4},
        # long sessions end, others of their length begin
        {"name": "turn over 4 x 131072", "op": "pages", "kind": "turnover", "sessions": 4,
         "held": 131072},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "mask", "accept", "pages", "pages"])
    q_heads, kv_heads = rng.choice([(24, 4), (24, 4), (32, 8), (16, 2), (8, 8), (12, 3), (20, 5),
                                    (16, 4), (8, 4)])
    if op == "attend":
        n = rng.randint(1, 8)
        nodes = rng.choice([rng.randint(1, 8), _log_int(rng, 2, 64), _log_int(rng, 8, 128)])
        # at most the tokens of the largest listed case, and its (row, key) pairs
        most = min(4 * 131072 // n, 4 * 131072 * 24 * 64 // (nodes * q_heads * n),
                   4 * 131072 * 4 // kv_heads // n)
        held = [_log_int(rng, 1, most) - 1 for _ in range(n)]
        return {"op": op, "held": ",".join(map(str, held)), "nodes": nodes, "q_heads": q_heads,
                "kv_heads": kv_heads}
    if op == "mask":
        return {"op": op, "sessions": _log_int(rng, 1, 128), "nodes": _log_int(rng, 1, 256)}
    if op == "accept":
        return {"op": op, "sessions": _log_int(rng, 1, 64), "nodes": _log_int(rng, 1, 64),
                "most": _log_int(rng, 100, 4000), "kv_heads": kv_heads}
    kind = rng.choice(["reserve", "branch", "turnover"])
    if kind == "reserve":
        return {"op": op, "kind": kind, "sessions": _log_int(rng, 1, 256),
                "most": _log_int(rng, 100, 32768), "tokens": _log_int(rng, 1, 256)}
    if kind == "branch":
        m = rng.randint(1, 4)
        return {"op": op, "kind": kind, "sessions": m, "held": _log_int(rng, 1, 100000 // m),
                "children": rng.randint(1, 12), "tokens": _log_int(rng, 1, 300),
                "kv_heads": min(kv_heads, 4)}
    m = rng.randint(1, 16)
    return {"op": op, "kind": kind, "sessions": m, "held": _log_int(rng, 1, 4 * 131072 // m)}


def _pages_of(tokens):
    return (tokens + PAGE - 1) // PAGE


def work(case):
    """Bytes and operations one pass cannot do without."""
    op = case["op"]
    if op == "attend":
        held, n, hq, H = _ints(case["held"]), case["nodes"], case["q_heads"], case["kv_heads"]
        S, W = len(held), (n + 31) // 32
        # a node sees the cached tokens and at least itself
        pairs = sum(held) * n * hq + S * n * hq
        return {"bytes": (sum(held) + S * n) * H * 144 + S * n * (hq * (72 + 2 * D) + 4 * W),
                "flops": 4 * D * pairs}
    if op == "mask":
        S, n = case["sessions"], case["nodes"]
        return {"bytes": S * (n * (4 + 4 * ((n + 31) // 32) + 12) + 4), "flops": S * n}
    if op == "accept":
        S, n = case["sessions"], case["nodes"]
        moved = S * min(2, n - 1)  # a path's first node is mostly in its place
        return {"bytes": S * (12 * n + 20) + moved * case["kv_heads"] * 288, "flops": S * n}
    S = case["sessions"]
    if case["kind"] == "reserve":
        fresh = S * case["tokens"] / PAGE  # pages taken and given back: table, count, list
        return {"bytes": 2 * (16 * S + 12 * fresh), "flops": 0}
    if case["kind"] == "turnover":
        return {"bytes": 2 * (16 * S + 12 * S * _pages_of(case["held"])), "flops": 0}
    # a child's pages: its table row read and written, the shared counts up and down
    k, held = case["children"], _pages_of(case["held"])
    copies = (k + 1) * 2 * 9216 * case["kv_heads"] if case["held"] % PAGE else 0
    return {"bytes": S * (k * held * 8 + held * 16 + copies), "flops": 0}


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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _block_table(lens, g, spare=3):
    """Pages of the sequences scattered over a pool: (table [S, P] int32, pages in the pool)."""
    pages = [_pages_of(n) for n in lens]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=g, device=DEV).int()
    table = torch.zeros(len(lens), max(1, max(pages)), dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n]
        at += n
    return table, total


def _trees(S, n, g):
    """Parents [S, n] of drafted trees: node 0 hangs on the cache, a later one on an earlier node,
    rather on an early or on the last one; a few trees have fewer nodes than there is room for."""
    i = torch.arange(n, device=DEV)
    u = torch.rand(S, n, generator=g, device=DEV)
    chain = torch.rand(S, n, generator=g, device=DEV) < 0.4
    parents = torch.where(chain, i - 1, (u * u * i).long())
    parents[:, 0] = -1
    fewer = torch.rand(S, 1, generator=g, device=DEV) < 0.2
    count = (n * (0.5 + 0.5 * torch.rand(S, 1, generator=g, device=DEV))).long().clamp(min=1)
    return torch.where(fewer & (i >= count), -2, parents).int()


def _ancestors(parents):
    """Whether node j is node i or above it, [S, n, n]; a node without a way up sees nothing."""
    S, n = parents.shape
    i = torch.arange(n, device=DEV)
    valid = (parents >= -1) & (parents < i)
    # node n stands for the cache, node n + 1 for nowhere
    up = torch.where(valid, torch.where(parents == -1, n, parents), n + 1).long()
    up = torch.cat([up, torch.tensor([[n, n + 1]], device=DEV).expand(S, 2)], 1)
    sees = torch.zeros(S, n + 2, n + 2, dtype=torch.bool, device=DEV)
    sees.diagonal(dim1=1, dim2=2).fill_(True)
    step = 1
    while step <= n:  # the sets of nodes at most 2 step - 1 levels up
        sees = sees | sees.gather(1, up[:, :, None].expand(S, n + 2, n + 2))
        up = up.gather(1, up)
        step *= 2
    rooted = sees[:, :n, n]
    return sees[:, :n, :n] & rooted[:, :, None]


def _pack_bits(sees):
    """[S, n, n] truth values as int32 words [S, n, ceil(n / 32)], node j at bit j % 32 of word j / 32."""
    S, n, _ = sees.shape
    W = (n + 31) // 32
    bits = torch.zeros(S, n, W * 32, dtype=torch.int64, device=DEV)
    bits[:, :, :n] = sees.long()
    words = (bits.view(S, n, W, 32) << torch.arange(32, device=DEV)).sum(3)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()


def _prepare_attend(case, g):
    held, n, Hq, H = _ints(case["held"]), case["nodes"], case["q_heads"], case["kv_heads"]
    lens = [h + n for h in held]
    table, total = _block_table(lens, g)
    pool = torch.zeros(total, 9216 * H, dtype=torch.uint8, device=DEV)
    queries = []
    for s, t in enumerate(lens):
        # most keys are noise to the queries; a few (and the first ones) lie along the direction
        # that the head looks for, and gather most of the weight
        p = _pages_of(t)
        look = torch.randn(H, 1, D, generator=g, device=DEV)
        heavy = (torch.rand(H, p * PAGE, 1, generator=g, device=DEV) < 0.01).float()
        heavy[:, :4] = 1
        k = torch.randn(H, p * PAGE, D, generator=g, device=DEV) + 0.5 * heavy * look
        kc, ks = _encode(k)
        vc, vs = _encode(torch.randn(H, p * PAGE, D, generator=g, device=DEV))
        pool[table[s, :p].long()] = _pack_pages(kc, ks, vc, vs)
        q = 1.3 * torch.randn(n, H, Hq // H, D, generator=g, device=DEV) + 0.6 * look
        queries.append(q.reshape(n, Hq, D))
    q_codes, q_scales = _encode(torch.cat(queries))
    return {"pool": pool, "table": table, "q_codes": q_codes, "q_scales": q_scales,
            "mask": _pack_bits(_ancestors(_trees(len(lens), n, g))), "held": _i32(held),
            "out": torch.zeros(len(lens) * n, Hq, D, dtype=torch.bfloat16, device=DEV)}


def _prepare_mask(case, g):
    S, n = case["sessions"], case["nodes"]
    held = torch.randint(0, 131072, (S,), generator=g, device=DEV, dtype=torch.int32)
    new = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"parents": _trees(S, n, g), "held": held,
            # behind an eviction the next position lies past the next slot
            "first": held + torch.randint(0, 9999, (S,), generator=g, device=DEV, dtype=torch.int32),
            "mask": new(S, n, (n + 31) // 32), "seqs": new(S * n), "slots": new(S * n),
            "positions": new(S * n)}


def _prepare_accept(case, g):
    S, n, H = case["sessions"], case["nodes"], case["kv_heads"]
    held = torch.randint(0, case["most"], (S,), generator=g, device=DEV, dtype=torch.int32)
    table, total = _block_table([case["most"] + n] * S, g)
    parents = _trees(S, n, g)
    i = torch.arange(n, device=DEV)
    draft = torch.randint(0, VOCAB, (S, n), generator=g, device=DEV, dtype=torch.int32)
    # the model agrees with one child in three of four nodes that have some
    luck = torch.rand(S, n, generator=g, device=DEV)
    luck = torch.where((parents >= 0) & (parents < i), luck, torch.zeros_like(luck))
    best = torch.zeros(S, n, device=DEV).scatter_reduce(1, parents.long().clamp(min=0), luck, "amax")
    picked = (luck > 0) & (luck == best.gather(1, parents.long().clamp(min=0)))
    target = torch.randint(0, VOCAB, (S, n), generator=g, device=DEV, dtype=torch.int32)
    agrees = torch.rand(S, n, generator=g, device=DEV) < 0.75
    child = torch.full((S, n + 1), -1, dtype=torch.int64, device=DEV)
    child.scatter_(1, torch.where(picked, parents.long(), n), i.expand(S, n))
    child = child[:, :n]
    target = torch.where(agrees & (child >= 0), draft.gather(1, child.clamp(min=0)), target)
    return {"pool": torch.randint(0, 256, (total, 9216 * H), generator=g, device=DEV,
                                  dtype=torch.uint8),
            "table": table, "parents": parents, "draft": draft, "target": target,
            "expected": draft[:, 0].clone(), "held": held,
            "path": torch.full((S, n), -1, dtype=torch.int32, device=DEV),
            "count": torch.zeros(S, dtype=torch.int32, device=DEV),
            "next": torch.zeros(S, dtype=torch.int32, device=DEV),
            "lens": torch.zeros(S, dtype=torch.int32, device=DEV), "row_bytes": _row_bytes(H)}


def _prepare_pages(case, g):
    kind, m = case["kind"], case["sessions"]
    if kind == "reserve":
        most = case["most"]
        lens = torch.exp(torch.rand(m, generator=g, device=DEV) * math.log(most)).long().clamp(1, most)
        room, children = case["tokens"], 0
    else:
        lens = torch.full((m,), case["held"], device=DEV)
        most = case["held"]
        room, children = case.get("tokens", 0), case.get("children", 0)
    S = m * (1 + children)
    lens = lens.repeat(1 + children)  # the parents' rows first, then their first children's, ...
    P = _pages_of(most + room)
    held = (lens + PAGE - 1) // PAGE
    held[m:] = 0
    # room for what a pass takes, and a few pages more
    spare = S * (2 + _pages_of(room)) + 5
    if kind == "turnover":
        spare += m * P
    used = m * P
    total = used + spare
    order = torch.randperm(total, generator=g, device=DEV).int()
    at = torch.arange(P, device=DEV)
    mine = at < held[:, None]
    table = torch.full((S, P), -1, dtype=torch.int32, device=DEV)
    table[:m] = torch.where(mine[:m], order[:used].view(m, P), -1)
    refs = torch.zeros(total + 1, dtype=torch.int32, device=DEV)
    refs[torch.where(mine, table, total).long()] = 1
    refs = refs[:total].contiguous()
    free = torch.zeros(total, dtype=torch.int32, device=DEV)
    rest = order[refs[order.long()] == 0]
    free[:rest.numel()] = rest
    state = {"table": table, "refs": refs, "free": free, "count": _i32([rest.numel()]),
             "held": held.int(), "lens": lens.int(), "none": torch.zeros_like(lens).int(),
             "copies": torch.zeros(S, 2, dtype=torch.int32, device=DEV),
             "copies_after": torch.zeros(S, 2, dtype=torch.int32, device=DEV)}
    state["more"] = state["lens"] + room
    if kind == "branch":
        state["kept"] = torch.cat([state["lens"][:m], state["none"][m:]])
        state["from"] = torch.arange(m, device=DEV).repeat(children).int()
        state["to"] = torch.arange(m, S, device=DEV).int()
        state["pool"] = torch.randint(0, 256, (total, 9216 * case["kv_heads"]), generator=g,
                                      device=DEV, dtype=torch.uint8)
    return state


def prepare(case, seed):
    make = {"attend": _prepare_attend, "mask": _prepare_mask, "accept": _prepare_accept,
            "pages": _prepare_pages}[case["op"]]
    state = make(case, _generator(seed))
    state["case"] = case
    if own:  # the library's handles that a serving program keeps: layout, status word, the step's plan
        import bit_kv_cache_03_gb300 as kv
        H = case.get("kv_heads", 4)
        state["kv"] = kv
        state["layout"] = kv.make_layout(case.get("q_heads", H), H, D, PAGE, 0)
        state["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if case["op"] == "attend":
            L, n = state["layout"], case["nodes"]
            lens = [h + n for h in _ints(case["held"])]
            chunk = PAGE if case["q_heads"] // H * n <= 8 and H <= 4 else 2 * PAGE
            size = kv.kv_nvfp4_plan_workspace_bytes(L, lens, n, False, chunk)
            state["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
            state["plan"] = kv.kv_nvfp4_plan(L, lens, n, False, chunk, state["workspace"], size)
        if case["op"] == "pages":
            size = kv.kv_nvfp4_pages_workspace_bytes(state["refs"].numel())
            state["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
            state["pages"] = kv.make_pages(state["table"], state["held"], state["refs"],
                                           state["free"], state["count"], state["workspace"])
    return state


# ---- one pass ----------------------------------------------------------------------------------

def _results(s):
    case = s["case"]
    names = {"attend": ["out"], "mask": ["mask", "seqs", "slots", "positions"],
             "accept": ["pool", "path", "count", "next", "lens"],
             "pages": ["table", "held", "refs", "free", "count", "copies", "copies_after"]}[case["op"]]
    return {name: s[name] for name in names + ["pool"] * (case.get("kind") == "branch")}


def _own(s):
    kv, case = s["kv"], s["case"]
    if case["op"] == "attend":
        kv.kv_nvfp4_tree_attn(
            s["layout"], s["plan"], s["workspace"], s["q_codes"], s["q_scales"], s["mask"],
            1.0 / math.sqrt(D), s["pool"], s["pool"].shape[0], s["table"], s["table"].shape[1],
            s["out"], s["status"])
    elif case["op"] == "mask":
        kv.kv_nvfp4_tree_mask(s["parents"], case["sessions"], case["nodes"], s["held"], s["first"],
                              s["mask"], s["seqs"], s["slots"], s["positions"], s["status"])
    elif case["op"] == "accept":
        kv.kv_nvfp4_tree_accept(
            s["layout"], s["parents"], s["draft"], s["target"], s["expected"], case["sessions"],
            case["nodes"], s["held"], s["table"], s["table"].shape[1], s["pool"].shape[0], s["pool"],
            s["path"], s["count"], s["next"], s["lens"], s["status"])
    elif case["kind"] == "reserve":
        kv.kv_nvfp4_pages_resize(s["pages"], s["lens"], s["more"], s["copies"], s["status"])
        kv.kv_nvfp4_pages_resize(s["pages"], s["lens"], s["lens"], s["copies_after"], s["status"])
    elif case["kind"] == "turnover":
        kv.kv_nvfp4_pages_resize(s["pages"], s["none"], s["none"], s["copies"], s["status"])
        kv.kv_nvfp4_pages_resize(s["pages"], s["none"], s["lens"], s["copies_after"], s["status"])
    else:
        n = s["to"].shape[0]
        kv.kv_nvfp4_pages_fork(s["pages"], s["from"], s["to"], s["lens"][-n:], n, s["status"])
        kv.kv_nvfp4_pages_resize(s["pages"], s["lens"], s["more"], s["copies"], s["status"])
        kv.kv_nvfp4_copy_pages(s["layout"], s["pool"], s["pool"].shape[0], s["copies"],
                               s["copies"].shape[0], s["status"])
        kv.kv_nvfp4_pages_resize(s["pages"], s["kept"], s["kept"], s["copies_after"], s["status"])
    return _results(s)


def _plain_attend(s):
    case = s["case"]
    H, Hq, n = case["kv_heads"], case["q_heads"], case["nodes"]
    S, P = s["table"].shape
    R, T = Hq // H * n, P * PAGE
    kc, ks, vc, vs = _unpack_pages(s["pool"][s["table"].long()], H)
    q = _decode(s["q_codes"], s["q_scales"])
    q = q.view(S, n, H, Hq // H, D).transpose(1, 2).reshape(S, H, R, D)
    scores = q @ _decode(kc, ks).transpose(2, 3) * (1.0 / math.sqrt(D))
    node = torch.arange(T, device=DEV) - s["held"].long()[:, None]  # of each slot, [S, T]
    bits = (s["mask"][..., None] >> torch.arange(32, device=DEV) & 1).flatten(2)[:, :, :n] != 0
    among = bits.gather(2, node.clamp(0, n - 1)[:, None].expand(S, n, T))
    sees = (node < 0)[:, None] | (among & (node < n)[:, None])  # [S, n, T]
    hidden = ~sees.repeat_interleave(Hq // H, 1)[:, None]
    scores = scores.masked_fill(hidden, -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    # a hidden key takes no part, whatever its value
    out = (p @ _decode(vc, vs)).view(S, H, n, Hq // H, D).transpose(1, 2).reshape(S * n, Hq, D)
    s["out"].copy_(out.bfloat16())


def _plain_mask(s):
    S, n = s["parents"].shape
    sees = _ancestors(s["parents"])
    depth = sees.sum(2).int()
    node = torch.arange(n, device=DEV, dtype=torch.int32)
    s["mask"].copy_(_pack_bits(sees))
    s["seqs"].copy_(torch.arange(S, device=DEV, dtype=torch.int32).repeat_interleave(n))
    s["slots"].copy_((s["held"][:, None] + node).flatten())
    s["positions"].copy_((s["first"][:, None] + (depth - 1).clamp(min=0)).flatten())


def _plain_accept(s):
    parents, draft, S, n = s["parents"].long(), s["draft"], *s["parents"].shape
    i = torch.arange(n, device=DEV)
    valid = (parents >= -1) & (parents < i)
    # the first child that a node's target names, n where there is none; row n is the cache
    wants = torch.cat([s["target"], s["expected"][:, None]], 1)
    under = torch.where(valid, torch.where(parents == -1, n, parents), n + 1)
    fits = (under[:, None] == torch.arange(n + 1, device=DEV)[:, None]) & \
        (draft[:, None] == wants[:, :, None])  # [S, n + 1, n]
    child = torch.where(fits, i, n).amin(2)
    # the path's nodes by doubling: hop[k] is the node after `step` steps from k, n + 1 for none
    hop = torch.where(child == n, n + 1, child)
    hop = torch.cat([hop, torch.full((S, 1), n + 1, device=DEV)], 1)
    path, step = hop[:, n:n + 1], 1
    while path.shape[1] < n:
        path = torch.cat([path, hop.gather(1, path)], 1)
        hop = hop.gather(1, hop)
    path = path[:, :n]
    count = (path < n).sum(1)
    last = path.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0]
    at = torch.where(count > 0, last, n)
    s["path"].copy_(torch.where(path < n, path, s["path"].long()))
    s["count"].copy_(count)
    s["next"].copy_(wants.gather(1, at[:, None])[:, 0])
    held = s["held"].long()
    s["lens"].copy_(held + count)
    # the path's rows move behind the cache; the others write where they stand
    table, bytes_of = s["table"].long(), s["row_bytes"]
    flat, block = s["pool"].view(-1), s["pool"].shape[1]
    old = held[:, None] + torch.where(path < n, path, i)
    new = (held[:, None] + i).expand_as(old)
    stays = (path >= n) & (i[None] < n)
    src = torch.where(stays, new, old)

    def place(slot):  # [S, n, H, 144]
        page = table.gather(1, slot // PAGE)
        return (page * block)[:, :, None, None] + bytes_of[:, slot % PAGE].permute(1, 2, 0, 3)
    flat[place(new)] = flat[place(src)]


def _plain_resize(s, keep, room, copies):
    table, refs, free, count, held = (s[k] for k in ("table", "refs", "free", "count", "held"))
    S, P = table.shape
    pages = refs.shape[0]
    j = torch.arange(P, device=DEV)
    full, kept = (keep // PAGE)[:, None], ((keep + PAGE - 1) // PAGE)[:, None]
    need, have = ((room + PAGE - 1) // PAGE)[:, None], held[:, None]
    old = table.long().clamp(min=0)
    shared = (j >= full) & (j < torch.minimum(have, need)) & (refs[old] > 1)
    drop = shared | ((j >= need) & (j < have))
    take = shared | ((j >= have) & (j < need))
    demand = take.sum(1)
    ok = ((demand == 0) | (demand.cumsum(0) <= count))[:, None]  # in the order of the sequences
    drop, take = drop & ok, take & ok
    rank = take.flatten().cumsum(0).view(S, P) - 1
    fresh = free[(count - 1 - rank).clamp(min=0)]
    copied = shared & take & (j < kept)
    pair = torch.stack([table, fresh], 2)
    none = torch.full_like(pair[:, 0], -1)
    at = (copied * j).sum(1)
    copies.copy_(torch.where(copied.any(1)[:, None], pair[torch.arange(S, device=DEV), at], none))
    wide = torch.cat([refs, refs.new_zeros(1)])  # a place for what does not count
    wide.index_add_(0, torch.where(drop, old, pages).flatten(), drop.flatten().int(), alpha=-1)
    wide[torch.where(take, fresh.long(), pages)] = 1
    refs.copy_(wide[:pages])
    # a page is free when its last holder in the order drops it
    order = torch.arange(S * P, device=DEV).view(S, P)
    last = torch.full((pages + 1,), -1, device=DEV).scatter_reduce_(
        0, torch.where(drop, old, pages).flatten(), order.flatten(), "amax")
    freed = drop & (refs[old] == 0) & (last[old] == order)
    left = count - take.sum()
    spot = (left + freed.flatten().cumsum(0).view(S, P) - 1).long()
    longer = torch.cat([free, free.new_zeros(1)])
    longer[torch.where(freed, spot, pages)] = table
    free.copy_(longer[:pages])
    count.copy_(left + freed.sum())
    table.copy_(torch.where(take, fresh, torch.where(drop, -1, table)))
    held.copy_(torch.where(ok[:, 0], need[:, 0], held))


def _plain_fork(s, src, dst, lens):
    table, refs, held = s["table"], s["refs"], s["held"]
    j = torch.arange(table.shape[1], device=DEV)
    have = (lens + PAGE - 1) // PAGE
    mine = j < have[:, None]
    rows = torch.where(mine, table[src.long()], -1)
    wide = torch.cat([refs, refs.new_zeros(1)])
    wide.index_add_(0, torch.where(mine, rows, refs.shape[0]).flatten(), mine.flatten().int())
    refs.copy_(wide[:-1])
    table[dst.long()] = rows
    held[dst.long()] = have


def _plain_pages(s):
    kind = s["case"]["kind"]
    if kind == "reserve":
        _plain_resize(s, s["lens"], s["more"], s["copies"])
        _plain_resize(s, s["lens"], s["lens"], s["copies_after"])
    elif kind == "turnover":
        _plain_resize(s, s["none"], s["none"], s["copies"])
        _plain_resize(s, s["none"], s["lens"], s["copies_after"])
    else:
        _plain_fork(s, s["from"], s["to"], s["lens"][-s["to"].shape[0]:])
        _plain_resize(s, s["lens"], s["more"], s["copies"])
        src, dst = s["copies"].long().unbind(1)  # a pair of -1 writes a page's own bytes
        own_page = s["table"][0, 0].long()
        src, dst = torch.where(dst < 0, own_page, src), torch.where(dst < 0, own_page, dst)
        s["pool"][dst] = s["pool"][src]
        _plain_resize(s, s["kept"], s["kept"], s["copies_after"])


def run(state):
    if own:
        return _own(state)
    {"attend": _plain_attend, "mask": _plain_mask, "accept": _plain_accept,
     "pages": _plain_pages}[state["case"]["op"]](state)
    return _results(state)


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
    if case["op"] != "attend":  # page ids, masks, tokens and moved bytes: no value but their own
        return None
    s = prepare(case, seed)
    H, Hq, n, held = case["kv_heads"], case["q_heads"], case["nodes"], _ints(case["held"])
    G, offsets = Hq // H, _row_bytes(H)
    out = torch.zeros(len(held) * n, Hq, D, dtype=torch.float64, device=DEV)
    bit = torch.arange(n, device=DEV)
    for b, base in enumerate(held):
        t = torch.arange(base + n, device=DEV)
        place = s["table"][b].long()[t // PAGE] * (9216 * H)
        words = s["mask"][b].long()[:, bit // 32]
        below = torch.ones(n, base, dtype=torch.bool, device=DEV)
        sees = torch.cat([below, torch.bitwise_right_shift(words, bit % 32) % 2 == 1], 1)
        mine = slice(b * n, (b + 1) * n)
        for h in range(H):
            row = s["pool"].view(-1)[place[:, None] + offsets[h, t % PAGE]]
            k, v = _value64(row[:, :64], row[:, 64:72]), _value64(row[:, 72:136], row[:, 136:])
            for g in range(h * G, h * G + G):
                q = _value64(s["q_codes"][mine, g], s["q_scales"][mine, g])
                score = torch.where(sees, q @ k.T / math.sqrt(D), -math.inf)
                p = torch.nan_to_num(torch.softmax(score, 1))  # 0 for a row that sees nothing
                out[mine, g] = p @ v
    return {"out": out}
