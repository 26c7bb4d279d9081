"""Workloads of the calls that check a tree of drafted tokens on the position-free page pool.

Four operators, each in a plain form (elementary torch operations) and through the package:

``tables``     positions of a tree's nodes, and for each the nodes it goes on from, out of their parents
``attention``  the nodes of every request's tree over its pages and over their own branches
``accept``     the branch that the model's own choices confirm: the new lengths, and the pages it leaves unused
``keep``       that branch's keys and values moved together in the pages, layer by layer

A request holds ``seq`` tokens in the pages ``block_table[b]`` lists, 16 to a page; token 16 p + r sits
at position ``page_pos[b][p] + r``.  Its ``new`` drafted tokens take the slots behind, a parent before
its children; node t goes on from node ``parent[t]`` of the same request, or from the last token held
(-1).  A node's position follows from its depth, not from its slot, and it sees the held tokens, itself
and the nodes it goes on from.  Keys are stored unrotated, so the branch that is kept moves bit for bit.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 16
DEV = "cuda"
VOCAB = 32000
# (query heads, kv heads, head dim) of the workloads and of the tests
SHAPES = ((8, 2, 64), (32, 8, 128), (64, 8, 128), (12, 3, 64), (24, 12, 128), (16, 2, 128), (4, 4, 64))


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one step's trees of a batch that decodes: 64 requests, 16 nodes each
        dict(name="tables_step", op="tables", reqs=64, new_lo=16, new_hi=16, width=4, hq=64, hkv=8, d=128, ctx_lo=1000,
             ctx_hi=2000, mix=1),
        # many requests whose drafts differ in size, the largest trees among them
        dict(name="tables_large", op="tables", reqs=512, new_lo=0, new_hi=256, width=40, hq=32, hkv=8, d=128, ctx_lo=0,
             ctx_hi=1000, mix=2),
        # latency: a small tree behind a short context, small heads
        dict(name="tree_tiny", op="attention", reqs=1, new_lo=7, new_hi=7, width=3, hq=8, hkv=2, d=64, ctx_lo=579,
             ctx_hi=579, mix=3),
        # one request of the Llama-3-8B-shaped layer, a tree of 26 nodes behind 4 k tokens
        dict(name="tree_layer", op="attention", reqs=1, new_lo=26, new_hi=26, width=5, hq=32, hkv=8, d=128, ctx_lo=4161,
             ctx_hi=4161, mix=4),
        # one long request, 64 nodes
        dict(name="tree_long", op="attention", reqs=1, new_lo=64, new_hi=64, width=8, hq=32, hkv=8, d=128, ctx_lo=32897,
             ctx_hi=32897, mix=5),
        # the 70B-shaped batch behind its fused prefill: 64 requests over shared spans, 16 nodes each,
        # stale copies of the recomputed tokens excluded
        dict(name="tree_shared", op="attention", reqs=64, new_lo=16, new_hi=16, width=4, hq=64, hkv=8, d=128, spans=16,
             span_len=1024, pool=256, zipf=1.0, pct=10, query=128, mix=6),
        # ragged requests, trees of 1 to 64 nodes
        dict(name="tree_ragged", op="attention", reqs=48, new_lo=1, new_hi=64, width=6, hq=32, hkv=8, d=128, ctx_lo=100,
             ctx_hi=9000, mix=7),
        # the largest trees behind short contexts: several row tiles a request
        dict(name="tree_wide", op="attention", reqs=12, new_lo=200, new_hi=256, width=60, hq=64, hkv=8, d=128, ctx_lo=500,
             ctx_hi=4000, mix=8),
        # one step's branches, 64 requests
        dict(name="accept_step", op="accept", reqs=64, new_lo=16, new_hi=16, width=4, hq=64, hkv=8, d=128, ctx_lo=1000,
             ctx_hi=2000, hit=0.7, roots=0, mix=9),
        # many requests, the largest trees, several candidates for the first token
        dict(name="accept_large", op="accept", reqs=512, new_lo=0, new_hi=256, width=40, hq=32, hkv=8, d=128, ctx_lo=0,
             ctx_hi=1000, hit=0.85, roots=1, mix=10),
        # the kept branch of one request in every layer of a small model
        dict(name="keep_one", op="keep", reqs=1, new_lo=26, new_hi=26, width=5, hq=32, hkv=8, d=128, ctx_lo=400, ctx_hi=400,
             hit=0.95, roots=0, layers=32, mix=28),
        # the kept branches of 128 requests in every layer
        dict(name="keep_batch", op="keep", reqs=128, new_lo=60, new_hi=64, width=6, hq=64, hkv=8, d=128, ctx_lo=50,
             ctx_hi=200, hit=0.95, roots=0, layers=32, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "attention", "attention", "attention", "accept", "keep"])
    hq, hkv, d = rng.choice(SHAPES)
    nodes = _log_int(rng, 1, 256)
    c = dict(op=op, hq=hq, hkv=hkv, d=d, new_lo=rng.choice([0, 1, (nodes + 1) // 2, nodes]), new_hi=nodes,
             width=_log_int(rng, 1, 64), mix=rng.randrange(1 << 30))
    if op in ("tables", "accept"):
        c = dict(c, reqs=_log_int(rng, 1, 512), ctx_lo=0, ctx_hi=_log_int(rng, 1, 1000))
        return c if op == "tables" else dict(c, hit=rng.uniform(0.3, 0.95), roots=rng.randint(0, 1))
    if op == "keep":
        reqs = _log_int(rng, 1, 64)
        return dict(c, reqs=reqs, ctx_lo=0, ctx_hi=_log_int(rng, 16, 400), hit=rng.uniform(0.5, 0.95), roots=0,
                    layers=_log_int(rng, 1, 32))
    # scores of the batch, and its keys as 32-bit numbers, stay below those of the largest listed case
    if rng.random() < 0.25:
        reqs, spans = _log_int(rng, 1, 32), rng.randint(1, 8)
        c = dict(c, new_lo=1, new_hi=min(nodes, 64), reqs=reqs, spans=spans, span_len=16 * rng.randint(1, 32),
                 pool=rng.choice([16, 32, 64]), zipf=rng.choice([1.0, 1.1]), pct=rng.choice([5, 10, 15, 30]),
                 query=rng.randint(1, 128))
        return c
    reqs = _log_int(rng, 1, 64)
    room = min(300_000_000 // (reqs * hq * nodes), 400_000 // (reqs * hkv))
    return dict(c, reqs=reqs, ctx_lo=1 if rng.random() < 0.3 else 0, ctx_hi=_log_int(rng, 16, max(17, min(33000, room))))


def _shape(case):
    """Lengths, pages and trees of a case, from its own numbers."""
    rng = random.Random(case["mix"])
    reqs = []
    for b in range(case["reqs"]):
        r = dict(new=rng.randint(case["new_lo"] if b else max(1, case["new_lo"]), case["new_hi"]), shared=[], n_sel=0, k=0, cached=0,
                 pos0=rng.randrange(4096))
        if "spans" in case:
            pages = case["span_len"] // PAGE
            weights = [(i + 1.0) ** -case["zipf"] for i in range(case["pool"])]
            for _ in range(case["spans"]):
                i = rng.choices(range(case["pool"]), weights)[0]
                weights[i] = 0.0
                r["shared"].append((i * pages, pages))
            r["k"] = -(-case["pct"] * case["span_len"] // 100)
            r["n_sel"] = case["spans"] * r["k"]
            r["cached"] = case["spans"] * case["span_len"]
            r["seq"] = r["cached"] + r["n_sel"] + case["query"]
        else:
            r["seq"] = rng.randint(case["ctx_lo"], case["ctx_hi"])
        # a node goes on from one of the `width` before it
        r["parent"] = [-1 if t == 0 or (case.get("roots") and rng.random() < 2 / (t + 2))
                       else rng.randrange(max(0, t - case["width"]), t) for t in range(r["new"])]
        depth = []
        for p in r["parent"]:
            depth.append(0 if p < 0 else depth[p] + 1)
        r["depth"] = depth
        reqs.append(r)
    return reqs


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _tokens(case, reqs):
    """Drafted tokens and the model's choices behind each row: the choice behind a node is one of its
    children's tokens in a share `hit` of the cases."""
    rng = random.Random(case["mix"] + 1)
    draft, choice, first = [], [], []
    for r in reqs:
        tok = [rng.randrange(VOCAB) for _ in range(r["new"])]
        kids = [[] for _ in range(r["new"] + 1)]
        for t, p in enumerate(r["parent"]):
            kids[p].append(t)              # (-1: the last list, of the first tokens)
        said = [tok[rng.choice(k)] if k and rng.random() < case["hit"] else rng.randrange(VOCAB) for k in kids]
        draft += tok
        choice += said[:-1]
        first.append(said[-1])
    return draft, choice, first


def work(case):
    reqs = _shape(case)
    n, rows = len(reqs), sum(r["new"] for r in reqs)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    words = (max(1, max(r["new"] for r in reqs)) + 31) // 32
    if case["op"] == "tables":
        # lengths, first positions and parents in; positions and bits out
        return {"bytes": 4 * (3 * n + rows + rows + rows * words), "flops": 0}
    if case["op"] == "accept":
        # lengths, parents, tokens and choices in; branches, numbers kept, next tokens, lengths out
        return {"bytes": 4 * (2 * n + 3 * rows + rows + 3 * n), "flops": 0}
    if case["op"] == "keep":
        moved = _moved(case, reqs)
        # the branches in; keys and values read and written
        return {"bytes": 4 * (n + rows) + moved * hkv * d * 2 * 2 * 2 * case["layers"], "flops": 0}
    slots, private, keys = set(), 0, 0
    for r in reqs:
        for first, m in r["shared"]:
            slots.update(range(first, first + m))
        private += r["seq"] + r["new"] - r["cached"]
        keys += r["new"] * (r["seq"] - r["n_sel"]) + sum(r["depth"]) + r["new"]
    tokens = private + PAGE * len(slots)
    return {"bytes": tokens * hkv * d * 4 + rows * hq * d * 4, "flops": keys * hq * d * 4}


def _moved(case, reqs):
    """Tokens of the kept branches that do not sit where they belong already."""
    draft, choice, first = _tokens(case, reqs)
    moved = base = 0
    for b, r in enumerate(reqs):
        at, said, place = -1, first[b] if case["roots"] else None, 0
        for t, p in enumerate(r["parent"]):
            if p == at and (said is None or draft[base + t] == said):
                moved += t != place
                at, said, place = t, choice[base + t], place + 1
        base += r["new"]
    return moved


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    reqs = _shape(case)
    n, hq, hkv, d, op = len(reqs), case["hq"], case["hkv"], case["d"], case["op"]
    host = random.Random(seed * 1000003 + case["mix"])
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    rows, nodes = sum(r["new"] for r in reqs), max(1, max(r["new"] for r in reqs))
    max_pages = max(1, max(_pages(r["seq"] + r["new"]) for r in reqs))
    shared_pages = case["pool"] * case["span_len"] // PAGE if "spans" in case else 0
    n_phys = shared_pages + sum(_pages(r["seq"] + r["new"]) - r["cached"] // PAGE for r in reqs) + 7
    order = list(range(shared_pages, n_phys))
    host.shuffle(order)
    table = torch.zeros((n, max_pages), dtype=torch.int32)
    page_pos = torch.zeros((n, max_pages), dtype=torch.int32)
    start, at, top = [], 0, 0
    for b, r in enumerate(reqs):
        if op in ("tables", "accept"):     # (whose results are whole numbers: other positions a seed)
            r["pos0"] = host.randrange(4096)
        pages = [p for first, m in r["shared"] for p in range(first, first + m)]
        private = _pages(r["seq"]) - len(pages)
        pages += order[at: at + private]
        at += private
        pos = torch.arange(len(pages), dtype=torch.int32) * PAGE + r["pos0"]
        # behind the shared spans: the recomputed tokens' slots, then the query at its own positions
        pos[r["cached"] // PAGE:] -= r["n_sel"]
        table[b, : len(pages)] = torch.tensor(pages, dtype=torch.int32)
        page_pos[b, : len(pages)] = pos
        start.append(r["pos0"] + r["seq"] - r["n_sel"])
        top = max(top, start[-1] + r["new"])
    ints = lambda x: torch.tensor(x, dtype=torch.int32).to(DEV)
    free = ints(order[at:])
    # the tables that a step's chunk of new tokens leaves: pages of the tree's slots, the rows' places
    taken = 0
    for b, r in enumerate(reqs):
        first, last = _pages(r["seq"]), _pages(r["seq"] + r["new"])
        for p in range(first, last):
            table[b, p] = order[at + taken]
            page_pos[b, p] = start[b] + p * PAGE - r["seq"]
            taken += 1
    rows_of = [(b, t) for b, r in enumerate(reqs) for t in range(r["new"])] or [(0, 0)]
    s = dict(case=case, reqs=reqs, n=n, rows=rows, nodes=nodes, max_pages=max_pages, n_phys=n_phys, taken=taken,
             theta=1e4 if d == 64 else 5e5, max_pos=top + 2 * PAGE, words=(nodes + 31) // 32,
             seq=ints([r["seq"] for r in reqs]), new=ints([r["new"] for r in reqs]), start=ints(start),
             row_req=ints([b for b, _ in rows_of]).long(), row_node=ints([t for _, t in rows_of]).long(),
             parent=ints([p for r in reqs for p in r["parent"]] or [0]), table=table.to(DEV), page_pos=page_pos.to(DEV),
             free=free, head=ints([0]))
    normal = lambda shape: torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    if op in ("accept", "keep"):
        draft, choice, first = _tokens(case, reqs)
        # (other tokens a seed, the same ones equal)
        turn = host.randrange(VOCAB)
        s["draft"], s["choice"], s["first"] = (ints([(x + turn) % VOCAB for x in v or [0]]) for v in (draft, choice, first))
    if op == "keep":
        # every layer's pool, the drafted tokens' keys and values in their slots
        s["k_all"] = torch.empty((case["layers"], n_phys, hkv, PAGE, d), dtype=torch.bfloat16, device=DEV)
        s["v_all"] = torch.empty_like(s["k_all"])
        for pools in (s["k_all"], s["v_all"]):
            for i in range(case["layers"]):
                pools[i] = normal(pools[i].shape)
        s["path"] = _plain_accept(s)["path"]        # of the step before
    if op == "attention":
        # whole pools of standard normal draws, slots behind a sequence's end included: stale values
        s["k_pool"] = torch.empty((n_phys, hkv, PAGE, d), dtype=torch.bfloat16, device=DEV)
        s["v_pool"] = torch.empty_like(s["k_pool"])
        for pool in (s["k_pool"], s["v_pool"]):
            for i in range(0, n_phys, 4096):
                pool[i: i + 4096] = normal(pool[i: i + 4096].shape)
        s["q"] = normal((max(1, rows), hq, d))
        s["excl"] = None
        if "spans" in case:
            bits = torch.zeros((n, max_pages, PAGE), dtype=torch.int32)
            for b, r in enumerate(reqs):
                flat = bits[b].view(-1)
                for i in range(len(r["shared"])):
                    flat[torch.tensor(host.sample(range(case["span_len"]), r["k"]), dtype=torch.int64)
                         + i * case["span_len"]] = 1
            word = (bits << torch.arange(PAGE, dtype=torch.int32)).sum(-1)
            s["excl"] = torch.where(word >= 32768, word - 65536, word).to(torch.int16).to(DEV)
    # what a program has before these calls: the layout with the chunk's tables, the tree's buffers, the model's
    # cos/sin rows (which the plain form works out within its pass)
    if own:
        _own_prepare(s)
    return s


def _own_prepare(s):
    import position_independent_kv_critical_gb300 as pcf
    case, op = s["case"], s["case"]["op"]
    L = pcf.ChunkLayout(s["n"], case["hq"], case["hkv"], case["d"], s["n_phys"], s["max_pos"], max_pages=s["max_pages"],
                        max_rows=max(1, s["rows"]), max_chunk=s["nodes"])
    L.block_table.copy_(s["table"])
    L.page_pos.copy_(s["page_pos"])
    tree = pcf.DraftTree(L)
    s["pcf"], s["L"], s["tree"] = pcf, L, tree
    s["seq_out"], s["head_out"] = torch.zeros_like(s["seq"]), torch.zeros_like(s["head"])
    pcf.chunk_tables(L, s["seq"], s["new"], s["free"], s["head"], s["seq_out"], s["head_out"], next_pos=s["start"])
    s["first_of"] = s.get("first") if case.get("roots") else None
    if op == "attention":
        s["rope"] = pcf.rope_table(case["d"], s["theta"], s["max_pos"]).to(DEV)
        s["out"] = torch.zeros((max(1, s["rows"]), case["hq"], case["d"]), dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.empty(max(16, tree.attention_workspace_bytes()), dtype=torch.uint8, device=DEV)
    if op == "keep":
        _own_accept(s)
        s["k_pools"], s["v_pools"] = list(s["k_all"]), list(s["v_all"])


# ------------------------------------------------------------------------------------ passes
def run(state):
    op = state["case"]["op"]
    if own:
        L, tree, pcf = state["L"], state["tree"], state["pcf"]
        if op == "tables":
            pcf.tree_tables(L, tree, state["parent"])
            return {"row_pos": tree.row_pos, "seen": tree.seen}
        if op == "accept":
            return _own_accept(state)
        if op == "keep":
            pcf.tree_keep(L, tree, state["k_pools"], state["v_pools"])
            return {"k": state["k_all"], "v": state["v_all"]}
        # (a step's tables and its first layer: like the plain form, the pass starts from the trees' parents)
        pcf.tree_tables(L, tree, state["parent"])
        pcf.tree_attention(L, tree, state["q"], state["k_pool"], state["v_pool"], state["rope"], state["out"], state["ws"],
                           excl=state["excl"])
        return {"out": state["out"]}
    if op == "tables":
        return _plain_tables(state)
    if op == "accept":
        return _plain_accept(state)
    return _plain_keep(state) if op == "keep" else _plain_attention(state)


def _own_accept(s):
    # (from the trees' parents too)
    tree = s["tree"]
    s["pcf"].tree_tables(s["L"], tree, s["parent"])
    s["pcf"].tree_accept(s["L"], tree, s["parent"], s["draft"], s["choice"], s["free"], s["seq_out"], s["head_out"],
                         root_choice=s["first_of"])
    return {"path": tree.path, "kept": tree.n_kept, "next": tree.next_token, "seq": s["seq_out"], "free": s["free"],
            "head": s["head_out"]}


def _by_request(s, x, fill):
    """x [rows, ...] as [requests, nodes, ...]."""
    full = torch.full((s["n"], s["nodes"]) + x.shape[1:], fill, dtype=x.dtype, device=DEV)
    if s["rows"]:
        full[s["row_req"], s["row_node"]] = x[: s["rows"]]
    return full


def _branches(s):
    """[requests, nodes, nodes]: whether node t is, or goes on from, node u."""
    parent = _by_request(s, s["parent"], -1)
    u = torch.arange(s["nodes"], device=DEV)
    seen = ((u[:, None] == u) | (parent[..., None] == u)).float()
    for _ in range((s["nodes"] - 1).bit_length()):         # twice as many steps back each time
        seen = torch.matmul(seen, seen).clamp_(max=1.0)
    return parent, seen > 0.5


def _plain_tables(s):
    _, seen = _branches(s)
    rows = max(1, s["rows"])
    row_pos = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    words = torch.zeros((rows, s["words"]), dtype=torch.int32, device=DEV)
    if s["rows"]:
        b, t = s["row_req"], s["row_node"]
        mine = seen[b, t]
        row_pos[:] = s["start"][b] + mine.sum(-1) - 1
        bits = torch.nn.functional.pad(mine, (0, s["words"] * 32 - s["nodes"])).view(rows, s["words"], 32).long()
        words[:] = (bits << torch.arange(32, device=DEV)).sum(-1).to(torch.int32)
    return {"row_pos": row_pos, "seen": words}


def _plain_accept(s):
    parent, seen = _branches(s)
    nodes, n = s["nodes"], s["n"]
    u = torch.arange(nodes, device=DEV)
    live = u < s["new"][:, None]
    draft, choice = _by_request(s, s["draft"], -1), _by_request(s, s["choice"], -1)
    said = torch.gather(choice, 1, parent.clamp(min=0).long())
    if s["case"]["roots"]:
        hit = draft == torch.where(parent < 0, s["first"][:, None].expand_as(said), said)
        nobody = s["first"]
    else:
        hit = torch.where(parent < 0, u == 0, draft == said)           # the first node is certain
        nobody = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    hit = hit & live
    # of siblings with the same token the first one
    twin = (parent[:, :, None] == parent[:, None, :]) & hit[:, None, :] & (u[None, :] < u[:, None])
    hit = hit & ~twin.any(-1)
    kept = live & ~(seen & ~hit[:, None, :]).any(-1)
    count = kept.sum(-1).to(torch.int32)
    place = torch.cumsum(kept, -1) - 1
    path = torch.full((n, nodes + 1), -1, dtype=torch.int32, device=DEV)
    path.scatter_(1, torch.where(kept, place, nodes), u.to(torch.int32).expand(n, nodes))
    rows = torch.full((max(1, s["rows"]),), -1, dtype=torch.int32, device=DEV)
    if s["rows"]:
        rows[:] = path[:, :nodes][s["row_req"], s["row_node"]]
    last = torch.where(kept, u, -1).amax(-1)
    token = torch.where(count > 0, torch.gather(choice, 1, last.clamp(min=0)[:, None])[:, 0], nobody)
    # pages that the shorter requests do not need go back to the end of what was taken
    seq, new = s["seq"], s["new"]
    held, enough, all_ = _pages(seq), _pages(seq + count), _pages(seq + new)
    p = torch.arange(s["max_pages"], device=DEV)
    back = (p >= enough[:, None]) & (p < all_[:, None])
    at = (torch.cumsum(back.view(-1), 0) - 1).view(back.shape) + s["head"] + (enough - held).sum()
    free = torch.cat([s["free"], s["free"][:1]])                       # (one more for what does not go back)
    free.scatter_(0, torch.where(back, at, s["free"].numel()).view(-1), s["table"].view(-1))
    head = (s["head"] + (enough - held).sum()).to(torch.int32)
    return {"path": rows, "kept": count, "next": token, "seq": seq + count, "free": free[:-1], "head": head}


def _plain_keep(s):
    b, t, path = s["row_req"], s["row_node"], s["path"]
    moves = path >= 0
    b, t, path = b[moves], t[moves], path[moves]
    place = lambda at: s["table"][b, at // PAGE].long() * PAGE + at % PAGE
    src, dst = place(s["seq"][b] + path), place(s["seq"][b] + t)
    for pools in (s["k_all"], s["v_all"]):
        pools[:, dst // PAGE, :, dst % PAGE] = pools[:, src // PAGE, :, src % PAGE]
    return {"k": s["k_all"], "v": s["v_all"]}


def _angles(pos, d, theta):
    """cos and sin of every position and frequency: 64-bit angles, 32-bit results."""
    inv = theta ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    a = pos.to(torch.float64)[..., None] * inv
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, pos, d, theta):
    """x [requests, tokens, heads, d] (32 bits): dimension i turns with i + d/2."""
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    c, s = (a[:, :, None] for a in _angles(pos, d, theta))
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, g = case["hq"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    n, nodes, slots, theta = s["n"], s["nodes"], s["max_pages"] * PAGE, s["theta"]
    _, seen = _branches(s)
    depth = seen.sum(-1) - 1
    j = torch.arange(slots, device=DEV)
    pos = s["page_pos"][:, j // PAGE] + j % PAGE
    node = j - s["seq"][:, None]                                        # the tree's node in a slot behind the held ones
    inside = node.clamp(0, nodes - 1).long()
    place = s["start"][:, None] + depth
    tail = node >= 0
    pos = torch.where(tail, torch.gather(place, 1, inside), pos)
    there = tail & (node < s["new"][:, None])
    branch = torch.gather(seen, 2, inside[:, None].expand(n, nodes, slots)) & there[:, None]
    ok = torch.where(tail[:, None], branch, True)
    if s["excl"] is not None:
        out_of = ((s["excl"].int()[..., None] >> torch.arange(PAGE, device=DEV)) & 1).view(n, slots)
        ok = ok & (out_of == 0)[:, None]
    pages = s["table"].long()
    k = s["k_pool"][pages].transpose(2, 3).reshape(n, slots, hkv, d).float()
    k = _rotate(k, pos, d, theta).transpose(1, 2)                       # [requests, kv heads, slots, d]
    v = s["v_pool"][pages].transpose(1, 2).reshape(n, hkv, slots, d).float()
    q = _rotate(_by_request(s, s["q"], 0).float(), place, d, theta)
    q = q.view(n, nodes, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * nodes, d)
    w = torch.matmul(q, k.transpose(2, 3)).div_(math.sqrt(d)).view(n, hkv, g, nodes, slots)
    w.masked_fill_(~ok[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(n, hkv, g * nodes, slots), v).view(n, hkv, g, nodes, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, nodes, hq, d).to(torch.bfloat16)
    out = torch.zeros((max(1, s["rows"]), hq, d), dtype=torch.bfloat16, device=DEV)
    if s["rows"]:
        out[:] = o[s["row_req"], s["row_node"]]
    return {"out": out}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    keep = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    op, reqs = case["op"], s["reqs"]
    whole = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)
    start = s["start"].tolist()
    ups = []                                  # every node with the nodes it goes on from, itself last
    for r in reqs:
        mine = []
        for t, p in enumerate(r["parent"]):
            mine.append((mine[p] if p >= 0 else []) + [t])
        ups.append(mine)
    if op == "tables":
        pos, bits = [], []
        for b, mine in enumerate(ups):
            for up in mine:
                pos.append(start[b] + len(up) - 1)
                mask = sum(1 << u for u in up)
                word = [(mask >> 32 * w) & 0xFFFFFFFF for w in range(s["words"])]
                bits.append([x - (1 << 32) if x >> 31 else x for x in word])
        return {"row_pos": whole(pos or [-1]), "seen": whole(bits or [[0] * s["words"]])}
    if op in ("accept", "keep"):
        got = _exact_accept(s, ups)
        if op == "accept":
            return {k: whole(v) for k, v in got.items()}
        k, v = s["k_all"].double(), s["v_all"].double()
        at = s["table"].cpu()
        base = 0
        for b, r in enumerate(reqs):
            for i in range(got["kept"][b]):
                t = got["path"][base + i]
                if t == i:
                    continue
                a, z = r["seq"] + t, r["seq"] + i
                pa, pz = int(at[b, a // PAGE]), int(at[b, z // PAGE])
                for pool in (k, v):
                    pool[:, pz, :, z % PAGE] = pool[:, pa, :, a % PAGE].clone()
            base += r["new"]
        return {"k": k, "v": v}
    if work(case)["flops"] > 4e12:
        return None
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    freq = torch.tensor([s["theta"] ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=DEV)

    def turned(x, pos):
        """x [tokens, heads, d] in 64 bits as d/2 complex numbers, turned by position x frequency."""
        z = torch.complex(x[..., : d // 2].double(), x[..., d // 2:].double())
        a = pos.double()[:, None] * freq
        return z * torch.polar(torch.ones_like(a), a)[:, None]

    out = torch.zeros((max(1, s["rows"]), hq, d), dtype=torch.float64, device=DEV)
    base = 0
    for b, r in enumerate(reqs):
        T, n = r["new"], r["seq"] + r["new"]
        if T == 0:
            continue
        j = torch.arange(n, device=DEV)
        page = s["table"][b].long()[j // PAGE]
        pos = s["page_pos"][b].long()[j // PAGE] + j % PAGE
        mine = torch.tensor([start[b] + x for x in r["depth"]], device=DEV)
        pos[r["seq"]:] = mine
        hidden = torch.zeros((T, n), dtype=torch.bool)
        hidden[:, r["seq"]:] = True
        for t, up in enumerate(ups[b]):
            hidden[t, [r["seq"] + u for u in up]] = False
        hidden = hidden.to(DEV)
        if s["excl"] is not None:
            hidden |= (((s["excl"][b].long()[j // PAGE] & 65535) >> (j % PAGE)) % 2 == 1)[None]
        for h in range(hkv):
            zk = turned(s["k_pool"][page, h, j % PAGE][:, None], pos)[:, 0]
            v = s["v_pool"][page, h, j % PAGE].double()
            zq = turned(s["q"][base: base + T, h * g: (h + 1) * g], mine)
            score = torch.einsum("tgi,ji->tgj", zq.real, zk.real) + torch.einsum("tgi,ji->tgj", zq.imag, zk.imag)
            score = (score * d ** -0.5).masked_fill(hidden[:, None], -math.inf)
            lse = torch.logsumexp(score, -1, keepdim=True)
            p = torch.where(lse == -math.inf, torch.zeros_like(score), torch.exp(score - lse))
            out[base: base + T, h * g: (h + 1) * g] = torch.einsum("tgj,jd->tgd", p, v)
        base += T
    return {"out": out}


def _exact_accept(s, ups):
    """The branches walked node by node on the host."""
    seq, draft, choice, first = (s[k].tolist() for k in ("seq", "draft", "choice", "first"))
    table, free, head = s["table"].tolist(), s["free"].tolist(), int(s["head"].item())
    path, kept, token, length, back = [], [], [], [], []
    used = base = 0
    for b, r in enumerate(s["reqs"]):
        at, said = -1, first[b] if s["case"]["roots"] else None
        mine = []
        while True:
            hits = [t for t in range(r["new"]) if r["parent"][t] == at and (said is None or draft[base + t] == said)]
            if not hits:
                break
            at = hits[0]
            said = choice[base + at]
            mine.append(at)
        path += mine + [-1] * (r["new"] - len(mine))
        kept.append(len(mine))
        token.append(-1 if said is None else said)
        length.append(seq[b] + len(mine))
        used += _pages(length[-1]) - _pages(seq[b])
        back += table[b][_pages(length[-1]): _pages(seq[b] + r["new"])]
        base += r["new"]
    free[head + used: head + used + len(back)] = back
    return {"path": path or [-1], "kept": kept, "next": token, "seq": length, "free": free, "head": [head + used]}
