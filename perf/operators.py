"""Workloads of the calls that continue a request on the position-free page pool.

Three operators, each in a plain form (elementary torch operations) and through the package:

``tables``     block tables, page positions and slot maps from request lengths, on the GPU
``append``     new keys and values into the pages the slot map names
``attention``  a chunk of new tokens of every request over its pages (one token: decoding)

A request holds ``seq`` tokens in the pages ``block_table[b]`` lists, 16 to a page; token 16 p + r
sits at logical position ``page_pos[b][p] + r``.  A chunk brings ``new`` tokens, which take the
slots behind; the pages it starts come from a list of free pages, in request order.  Keys are
stored unrotated and rotated to their position when they are used.  ``excl`` marks slots that take
no part: cached copies of recomputed tokens, whose fresh keys and values sit in the request's own
pages behind the shared ones.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 16
DEV = "cuda"
# (query heads, kv heads, head dim) of the workloads and of the tests
SHAPES = ((8, 2, 64), (32, 8, 128), (64, 8, 128), (12, 3, 64), (24, 12, 128), (16, 2, 128), (4, 4, 64))


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step's tables: every request adds a token, few start a page
        dict(name="tables_step", op="tables", reqs=64, hq=64, hkv=8, d=128, ctx_lo=16384, ctx_hi=20480, new_lo=1,
             new_hi=1, mix=1),
        # a step of continuous batching with many requests: idle ones, decoding ones, long chunks
        dict(name="tables_chunks", op="tables", reqs=512, hq=32, hkv=8, d=128, ctx_lo=0, ctx_hi=4096, new_lo=0,
             new_hi=127, mix=2),
        # one decoding step's keys and values of one layer, 64 requests
        dict(name="append_step", op="append", reqs=64, hq=64, hkv=8, d=128, ctx_lo=1000, ctx_hi=2000, new_lo=1,
             new_hi=1, fused=0, mix=3),
        # after the fused prefill of 32 requests over shared spans: the recomputed tokens (moved to
        # the slots behind the spans) and the query tokens of each
        dict(name="append_fused", op="append", reqs=32, hq=32, hkv=8, d=128, spans=10, span_len=1024, pool=64,
             zipf=1.1, pct=15, query=64, fused=1, mix=4),
        # latency: one small request decodes
        dict(name="decode_tiny", op="attention", reqs=1, hq=8, hkv=2, d=64, ctx_lo=579, ctx_hi=579, new_lo=1,
             new_hi=1, mix=5),
        # one request of the Llama-3-8B-shaped layer decodes behind 4 k tokens
        dict(name="decode_layer", op="attention", reqs=1, hq=32, hkv=8, d=128, ctx_lo=4161, ctx_hi=4161, new_lo=1,
             new_hi=1, mix=6),
        # one long request decodes
        dict(name="decode_long", op="attention", reqs=1, hq=32, hkv=8, d=128, ctx_lo=32897, ctx_hi=32897, new_lo=1,
             new_hi=1, mix=7),
        # 64 requests of the 70B-shaped batch decode after their fused prefill over shared spans
        dict(name="decode_shared", op="attention", reqs=64, hq=64, hkv=8, d=128, spans=16, span_len=1024, pool=256,
             zipf=1.0, pct=10, query=128, new_lo=1, new_hi=1, mix=8),
        # draft tokens of ragged requests are checked
        dict(name="draft", op="attention", reqs=48, hq=32, hkv=8, d=128, ctx_lo=100, ctx_hi=9000, new_lo=1, new_hi=4,
             mix=9),
        # short chunks (a next turn's question) behind cached contexts, ragged, small heads
        dict(name="chunk_short", op="attention", reqs=9, hq=8, hkv=2, d=64, ctx_lo=0, ctx_hi=1500, new_lo=17,
             new_hi=200, mix=10),
        # continuous batching: most requests decode while some bring a chunk
        dict(name="mixed", op="attention", reqs=32, hq=32, hkv=8, d=128, ctx_lo=200, ctx_hi=8000, new_lo=1, new_hi=1,
             long=6, long_new_lo=100, long_new_hi=700, mix=11),
        # a long document's next chunk
        dict(name="chunk_long", op="attention", reqs=1, hq=32, hkv=8, d=128, ctx_lo=32768, ctx_hi=32768, new_lo=2048,
             new_hi=2048, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "attention"])
    hq, hkv, d = rng.choice(SHAPES)
    mix = rng.randrange(1 << 30)
    c = dict(op=op, hq=hq, hkv=hkv, d=d, mix=mix)
    if op == "tables":
        reqs = _log_int(rng, 1, 1024)
        hi = _log_int(rng, 1, max(1, min(2000, 40000 // reqs)))
        return dict(c, reqs=reqs, ctx_lo=0, ctx_hi=_log_int(rng, 16, 20000), new_lo=rng.choice([0, 1]), new_hi=hi)
    if op == "append":
        if rng.random() < 0.4:
            return dict(c, reqs=_log_int(rng, 1, 16), spans=rng.randint(1, 8), span_len=16 * rng.randint(1, 48),
                        pool=16, zipf=1.1, pct=rng.choice([5, 10, 15, 20, 30]), query=rng.randint(1, 128), fused=1)
        reqs = _log_int(rng, 1, 256)
        return dict(c, reqs=reqs, ctx_lo=0, ctx_hi=_log_int(rng, 16, 2000), new_lo=rng.choice([0, 1]),
                    new_hi=_log_int(rng, 1, 128), fused=0)
    kind = rng.choice(["decode", "shared", "draft", "chunk", "mixed"])
    room = 500000 // hkv                       # tokens of context of the whole batch
    if kind == "shared":
        reqs = _log_int(rng, 1, 32)
        spans = rng.randint(1, 12)
        return dict(c, reqs=reqs, spans=spans, span_len=16 * max(1, min(64, room // (reqs * spans * 16))),
                    pool=rng.choice([16, 32, 64]), zipf=rng.choice([1.0, 1.1]), pct=rng.choice([5, 10, 15, 30]),
                    query=rng.randint(1, 128), new_lo=1, new_hi=1)
    if kind == "chunk":
        reqs = _log_int(rng, 1, 12)
        hi = _log_int(rng, 20, 1000)
        return dict(c, reqs=reqs, ctx_lo=0, ctx_hi=_log_int(rng, 16, max(17, min(16000, room // reqs))),
                    new_lo=hi // 5 + 1, new_hi=hi)
    reqs = _log_int(rng, 1, 128)
    c = dict(c, reqs=reqs, ctx_lo=1, ctx_hi=_log_int(rng, 16, max(17, min(33000, 2 * room // reqs))))
    if kind == "mixed":
        return dict(c, new_lo=0, new_hi=1, long=rng.randint(1, min(6, reqs)), long_new_lo=10, long_new_hi=400)
    return dict(c, new_lo=1, new_hi=1 if kind == "decode" else 4)


def _shape(case):
    """Lengths and pages of a case, from its own numbers: per request the tokens held, the new
    tokens, the shared spans drawn (first page, pages), the recomputed tokens, the first position."""
    rng = random.Random(case["mix"])
    reqs = []
    if "spans" in case:
        sp = case["span_len"] // PAGE
        weights = [(r + 1.0) ** -case["zipf"] for r in range(case["pool"])]
        k = -(-case["pct"] * case["span_len"] // 100)
        for _ in range(case["reqs"]):
            w, ids = list(weights), []
            for _ in range(case["spans"]):
                i = rng.choices(range(case["pool"]), w)[0]
                w[i] = 0.0
                ids.append(i)
            cached, n_sel = case["spans"] * case["span_len"], case["spans"] * k
            rows = n_sel + case["query"]
            if case["op"] == "append":
                seq, new = cached, rows
            else:
                seq, new = cached + rows, rng.randint(case["new_lo"], case["new_hi"])
            reqs.append(dict(seq=seq, new=new, shared=[(i * sp, sp) for i in ids], n_sel=n_sel, k=k, cached=cached,
                             pos0=rng.randrange(4096)))
        return reqs
    n_long = case.get("long", 0)
    longs = set(rng.sample(range(case["reqs"]), n_long))
    for b in range(case["reqs"]):
        many = "long_new" if b in longs else "new"
        new = rng.randint(case[many + "_lo"], case[many + "_hi"])
        reqs.append(dict(seq=rng.randint(case["ctx_lo"], case["ctx_hi"]), new=new, shared=[], n_sel=0, k=0, cached=0,
                         pos0=rng.randrange(4096)))
    return reqs


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    reqs = _shape(case)
    n = len(reqs)
    rows = sum(r["new"] for r in reqs)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "tables":
        taken = sum(_pages(r["seq"] + r["new"]) - _pages(r["seq"]) for r in reqs)
        # lengths, last page's position and the pages taken in; table entries, slots, positions, offsets out
        return {"bytes": 4 * (2 * n + n + taken + 2 * taken + 2 * rows + 2 * n + 1), "flops": 0}
    if case["op"] == "append":
        moved = sum(r["n_sel"] for r in reqs)
        return {"bytes": rows * (4 * hkv * d * 2 + 8), "flops": moved * hkv * d * 3}
    slots = set()
    kept = 0
    keys = 0
    for r in reqs:
        shared = r["shared"]
        private = r["seq"] + r["new"] - r["cached"]
        for first, m in shared:
            slots.update(range(first, first + m))
        kept += private
        ctx = r["seq"] - r["n_sel"]
        keys += r["new"] * ctx + r["new"] * (r["new"] + 1) // 2
    tokens = kept + PAGE * len(slots)
    return {"bytes": tokens * hkv * d * 4 + rows * hq * d * 4, "flops": keys * hq * d * 4}


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    reqs = _shape(case)
    n, hq, hkv, d = len(reqs), case["hq"], case["hkv"], case["d"]
    host = random.Random(seed * 1000003 + case["mix"])
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    rows = sum(r["new"] for r in reqs)
    max_pages = max(1, max(_pages(r["seq"] + r["new"]) for r in reqs))
    shared_pages = case["pool"] * case["span_len"] // PAGE if "spans" in case else 0
    private = sum(_pages(r["seq"]) - r["cached"] // PAGE for r in reqs)
    taken = sum(_pages(r["seq"] + r["new"]) - _pages(r["seq"]) for r in reqs)
    n_phys = shared_pages + private + taken + 7
    order = list(range(shared_pages, n_phys))
    host.shuffle(order)
    table = torch.zeros((n, max_pages), dtype=torch.int32)
    page_pos = torch.zeros((n, max_pages), dtype=torch.int32)
    next_pos = torch.zeros(n, dtype=torch.int32)
    at, top = 0, 0
    for b, r in enumerate(reqs):
        pages = [p for first, m in r["shared"] for p in range(first, first + m)]
        own_pages = _pages(r["seq"]) - len(pages)
        pages += order[at: at + own_pages]
        at += own_pages
        pos = torch.arange(len(pages), dtype=torch.int32) * PAGE + r["pos0"]
        # behind the shared spans: the recomputed tokens' slots, then the query at its own positions
        pos[r["cached"] // PAGE:] -= r["n_sel"]
        table[b, : len(pages)] = torch.tensor(pages, dtype=torch.int32)
        page_pos[b, : len(pages)] = pos
        next_pos[b] = r["pos0"] + r["seq"] - r["n_sel"]
        top = max(top, r["pos0"] + r["seq"] + r["new"])
    free = torch.tensor(order[at:] + [0] * 9, dtype=torch.int32)       # the list's end is never reached
    s = dict(case=case, reqs=reqs, n=n, rows=rows, max_pages=max_pages, n_phys=n_phys,
             theta=1e4 if d == 64 else 5e5, max_pos=top + 2 * PAGE,
             seq=torch.tensor([r["seq"] for r in reqs], dtype=torch.int32).to(DEV),
             new=torch.tensor([r["new"] for r in reqs], dtype=torch.int32).to(DEV),
             table=table.to(DEV), page_pos=page_pos.to(DEV), next_pos=next_pos.to(DEV), free=free.to(DEV),
             free_head=torch.zeros(1, dtype=torch.int32, device=DEV))
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    op = case["op"]
    if op != "tables":
        # whole pools of standard normal draws, slots behind a sequence's end included: stale values
        s["k_pool"] = torch.empty((n_phys, hkv, PAGE, d), dtype=torch.bfloat16, device=DEV)
        s["v_pool"] = torch.empty_like(s["k_pool"])
        for t in (s["k_pool"], s["v_pool"]):
            for i in range(0, n_phys, 4096):
                t[i: i + 4096].copy_(torch.randn(t[i: i + 4096].shape, generator=gen, device=DEV))
    if op == "append":
        # rows of one product's output, queries first: keys and values are columns of it
        s["qkv"] = normal(max(1, rows), (hq + 2 * hkv) * d).view(max(1, rows), hq + 2 * hkv, d)
        s["k_new"], s["v_new"] = s["qkv"][:, hq: hq + hkv], s["qkv"][:, hq + hkv:]
        s["move"] = None
        if case["fused"]:
            pos = []
            for r in reqs:
                for i in range(len(r["shared"])):
                    span = case["span_len"]
                    pos += [r["pos0"] + i * span + j for j in sorted(host.sample(range(span), r["k"]))]
                pos += range(r["pos0"] + r["cached"], r["pos0"] + r["cached"] + case["query"])
            s["move"] = torch.tensor(pos, dtype=torch.int32).to(DEV)
    excl = None
    if op == "attention":
        s["q"] = normal(max(1, rows), hq, d)
        if "spans" in case:
            bits = torch.zeros((n, max_pages, PAGE), dtype=torch.int32)
            for b, r in enumerate(reqs):
                flat = bits[b].view(-1)
                for i in range(len(r["shared"])):
                    flat[torch.tensor(host.sample(range(case["span_len"]), r["k"]), dtype=torch.int64)
                         + i * case["span_len"]] = 1
            words = (bits << torch.arange(PAGE, dtype=torch.int32)).sum(-1)
            excl = torch.where(words >= 32768, words - 65536, words).to(torch.int16).to(DEV)
        s["excl"] = excl
    # what a program keeps from call to call
    if own:
        import position_independent_kv_critical_gb300 as pcf
        max_chunk = max(1, max(r["new"] for r in reqs))
        L = pcf.ChunkLayout(n, hq, hkv, d, n_phys, s["max_pos"], max_pages=max_pages, max_rows=max(1, rows),
                            max_chunk=max_chunk)
        L.block_table.copy_(s["table"])
        L.page_pos.copy_(s["page_pos"])
        s["pcf"], s["L"] = pcf, L
        s["seq_out"] = torch.zeros_like(s["seq"])
        s["head_out"] = torch.zeros_like(s["free_head"])
        if op != "tables":
            _own_tables(s)
            s["rope"] = pcf.rope_table(d, s["theta"], s["max_pos"]).to(DEV)
        if op == "attention":
            s["out"] = torch.zeros((max(1, rows), hq, d), dtype=torch.bfloat16, device=DEV)
            s["ws"] = torch.empty(max(16, L.attention_workspace_bytes()), dtype=torch.uint8, device=DEV)
    if op != "tables":
        t = _plain_tables(s)
        s["slot_map"], s["row_pos"], s["table_all"], s["pos_all"] = (t["slot_map"], t["row_pos"], t["block_table"],
                                                                     t["page_pos"])
    return s


# ------------------------------------------------------------------------------------ passes
def run(state):
    op = state["case"]["op"]
    if own:
        L, pcf = state["L"], state["pcf"]
        if op == "tables":
            return _own_tables(state)
        if op == "append":
            pcf.append_kv(L, state["k_new"], state["v_new"], state["k_pool"], state["v_pool"], rope=state["rope"],
                          row_pos=state["move"])
            return {"k_pool": state["k_pool"], "v_pool": state["v_pool"]}
        pcf.chunk_attention(L, state["q"], state["k_pool"], state["v_pool"], state["rope"], state["out"], state["ws"],
                            excl=state["excl"])
        return {"out": state["out"]}
    if op == "tables":
        return _plain_tables(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state)


def _own_tables(s):
    L = s["L"]
    s["pcf"].chunk_tables(L, s["seq"], s["new"], s["free"], s["free_head"], s["seq_out"], s["head_out"],
                          next_pos=s["next_pos"])
    return {"block_table": L.block_table, "page_pos": L.page_pos, "slot_map": L.slot_map, "row_pos": L.row_pos,
            "row_base": L.row_base, "seq": s["seq_out"], "free_head": s["head_out"]}


def _plain_tables(s):
    rows, max_pages = max(1, s["rows"]), s["max_pages"]
    seq, new = s["seq"], s["new"]
    before = (seq + PAGE - 1) // PAGE
    after = (seq + new + PAGE - 1) // PAGE
    ends = torch.cumsum(after - before, 0)
    p = torch.arange(max_pages, device=DEV, dtype=torch.int32)[None]
    fresh = (p >= before[:, None]) & (p < after[:, None])
    rank = s["free_head"].long() + (ends - (after - before))[:, None] + p - before[:, None]
    table = torch.where(fresh, s["free"][rank.clamp(0, s["free"].numel() - 1)], s["table"])
    start = s["next_pos"]
    page_pos = torch.where(fresh, start[:, None] + p * PAGE - seq[:, None], s["page_pos"])
    row_base = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)])
    i = torch.arange(rows, device=DEV)
    live = i < row_base[-1]
    b = torch.searchsorted(row_base[1:], i, right=True).clamp(max=s["n"] - 1)
    t = i - row_base[b]
    slot = seq[b] + t
    page = table[b, (slot // PAGE).clamp(0, max_pages - 1)].long()
    slot_map = torch.where(live, page * PAGE + slot % PAGE, -1)
    row_pos = torch.where(live, start[b] + t, -1)
    return {"block_table": table, "page_pos": page_pos.to(torch.int32), "slot_map": slot_map.to(torch.int32),
            "row_pos": row_pos.to(torch.int32), "row_base": row_base.to(torch.int32), "seq": seq + new,
            "free_head": (s["free_head"] + ends[-1]).to(torch.int32)}


def _angles(pos, d, theta):
    """cos and sin of every position and frequency: 64-bit angles, 32-bit results."""
    inv = theta ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
    a = pos.to(torch.float64)[:, None] * inv[None]
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin):
    """x [tokens, heads, d] (32 bits): dimension i turns with i + d/2."""
    h = x.shape[-1] // 2
    lo, hi, c, s = x[..., :h], x[..., h:], cos[:, None], sin[:, None]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)


def _plain_append(s):
    if s["rows"] == 0:
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    slot = s["slot_map"].long()
    page, r = slot // PAGE, slot % PAGE
    k = s["k_new"]
    if s["move"] is not None:
        cos, sin = _angles(s["move"] - s["row_pos"], s["case"]["d"], s["theta"])
        k = _rotate(k.float(), cos, sin).to(torch.bfloat16)
    s["k_pool"][page, :, r] = k
    s["v_pool"][page, :, r] = s["v_new"]
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.zeros((max(1, s["rows"]), hq, d), dtype=torch.bfloat16, device=DEV)
    sixteen = torch.arange(PAGE, device=DEV, dtype=torch.int32)
    base = 0
    for b, r in enumerate(s["reqs"]):
        T, n = r["new"], r["seq"] + r["new"]
        if T == 0:
            continue
        np_ = _pages(n)
        pages = s["table_all"][b, :np_].long()
        pos = (s["pos_all"][b, :np_, None] + sixteen).reshape(-1)[:n]
        cos, sin = _angles(pos, d, s["theta"])
        k = _rotate(s["k_pool"][pages].transpose(1, 2).reshape(-1, hkv, d)[:n].float(), cos, sin)
        v = s["v_pool"][pages].transpose(1, 2).reshape(-1, hkv, d)[:n].float()
        cos, sin = _angles(s["row_pos"][base: base + T], d, s["theta"])
        q = _rotate(s["q"][base: base + T].float(), cos, sin)
        j = torch.arange(n, device=DEV)
        seen = j[None] <= r["seq"] + torch.arange(T, device=DEV)[:, None]
        if s["excl"] is not None:
            gone = ((s["excl"][b, :np_, None].int() >> sixteen) & 1).reshape(-1)[:n]
            seen = seen & (gone == 0)[None]
        step = max(1, (1 << 28) // (T * g * n))               # kv heads at a time
        for h in range(0, hkv, step):
            e = min(hkv, h + step)
            kh, vh = k[:, h:e].transpose(0, 1), v[:, h:e].transpose(0, 1)            # [heads, n, d]
            qh = q[:, h * g: e * g].reshape(T, e - h, g, d).permute(1, 2, 0, 3).reshape(e - h, g * T, d)
            w = torch.matmul(qh, kh.transpose(1, 2)) / math.sqrt(d)
            w = w.view(e - h, g, T, n).masked_fill_(~seen, -math.inf)
            top = w.amax(-1, keepdim=True)
            w = torch.exp_(w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)))
            total = w.sum(-1, keepdim=True)
            o = torch.matmul(w.view(e - h, g * T, n), vh).view(e - h, g, T, d)
            o = o / torch.where(total == 0, torch.ones_like(total), total)
            out[base: base + T, h * g: e * g] = o.permute(2, 0, 1, 3).reshape(T, (e - h) * g, d).to(torch.bfloat16)
        base += T
    return {"out": out}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    keep = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    op, reqs, d, hkv, hq = case["op"], s["reqs"], case["d"], case["hkv"], case["hq"]
    if op == "tables":
        return _exact_tables(s)
    if op == "attention" and work(case)["flops"] > 4e12:
        return None
    freq = torch.tensor([s["theta"] ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device=DEV)

    def turned(x, pos):
        """x [tokens, heads, d] in 64 bits as d/2 complex numbers, turned by position x frequency."""
        z = torch.complex(x[..., : d // 2].double(), x[..., d // 2:].double())
        a = pos.double()[:, None] * freq
        return z * torch.polar(torch.ones_like(a), a)[:, None]

    t = _exact_tables(s)
    slots, where = t["slot_map"].long(), t["row_pos"]
    if op == "append":
        k, v = s["k_pool"].double(), s["v_pool"].double()
        if s["rows"]:
            new = s["k_new"].double()
            if s["move"] is not None:
                z = turned(s["k_new"], s["move"] - where)
                new = torch.cat([z.real, z.imag], -1)
            flat = lambda x: x.permute(0, 2, 1, 3).reshape(-1, hkv, d)
            kf, vf = flat(k), flat(v)
            kf[slots], vf[slots] = new, s["v_new"].double()
            back = lambda x: x.view(s["n_phys"], PAGE, hkv, d).permute(0, 2, 1, 3)
            k, v = back(kf), back(vf)
        return {"k_pool": k, "v_pool": v}
    out = torch.zeros((max(1, s["rows"]), hq, d), dtype=torch.float64, device=DEV)
    g, base = hq // hkv, 0
    for b, r in enumerate(reqs):
        T, n = r["new"], r["seq"] + r["new"]
        if T == 0:
            continue
        j = torch.arange(n, device=DEV)
        page = t["block_table"][b].long()[j // PAGE]
        pos = t["page_pos"][b].long()[j // PAGE] + j % PAGE
        hidden = torch.zeros(n, dtype=torch.bool, device=DEV)
        if s["excl"] is not None:
            hidden = ((s["excl"][b].long()[j // PAGE] & 65535) >> (j % PAGE)) % 2 == 1
        for h in range(hkv):
            zk = turned(s["k_pool"][page, h, j % PAGE][:, None], pos)[:, 0]
            v = s["v_pool"][page, h, j % PAGE].double()
            for first in range(0, T, 256):
                m = min(256, T - first)
                some = slice(base + first, base + first + m)
                zq = turned(s["q"][some, h * g: (h + 1) * g], where[some])
                score = (torch.einsum("tgi,ji->tgj", zq.real, zk.real) + torch.einsum("tgi,ji->tgj", zq.imag, zk.imag))
                score = score * d ** -0.5
                late = j[None] > r["seq"] + first + torch.arange(m, device=DEV)[:, None]
                score = score.masked_fill((late | hidden)[:, None], -math.inf)
                top = score.amax(-1)
                lse = torch.logsumexp(score, -1)
                p = torch.exp(score - lse[..., None])
                p = torch.where((top == -math.inf)[..., None], torch.zeros_like(p), p)
                out[some, h * g: (h + 1) * g] = torch.einsum("tgj,jd->tgd", p, v)
        base += T
    return {"out": out}


def _exact_tables(s):
    """The tables from the lists themselves, request by request on the host."""
    seq, new, free = s["seq"].tolist(), s["new"].tolist(), s["free"].tolist()
    table, pos, start = s["table"].cpu().clone(), s["page_pos"].cpu().clone(), s["next_pos"].tolist()
    head = int(s["free_head"].item())
    slot_map, row_pos, row_base = [], [], [0]
    for b in range(s["n"]):
        ids, at = table[b].tolist(), pos[b].tolist()
        for i in range(new[b]):
            slot = seq[b] + i
            if slot % PAGE == 0:
                ids[slot // PAGE], at[slot // PAGE] = free[head], start[b] + i
                head += 1
            slot_map.append(ids[slot // PAGE] * PAGE + slot % PAGE)
            row_pos.append(start[b] + i)
        table[b], pos[b] = torch.tensor(ids, dtype=torch.int32), torch.tensor(at, dtype=torch.int32)
        row_base.append(len(slot_map))
    if not slot_map:
        slot_map, row_pos = [-1], [-1]
    whole = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)
    return {"block_table": table.to(DEV), "page_pos": pos.to(DEV), "slot_map": whole(slot_map),
            "row_pos": whole(row_pos), "row_base": whole(row_base), "seq": whole([a + c for a, c in zip(seq, new)]),
            "free_head": whole([head])}
