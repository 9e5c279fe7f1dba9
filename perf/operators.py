"""The serving operators on a quantised history cache: cases, inputs, plain forms and exact values.

Five operators share one paged cache of keys and values in MXFP8 (E4M3 elements, one power-of-two
scale for 32 of them along head_dim): writing rows into it, reading rows back, averaging the keys of
each full page, selecting pages for a query by their mean key, and attention of new queries (single
tokens, chunks, trees of drafted tokens, candidates) over it.

A case is a dict of plain values:
  op         write, read, summarize, select or attend
  batch      sequences; kv_heads, group: heads = kv_heads * group query heads; head_dim; page: slots a page
  len_lo/hi  cached slots of a sequence before the call, uniform
  rows_lo/hi rows a sequence brings (write, read: rows moved; select, attend: queries), uniform
  block, window  the block rule; topk: pages selected for a query (0: none)
  shape      chain (rows follow one another), tree (each drafted row has one parent), candidates
             (rows that see the history and themselves)
  dtype      of the dense rows (bf16 or f32)
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BASE = dict(batch=1, kv_heads=8, group=1, head_dim=128, page=64, len_lo=0, len_hi=0, rows_lo=1, rows_hi=1, block=256,
             window=2, topk=0, shape="chain", dtype="bf16")


def _case(name, op, **kw):
    return dict(_BASE, name=name, op=op, **kw)


def listed():
    return [
        # serving: one new event for each of 256 histories of 64 to 4096 events
        _case("write_event", "write", batch=256, len_lo=64, len_hi=4096),
        # filling the cache with whole jagged histories
        _case("write_histories", "write", batch=256, rows_lo=64, rows_hi=4096),
        # a window of each history back as dense rows, for a dense kernel or another cache
        _case("read_window", "read", batch=256, len_lo=64, len_hi=4096, rows_lo=1, rows_hi=512),
        # whole short histories back in float32, head_dim 64
        _case("read_f32", "read", batch=64, kv_heads=4, head_dim=64, page=16, len_lo=1024, len_hi=1024, rows_lo=1,
              rows_hi=1024, dtype="f32"),
        # the page that each history has just filled
        _case("summarize_step", "summarize", batch=256, len_lo=64, len_hi=4096, rows_lo=64, rows_hi=64),
        # all pages of long histories
        _case("summarize_long", "summarize", batch=8, len_lo=32768, len_hi=32768, rows_lo=32768, rows_hi=32768),
        # one event looks for its pages, short histories in small pages
        _case("select_event", "select", batch=64, kv_heads=4, head_dim=64, page=16, len_lo=1, len_hi=1024, block=128,
              window=1, topk=8),
        # trees of drafted events over long histories
        _case("select_tree", "select", batch=8, len_lo=16384, len_hi=32768, rows_lo=17, rows_hi=64, block=512,
              window=1, topk=32, shape="tree"),
        # one event for each of 256 histories under the block rule
        _case("event_window", "attend", batch=256, len_lo=64, len_hi=4096),
        # one event over the whole of long histories, four query heads for a key/value head
        _case("event_long", "attend", batch=16, group=4, len_lo=24576, len_hi=32767, block=512, window=65),
        # trees of drafted events under the block rule, ragged
        _case("tree_window", "attend", batch=64, page=32, len_lo=64, len_hi=32768, rows_lo=5, rows_hi=64, block=512,
              window=4, shape="tree"),
        # candidates scored against their own block and selected pages of long histories
        _case("candidates_selected", "attend", batch=16, group=2, len_lo=16384, len_hi=32768, rows_lo=33, rows_hi=64,
              block=512, window=1, topk=32, shape="candidates"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(["write", "read", "summarize", "select", "attend", "attend", "attend"])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = spread(1, 8)
    batch = spread(1, 256)
    cap = max(256, min(32768, (1 << 28) // (batch * kv_heads * head_dim)))
    page = rng.choice([16, 32, 64, 128])
    len_hi = spread({"summarize": page, "select": 2 * page}.get(op, 1), cap)
    least = {"read": 1, "summarize": page}.get(op, 0)
    len_lo = rng.choice([least, len_hi, rng.randint(least, len_hi)])
    c = dict(_BASE, op=op, batch=batch, kv_heads=kv_heads, head_dim=head_dim, page=page,
             len_lo=len_lo, len_hi=len_hi, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("write", "read"):
        c["rows_hi"] = spread(1, cap)
        c["rows_lo"] = rng.choice([1, rng.randint(1, c["rows_hi"])])
    elif op == "summarize":
        c["rows_lo"] = c["rows_hi"] = rng.choice([page, len_hi])
        c["dtype"] = "bf16"
    else:
        c["dtype"] = "bf16"
        c["group"] = rng.choice([1, 1, 2, 3, 4, 8])
        c["shape"] = rng.choice(["chain", "tree", "candidates"])
        c["rows_hi"] = rng.choice([1, spread(1, 64)])
        if op == "attend" and c["shape"] == "chain" and rng.random() < 0.3:
            c["rows_hi"] = spread(64, 512)  # a chunk of a prompt
            c["batch"] = min(batch, 16)
        c["block"] = rng.choice([1, 64, 128, 256, 512, spread(1, 600)])
        c["window"] = spread(1, 64)
        c["topk"] = rng.choice([0, 0, spread(1, 64)])
        if op == "select":
            c["block"], c["topk"] = min(c["block"], len_hi // 2), spread(1, 64)
            c["window"] = spread(1, max(1, len_hi // (2 * c["block"])))
        pairs = c["batch"] * kv_heads * c["group"] * (len_hi + c["rows_hi"])
        c["rows_hi"] = max(1, min(c["rows_hi"], (1 << 25) // pairs))
        c["rows_lo"] = rng.randint(1, c["rows_hi"])
    return c


# ----------------------------------------------------------------- inputs ---

def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, dtype=torch.int64)


def _offsets(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)])


def _random_pages(gd, shape):
    """Element codes (E4M3) and scale codes (E8M0) of quantised normal rows, for a pool of `shape`."""
    pages, kh, s, d = shape
    el = torch.empty(shape, dtype=torch.uint8, device=DEV)
    sc = torch.empty((pages, kh, s, d // 32), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (kh * s * d))
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i), kh, s, d), generator=gd, device=DEV)
        a, b = _quantize(x)
        el[i:i + step], sc[i:i + step] = a.view(torch.uint8), b
    return el, sc


def _tree(c, g, n, n_max):
    """Parents of drafted rows as visibility [batch, n_max, n_max] and each row's depth, on the CPU."""
    B = c["batch"]
    if c["shape"] == "candidates":
        return torch.eye(n_max, dtype=torch.bool).expand(B, -1, -1).clone(), torch.zeros(B, n_max, dtype=torch.int64)
    sees = torch.zeros(B, n_max, n_max, dtype=torch.bool)
    depth = torch.zeros(B, n_max, dtype=torch.int64)
    at = torch.arange(B)
    for j in range(n_max):
        parent = (j - 1 - torch.randint(0, 4, (B,), generator=g)).clamp(min=-1)
        has = parent >= 0
        p = parent.clamp(min=0)
        sees[:, j] = sees[at, p] & has[:, None]
        sees[:, j, j] = True
        depth[:, j] = torch.where(has, depth[at, p] + 1, torch.zeros_like(p))
    return sees, depth


def _words(bits):
    """Truth values [..., n] as int32 words [..., ceil(n / 32)], bit j of word w for value 32 w + j."""
    n = bits.shape[-1]
    pad = torch.nn.functional.pad(bits, (0, -n % 32)).unflatten(-1, (-1, 32)).to(torch.int64)
    w = (pad << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    c = dict(_BASE, **case)
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)
    B, KH, G, D, S, op = c["batch"], c["kv_heads"], c["group"], c["head_dim"], c["page"], c["op"]
    # the batch's lengths are the case's; which sequence has which comes from the seed
    sizes = torch.Generator().manual_seed(17)
    lens = _ints(sizes, c["len_lo"], c["len_hi"], B)
    n = _ints(sizes, c["rows_lo"], c["rows_hi"], B)
    shuffle = torch.randperm(B, generator=g)
    lens, n = lens[shuffle], n[shuffle]
    if op == "read":  # the last rows of each history
        n = torch.minimum(n, lens)
    if op == "summarize":  # the slots from `starts` on have just been written
        n = torch.minimum(n, lens)
    starts = lens - n if op in ("read", "summarize") else lens
    ends = torch.maximum(lens, starts + n)
    n_max, max_slots = max(1, int(n.max())), max(1, int(ends.max()))
    max_pages = -(-max_slots // S)
    need = -(-ends // S)
    pages = int(need.sum()) + 1
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, max_pages), -1, dtype=torch.int64)
    live = torch.arange(max_pages)[None] < need[:, None]
    table[live] = order[:int(need.sum())]
    offs = _offsets(n)
    rows = int(offs[-1])
    i32 = lambda t: t.to(torch.int32).to(DEV)  # noqa: E731
    s = dict(case=c, rows=rows, n_max=n_max, max_slots=max_slots, max_pages=max_pages, pages=pages, table=i32(table),
             offs=i32(offs), starts=i32(starts), ends=i32(ends), lens=i32(lens),
             seq=torch.repeat_interleave(torch.arange(B), n).to(DEV))
    shape = (pages, KH, S, D)
    s["touched"] = int((need - starts // S).max())
    if op == "write":
        s["k_pages"], s["v_pages"] = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in "kv")
        s["k_scales"], s["v_scales"] = (torch.zeros(shape[:3] + (D // 32,), dtype=torch.uint8, device=DEV) for _ in "kv")
        s["k"], s["v"] = (torch.randn((rows, KH, D), generator=gd, device=DEV).to(_DT[c["dtype"]]) for _ in "kv")
    elif op == "select":  # reads the summaries and the page table alone
        s["k_pages"], s["v_pages"] = (torch.empty(shape, dtype=torch.uint8, device=DEV) for _ in "kv")
        s["k_scales"], s["v_scales"] = (torch.empty(shape[:3] + (D // 32,), dtype=torch.uint8, device=DEV) for _ in "kv")
    else:
        s["k_pages"], s["k_scales"] = _random_pages(gd, shape)
        s["v_pages"], s["v_scales"] = _random_pages(gd, shape)
    if op in ("select", "attend"):
        # queries of one sequence share its context: a common part and their own
        q = torch.randn((B, KH * G, D), generator=gd, device=DEV)[s["seq"]]
        q = q + torch.randn((rows, KH * G, D), generator=gd, device=DEV)
        s["q"] = (q * 0.7).to(torch.bfloat16)
        t = torch.arange(rows) - torch.repeat_interleave(offs[:-1], n)
        bseq = torch.repeat_interleave(torch.arange(B), n)
        if c["shape"] == "chain":
            s["tree"], s["positions"] = None, None
            pos = lens[bseq] + t
        else:
            sees, depth = _tree(c, g, n, n_max)
            s["tree"] = _words(sees[bseq, t]).to(DEV)
            pos = lens[bseq] + depth[bseq, t]
            s["positions"] = i32(pos)
        s["row"] = t.to(DEV)
        s["pos"] = pos.to(DEV)
        low = _window_start(lens, c)  # no row of the sequence sees an earlier cached slot by the rule
        s["low"], s["reach"] = low.to(DEV), max(1, int((ends - low).max()))
    if op == "select":
        s["summaries"] = torch.randn((pages, KH, D), generator=gd, device=DEV) / math.sqrt(S)
    s["mask"] = None
    if op == "attend" and c["topk"]:
        # each query picks topk of a sequence's pool of 1.5 topk pages, head by head
        k = min(c["topk"], max_pages)
        pool = min(max_pages, k + (k + 1) // 2)
        score = torch.rand((B, KH, max_pages), generator=gd, device=DEV)
        score.masked_fill_(torch.arange(max_pages, device=DEV)[None, None] >= (s["lens"] // S)[:, None, None], -1.0)
        best = score.topk(pool, dim=-1)[1]
        mine = torch.rand((rows, KH, pool), generator=gd, device=DEV).topk(k, dim=-1)[1]
        chosen = best[s["seq"]].gather(-1, mine)
        bits = torch.zeros((rows, KH, max_pages), dtype=torch.bool, device=DEV)
        s["mask"] = _words(bits.scatter_(-1, chosen, True))
    # buffers that a serving program keeps for the results
    if op == "read":
        s["k"], s["v"] = (torch.empty((rows, KH, D), dtype=_DT[c["dtype"]], device=DEV) for _ in "kv")
    elif op == "summarize":
        s["out"] = torch.zeros((pages, KH, D), device=DEV)
    elif op == "select":
        s["out"] = torch.empty((rows, KH, -(-max_pages // 32)), dtype=torch.int32, device=DEV)
    elif op == "attend":
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((KH * G, rows), device=DEV)
    if own:
        s["own"] = _own_state(s)
    return s


# ------------------------------------------------------------ plain forms ---

def _window_start(pos, c):
    """First position that the block rule shows to a query at `pos`."""
    first = torch.div(pos, c["block"], rounding_mode="floor") - (c["window"] - 1)
    return first.clamp(min=0) * c["block"]


def _quantize(x):
    """MXFP8 along the last axis: (E4M3 values in x's shape, E8M0 codes)."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, torch.full_like(amax, -8, dtype=torch.int32)).clamp(-127, 127)
    v = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return v.flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def _dequantize(el, sc):
    v = el.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return torch.ldexp(v, sc.to(torch.int32).unsqueeze(-1) - 127).flatten(-2)


def _slots(s, seq, slot):
    """Page and row within it of slots (any shape, with their sequences); where a slot has no page, page 0."""
    S = s["case"]["page"]
    page = s["table"][seq, (slot // S).clamp(0, s["max_pages"] - 1)].long()
    return page.clamp(min=0), slot % S


def _row_slots(s):
    first = s["offs"][:-1].long()[s["seq"]]
    slot = s["starts"].long()[s["seq"]] + torch.arange(s["rows"], device=DEV) - first
    return _slots(s, s["seq"], slot)


def _plain_write(s):
    page, at = _row_slots(s)
    for x, el, sc in ((s["k"], s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
        a, b = _quantize(x)
        el[page, :, at] = a.view(torch.uint8)
        sc[page, :, at] = b


def _plain_read(s):
    page, at = _row_slots(s)
    dt = _DT[s["case"]["dtype"]]
    return [_dequantize(el[page, :, at], sc[page, :, at]).to(dt)
            for el, sc in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"]))]


def _plain_summarize(s):
    c = s["case"]
    S = c["page"]
    at = (s["starts"].long() // S)[:, None] + torch.arange(s["touched"], device=DEV)
    full = (at + 1) * S <= s["ends"].long()[:, None]
    out = torch.zeros((s["pages"] + 1, c["kv_heads"], c["head_dim"]), device=DEV)
    page = s["table"].long().gather(1, at.clamp(max=s["max_pages"] - 1))
    page = torch.where(full, page, torch.full_like(at, -1)).flatten()
    mean = _dequantize(s["k_pages"][page.clamp(min=0)], s["k_scales"][page.clamp(min=0)]).mean(2)
    out[torch.where(page >= 0, page, torch.full_like(page, s["pages"]))] = mean
    return out[:-1]


def _plain_select(s):
    c = s["case"]
    S, k, P = c["page"], min(c["topk"], s["max_pages"]), s["max_pages"]
    q = s["q"].double().unflatten(1, (c["kv_heads"], c["group"])).sum(2)
    mean = s["summaries"][s["table"].long().clamp(min=0)].double()  # [batch, pages, kv_heads, D]
    qp = torch.zeros((c["batch"], s["n_max"], c["kv_heads"], c["head_dim"]), dtype=torch.float64, device=DEV)
    qp[s["seq"], s["row"]] = q
    score = torch.matmul(qp.transpose(1, 2), mean.permute(0, 2, 3, 1)).transpose(1, 2)[s["seq"], s["row"]]
    at = torch.arange(P, device=DEV)
    ok = (at * S < _window_start(s["pos"], c)[:, None]) & ((at + 1) * S <= s["lens"].long()[s["seq"]][:, None])
    score = torch.where(ok[:, None], score, torch.full_like(score, -math.inf))
    best = score.sort(dim=-1, descending=True, stable=True)[1][..., :k]
    bits = torch.zeros(score.shape, dtype=torch.bool, device=DEV).scatter_(-1, best, True) & ok[:, None]
    return _words(bits)


def _plain_attend(s):
    c = s["case"]
    B, KH, G, D, S, n = c["batch"], c["kv_heads"], c["group"], c["head_dim"], c["page"], s["n_max"]
    lens = s["lens"].long()
    if s["mask"] is None:
        slot = s["low"][:, None] + torch.arange(s["reach"], device=DEV)
    else:
        slot = torch.arange(s["max_slots"], device=DEV).expand(B, -1)
    R = slot.shape[1]
    page, at = _slots(s, torch.arange(B, device=DEV)[:, None], slot)
    k = _dequantize(s["k_pages"][page, :, at], s["k_scales"][page, :, at])  # [B, R, KH, D]
    v = _dequantize(s["v_pages"][page, :, at], s["v_scales"][page, :, at])
    seq, row = s["seq"], s["row"]
    q = torch.zeros((B, n, KH, G, D), device=DEV)
    q[seq, row] = s["q"].float().unflatten(1, (KH, G))
    pos = torch.full((B, n), -1, dtype=torch.int64, device=DEV)
    pos[seq, row] = s["pos"]
    low = _window_start(pos, c)
    draft = slot - lens[:, None]                                            # the drafted row in a slot
    kpos = torch.where(draft < 0, slot, pos.gather(1, draft.clamp(0, n - 1)))
    rule = (kpos[:, None] <= pos[..., None]) & (kpos[:, None] >= low[..., None])    # [B, n, R]
    if s["tree"] is None:
        edge = draft[:, None] <= torch.arange(n, device=DEV)[None, :, None]
    else:
        words = torch.zeros((B, n, s["tree"].shape[-1]), dtype=torch.int64, device=DEV)
        words[seq, row] = s["tree"].long()
        d = draft.clamp(0, n - 1)[:, None].expand(B, n, R)
        edge = (words.gather(2, d // 32) >> (d % 32)) & 1 > 0
    there = draft < s["offs"].diff().long()[:, None]
    sees = (rule & ((draft < 0)[:, None] | edge) & there[:, None])[:, :, None].expand(B, n, KH, R)
    if s["mask"] is not None:
        words = torch.zeros((B, n, KH, s["mask"].shape[-1]), dtype=torch.int64, device=DEV)
        words[seq, row] = s["mask"].long()
        p = slot // S
        w = words.gather(3, (p // 32)[:, None, None].expand(B, n, KH, R))
        old = (draft < 0)[:, None] & (slot[:, None] <= pos[..., None])
        sees = sees | ((w >> (p % 32)[:, None, None]) & 1 > 0) & old[:, :, None]
    sees = sees.permute(0, 2, 1, 3).repeat_interleave(G, 2)                # [B, KH, n G, R]
    qq = q.permute(0, 2, 1, 3, 4).reshape(B, KH, n * G, D)
    score = torch.matmul(qq, k.permute(0, 2, 3, 1)) / math.sqrt(D)
    score = score.masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.transpose(1, 2)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1)
    out = out.reshape(B, KH, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, KH * G, D)[seq, row]
    lse = lse.reshape(B, KH, n, G).permute(0, 2, 1, 3).reshape(B, n, KH * G)[seq, row]
    return out.to(torch.bfloat16), lse.t().contiguous()


# -------------------------------------------------- the framework's calls ---

def _own_state(s):
    """What a program that serves keeps: the cache's handle and the attention's workspace."""
    import block_sparse_attention_kunlun_b200 as ba
    c = s["case"]
    o = {"ba": ba, "cache": ba.HistoryCache(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"])}
    if c["op"] == "attend":
        need = ba.ba_cache_fwd_workspace_size(o["cache"], ba.make_problem(s["q"], s["offs"]), c["block"], c["window"])
        o["workspace"] = ba.workspace_for(need, DEV)
    return o


def _run_own(s):
    c, o = s["case"], s["own"]
    ba, cache = o["ba"], o["cache"]
    if c["op"] == "write":
        ba.cache_write(cache, s["k"], s["v"], s["offs"], s["starts"])
    elif c["op"] == "read":
        return ba.cache_read(cache, s["offs"], s["starts"], s["rows"], k=s["k"], v=s["v"])
    elif c["op"] == "summarize":
        return ba.cache_summarize(cache, s["starts"], s["ends"], s["out"])
    elif c["op"] == "select":
        return ba.cache_select(cache, s["q"], s["offs"], s["lens"], s["summaries"], c["block"], c["window"], c["topk"],
                               positions=s["positions"], page_mask=s["out"])
    else:
        return ba.cache_attention_fwd(cache, s["q"], s["offs"], s["lens"], c["block"], c["window"],
                                      positions=s["positions"], tree_mask=s["tree"], page_mask=s["mask"],
                                      out=s["out"], lse=s["lse"], workspace=o["workspace"])


def run(state):
    c = state["case"]
    if own:
        r = _run_own(state)
    else:
        r = {"write": _plain_write, "read": _plain_read, "summarize": _plain_summarize, "select": _plain_select,
             "attend": _plain_attend}[c["op"]](state)
    if c["op"] == "write":  # the cache's own buffers, as the values they stand for
        return [state["k_pages"].view(torch.float8_e4m3fn), state["k_scales"].view(torch.float8_e8m0fnu),
                state["v_pages"].view(torch.float8_e4m3fn), state["v_scales"].view(torch.float8_e8m0fnu)]
    return r


# ------------------------------------------------------------------- work ---

def work(case):
    c = dict(_BASE, **case)
    B, KH, G, D, S = c["batch"], c["kv_heads"], c["group"], c["head_dim"], c["page"]
    cached = 2 * (D + D // 32)                    # bytes of one slot's key and value, a head
    mean_len, mean_rows = (c["len_lo"] + c["len_hi"]) / 2, (c["rows_lo"] + c["rows_hi"]) / 2
    esz = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("write", "read"):
        rows = B * (mean_rows if c["op"] == "write" else min(mean_rows, max(mean_len, 1)))
        return {"bytes": rows * KH * (2 * D * esz + cached) + 8 * B, "flops": 2 * rows * KH * D}
    if c["op"] == "summarize":
        pages = max(1.0, B * min(mean_rows, mean_len) / S)
        return {"bytes": pages * KH * (S * cached / 2 + 4 * D), "flops": pages * KH * S * D}
    rows = B * mean_rows
    lengths = [c["len_lo"] + (c["len_hi"] - c["len_lo"]) * (i + 0.5) / 64 for i in range(64)]
    start = [max(0, int(x) // c["block"] - c["window"] + 1) * c["block"] for x in lengths]
    if c["op"] == "select":
        pages = B * sum(min(-(-w // S), int(x) // S) for w, x in zip(start, lengths)) / 64
        return {"bytes": pages * KH * 4 * D + rows * KH * (G * D * 2 + 4 * -(-c["len_hi"] // S // 32)) + 8 * B,
                "flops": max(1.0, 2 * D * KH * pages * mean_rows)}
    near = sum(x - w for w, x in zip(start, lengths)) / 64
    far = sum(min(w, c["topk"] * S) for w in start) / 64 if c["topk"] else 0.0
    union = sum(min(w, c["topk"] * S * (1 if mean_rows == 1 else 1.5)) for w in start) / 64 if c["topk"] else 0.0
    drafts = {"chain": (mean_rows + 1) / 2, "tree": min(mean_rows, 2 + mean_rows / 3), "candidates": 1.0}[c["shape"]]
    return {"bytes": B * KH * (near + union + mean_rows) * cached + rows * KH * G * (4 * D + 4),
            "flops": 4 * D * rows * KH * G * (near + far + drafts)}


# ------------------------------------------------- exact values, 64 bits ---

def _exact_codes(x):
    """Elements and scales of x's 32-value blocks as numbers in 64 bits."""
    b = x.double().reshape(x.shape[:-1] + (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))) - 8
    scale = torch.exp2(e.clamp(-127, 127))
    y = b / scale
    quantum = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = (torch.round(y / quantum) * quantum).clamp(-448, 448)
    return y.reshape(x.shape), scale.squeeze(-1)


def _exact_rows(el, sc):
    """Cached rows [..., D] as numbers in 64 bits, from the codes' fields."""
    c = el.to(torch.int64)
    ef, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ef > 0, (1 + m / 8) * torch.exp2((ef - 7).double()), m / 8 * 2.0 ** -6)
    v = torch.where(c >= 128, -mag, mag)
    return v * torch.exp2(sc.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    S, KH, G, D = c["page"], c["kv_heads"], c["group"], c["head_dim"]
    table, offs = s["table"].long().cpu(), s["offs"].tolist()
    starts, lens, ends = s["starts"].tolist(), s["lens"].tolist(), s["ends"].tolist()
    if c["op"] == "write":
        got = []
        for x, el, sc in ((s["k"], s["k_pages"], s["k_scales"]), (s["v"], s["v_pages"], s["v_scales"])):
            pool, scales = torch.zeros(el.shape, dtype=torch.float64, device=DEV), torch.zeros(sc.shape, dtype=torch.float64, device=DEV)
            scales += 2.0 ** -127  # what a scale code of zero stands for
            for b in range(c["batch"]):
                t = torch.arange(starts[b], starts[b] + offs[b + 1] - offs[b])
                a, e = _exact_codes(x[offs[b]:offs[b + 1]])
                page, at = table[b, t // S].to(DEV), (t % S).to(DEV)
                pool[page, :, at], scales[page, :, at] = a, e
            got += [pool, scales]
        return got
    if c["op"] == "read":
        got = []
        for el, sc in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])):
            parts = []
            for b in range(c["batch"]):
                t = torch.arange(starts[b], starts[b] + offs[b + 1] - offs[b])
                page, at = table[b, t // S].to(DEV), (t % S).to(DEV)
                parts.append(_exact_rows(el[page, :, at], sc[page, :, at]))
            got.append(torch.cat(parts))
        return got
    if c["op"] == "summarize":
        out = torch.zeros((s["pages"], KH, D), dtype=torch.float64, device=DEV)
        for b in range(c["batch"]):
            for p in range(starts[b] // S, ends[b] // S):
                page = int(table[b, p])
                out[page] = _exact_rows(s["k_pages"][page], s["k_scales"][page]).sum(1) / S
        return out
    if c["op"] == "select":
        return None
    tree = None if s["tree"] is None else s["tree"].tolist()
    outs, lses = [], []
    for b in range(c["batch"]):
        lo, hi = offs[b], offs[b + 1]
        n = hi - lo
        t = torch.arange(lens[b] + n)
        page, at = table[b, t // S].to(DEV), (t % S).to(DEV)
        pos = s["pos"][lo:hi]
        first = (pos // c["block"] - c["window"] + 1).clamp(min=0) * c["block"]
        old = torch.arange(lens[b], device=DEV)
        near = (old[None] >= first[:, None]) & (old[None] <= pos[:, None])
        if tree is None:
            among = torch.ones(n, n, dtype=torch.bool).tril()
        else:
            among = torch.tensor([[bool((tree[lo + i][j // 32] >> (j % 32)) & 1) for j in range(n)] for i in range(n)])
        among = among.to(DEV) & (pos[None] >= first[:, None]) & (pos[None] <= pos[:, None])
        for h in range(KH):
            seen = near
            if s["mask"] is not None:
                w = s["mask"][lo:hi, h].long()[:, (old // S) // 32]
                seen = seen | (((w >> ((old // S) % 32)[None]) & 1) > 0) & (old[None] <= pos[:, None])
            vis = torch.cat([seen, among], 1)
            k, v = (_exact_rows(el[page, h, at], sc[page, h, at])
                    for el, sc in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
            for g in range(G):
                q = s["q"][lo:hi, h * G + g].double()
                x = (q @ k.t() / math.sqrt(D)).masked_fill(~vis, -math.inf)
                lse = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[:, None]) if bool(vis.any(1).all()) else torch.nan_to_num(torch.exp(x - lse[:, None]))
                outs.append((lo, h * G + g, p @ v))
                lses.append((lo, h * G + g, lse))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros((KH * G, s["rows"]), dtype=torch.float64, device=DEV)
    for (lo, h, o), (_, _, x) in zip(outs, lses):
        out[lo:lo + o.shape[0], h] = o
        lse[h, lo:lo + o.shape[0]] = x
    return out, lse
