"""The operators over a paged K/V cache, as cases that can be timed and checked.

Four kinds of case:
  attn    softmax attention of each sequence's newest rows over its whole paged cache (decode, verify, prefill chunk);
  window  the same where a row sees the last `window` tokens and the first `sinks` tokens of its sequence only;
  append  new tokens' K and V written into the pages (quantized when the cache holds E4M3 codes);
  fork    children of a beam: the page lists of the last step's children are freed and the parents' are forked again;
  compact pages in use moved to the lowest page numbers after sequences have ended.

A cache layer is two arrays of pages, [n_pages, kv_heads, page, dim] (order "head") or [n_pages, page, kv_heads, dim]
(order "token"); a sequence's tokens lie in the pages that its row of the page table names.  With fp8 state the
arrays hold E4M3 codes and a (K, V) pair of f16 scales for each head and token.
"""
import math
import random

import torch

own = False

#: 24 query heads over 2 KV heads, head_dim 256 or 128: the shapes of this repository's workloads.
HQ, HKV = 24, 2


def listed():
    base = {"hq": HQ, "hkv": HKV}
    return [
        # The first tokens of a chat: one short sequence, where the launches are what counts.
        {"name": "decode short bf16", "op": "attn", "dtype": "bf16", "dim": 128, "page": 16, "order": "head", "seqs": 1, "len_lo": 517,
         "len_hi": 517, "rows_lo": 1, "rows_hi": 1, "window": 0, "sinks": 0, "shape": 1, **base},
        # The decode workload's context.
        {"name": "decode 65k bf16", "op": "attn", "dtype": "bf16", "dim": 256, "page": 64, "order": "head", "seqs": 1, "len_lo": 65536,
         "len_hi": 65536, "rows_lo": 1, "rows_hi": 1, "window": 0, "sinks": 0, "shape": 2, **base},
        # The verify workload: four speculative rows at 261,120 tokens.
        {"name": "verify 261k bf16", "op": "attn", "dtype": "bf16", "dim": 256, "page": 128, "order": "token", "seqs": 1, "len_lo": 261120,
         "len_hi": 261120, "rows_lo": 4, "rows_hi": 4, "window": 0, "sinks": 0, "shape": 3, **base},
        # A serving batch of ragged contexts with quantized state, some sequences with one row and some with several.
        {"name": "ragged batch fp8", "op": "attn", "dtype": "fp8", "dim": 256, "page": 32, "order": "head", "seqs": 16, "len_lo": 4096,
         "len_hi": 262144, "rows_lo": 1, "rows_hi": 4, "window": 0, "sinks": 0, "shape": 4, **base},
        # A prompt's chunk of 2,048 rows over what came before it.
        {"name": "prefill chunk bf16", "op": "attn", "dtype": "bf16", "dim": 128, "page": 64, "order": "head", "seqs": 1, "len_lo": 16384,
         "len_hi": 16384, "rows_lo": 2048, "rows_hi": 2048, "window": 0, "sinks": 0, "shape": 5, **base},
        # Decode of a full batch in the sliding-window layers of a model.
        {"name": "window decode bf16", "op": "window", "dtype": "bf16", "dim": 128, "page": 32, "order": "head", "seqs": 64, "len_lo": 900,
         "len_hi": 65536, "rows_lo": 1, "rows_hi": 1, "window": 4096, "sinks": 4, "shape": 6, **base},
        # The prefill workload's chunk (2,048 rows at a prefix of 100,352 tokens) in a sliding-window layer.
        {"name": "window prefill bf16", "op": "window", "dtype": "bf16", "dim": 256, "page": 64, "order": "head", "seqs": 1, "len_lo": 102400,
         "len_hi": 102400, "rows_lo": 2048, "rows_hi": 2048, "window": 4096, "sinks": 64, "shape": 7, **base},
        # Full precision, odd sizes: a small mixed batch as a check against a reference runs it.
        {"name": "window ragged f32", "op": "window", "dtype": "f32", "dim": 256, "page": 16, "order": "token", "seqs": 5, "len_lo": 301,
         "len_hi": 4099, "rows_lo": 1, "rows_hi": 37, "window": 1001, "sinks": 5, "shape": 8, **base},
        # The cache write of a decode or verify step of a full batch; K and V are slices of one fused projection.
        {"name": "append batch bf16", "op": "append", "dtype": "bf16", "dim": 128, "page": 16, "order": "head", "seqs": 64, "len_lo": 100,
         "len_hi": 4000, "rows_lo": 1, "rows_hi": 4, "window": 0, "sinks": 0, "shape": 9, **base},
        # The cache write of a prompt's chunk, quantized.
        {"name": "append chunk fp8", "op": "append", "dtype": "fp8", "dim": 256, "page": 64, "order": "head", "seqs": 1, "len_lo": 4099,
         "len_hi": 4099, "rows_lo": 2048, "rows_hi": 2048, "window": 0, "sinks": 0, "shape": 10, **base},
        # One step of a beam search over 12 layers: 8 parents of up to 16k tokens, 4 children each.
        {"name": "fork beams bf16", "op": "fork", "dtype": "bf16", "dim": 128, "page": 16, "order": "head", "seqs": 8, "children": 4,
         "len_lo": 1000, "len_hi": 16000, "layers": 12, "pool": 6000, "shape": 11, **base},
        # A pool of 12 layers of which two thirds of the sequences have ended.
        {"name": "compact pool bf16", "op": "compact", "dtype": "bf16", "dim": 256, "page": 64, "order": "head", "seqs": 24, "children": 0,
         "len_lo": 500, "len_hi": 8000, "layers": 12, "pool": 1500, "shape": 12, **base},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "window", "window", "append", "fork", "compact"])
    dim = rng.choice([128, 256])
    page = rng.choice([16, 32, 64, 128])
    order = rng.choice(["head", "token"])
    case = {"op": op, "dim": dim, "page": page, "order": order, "hq": HQ, "hkv": HKV, "shape": rng.randrange(1 << 30)}
    if op in ("fork", "compact"):
        hi = _log(rng, 64, 16000 if op == "fork" else 8000)
        seqs = rng.randint(1, 8) if op == "fork" else rng.randint(3, 24)
        children = rng.randint(1, 4) if op == "fork" else 0
        # Room for every sequence and the children's own last pages.
        pool = seqs * (-(-hi // page)) + seqs * children + rng.randint(0, 40)
        layers = rng.randint(1, 12)
        while layers > 1 and pool * page * dim * layers > 1500 * 64 * 256 * 12:
            layers -= 1
        return {**case, "dtype": "bf16", "seqs": seqs, "children": children, "len_lo": max(1, hi // 5), "len_hi": hi, "layers": layers, "pool": pool}
    dtype = rng.choice(["bf16", "bf16", "fp8", "f32"])
    window = sinks = 0
    if op == "window":
        window, sinks = _log(rng, 1, 8192), rng.choice([0, rng.randint(1, 128)])
    kind = rng.choice(["decode", "verify", "chunk"])
    if op == "append":
        rows = {"decode": 1, "verify": rng.randint(2, 8), "chunk": _log(rng, 9, 2048)}[kind]
        seqs = _log(rng, 1, 64) if kind != "chunk" else rng.randint(1, 3)
        hi = max(rows, _log(rng, 16, 4000))
        return {**case, "dtype": dtype, "seqs": seqs, "len_lo": max(rows, hi // 7), "len_hi": hi, "rows_lo": max(1, rows // 2), "rows_hi": rows,
                "window": 0, "sinks": 0}
    if kind == "chunk":
        rows = _log(rng, 9, 2048 if dtype != "f32" else 256)
        seqs = rng.randint(1, 2)
        hi = max(rows, _log(rng, 16, 16384 if window == 0 and dtype != "f32" else 8000))
    else:
        rows = 1 if kind == "decode" else rng.randint(2, 8)
        seqs = _log(rng, 1, 64)
        hi = max(rows, _log(rng, 16, min(262144, 524288 // seqs) if dtype != "f32" else 60000 // seqs))
    return {**case, "dtype": dtype, "seqs": seqs, "len_lo": max(rows, hi // 20), "len_hi": hi, "rows_lo": max(1, rows // 3), "rows_hi": rows,
            "window": window, "sinks": sinks}


def sizes(case):
    """(tokens, rows) of each sequence: the case's own, whatever the seed of its values."""
    rng = random.Random(case["shape"])
    lens = [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    rows = [min(n, rng.randint(case["rows_lo"], case["rows_hi"])) if "rows_lo" in case else 0 for n in lens]
    return lens, rows


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _encode(x):
    """E4M3 codes (as bytes) and f16 scales of f32 rows: scale = f16(f32(amax / 448)), codes nearest to f32(x / scale)."""
    scale = (x.abs().amax(-1, keepdim=True) / 448.0).half()
    s = scale.float()
    y = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _pages_of(x, page, order):
    """Pages [n, kv_heads, page, dim] as they lie in memory: "token" order keeps a token's heads side by side."""
    return x if order == "head" else x.transpose(1, 2).contiguous().transpose(1, 2)


def prepare(case, seed):
    g = _gen(seed)
    dim, page, hkv, hq = case["dim"], case["page"], case["hkv"], case["hq"]
    lens, rows = sizes(case)
    counts = [-(-n // page) for n in lens]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if case["op"] in ("fork", "compact"):
        return _prepare_pages(case, g, lens, counts, rand)
    n_pages = sum(counts) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    ld = max(counts) + 2
    table = torch.full((len(lens), ld), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = perm[at:at + c]
        at += c
    total = sum(rows)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    st = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "row_start": torch.tensor(starts, dtype=torch.int32, device="cuda"), "max_rows": max(rows), "scale": None}
    pages = [rand(n_pages, hkv, page, dim) for _ in range(2)]
    if case["dtype"] == "fp8":
        codes, scales = zip(*[_encode(x) for x in pages])
        pages = [_pages_of(c, page, case["order"]) for c in codes]
        st["scale"] = _pages_of(torch.cat(scales, -1), page, case["order"])
    else:
        kind = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        pages = [_pages_of(x.to(kind), page, case["order"]) for x in pages]
    st["k"], st["v"] = (x.view(torch.float8_e4m3fn) if case["dtype"] == "fp8" else x for x in pages)
    act = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    if case["op"] == "append":
        # One fused projection per row: queries, then keys, then values.
        fused = rand(total, hq + 2 * hkv, dim).to(act)
        st["k_new"], st["v_new"] = fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        return st
    # Heads from nearly uniform to sharply peaked attention.
    heat = torch.linspace(0.5, 3.0, hq, device="cuda")[None, :, None]
    st["q"] = (rand(total, hq, dim) * heat).to(act)
    # Keys that any row can see, at most: what a program knows when it sizes its buffers.
    w, s = case["window"], case["sinks"]
    st["span"] = max(lens) if not w else max(min(n, s + w + r) for n, r in zip(lens, rows))
    return st


def _prepare_pages(case, g, lens, counts, rand):
    dim, page, hkv, n_pages = case["dim"], case["page"], case["hkv"], case["pool"]
    layers, seqs, kids = case["layers"], case["seqs"], case["children"]
    k, v = (torch.empty(layers, n_pages, hkv, page, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(layers):
        k[i], v[i] = rand(n_pages, hkv, page, dim), rand(n_pages, hkv, page, dim)
    if case["order"] == "token":
        k, v = (x.transpose(2, 3).contiguous().transpose(2, 3) for x in (k, v))
    rng = random.Random(case["shape"] + 1)
    # For "compact", two of three sequences have ended and their pages are free again.
    live = [i for i in range(seqs) if case["op"] == "fork" or i % 3 == 0]
    slots = seqs * (1 + kids)
    table = torch.full((slots, max(counts) + 1), -1, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    length = torch.zeros(slots, dtype=torch.int32)
    order = list(range(n_pages))
    rng.shuffle(order)
    if sum(counts) > n_pages:  # a pool that all of them would not have fitted into at once: as many as fit
        room, kept = n_pages - seqs * kids, []
        for i in live:
            if counts[i] <= room:
                kept.append(i)
                room -= counts[i]
        live = kept
    at = 0
    for i in live:
        ids = torch.tensor(order[at:at + counts[i]], dtype=torch.int32)
        table[i, :counts[i]] = ids
        refs[ids.long()] = 1
        length[i] = lens[i]
        at += counts[i]
    st = {"case": case, "k": k, "v": v, "table": table.cuda(), "refs": refs.cuda(), "lens": length.cuda()}
    if case["op"] == "fork":
        src = [i for i in live for _ in range(kids)]
        st["src"] = torch.tensor(src, dtype=torch.int32, device="cuda")
        st["dst"] = torch.arange(seqs, seqs + len(src), dtype=torch.int32, device="cuda")
    else:
        # A serving loop meets a scattered pool whenever sequences have ended; here each pass puts the
        # scattered bookkeeping back first (three copies of some kilobytes, beside the pages that move).
        st["was"] = [st[x].clone() for x in ("table", "refs", "lens")]
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    if op in ("attn", "window"):
        return _attend(st)
    if op == "append":
        return _append(st)
    return _fork(st) if op == "fork" else _compact(st)


# ---------------------------------------------------------------- the framework's calls


def _run_own(st, op):
    import indexed_sparse_attention_gb300 as qsa

    case = st["case"]
    if op in ("attn", "window"):
        if "step" not in st:
            batch = qsa.PagedBatch(st["table"], st["lens"], st["row_start"], n_rows=st["q"].shape[0], max_rows=st["max_rows"])
            cache = qsa.PagedCache(st["k"], st["v"], kv_scale=st["scale"])
            st["step"] = qsa.PagedStep(cache, batch, st["q"], out_dtype=st["q"].dtype, window=case["window"], n_sinks=case["sinks"])
        out, lse = st["step"].attend()
        return {"out": out, "lse": lse}
    if op == "append":
        if "batch" not in st:
            st["batch"] = qsa.PagedBatch(st["table"], st["lens"], st["row_start"], n_rows=st["k_new"].shape[0], max_rows=st["max_rows"])
            st["cache"] = qsa.PagedCache(st["k"], st["v"], kv_scale=st["scale"])
        qsa.paged_append(st["cache"], st["batch"], st["k_new"], st["v_new"])
        return _state(st)
    if "pages" not in st:
        caches = [qsa.PagedCache(st["k"][i], st["v"][i]) for i in range(case["layers"])]
        st["pages"] = qsa.PagePool(st["table"], st["lens"], st["refs"], caches)
    if op == "fork":
        st["pages"].free(st["dst"])
        st["pages"].fork(st["src"], st["dst"])
    else:
        _scatter(st)
        st["pages"].compact()
    return _state(st)


# ---------------------------------------------------------------- plain forms


def _state(st):
    keys = ("k", "v", "scale", "table", "lens", "refs")
    return {x: st[x] for x in keys if st.get(x) is not None}


def _scatter(st):
    for name, was in zip(("table", "refs", "lens"), st["was"]):
        st[name].copy_(was)


def _attend(st):
    case = st["case"]
    dim, page, hkv, hq = case["dim"], case["page"], case["hkv"], case["hq"]
    w, s, group, n = case["window"], case["sinks"], hq // hkv, case["seqs"]
    lens, start, most = st["lens"].long(), st["row_start"].long(), st["max_rows"]
    rows = start[1:] - start[:-1]
    # The keys of each sequence that any of its rows sees, padded to the longest: its first tokens, then the last.
    j = torch.arange(st["span"], device="cuda")
    if w:
        low = (lens - rows - w + 1).clamp(min=s)
        pos = torch.where(j < s, j, low[:, None] + (j - s))
    else:
        pos = j.expand(n, -1)
    there = pos < lens[:, None]
    safe = torch.where(there, pos, torch.zeros_like(pos))
    ids, slot = torch.gather(st["table"], 1, safe // page).long(), safe % page
    kv = []
    for x, which in ((st["k"], 0), (st["v"], 1)):  # K, then V
        x = x[ids, :, slot] if x.dtype != torch.float8_e4m3fn else x.view(torch.uint8)[ids, :, slot].view(torch.float8_e4m3fn)
        x = x.float()
        kv.append(x if st["scale"] is None else x * st["scale"][ids, :, slot, which:which + 1].float())
    k, v = (x.transpose(1, 2) for x in kv)  # [sequences, kv_heads, keys, dim]
    # Each sequence's rows, padded to the most that one has.
    r = torch.arange(most, device="cuda")
    at = (start[:-1, None] + r).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[at].reshape(n, most, hkv, group, dim).transpose(1, 2).reshape(n, hkv, most * group, dim)
    logits = (q @ k.transpose(2, 3)) / math.sqrt(dim)
    place = (lens - rows)[:, None] + r  # [sequences, rows]
    seen = there[:, None] & (pos[:, None] <= place[:, :, None])
    if w:
        seen &= (pos[:, None] > place[:, :, None] - w) | (pos[:, None] < s)
    seen = seen[:, None, :, None].expand(-1, 1, -1, group, -1).reshape(n, 1, most * group, -1)
    logits.masked_fill_(~seen, float("-inf"))
    top = logits.amax(-1, keepdim=True)
    e = (logits - torch.where(top.isfinite(), top, torch.zeros_like(top))).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.where(total > 0, (e @ v) / total, torch.zeros((), device="cuda"))
    lse = (top + total.log())[..., 0]
    real = (r < rows[:, None]).reshape(-1)
    back = lambda x: x.reshape(n, hkv, most, group, -1).transpose(1, 2).reshape(n * most, hq, -1)[real]  # noqa: E731
    return {"out": back(out).to(st["q"].dtype), "lse": back(lse)[..., 0]}


def _append(st):
    page = st["case"]["page"]
    lens, start = st["lens"].long(), st["row_start"].long()
    row = torch.arange(st["k_new"].shape[0], device="cuda")
    seq = torch.searchsorted(start, row, right=True) - 1
    pos = lens[seq] - (start[seq + 1] - row)
    ids, slot = st["table"][seq, pos // page].long(), pos % page
    if st["scale"] is None:
        st["k"][ids, :, slot], st["v"][ids, :, slot] = st["k_new"], st["v_new"]
        return _state(st)
    (kc, ks), (vc, vs) = _encode(st["k_new"].float()), _encode(st["v_new"].float())
    st["k"].view(torch.uint8)[ids, :, slot], st["v"].view(torch.uint8)[ids, :, slot] = kc, vc
    st["scale"][ids, :, slot] = torch.cat((ks, vs), -1)
    return _state(st)


def _fork(st):
    page, table, lens, refs = st["case"]["page"], st["table"], st["lens"], st["refs"]
    src, dst = st["src"].long(), st["dst"].long()
    # Free what the children held: one user less for each page, and empty rows.
    col = torch.arange(table.shape[1], device="cuda")
    held = table[dst][col < ((lens[dst] + page - 1) // page)[:, None]].long()
    refs.index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    table[dst], lens[dst] = -1, 0
    # Fork: whole pages are shared, a last page that is not full is copied to the lowest free page.
    size, full, tail = lens[src], lens[src] // page, lens[src] % page
    shared = col < full[:, None]
    row = torch.where(shared, table[src], torch.full_like(table[src], -1))
    refs.index_add_(0, row[shared].long(), torch.ones_like(row[shared]))
    part = (tail > 0).nonzero()[:, 0]
    new = (refs == 0).nonzero()[:part.numel(), 0]
    old = table[src[part], full[part].long()].long()
    row[part, full[part].long()] = new.to(torch.int32)
    refs[new] = 1
    table[dst], lens[dst] = row, size
    tok = torch.arange(page, device="cuda") < tail[part][:, None]
    tok = tok[None, :, None, :, None]
    st["k"][:, new] = torch.where(tok, st["k"][:, old], st["k"][:, new])
    st["v"][:, new] = torch.where(tok, st["v"][:, old], st["v"][:, new])
    return _state(st)


def _compact(st):
    _scatter(st)
    table, refs = st["table"], st["refs"]
    n = refs.numel()
    used = refs > 0
    ids = torch.arange(n, device="cuda")
    most = used.sum()
    old, new = (used & (ids >= most)).nonzero()[:, 0], (~used & (ids < most)).nonzero()[:, 0]
    st["k"][:, new], st["v"][:, new] = st["k"][:, old], st["v"][:, old]
    to = ids.clone()
    to[old] = new
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table))
    refs[new], refs[old] = refs[old], 0
    return _state(st)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    lens, rows = sizes(case)
    dim, page, hkv, hq = case["dim"], case["page"], case["hkv"], case["hq"]
    if case["op"] in ("fork", "compact"):
        return _work_pages(case, lens)
    width, extra = {"bf16": (2, 0), "fp8": (1, 2), "f32": (4, 0)}[case["dtype"]]
    act = 4 if case["dtype"] == "f32" else 2
    token = 2 * hkv * (dim * width + extra)  # K and V of one token, scales among them
    total = sum(rows)
    if case["op"] == "append":
        return {"bytes": total * (2 * hkv * dim * act + token), "flops": 0}
    w, s = case["window"], case["sinks"]
    keys = products = 0
    for n, r in zip(lens, rows):
        low = max(0, n - r - w + 1) if w else 0
        keys += n - low + min(s, low)
        for p in range(n - r, n):
            first = max(0, p - w + 1) if w else 0
            products += p + 1 - first + min(s, first)
    table = sum(-(-n // page) for n in lens) * 4 if not w else keys // page * 4
    return {"bytes": keys * token + table + total * hq * (2 * dim * act + 4), "flops": 4 * dim * hq * products}


def _work_pages(case, lens):
    page, token = case["page"], 2 * case["hkv"] * case["dim"] * 2
    if case["op"] == "fork":
        kids = case["children"]
        pages = kids * sum(-(-n // page) for n in lens)
        tails = kids * sum(n % page for n in lens)
        # Freeing reads and clears a table entry and changes a count; forking reads and writes one and changes a count.
        return {"bytes": case["layers"] * tails * token * 2 + pages * (8 + 8 + 8 + 8), "flops": 0}
    live = [n for i, n in enumerate(lens) if i % 3 == 0]
    used, pool = sum(-(-n // page) for n in live), case["pool"]
    moved = used * max(0, pool - used) // pool  # pages that lie above the first `used`, in the mean
    return {"bytes": case["layers"] * moved * page * token * 2 + used * 8 + pool * 4, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # pages, counts and page numbers are moved, not computed
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st) if st["scale"] is not None else None
    lens, rows = sizes(case)
    dim, page, hkv, hq = case["dim"], case["page"], case["hkv"], case["hq"]
    out, lse, at = [], [], 0
    for i, (n, r) in enumerate(zip(lens, rows)):
        pages = st["table"][i, :-(-n // page)].long()
        k, v = (x.view(torch.uint8)[pages].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[pages] for x in (st["k"], st["v"]))
        q = st["q"][at:at + r].double()
        at += r
        p = torch.arange(n - r, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None, :]
        ok = t <= p
        if case["window"]:
            ok &= (t + case["window"] > p) | (t < case["sinks"])
        heads_o, heads_l = [], []
        for h in range(hkv):
            kh, vh = (x[:, h].double().reshape(-1, dim)[:n] for x in (k, v))
            if st["scale"] is not None:
                sc = st["scale"][pages][:, h].double().reshape(-1, 2)[:n]
                kh, vh = kh * sc[:, :1], vh * sc[:, 1:]
            g = hq // hkv
            z = torch.einsum("rgd,td->rgt", q[:, h * g:(h + 1) * g], kh) * dim ** -0.5
            z = z.masked_fill(~ok[:, None, :], -math.inf)
            lz = torch.logsumexp(z, -1)
            heads_l.append(lz)
            heads_o.append(torch.einsum("rgt,td->rgd", torch.exp(z - lz[..., None]), vh))
        out.append(torch.cat(heads_o, 1))
        lse.append(torch.cat(heads_l, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _exact_append(st):
    page = st["case"]["page"]
    lens, rows = sizes(st["case"])
    k, v, scale = st["k"].view(torch.uint8).clone(), st["v"].view(torch.uint8).clone(), st["scale"].clone()
    places = [(i, n - r + j) for i, (n, r) in enumerate(zip(lens, rows)) for j in range(r)]
    seq = torch.tensor([a for a, _ in places], device="cuda")
    pos = torch.tensor([b for _, b in places], device="cuda")
    ids, slot = st["table"][seq, pos // page].long(), pos % page
    for which, (to, x) in enumerate(((k, st["k_new"]), (v, st["v_new"]))):
        x = x.double()
        sc = (x.abs().amax(-1) / 448).float().half()
        y = (x / sc.double()[..., None]).nan_to_num(0.0).clamp(-448, 448)
        to[ids, :, slot] = y.float().to(torch.float8_e4m3fn).view(torch.uint8)
        scale[ids, :, slot, which] = sc
    return {"k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "scale": scale, "table": None, "lens": None}
