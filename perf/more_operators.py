"""Rotary positions and caches held in 4 bits, as cases that can be timed and checked.

Four kinds of case:
  rotate  the rotation of query rows by their positions (halves or neighbouring pairs, part of the head, scaled frequencies);
  append  a step's rows into the pages of a cache, K rotated on the way and Q beside it (f32, bf16, fp8 and 4-bit caches);
  read    rows of a 4-bit cache back out of its pages;
  attn    attention of each sequence's newest rows over its 4-bit cache, whole or through a sliding window.

A cache layer is two arrays of pages, [n_pages, kv_heads, page, dim] (order "head") or [n_pages, page, kv_heads, dim] (order
"token"); a sequence's tokens lie in the pages that its row of the page table names.  With 4-bit state a row of `dim`
channels is dim / 32 blocks: value = code * scale + minimum with codes 0 .. 15 and an f16 pair for each block; channel
32 g + 4 n + j of a row is nibble j (low first) of its 16-bit unit n * (dim / 32) + g.
"""
import math
import random

import torch

own = False

#: 24 query heads over 2 KV heads, head_dim 256 or 128: the shapes of this repository's workloads.
HQ, HKV = 24, 2
NEAR = {"scaling": "none", "factor": 1.0}
#: Contexts stretched by parts, as for 32 times the 8,192 tokens of a first training.
FAR = {"scaling": "parts", "factor": 32.0}
ORIGINAL = 8192


def listed():
    base = {"hq": HQ, "hkv": HKV, "base": 1e6}
    step = {"page": 16, "order": "head", "window": 0, "sinks": 0}
    return [
        # The queries of a decode step of a full batch, rotated by themselves.
        {"name": "rotate step bf16", "op": "rotate", "dtype": "bf16", "dim": 128, "rot": 128, "pairs": False, "seqs": 64, "len_lo": 100,
         "len_hi": 65536, "rows_lo": 1, "rows_hi": 1, "shape": 1, **base, **NEAR},
        # Queries of a long prompt, the first quarter of each head rotated, positions past the first training's context.
        {"name": "rotate prompt part bf16", "op": "rotate", "dtype": "bf16", "dim": 256, "rot": 64, "pairs": True, "seqs": 2, "len_lo": 100352,
         "len_hi": 261120, "rows_lo": 8192, "rows_hi": 8192, "shape": 2, **base, **FAR},
        # The rows of a decode or verify step of a full batch into a bf16 cache, all three from one fused projection.
        {"name": "append step bf16", "op": "append", "dtype": "bf16", "dim": 128, "rot": 128, "pairs": False, "seqs": 64, "len_lo": 100,
         "len_hi": 4000, "rows_lo": 1, "rows_hi": 4, "shape": 3, **base, **NEAR, **step},
        # A prompt's chunk into a 4-bit cache (and its rows read back: what is held in 4 bits).
        {"name": "append chunk q4", "op": "append", "dtype": "q4", "dim": 256, "rot": 256, "pairs": False, "seqs": 1, "len_lo": 102400,
         "len_hi": 102400, "rows_lo": 2048, "rows_hi": 2048, "shape": 4, **base, **FAR, **step, "page": 64},
        # The same for fp8, ragged prompts of odd lengths, neighbouring channels paired.
        {"name": "append prompts fp8", "op": "append", "dtype": "fp8", "dim": 128, "rot": 64, "pairs": True, "seqs": 5, "len_lo": 301,
         "len_hi": 4099, "rows_lo": 301, "rows_hi": 2047, "shape": 5, **base, **NEAR, **step, "order": "token"},
        # A cached prefix handed to something that takes bf16.
        {"name": "read prefix q4", "op": "read", "dtype": "q4", "dim": 256, "seqs": 1, "len_lo": 65536, "len_hi": 65536, "rows_lo": 65536,
         "rows_hi": 65536, "shape": 6, **base, **step, "page": 64},
        # The newest rows of a batch, as a check reads them.
        {"name": "read step q4", "op": "read", "dtype": "q4", "dim": 128, "seqs": 16, "len_lo": 100, "len_hi": 4000, "rows_lo": 1, "rows_hi": 4,
         "shape": 7, **base, **step, "order": "token"},
        # The first tokens of a chat: one short sequence, where the launches are what counts.
        {"name": "decode short q4", "op": "attn", "dtype": "q4", "dim": 128, "seqs": 1, "len_lo": 517, "len_hi": 517, "rows_lo": 1,
         "rows_hi": 1, "shape": 8, **base, **step},
        # The decode workload's context.
        {"name": "decode 65k q4", "op": "attn", "dtype": "q4", "dim": 256, "seqs": 1, "len_lo": 65536, "len_hi": 65536, "rows_lo": 1,
         "rows_hi": 1, "shape": 9, **base, **step, "page": 64},
        # The verify workload: four speculative rows at 261,120 tokens.
        {"name": "verify 261k q4", "op": "attn", "dtype": "q4", "dim": 256, "seqs": 1, "len_lo": 261120, "len_hi": 261120, "rows_lo": 4,
         "rows_hi": 4, "shape": 10, **base, **step, "page": 128, "order": "token"},
        # A serving batch of ragged contexts, one row each.
        {"name": "ragged decode q4", "op": "attn", "dtype": "q4", "dim": 256, "seqs": 16, "len_lo": 4096, "len_hi": 262144, "rows_lo": 1,
         "rows_hi": 1, "shape": 11, **base, **step, "page": 32},
        # A prompt's chunk of 2,048 rows over what came before it.
        {"name": "prefill chunk q4", "op": "attn", "dtype": "q4", "dim": 128, "seqs": 1, "len_lo": 16384, "len_hi": 16384, "rows_lo": 2048,
         "rows_hi": 2048, "shape": 12, **base, **step, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "read", "attn", "attn", "attn"])
    dim = rng.choice([128, 256])
    case = {"op": op, "dim": dim, "hkv": HKV, "hq": rng.choice([24, 24, 16, 2, 32]), "base": rng.choice([1e4, 1e6, 5e5]), "shape": rng.randrange(1 << 30)}
    if op in ("rotate", "append"):
        case |= {"rot": rng.choice([dim, dim, dim // 2, 32, 16 * rng.randint(1, dim // 16)]), "pairs": rng.random() < 0.5}
        case |= {"scaling": rng.choice(["none", "linear", "parts"]), "factor": round(rng.uniform(1.0, 40.0), 2)}
    if op == "rotate":
        rows = _log(rng, 1, 8192)
        hi = _log(rng, rows, 1 << 20)
        return {**case, "dtype": rng.choice(["bf16", "f32"]), "seqs": rng.randint(1, 2), "len_lo": max(rows, hi // 3), "len_hi": hi, "rows_lo": rows, "rows_hi": rows}
    case |= {"page": rng.choice([16, 32, 64, 128, 256]), "order": rng.choice(["head", "token"]), "window": 0, "sinks": 0}
    kind = rng.choice(["decode", "verify", "chunk"])
    rows = {"decode": 1, "verify": rng.randint(2, 8), "chunk": _log(rng, 9, 2048)}[kind]
    seqs = _log(rng, 1, 64) if kind != "chunk" else rng.randint(1, 3)
    if op == "append":
        hi = max(rows, _log(rng, 16, 4000))
        return {**case, "dtype": rng.choice(["q4", "q4", "q4", "bf16", "fp8", "f32"]), "seqs": seqs, "len_lo": max(rows, hi // 7), "len_hi": hi,
                "rows_lo": max(1, rows // 2), "rows_hi": rows}
    if op == "read":
        rows = _log(rng, 1, 16384)
        hi = max(rows, _log(rng, 16, 20000))
        return {**case, "dtype": "q4", "seqs": rng.randint(1, 4), "len_lo": max(rows, hi // 2), "len_hi": hi, "rows_lo": max(1, rows // 2), "rows_hi": rows}
    case["hq"] = rng.choice([24, 24, 16, 2])
    if rng.random() < 0.4:
        case |= {"window": _log(rng, 1, 8192), "sinks": rng.choice([0, rng.randint(1, 128)])}
    if kind == "chunk":
        hi = max(rows, _log(rng, 16, 16384))
        seqs = rng.randint(1, 2)
    else:
        hi = max(rows, _log(rng, 16, min(262144, 524288 // seqs)))
    return {**case, "dtype": "q4", "seqs": seqs, "len_lo": max(rows, hi // 20), "len_hi": hi, "rows_lo": max(1, rows // 3), "rows_hi": rows}


def sizes(case):
    """(tokens, rows) of each sequence: the case's own, whatever the seed of its values."""
    rng = random.Random(case["shape"])
    lens = [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    return lens, [min(n, rng.randint(case["rows_lo"], case["rows_hi"])) for n in lens]


def _pages_of(x, order):
    """Pages [n, kv_heads, page, dim] as they lie in memory: "token" order keeps a token's heads side by side."""
    return x if order == "head" else x.transpose(1, 2).contiguous().transpose(1, 2)


def _encode4(x):
    """Codes as bytes [..., dim / 2] and (scale, minimum) pairs [..., dim / 32, 2] of f32 rows."""
    dim = x.shape[-1]
    b = x.reshape(*x.shape[:-1], dim // 32, 32)
    low, high = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
    least, scale = low.half(), ((high - low) / 15.0).half()
    s = scale.float()
    c = torch.where(s > 0, (b - least.float()) / s, torch.zeros_like(b)).round().clamp(0, 15).to(torch.uint8)
    c = c.reshape(*x.shape[:-1], dim // 32, 8, 2, 2).transpose(-4, -3)  # [..., n, g, byte, nibble]
    return (c[..., 0] | (c[..., 1] << 4)).reshape(*x.shape[:-1], dim // 2), torch.cat((scale, least), -1)


def _decode4(codes, pairs):
    """The f32 rows that codes and pairs stand for."""
    g = pairs.shape[-2]
    c = codes.reshape(*codes.shape[:-1], 8, g, 2).transpose(-3, -2)
    c = torch.stack((c & 15, c >> 4), -1).reshape(*codes.shape[:-1], g, 32).float()
    return (c * pairs[..., :1].float() + pairs[..., 1:].float()).reshape(*codes.shape[:-1], 32 * g)


def _encode8(x):
    """E4M3 codes (as bytes) and f16 scales of f32 rows."""
    scale = (x.abs().amax(-1, keepdim=True) / 448.0).half()
    s = scale.float()
    y = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dim, hkv, hq = case["dim"], case["hkv"], case["hq"]
    lens, rows = sizes(case)
    total = sum(rows)
    act = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    # Heads from nearly uniform to sharply peaked attention.
    heat = torch.linspace(0.5, 3.0, hq, device="cuda")[None, :, None]
    st = {"case": case}
    if case["op"] == "rotate":
        st["x"] = (rand(total, hq, dim) * heat).to(act)
        st["positions"] = torch.cat([torch.arange(n - r, n, dtype=torch.int32) for n, r in zip(lens, rows)]).cuda()
        return st
    page = case["page"]
    counts = [-(-n // page) for n in lens]
    n_pages = sum(counts) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(counts) + 2), -1, dtype=torch.int32, device="cuda")
    starts, at = [0], 0
    for i, (c, r) in enumerate(zip(counts, rows)):
        table[i, :c] = perm[at:at + c]
        at += c
        starts.append(starts[-1] + r)
    st |= {"table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
           "row_start": torch.tensor(starts, dtype=torch.int32, device="cuda"), "rows": total, "max_rows": max(rows), "scale": None}
    # Keys of which some channels lie far from zero in all tokens, as they do behind a projection.
    lean = rand(hkv, 1, dim).pow(3) * 0.3
    pages = [rand(n_pages, hkv, page, dim) + lean, rand(n_pages, hkv, page, dim)]
    if case["dtype"] in ("q4", "fp8"):
        codes, scales = [], []
        for x in pages:
            c, s = _encode4(x) if case["dtype"] == "q4" else _encode8(x)
            codes.append(_pages_of(c, case["order"]))
            scales.append(s.reshape(*s.shape[:3], -1))
        st["scale"] = _pages_of(torch.cat(scales, -1), case["order"])
        pages = [c if case["dtype"] == "q4" else c.view(torch.float8_e4m3fn) for c in codes]
    else:
        pages = [_pages_of(x.to(act), case["order"]) for x in pages]
    st["k"], st["v"] = pages
    if case["op"] == "append":
        # One fused projection per row: queries, then keys, then values.
        fused = rand(total, hq + 2 * hkv, dim).to(act)
        st["q"], st["k_new"], st["v_new"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    elif case["op"] == "attn":
        st["q"] = (rand(total, hq, dim) * heat).to(act)
        # Keys that any row can see, at most: what a program knows when it sizes its buffers.
        w, s = case["window"], case["sinks"]
        st["span"] = max(lens) if not w else max(min(n, s + w + r) for n, r in zip(lens, rows))
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"rotate": _rotate_case, "append": _append, "read": _read, "attn": _attend}[op](st)


# ---------------------------------------------------------------- the framework's calls


def _rope_of(qsa, case):
    scaling = None
    if case["scaling"] == "linear":
        scaling = qsa.RopeScaling("linear", case["factor"])
    elif case["scaling"] == "parts":
        scaling = qsa.RopeScaling("parts", case["factor"], original_tokens=ORIGINAL)
    return qsa.Rope(case["rot"], base=case["base"], pairs=case["pairs"], scaling=scaling)


def _run_own(st, op):
    import indexed_sparse_attention_gb300 as qsa

    case = st["case"]
    if op == "rotate":
        if "rope" not in st:
            st["rope"], st["out"] = _rope_of(qsa, case), torch.empty_like(st["x"])
        qsa.rotate(st["rope"], st["positions"], st["x"], st["out"])
        return {"out": st["out"]}
    if "batch" not in st:
        st["batch"] = qsa.PagedBatch(st["table"], st["lens"], st["row_start"], n_rows=st["rows"], max_rows=st["max_rows"])
        st["cache"] = qsa.PagedCache(st["k"], st["v"], kv_scale=st["scale"], kv_dtype=qsa.Q4 if case["dtype"] == "q4" else None)
        if op == "append":
            st["rope"], st["q_out"] = _rope_of(qsa, case), torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
        if op in ("append", "read") and case["dtype"] == "q4":
            st["k_out"], st["v_out"] = (torch.empty(st["rows"], case["hkv"], case["dim"], dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if op == "attn":
            st["out"] = torch.empty_like(st["q"])
            st["ws"] = torch.empty(qsa.paged_attn_workspace_size(st["batch"], st["cache"].config(case["hq"], st["out"].dtype)), dtype=torch.uint8, device="cuda")
    if op == "attn":
        qsa.paged_attn(st["cache"], st["batch"], st["q"], st["out"], window=case["window"], n_sinks=case["sinks"], workspace=st["ws"])
        return {"out": st["out"]}
    if op == "append":
        qsa.paged_append(st["cache"], st["batch"], st["k_new"], st["v_new"], rope=st["rope"], q=st["q"], q_out=st["q_out"])
        if case["dtype"] != "q4":
            return {"q": st["q_out"], **_state(st)}
    qsa.paged_read(st["cache"], st["batch"], st["k_out"], st["v_out"])
    return {"k": st["k_out"], "v": st["v_out"], **({"q": st["q_out"]} if op == "append" else {})}


# ---------------------------------------------------------------- plain forms


def _state(st):
    return {x: st[x] for x in ("k", "v", "scale") if st[x] is not None}


def frequencies(case):
    """Angle per position of each rotated pair, and the factor on what is rotated."""
    inv = [case["base"] ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
    f = case["factor"]
    if case["scaling"] == "linear":
        return [w / f for w in inv], 1.0
    if case["scaling"] == "parts":
        # Channels that turn more than 32 times over the first training's context stay, those that turn less than
        # once are stretched, with a ramp between the two.
        keep = [min(1.0, max(0.0, (ORIGINAL * w / (2 * math.pi) - 1.0) / (32.0 - 1.0))) for w in inv]
        return [(1 - k) * w / f + k * w for w, k in zip(inv, keep)], 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _rotate(case, x, positions):
    """x [rows, heads, dim] rotated in 32 bits, from angles in 64."""
    inv, magnitude = frequencies(case)
    rot = case["rot"]
    angle = positions.double()[:, None, None] * torch.tensor(inv, dtype=torch.float64, device="cuda")
    cos, sin = (magnitude * angle.cos()).float(), (magnitude * angle.sin()).float()
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["pairs"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), -1).flatten(-2) if case["pairs"] else torch.cat((a, b), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _rotate_case(st):
    return {"out": _rotate(st["case"], st["x"], st["positions"]).to(st["x"].dtype)}


def _places(st):
    """Page, slot and position of each row."""
    page = st["case"]["page"]
    lens, start = st["lens"].long(), st["row_start"].long()
    row = torch.arange(st["rows"], device="cuda")
    seq = torch.searchsorted(start, row, right=True) - 1
    pos = lens[seq] - (start[seq + 1] - row)
    return st["table"][seq, pos // page].long(), pos % page, pos


def _append(st):
    case = st["case"]
    ids, slot, pos = _places(st)
    # The rows are rounded to the type that a row has, then stored (and quantized) as rows are.
    q = _rotate(case, st["q"], pos).to(st["q"].dtype)
    k, v = _rotate(case, st["k_new"], pos).to(st["q"].dtype), st["v_new"]
    if case["dtype"] in ("bf16", "f32"):
        st["k"][ids, :, slot], st["v"][ids, :, slot] = k, v
        return {"q": q, **_state(st)}
    encode = _encode4 if case["dtype"] == "q4" else _encode8
    (kc, ks), (vc, vs) = encode(k.float()), encode(v.float())
    st["k"].view(torch.uint8)[ids, :, slot], st["v"].view(torch.uint8)[ids, :, slot] = kc, vc
    st["scale"][ids, :, slot] = torch.cat((ks.flatten(2), vs.flatten(2)), -1)
    return {"q": q, **_state(st)} if case["dtype"] == "fp8" else {"q": q, **_read(st)}


def _rows_of(st, ids, slot):
    """K and V of tokens in pages `ids`, in 32 bits: [..., kv_heads, dim]."""
    pairs = st["scale"][ids, :, slot].unflatten(-1, (2, -1, 2))
    return [_decode4(x[ids, :, slot], pairs[..., i, :, :]) for i, x in enumerate((st["k"], st["v"]))]


def _read(st):
    ids, slot, _ = _places(st)
    k, v = _rows_of(st, ids, slot)
    return {"k": k.bfloat16(), "v": v.bfloat16()}


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
    k, v = (x.transpose(1, 2) for x in _rows_of(st, torch.gather(st["table"], 1, safe // page).long(), safe % page))
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
    real = (r < rows[:, None]).reshape(-1)
    return {"out": out.reshape(n, hkv, most, group, dim).transpose(1, 2).reshape(n * most, hq, dim)[real].to(st["q"].dtype)}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    lens, rows = sizes(case)
    dim, hkv, hq, total = case["dim"], case["hkv"], case["hq"], sum(sizes(case)[1])
    act = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotate":
        return {"bytes": total * (2 * hq * dim * act + 4), "flops": 3 * total * hq * case["rot"]}
    token = 2 * hkv * {"q4": dim * 5 // 8, "fp8": dim + 2, "bf16": 2 * dim, "f32": 4 * dim}[case["dtype"]]  # K and V, scales among them
    if case["op"] == "append":
        back = token + 2 * hkv * dim * 2 if case["dtype"] == "q4" else 0  # the rows are read back
        return {"bytes": total * (2 * hkv * dim * act + token + 2 * hq * dim * act + back), "flops": 3 * total * (hq + hkv) * case["rot"]}
    if case["op"] == "read":
        return {"bytes": total * (token + 2 * hkv * dim * 2), "flops": 2 * total * 2 * hkv * dim}
    w, s = case["window"], case["sinks"]
    keys = products = 0
    for n, r in zip(lens, rows):
        low = max(0, n - r - w + 1) if w else 0
        keys += n - low + min(s, low)
        for p in range(n - r, n):
            first = max(0, p - w + 1) if w else 0
            products += p + 1 - first + min(s, first)
    return {"bytes": keys * token + keys // case["page"] * 4 + total * hq * 2 * dim * act, "flops": 4 * dim * hq * products}


# ---------------------------------------------------------------- the definitions in 64 bits


def _turn64(case, x, pos):
    """Each pair as a complex number, turned."""
    inv, magnitude = frequencies(case)
    rot = case["rot"]
    x = x.double()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + rot // 2)
    turn = torch.polar(torch.full((), magnitude, dtype=torch.float64, device="cuda").expand(len(pos), rot // 2),
                       pos.double()[:, None] * torch.tensor(inv, dtype=torch.float64, device="cuda"))
    z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _stored64(x):
    """What rows are after 4 bits, in 64."""
    b = x.double().unflatten(-1, (-1, 32))
    low, high = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
    m, s = low.half().double(), ((high - low) / 15).half().double()
    c = ((b - m) / s).nan_to_num(0.0, 0.0, 0.0).round().clamp(0, 15)
    return (c * s + m).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    lens, rows = sizes(case)
    dim, hkv, hq = case["dim"], case["hkv"], case["hq"]
    if case["op"] == "rotate":
        return {"out": _turn64(case, st["x"], st["positions"])}
    page = case["page"]
    places = [(i, n - r + j) for i, (n, r) in enumerate(zip(lens, rows)) for j in range(r)]
    seq, pos = (torch.tensor(x, device="cuda") for x in zip(*places))
    if case["op"] == "append":
        ids, slot = st["table"][seq, pos // page].long(), pos % page
        q, k, v = _turn64(case, st["q"], pos), _turn64(case, st["k_new"], pos), st["v_new"].double()
        if case["dtype"] == "f32":
            kk, vv = st["k"].double(), st["v"].double()
            kk[ids, :, slot], vv[ids, :, slot] = k, v
            return {"q": q, "k": kk, "v": vv}
        k = k.bfloat16().double()
        if case["dtype"] == "q4":
            return {"q": q, "k": _stored64(k), "v": _stored64(v)}
        if case["dtype"] == "bf16":
            kk, vv = st["k"].double(), st["v"].double()
            kk[ids, :, slot], vv[ids, :, slot] = k, v
            return {"q": q, "k": kk, "v": vv}
        got, scale = [], st["scale"].clone()
        for which, (to, x) in enumerate(((st["k"], k), (st["v"], v))):
            sc = (x.abs().amax(-1) / 448).float().half()
            to = to.view(torch.uint8).clone()
            to[ids, :, slot] = (x / sc.double()[..., None]).nan_to_num(0.0).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
            scale[ids, :, slot, which] = sc
            got.append(to.view(torch.float8_e4m3fn))
        return {"q": q, "k": got[0], "v": got[1], "scale": scale}

    def values(i, n, h):
        """K and V of a sequence's first n tokens of one head, value by value."""
        pages = st["table"][i, :-(-n // page)].long()
        c = torch.arange(dim, device="cuda")
        g, unit = c // 32, (c % 32) // 4 * (dim // 32) + c // 32
        byte, shift = 2 * unit + (c % 4) // 2, 4 * (c % 2)
        pair = st["scale"][pages][:, h].reshape(-1, dim // 8)[:n].double()
        for which, x in enumerate((st["k"], st["v"])):
            code = (x[pages][:, h].reshape(-1, dim // 2)[:n][:, byte].int() >> shift) & 15
            at = which * dim // 16 + 2 * g
            yield code.double() * pair[:, at] + pair[:, at + 1]

    if case["op"] == "read":
        got = [[list(values(i, n, h)) for h in range(hkv)] for i, n in enumerate(lens)]
        pick = lambda which: torch.cat([torch.stack([got[i][h][which][n - r:] for h in range(hkv)], 1) for i, (n, r) in enumerate(zip(lens, rows))])  # noqa: E731
        return {"k": pick(0), "v": pick(1)}
    out, at = [], 0
    for i, (n, r) in enumerate(zip(lens, rows)):
        q = st["q"][at:at + r].double()
        at += r
        p = torch.arange(n - r, n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None, :]
        ok = t <= p
        if case["window"]:
            ok &= (t + case["window"] > p) | (t < case["sinks"])
        heads = []
        for h in range(hkv):
            k, v = values(i, n, h)
            g = hq // hkv
            z = torch.einsum("rgd,td->rgt", q[:, h * g:(h + 1) * g], k) * dim ** -0.5
            heads.append(torch.einsum("rgt,td->rgd", torch.softmax(z.masked_fill(~ok[:, None, :], -math.inf), -1), v))
        out.append(torch.cat(heads, 1))
    return {"out": torch.cat(out)}
