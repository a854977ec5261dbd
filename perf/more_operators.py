"""What is measured of the paged cache's serving forms: their cases, inputs, plain forms and exact values.

A paged cache holds one key row of d elements a position, shared by all heads; a row's first dv elements are also the
value.  `cache` is [pages, page_size, d], either bf16, or e4m3 codes with one fp32 scale (a power of two) for each run
of 128 elements of a row (`scales` [pages, page_size, ceil(d / 128)]).  `page_table` int32 [b, max_pages] names the
pages of each of b sequences in order; row r of a call belongs to sequence r // (rows // b).  The three operators:

  append  new rows [tokens, d] go into the cache at their positions (negative: a padding token, skipped), the
          elements `first` .. of each row rotated by the position's angles on the way: pairs (x, y) become
          (x cos - y sin, y cos + x sin), either neighbours or elements half of the rotated run apart; the same
          tokens' queries [tokens, h, d], where there are any, are rotated alike and returned in bf16 (a padding
          token's unrotated).  `rotation` fp32 [positions, rot] holds rot / 2 cosines, then rot / 2 sines, a row
          a position
  window  softmax(scale * q k^T) v over the last `window` positions below the row's exclusive end and the first
          `sinks` ones
  shared  the same over every position below the row's end, where the first `shared` positions are the same rows
          for all sequences (one long prefix, its pages in every sequence's table)

A row without positions gives zeros and a log-sum of -inf.
"""
import math

import torch

own = False

GROUP = 128          # elements of a row that share a scale
E4M3_MAX = 448.0
DEVICE = "cuda"

# Sizes are this repository's own (keys of 128, 192 and 512 elements, 64 heads, chunks of 701, 1024 and 4096 rows,
# contexts of 1000, 16384 and 204800), and generic ones around them.
_LISTED = [
    # one serving step: each of 32 sequences appends a token and has its queries rotated (latency counts)
    {"name": "append_step_32_h64_d512_fp8", "op": "append", "tokens": 32, "b": 32, "ctx": 16384, "d": 512, "rot": 64,
     "pairs": "halves", "h": 64, "src": "bf16", "cache": "fp8", "page": 32},
    # a prompt of 16384 tokens goes into an 8-bit cache, its queries elsewhere
    {"name": "append_prompt_16384_d512_fp8", "op": "append", "tokens": 16384, "b": 1, "ctx": 16384, "d": 512,
     "rot": 64, "pairs": "neighbours", "h": 0, "src": "bf16", "cache": "fp8", "page": 32},
    # chunks of three sequences with their queries, keys rotated whole, odd sizes, fp32 activations
    {"name": "append_chunk_3x1367_h24_d192", "op": "append", "tokens": 4101, "b": 3, "ctx": 5000, "d": 192,
     "rot": 192, "pairs": "halves", "h": 24, "src": "f32", "cache": "bf16", "page": 24},
    # a batch of chunks with the queries of 16 heads: the bandwidth of the card
    {"name": "append_batch_8x1024_h16_d512_fp8", "op": "append", "tokens": 8192, "b": 8, "ctx": 16384, "d": 512,
     "rot": 64, "pairs": "halves", "h": 16, "src": "bf16", "cache": "fp8", "page": 64},
    # one token of one sequence with a short window: the latency of a step
    {"name": "window_token_1x1000_d128", "op": "window", "rows": 1, "b": 1, "ctx": 1000, "window": 512, "sinks": 4,
     "h": 64, "d": 128, "dv": 128, "cache": "bf16", "page": 16, "lse": True},
    # one token of each of 32 sequences, contexts of up to 204800 positions of which a window is kept visible
    {"name": "window_step_32x204800_d512_fp8", "op": "window", "rows": 32, "b": 32, "ctx": 204800, "window": 4096,
     "sinks": 16, "h": 64, "d": 512, "dv": 512, "cache": "fp8", "page": 32, "lse": False},
    # a prompt's chunk of 1024 rows behind a long context
    {"name": "window_chunk_1024_h64_d512", "op": "window", "rows": 1024, "b": 1, "ctx": 16384, "window": 1024,
     "sinks": 4, "h": 64, "d": 512, "dv": 512, "cache": "bf16", "page": 16, "lse": False},
    # chunks of three sequences, fewer heads, odd sizes, padding rows
    {"name": "window_chunk_3x701_h24_d192", "op": "window", "rows": 2103, "b": 3, "ctx": 5000, "window": 1000,
     "sinks": 7, "h": 24, "d": 192, "dv": 128, "cache": "bf16", "page": 24, "lse": True},
    # one token of each of 4 sequences behind a short prefix: the latency of a step
    {"name": "shared_token_4x700_h16_d128", "op": "shared", "rows": 4, "b": 4, "shared": 688, "ctx": 100, "h": 16,
     "d": 128, "dv": 128, "cache": "bf16", "page": 16, "lse": True},
    # a batch of 64 sequences behind one prefix of 16384 positions, 8 bits
    {"name": "shared_step_64x16384_h16_d512_fp8", "op": "shared", "rows": 64, "b": 64, "shared": 16384, "ctx": 700,
     "h": 16, "d": 512, "dv": 512, "cache": "fp8", "page": 32, "lse": False},
    # samples drawn from one long document: 48 sequences, 204800 positions in common
    {"name": "shared_step_48x204800_h8_d128", "op": "shared", "rows": 48, "b": 48, "shared": 204800, "ctx": 2048,
     "h": 8, "d": 128, "dv": 128, "cache": "bf16", "page": 128, "lse": False},
    # a few new tokens of each of 16 sequences (drafts to be verified) behind a common prefix
    {"name": "shared_draft_16x5_h8_d320", "op": "shared", "rows": 80, "b": 16, "shared": 30000, "ctx": 1001, "h": 8,
     "d": 320, "dv": 256, "cache": "bf16", "page": 48, "lse": True},
]


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    most = {op: max(_cost(c) for c in _LISTED if c["op"] == op) for op in ("append", "window", "shared")}
    most_values = 2 ** 31  # fp32 values of the widest intermediate of a plain form
    while True:
        op = rng.choice(("append", "window", "window", "shared", "shared"))
        cache = rng.choice(("bf16", "fp8"))
        page = rng.choice((1, 8, 16, 24, 32, 48, 100, 128, 256))
        d = rng.choice((16, 64, 80, 96, 128, 128, 192, 256, 272, 320, 512, 512))
        h = rng.choice((1, 2, 4, 5, 8, 16, 24, 32, 48, 64, 96, 128))
        if op == "append":
            per, b = _log(rng, 1, 20000), _log(rng, 1, 64)
            c = {"op": op, "tokens": per * b, "b": b, "ctx": _log(rng, per, max(per, 204800)), "d": d,
                 "rot": rng.choice([r for r in (16, 32, 64, 80, 128, d) if r <= d]),
                 "pairs": rng.choice(("halves", "neighbours")), "h": h if rng.random() < 0.6 else 0,
                 "src": rng.choice(("bf16", "f32")), "cache": cache, "page": page}
            if b * (c["ctx"] + page) * d > most_values // 4 or c["tokens"] * d * max(1, c["h"]) > most_values // 4:
                continue
        else:
            per = 1 if rng.random() < 0.5 else _log(rng, 1, 2048)
            dv = d if rng.random() < 0.6 else max(8, (d // 2 + 7) // 8 * 8)
            b = _log(rng, 1, 128)
            c = {"op": op, "rows": per * b, "b": b, "h": h, "d": d, "dv": dv, "cache": cache, "page": page,
                 "lse": rng.random() < 0.5}
            if op == "window":
                c |= {"ctx": _log(rng, per, max(per, 204800)), "window": _log(rng, 1, 8192),
                      "sinks": rng.choice((0, 1, 4, 16, 128, 200))}
                seen, held = min(c["ctx"], c["window"] + per), c["ctx"]
            else:
                c |= {"ctx": _log(rng, per, max(per, 8192)), "shared": _log(rng, 1, 204800) // page * page}
                seen, held = c["shared"] + c["ctx"], c["shared"] // b + c["ctx"]
            if c["rows"] > 8192 or b * held * d > most_values // 2 or c["rows"] * h * seen > most_values // 2:
                continue
            if c["rows"] * h * d > most_values // 8 or b * (seen if op == "window" else c["ctx"]) * d > most_values // 4:
                continue
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------------------------------------ shapes
def _lengths(case):
    """Positions of each sequence (behind the shared ones), its new tokens among them: they differ, the first is the
    longest; and its padding rows, the last ones of every second sequence's chunk."""
    per = case["rows" if case["op"] != "append" else "tokens"] // case["b"]
    out = []
    for s in range(case["b"]):
        ctx = max(per, case["ctx"] - (s * 613) % (case["ctx"] // 2 + 1))
        out.append((ctx, min(per // 4, 5) if s % 2 else 0))
    return per, out


def _ends(case):
    """Exclusive end of each row's positions, causal within a sequence's chunk; 0 for padding."""
    per, lengths = _lengths(case)
    ends = []
    for ctx, pad in lengths:
        live = per - pad
        ends += [case.get("shared", 0) + ctx - live + i + 1 if i < live else 0 for i in range(per)]
    return ends


def _positions(case):
    """Position of each token, -1 for padding."""
    return [e - 1 for e in _ends(case)]


def _capacity(case):
    """Columns of the page table."""
    return -(-(case.get("shared", 0) + max(ctx for ctx, _ in _lengths(case)[1])) // case["page"])


def _spans(case):
    """Of each sequence the positions from `lo` on that its rows see besides the sinks, and their exclusive end."""
    per, lengths = _lengths(case)
    out = []
    for ctx, pad in lengths:
        first = ctx - (per - pad) + 1  # the first row's end
        out.append((max(0, first - case["window"]), ctx))
    return out


def work(case):
    d = case["d"]
    groups = -(-d // GROUP)
    row = d + 4 * groups if case["cache"] == "fp8" else 2 * d
    per, lengths = _lengths(case)
    if case["op"] == "append":
        src = 4 if case["src"] == "f32" else 2
        live = sum(per - pad for _, pad in lengths)
        marks, angles, upto = sorted((ctx - (per - pad), ctx) for ctx, pad in lengths), 0, 0
        for lo, hi in marks:  # distinct positions: a row of the table each
            angles += max(0, hi - max(lo, upto))
            upto = max(upto, hi)
        queries = case["tokens"] * case["h"] * d * (src + 2)
        # a product and a sum for each of a pair's two values, counted for rows and queries
        return {"bytes": live * (d * src + row) + 4 * case["tokens"] + 4 * case["rot"] * angles + queries,
                "flops": 3 * case["rot"] * live * (1 + case["h"])}
    ends = _ends(case)
    if case["op"] == "window":
        w, k = case["window"], case["sinks"]
        taken = sum(min(e, w) + min(max(0, e - w), k) for e in ends)
        distinct = sum(hi - lo + min(lo, k) for lo, hi in _spans(case))
    else:
        taken = sum(ends)
        distinct = case["shared"] + sum(ctx for ctx, _ in lengths)
    small = 4 * case["rows"] + (4 * case["rows"] * case["h"] if case["lse"] else 0)
    return {"bytes": distinct * row + case["rows"] * case["h"] * 2 * (d + case["dv"]) + small,
            "flops": taken * case["h"] * 2 * (d + case["dv"])}


# ------------------------------------------------------------------------------------------------ inputs
def _values(shape, gen):
    """Activations: normal, with runs of a row at different magnitudes."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    runs = -(-shape[-1] // GROUP)
    size = torch.exp(0.5 * torch.randn((*shape[:-1], runs), generator=gen, device=DEVICE))
    return x.mul_(size.repeat_interleave(GROUP, dim=-1)[..., : shape[-1]])


def _fill_cache(case, pages, gen):
    """A cache in use: every row written."""
    shape = (pages, case["page"], case["d"])
    if case["cache"] == "bf16":
        return _values(shape, gen).to(torch.bfloat16), None
    runs = -(-case["d"] // GROUP)
    power = torch.randint(-9, -6, (pages, case["page"], runs), generator=gen, device=DEVICE)
    scales = ((power + 127) << 23).to(torch.int32).view(torch.float32)  # 2^power, from its bits
    codes = torch.randn(shape, generator=gen, device=DEVICE).mul_(110).clamp_(-E4M3_MAX, E4M3_MAX)
    return codes.to(torch.float8_e4m3fn), scales


def _rotation(positions, rot):
    """Cosines and sines of a model's angles, formed in 64 bits (far positions lose their angle in 32)."""
    rate = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEVICE),
                     -torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    angle = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * rate
    return torch.cat((angle.cos(), angle.sin()), dim=1).float()


def prepare(case, seed):
    gen = torch.Generator(DEVICE)
    gen.manual_seed(seed)
    b, d, columns = case["b"], case["d"], _capacity(case)
    if case["op"] == "append":
        tokens = case["tokens"]
        src = torch.float32 if case["src"] == "f32" else torch.bfloat16
        pages = b * columns + 1  # the last one belongs to nobody
        state = {"case": case, "x": _values((tokens, d), gen).to(src),
                 "q": 1.5 * torch.randn((tokens, case["h"], d), generator=gen, device=DEVICE).to(src)
                 if case["h"] else None,
                 "positions": torch.tensor(_positions(case), dtype=torch.int32, device=DEVICE),
                 "page_table": torch.randperm(pages - 1, generator=gen, device=DEVICE).to(torch.int32).view(b, columns),
                 "rotation": _rotation(columns * case["page"], case["rot"]),
                 "first": d - case["rot"], "scales": None}
        state["cache"] = torch.zeros((pages, case["page"], d), dtype=torch.bfloat16, device=DEVICE)
        if case["cache"] == "fp8":
            state["cache"] = torch.zeros((pages, case["page"], d), dtype=torch.uint8,
                                         device=DEVICE).view(torch.float8_e4m3fn)
            state["scales"] = torch.ones((pages, case["page"], -(-d // GROUP)), device=DEVICE)
        return state
    common = case.get("shared", 0) // case["page"]  # whole pages
    pages = common + b * (columns - common) + 1
    cache, scales = _fill_cache(case, pages, gen)
    ids = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.cat((ids[:common].expand(b, -1), ids[common: pages - 1].view(b, columns - common)), dim=1)
    state = {"case": case, "cache": cache, "scales": scales, "page_table": table.contiguous()}
    q = 1.5 * torch.randn((case["rows"], case["h"], d), generator=gen, device=DEVICE)
    state["q"] = q.to(torch.bfloat16)
    state["end"] = torch.tensor(_ends(case), dtype=torch.int32, device=DEVICE)
    if case["op"] == "window":
        state["spans"] = torch.tensor(_spans(case), device=DEVICE)
    return state


# ------------------------------------------------------------------------------------------------ plain forms
def _rotate(x, state):
    """fp32 rows [tokens, .., d] with their run rotated; padding tokens' stay."""
    rot, first = state["case"]["rot"], state["first"]
    live = state["positions"] >= 0
    angles = state["rotation"][torch.where(live, state["positions"], 0)]
    angles = angles.view(-1, *(1,) * (x.dim() - 2), 2, rot // 2)
    live = live.view(-1, *(1,) * (x.dim() - 1))
    cos, sin = torch.where(live, angles[..., 0, :], 1.0), torch.where(live, angles[..., 1, :], 0.0)
    run = x[..., first: first + rot]
    shape = (2, rot // 2) if state["case"]["pairs"] == "halves" else (rot // 2, 2)
    at = -2 if state["case"]["pairs"] == "halves" else -1
    u, v = run.unflatten(-1, shape).unbind(at)
    turned = torch.stack((u * cos - v * sin, v * cos + u * sin), dim=at).flatten(-2)
    return torch.cat((x[..., :first], turned, x[..., first + rot:]), dim=-1)


def _quantise(x):
    """(codes, scales) of fp32 rows [..., d]: for each run of 128, the smallest power of two that brings its largest
    finite magnitude to 448 or less, and the values over it in e4m3."""
    d = x.shape[-1]
    runs = -(-d // GROUP)
    x = torch.nn.functional.pad(x, (0, runs * GROUP - d)).unflatten(-1, (runs, GROUP))
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=-1)
    mantissa, exponent = torch.frexp(amax)          # amax = mantissa * 2^exponent, 1/2 <= mantissa < 1
    power = exponent - 9 + (mantissa > 0.875).int()  # 448 = 0.875 * 2^9
    power = torch.where(amax > 0, power, -126).clamp(min=-126)
    scales = ((power + 127) << 23).to(torch.int32).view(torch.float32)  # 2^power, from its bits
    y = (x / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.flatten(-2)[..., :d].to(torch.float8_e4m3fn), scales


def _slots(state, positions):
    """Flat cache rows of positions [b, ...]."""
    page = state["case"]["page"]
    b = positions.shape[0]
    flat = positions.reshape(b, -1)
    return (torch.gather(state["page_table"].long(), 1, flat // page) * page + flat % page).view(positions.shape)


def _plain_append(state):
    cache, scales, b = state["cache"], state["scales"], state["case"]["b"]
    positions = state["positions"].long()
    live = (positions >= 0)[:, None]
    spare = cache.shape[0] * cache.shape[1] - 1  # a row of nobody's: padding writes back what it holds
    to = torch.where(live[:, 0], _slots(state, positions.clamp(min=0).view(b, -1)).flatten(), spare)
    x = _rotate(state["x"].float(), state)
    if scales is None:
        rows = cache.flatten(0, 1)
        rows[to] = torch.where(live, x.to(torch.bfloat16), rows[spare])
        got = {"cache": cache}
    else:
        codes, s = _quantise(x)
        rows, at = cache.view(torch.uint8).flatten(0, 1), scales.flatten(0, 1)
        rows[to] = torch.where(live, codes.view(torch.uint8), rows[spare])
        at[to] = torch.where(live, s, at[spare])
        got = {"cache": cache, "scales": scales}
    if state["q"] is not None:
        got["q"] = _rotate(state["q"].float(), state).to(torch.bfloat16)
    return got


def _rows32(state, slots):
    """Cache rows at flat slots, in fp32."""
    x = state["cache"].flatten(0, 1)[slots].float()
    if state["scales"] is not None:
        x *= state["scales"].flatten(0, 1)[slots].repeat_interleave(GROUP, dim=-1)[..., : x.shape[-1]]
    return x


def _outputs(case, parts):
    """Softmax over parts (scores with -inf where masked, values), and the log-sum."""
    top = torch.stack([s.amax(dim=-1, keepdim=True) for s, _ in parts]).amax(dim=0)
    top = top.clamp(min=torch.finfo(torch.float32).min)
    out = total = 0.0
    for s, v in parts:
        p = s.sub_(top).exp_()
        total = total + p.sum(dim=-1, keepdim=True)
        out = out + (p.flatten(0, 1) @ v).view(*p.shape[:2], -1) if v.dim() == 2 else out + p @ v
    out = out / torch.where(total > 0, total, 1.0)
    got = {"out": out.to(torch.bfloat16).view(case["rows"], case["h"], case["dv"])}
    if case["lse"]:
        got["lse"] = torch.where(total > 0, top + total.log(), -math.inf).view(case["rows"], case["h"])
    return got


def _plain_window(state):
    case = state["case"]
    b, h, d, dv = case["b"], case["h"], case["d"], case["dv"]
    lo, hi = state["spans"][:, :1], state["spans"][:, 1:]
    # each sequence's sinks that lie before its span, then the span, up to the longest one's length
    longest = case["sinks"] + min(case["ctx"], case["window"] + case["rows"] // b)
    at = torch.arange(longest, device=DEVICE)
    before = lo.clamp(max=case["sinks"])
    positions = torch.where(at < before, at, at - before + lo)
    known = positions < hi
    keys = _rows32(state, _slots(state, torch.where(known, positions, 0)))
    end = state["end"].view(b, -1, 1)
    p = positions[:, None, :]
    seen = (p < end) & ((p >= end - case["window"]) | (p < case["sinks"])) & known[:, None, :]
    q = state["q"].float().view(b, -1, d)
    s = torch.matmul(q, keys.transpose(1, 2)).mul_(1 / math.sqrt(d))
    s.view(b, -1, h, longest).masked_fill_(~seen[:, :, None, :], -math.inf)
    return _outputs(case, [(s, keys[..., :dv])])


def _plain_shared(state):
    case = state["case"]
    b, h, d, dv, common = case["b"], case["h"], case["d"], case["dv"], case["shared"]
    q = state["q"].float().view(b, -1, d)
    end = state["end"].view(b, -1, 1)
    parts = []
    own_at = torch.arange(common, max(common + 1, state["page_table"].shape[1] * case["page"]), device=DEVICE)
    own_at = own_at[: case["ctx"]]
    keys = _rows32(state, _slots(state, own_at.expand(b, -1)))
    s = torch.matmul(q, keys.transpose(1, 2)).mul_(1 / math.sqrt(d))
    s.view(b, -1, h, own_at.numel()).masked_fill_((own_at >= end)[:, :, None, :], -math.inf)
    parts.append((s, keys[..., :dv]))
    if common:
        at = torch.arange(common, device=DEVICE)
        keys = _rows32(state, _slots(state, at[None])[0])
        s = (q.flatten(0, 1) @ keys.T).view(b, -1, common).mul_(1 / math.sqrt(d))
        s.view(b, -1, h, common).masked_fill_((at >= end)[:, :, None, :], -math.inf)
        parts.append((s, keys[:, :dv]))
    return _outputs(case, parts)


def run(state):
    case = state["case"]
    if not own:
        return {"append": _plain_append, "window": _plain_window, "shared": _plain_shared}[case["op"]](state)
    import gather_radix_select_gb300 as sel
    if case["op"] == "append":
        q = sel.cache_append(state["x"], state["cache"], state["page_table"], state["positions"], state["rotation"],
                             scales=state["scales"], first=state["first"], interleaved=case["pairs"] == "neighbours",
                             q=state["q"])
        got = {"cache": state["cache"]}
        if state["scales"] is not None:
            got["scales"] = state["scales"]
        if q is not None:
            got["q"] = q
        return got
    seen = {"window": case["window"], "sinks": case["sinks"]} if case["op"] == "window" else {"shared": case["shared"]}
    out, lse = sel.cache_attention(state["q"], state["cache"], state["page_table"], scales=state["scales"],
                                   end=state["end"], dv=case["dv"], return_lse=case["lse"], **seen)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _power64(exponent):
    """2^exponent, from its bits (the card's exp2 and ldexp may be a rounding off)."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _turned64(case, s, x):
    """Rows [n, .., d] of live tokens at positions `at`, rotated by complex numbers of modulus about 1."""
    x, at = x
    rot, first, half = case["rot"], s["first"], case["rot"] // 2
    table = s["rotation"][at].double()
    z = torch.complex(table[:, :half], table[:, half:]).view(-1, *(1,) * (x.dim() - 2), half)
    x = x.double().clone()
    j = torch.arange(half, device=DEVICE)
    re, im = (first + j, first + half + j) if case["pairs"] == "halves" else (first + 2 * j, first + 2 * j + 1)
    w = torch.complex(x[..., re], x[..., im]) * z
    x[..., re], x[..., im] = w.real, w.imag
    return x


def _exact_append(case, s):
    d, page, b = case["d"], case["page"], case["b"]
    per = case["tokens"] // b
    where = _positions(case)
    live = torch.tensor([i for i, p in enumerate(where) if p >= 0], device=DEVICE, dtype=torch.long)
    at = torch.tensor([p for p in where if p >= 0], device=DEVICE, dtype=torch.long)
    to = s["page_table"][live // per, at // page].long() * page + at % page
    x = _turned64(case, s, (s["x"][live], at))
    rows = s["cache"].shape[0] * page
    held = torch.zeros((rows, d), dtype=torch.float64, device=DEVICE)
    got = {}
    if case["cache"] == "bf16":
        held[to] = x
    else:
        runs = -(-d // GROUP)
        scales = torch.ones((rows, runs), dtype=torch.float64, device=DEVICE)
        for g in range(runs):
            part = x[:, g * GROUP: (g + 1) * GROUP]
            mantissa, exponent = torch.frexp(part.abs().amax(dim=1) / E4M3_MAX)
            power = torch.where(mantissa > 0.5, exponent, exponent - 1)  # ceil(log2)
            scale = _power64(power.clamp(min=-126))
            y = part / scale[:, None]
            # e4m3: 3 bits behind the leading one, steps of 2^-9 below 2^-6; ties to even
            step = _power64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
            held[to, g * GROUP: g * GROUP + part.shape[1]] = torch.round(y / step) * step
            scales[to, g] = scale
        got["scales"] = scales.view(-1, page, runs)
    got = {"cache": held.view(-1, page, d), **got}
    if case["h"]:
        q = s["q"].double()
        step = max(1, 2 ** 26 // (case["h"] * d))
        for i in range(0, live.numel(), step):
            t = live[i: i + step]
            q[t] = _turned64(case, s, (s["q"][t], at[i: i + step]))
        got["q"] = q
    return got


def _exact_rows(case, s, seq, positions):
    """Rows of one sequence at a list of positions, in 64 bits."""
    page = s["page_table"][seq].long()[torch.div(positions, case["page"], rounding_mode="floor")]
    place = positions % case["page"]
    x = s["cache"][page, place].double()
    if s["scales"] is not None:
        element = torch.arange(case["d"], device=DEVICE) // GROUP
        x = x * s["scales"][page, place].double()[..., element]
    return x


def _exact_attend(case, s):
    rows, h, d, dv = case["rows"], case["h"], case["d"], case["dv"]
    per = rows // case["b"]
    out = torch.zeros((rows, h, dv), dtype=torch.float64, device=DEVICE)
    lse = torch.full((rows, h), -math.inf, dtype=torch.float64, device=DEVICE)
    ends = s["end"].tolist()
    for seq in range(case["b"]):
        for first in range(seq * per, (seq + 1) * per, 64):
            rows_now = [r for r in range(first, min(first + 64, (seq + 1) * per)) if ends[r] > 0]
            if not rows_now:
                continue
            most = max(ends[r] for r in rows_now)
            at = torch.arange(most, device=DEVICE)
            if case["op"] == "window":
                least = min(ends[r] for r in rows_now) - case["window"]
                at = at[(at < case["sinks"]) | (at >= least)]
            keys = _exact_rows(case, s, seq, at)
            step = max(1, 2 ** 27 // (at.numel() * h))
            for i in range(0, len(rows_now), step):
                r = torch.tensor(rows_now[i: i + step], device=DEVICE)
                z = torch.einsum("rhd,kd->rhk", s["q"][r].double(), keys) / math.sqrt(d)
                end = s["end"][r, None, None]
                bad = at >= end
                if case["op"] == "window":
                    bad = bad | ((at >= case["sinks"]) & (at < end - case["window"]))
                z = z.masked_fill(bad, -math.inf)
                lse[r] = torch.logsumexp(z, dim=-1)
                out[r] = torch.einsum("rhk,kd->rhd", torch.exp(z - lse[r][..., None]), keys[:, :dv])
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    # over about 20 s where 64-bit products run at about 1 TFLOP/s
    if case["op"] != "append" and work(case)["flops"] > 1.0e13:
        return None
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)
