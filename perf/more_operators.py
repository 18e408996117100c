"""More of the attention half's operators: inputs, one pass of each, and what a pass has to move and compute.

    norm_write     RMS norms of the query and key heads and rotary positions on fresh rows, q handed on, k and v written
                   into a paged cache
    chunk          the last tokens of every sequence over the paged cache that holds them already: proposed tokens that
                   are verified, prompts that arrive in pieces; causal, over everything before or over a sliding window
                   and a few first tokens that stay visible
    decode_window  one new token of every sequence over a sliding window and a few first tokens of the paged cache

A cache is k_pages [pages][kv heads][slots][d] and v_pages [pages][kv heads][d][slots], in bf16, fp16, or int8 with one
fp32 step for every token and head ([pages][kv heads][slots]).  A sequence's pages are named by its row of the block
table; with a window, pages that no query can see any more have been given back, and their entries are -1.  With own =
False a pass is plain torch arithmetic in 32 bits; with own = True it makes the package's calls.  exact() gives the same
outputs from the definitions in 64 bits."""
import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
SIZES = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}
EPS = 1e-6


# ------------------------------------------------------------------- cases ----

def _write(name, *, tokens, hq, hkv, d, src, q, cache, page, rot, mix):
    return {"name": name, "op": "norm_write", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "src": src, "q": q,
            "cache": cache, "page": page, "rot": rot, "mix": mix}


def _chunk(name, *, batch, new, context, hq, hkv, d, q, cache, page, mix, window=0, sinks=0):
    return {"name": name, "op": "chunk", "batch": batch, "new": new, "context": context, "hq": hq, "hkv": hkv, "d": d,
            "q": q, "cache": cache, "page": page, "window": window, "sinks": sinks, "mix": mix}


def _decode(name, *, batch, low, high, hq, hkv, d, q, cache, page, window, sinks, mix):
    return {"name": name, "op": "decode_window", "batch": batch, "low": low, "high": high, "hq": hq, "hkv": hkv, "d": d,
            "q": q, "cache": cache, "page": page, "window": window, "sinks": sinks, "mix": mix}


def listed():
    return [
        # the single-token step of one conversation: fp32 rows from the decode matvecs, nothing but latency
        _write("norm_write_one_token", tokens=1, hq=40, hkv=8, d=128, src="f32", q="f32", cache="bf16", page=64,
               rot=128, mix=1),
        # a middling batch of short prompts, 16-bit rows, narrow heads of which half turns, small pages
        _write("norm_write_d64", tokens=777, hq=14, hkv=2, d=64, src="bf16", q="bf16", cache="bf16", page=16, rot=32,
               mix=2),
        # packed prompts behind the prefill projections, 256-wide heads of which a quarter turns
        _write("norm_write_prompts_d256", tokens=8191, hq=24, hkv=4, d=256, src="f32", q="bf16", cache="bf16", page=64,
               rot=64, mix=3),
        # five proposed tokens of one conversation, verified at once: latency
        _chunk("chunk_verify_one", batch=1, new=5, context=700, hq=40, hkv=8, d=128, q="bf16", cache="bf16", page=64,
               mix=4),
        # the same for a serving batch with long contexts: a few rows for every key, so the cache's bytes count
        _chunk("chunk_verify_batch", batch=32, new=8, context=8000, hq=32, hkv=8, d=128, q="bf16", cache="bf16",
               page=16, mix=5),
        # pieces of long prompts: a few hundred new tokens each behind thousands, over an 8-bit cache
        _chunk("chunk_prefill_i8", batch=8, new=512, context=12000, hq=40, hkv=8, d=128, q="bf16", cache="i8", page=64,
               mix=6),
        # one large piece of one very long document: matrix work
        _chunk("chunk_long", batch=1, new=4096, context=28000, hq=40, hkv=8, d=128, q="bf16", cache="bf16", page=64,
               mix=7),
        # wide heads, few key heads, fp16
        _chunk("chunk_d256_f16", batch=4, new=700, context=4000, hq=24, hkv=4, d=256, q="f16", cache="f16", page=32,
               mix=8),
        # pieces of prompts in a layer with a sliding window
        _chunk("window_chunk", batch=3, new=2000, context=20000, hq=32, hkv=8, d=128, q="bf16", cache="bf16", page=64,
               window=1024, sinks=4, mix=9),
        # a windowed layer's step of one conversation, fp32 activations throughout: latency
        _decode("window_decode_one", batch=1, low=9001, high=9001, hq=40, hkv=8, d=128, q="f32", cache="bf16", page=64,
                window=1024, sinks=4, mix=10),
        # the same for a serving batch with lengths from a few tokens to the limit
        _decode("window_decode_batch", batch=64, low=3, high=131072, hq=32, hkv=8, d=128, q="bf16", cache="bf16",
                page=16, window=4096, sinks=4, mix=11),
        # a large batch of a small model over an 8-bit cache, a window that is no multiple of anything
        _decode("window_decode_i8_d64", batch=200, low=1, high=20000, hq=14, hkv=2, d=64, q="f32", cache="i8", page=16,
                window=700, sinks=33, mix=12),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 5, 6, 7, 8])
    d = rng.choice([64, 128, 256])
    heads = {"hq": hkv * group, "hkv": hkv, "d": d}
    page = rng.choice([16, 32, 64, 128, 256])
    mix = rng.randrange(1 << 30)
    op = rng.choice(["norm_write", "chunk", "chunk", "chunk", "decode_window", "decode_window"])
    sixteen = rng.choice(["bf16", "f16"])
    cache = rng.choice([sixteen, sixteen, "i8"])
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, _log(rng, 1, 200)])
    if op == "norm_write":
        case = _write("", tokens=_log(rng, 1, 8000), src=rng.choice(["f32", "f32", sixteen]),
                      q=rng.choice([sixteen, "f32"]), cache=sixteen, page=page, rot=rng.choice([0, d // 4, d // 2, d]),
                      mix=mix, **heads)
    elif op == "chunk":
        batch = _log(rng, 1, 32)
        if rng.random() < 0.6:
            window, sinks = 0, 0
        case = _chunk("", batch=batch, new=_log(rng, 1, 2000 // batch), context=_log(rng, 1, min(12000, 128000 // batch)),
                      q=sixteen, cache=cache, page=page, window=window, sinks=sinks, mix=mix, **heads)
    else:
        batch = _log(rng, 1, 200)
        high = _log(rng, 1, 131072)
        case = _decode("", batch=batch, low=_log(rng, 1, high), high=high, q=rng.choice([sixteen, "f32"]), cache=cache,
                       page=page, window=max(1, min(window, 262144 // batch)), sinks=sinks, mix=mix, **heads)
    del case["name"]
    return case


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every sequence; of single tokens: lengths spread over [low, high]
    on a logarithmic scale, the first one the longest."""
    rng = random.Random(case["mix"])
    if case["op"] == "decode_window":
        lens = [_log(rng, case["low"], case["high"]) for _ in range(case["batch"])]
        lens[0] = case["high"]
        return [1] * case["batch"], lens
    new = [rng.randint(max(1, case["new"] // 2), case["new"]) for _ in range(case["batch"])]
    old = [rng.randint(case["context"] // 2, case["context"]) for _ in range(case["batch"])]
    new[0] = case["new"]
    return new, [a + b for a, b in zip(new, old)]


def _hidden(case, new, length):
    """The tokens [first, end) of a sequence that none of its queries sees."""
    if not case["window"]:
        return 0, 0
    end = max(0, length - new - case["window"] + 1)
    return min(case["sinks"], end), end


def _pairs(case, new, length):
    """Query-key pairs that see each other."""
    total = 0
    for p in range(length - new, length):
        lo = max(0, p + 1 - case["window"]) if case["window"] else 0
        total += p + 1 - lo + min(case["sinks"], lo)
    return total


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    cell = d * SIZES[case["cache"]] + (4 if case["cache"] == "i8" else 0)
    if case["op"] == "norm_write":
        n, rot = case["tokens"], case["rot"]
        moved = n * ((hq + 2 * hkv) * d * SIZES[case["src"]] + hq * d * SIZES[case["q"]] + 2 * hkv * cell + 8)
        moved += n * rot * 4 + (n * 4 if rot else 0) + 2 * d * 4
        return {"bytes": moved, "flops": n * (hq + hkv) * (3 * rot + 4 * d)}
    new, lens = _lengths(case)
    seen = pairs = 0
    for a, n in zip(new, lens):
        first, end = _hidden(case, a, n)
        seen += n - (end - first)
        pairs += _pairs(case, a, n)
    return {"bytes": 2 * seen * hkv * cell + 2 * sum(new) * hq * d * SIZES[case["q"]], "flops": 4 * hq * d * pairs}


# ------------------------------------------------------------------ inputs ----

def _channels(gen, d):
    """A gain for every dimension of a head: a few of them several times the others, as trained keys have."""
    gain = torch.ones(d, device=DEVICE)
    gain[torch.randperm(d, generator=gen, device=DEVICE)[: max(1, d // 32)]] = 4.0
    return gain


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _quantised(x, dim):
    """int8 codes and fp32 steps of x along dim (one step for every token and head)."""
    top = x.abs().amax(dim=dim, keepdim=True)
    return torch.round(x * (127.0 / top)).to(torch.int8), (top / 127.0).squeeze(dim)


def _filled_cache(gen, case, pages):
    hkv, d, page = case["hkv"], case["d"], case["page"]
    k = _normal(gen, pages, hkv, page, d) * _channels(gen, d)
    v = _normal(gen, pages, hkv, d, page)
    if case["cache"] == "i8":
        k, ks = _quantised(k, 3)
        v, vs = _quantised(v, 2)
        return {"k": k, "v": v, "ks": ks, "vs": vs}
    dtype = DTYPES[case["cache"]]
    return {"k": k.to(dtype), "v": v.to(dtype), "ks": None, "vs": None}


def _tables(gen, held, page, spare):
    """Pages in a random order for the tokens [0, first) and [end, length) of every sequence of `held`, -1 for those in
    between that hold neither, and the number of pages of the cache."""
    rows = []
    for first, end, n in held:
        pages = max(1, -(-n // page))
        rows.append([not (-(-first // page) <= i < end // page) for i in range(pages)])
    total = sum(sum(r) for r in rows) + spare
    order = torch.randperm(total, generator=gen, device=DEVICE).to(torch.int32)
    width = max(len(r) for r in rows)
    mask = torch.tensor([r + [False] * (width - len(r)) for r in rows], device=DEVICE)
    table = torch.full(mask.shape, -1, dtype=torch.int32, device=DEVICE)
    table[mask] = order[: total - spare]
    return table, total


def _cumulated(lens):
    at, out = 0, [0]
    for n in lens:
        at += n
        out.append(at)
    return torch.tensor(out, dtype=torch.int32, device=DEVICE)


def _rope_table(positions, rot):
    """[positions][rot]: rot / 2 cosines, then rot / 2 sines."""
    half = rot // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEVICE) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=DEVICE)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32)


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed * 7919 + 17)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = {"case": case}
    if case["op"] == "norm_write":
        # whole prompts, each from its first position: about 1500 tokens apiece; a single token stands behind others
        page, tokens = case["page"], case["tokens"]
        new = [min(1500, tokens - at) for at in range(0, tokens, 1500)]
        lens = new if tokens > 1 else [777]
        table, pages = _tables(gen, [(0, 0, n) for n in lens], page, 3)
        positions = torch.cat([torch.arange(n - m, n, device=DEVICE) for m, n in zip(new, lens)])
        rows = torch.repeat_interleave(torch.arange(len(new), device=DEVICE), torch.tensor(new, device=DEVICE))
        s["slots"] = table[rows, positions // page].to(torch.int64) * page + positions % page
        s["positions"] = positions.to(torch.int32)
        s["rope"] = _rope_table(max(lens), case["rot"]) if case["rot"] else None
        # the stacked projection's rows, q, k and v views of them: magnitudes differ from token to token and head to
        # head, and a few channels stand out
        x = _normal(gen, tokens, hq + 2 * hkv, d)
        x *= torch.exp(_normal(gen, tokens, hq + 2 * hkv, 1))
        x[:, :hq + hkv] *= _channels(gen, d)
        x = x.to(DTYPES[case["src"]])
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        s["q_gain"], s["k_gain"] = (1.0 + 0.3 * _normal(gen, d) for _ in range(2))
        s["cache"] = _filled_cache(gen, case, pages)
        return s
    new, lens = _lengths(case)
    held = [_hidden(case, a, n) + (n,) for a, n in zip(new, lens)]
    s["table"], pages = _tables(gen, held, case["page"], 3)
    s["cache"] = _filled_cache(gen, case, pages)
    s["q"] = _normal(gen, sum(new), hq, d).to(DTYPES[case["q"]])
    s["new"], s["lens"] = new, lens
    s["cu"] = _cumulated(new)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import ternary_weight_ptq1_amd as P

        c = s["cache"]
        s["kv"] = P.KvCache(c["k"], c["v"], c["ks"], c["vs"])
    return s


# ----------------------------------------------------------- the plain form ----

def _normed(x, gain):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * gain


def _turned(x, positions, table):
    """Rotary positions on the first rot dimensions of x [tokens][heads][d]."""
    if table is None:
        return x
    half = table.shape[1] // 2
    row = table[positions.long()][:, None]
    cos, sin = row[..., :half], row[..., half:]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], dim=-1)


def _plain_write(s):
    case, cache = s["case"], s["cache"]
    q = _turned(_normed(s["q"], s["q_gain"]), s["positions"], s["rope"]).to(DTYPES[case["q"]])
    k = _turned(_normed(s["k"], s["k_gain"]), s["positions"], s["rope"])
    at, off = s["slots"] // case["page"], s["slots"] % case["page"]
    cache["k"][at, :, off] = k.to(cache["k"].dtype)
    cache["v"][at, :, :, off] = s["v"].to(cache["v"].dtype)
    return q, cache["k"], cache["v"]


def _plain_attention(s):
    """Sequences side by side, padded to the longest, as many at once as fit; of every sequence only the tokens that some
    query sees."""
    case, cache = s["case"], s["cache"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group, window, sinks = hq // hkv, case["window"], case["sinks"]
    lens, cu = s["seq_lens"].long(), s["cu"].long()
    new, cu = cu[1:] - cu[:-1], cu[:-1]
    hidden = [_hidden(case, a, n) for a, n in zip(s["new"], s["lens"])]
    most_new, most = max(s["new"]), max(n - (e - f) for (f, e), n in zip(hidden, s["lens"]))
    first = torch.tensor([f for f, _ in hidden], device=DEVICE)
    end = torch.tensor([e for _, e in hidden], device=DEVICE)
    out = torch.empty_like(s["q"])
    at_once = max(1, (1 << 28) // (most * hkv * d))
    rows = max(1, (1 << 29) // (min(at_once, len(s["lens"])) * hq * most))
    place = torch.arange(most, device=DEVICE)
    for b in range(0, len(s["lens"]), at_once):
        n, f, e = lens[b:b + at_once, None], first[b:b + at_once, None], end[b:b + at_once, None]
        tok = torch.where(place < f, place, place + (e - f))
        is_tok = tok < n
        at = torch.where(is_tok, tok, n - 1)
        pg, off = s["table"][b:b + at_once].gather(1, at // page).long(), at % page
        k, v = cache["k"][pg, :, off].float(), cache["v"][pg, :, :, off].float()
        if cache["ks"] is not None:
            k, v = k * cache["ks"][pg, :, off][..., None], v * cache["vs"][pg, :, off][..., None]
        k, v = k.permute(0, 2, 3, 1).contiguous(), v.transpose(1, 2).contiguous()
        for r in range(0, most_new, rows):
            i = torch.arange(r, min(most_new, r + rows), device=DEVICE)
            is_row = i < new[b:b + at_once, None]
            row = torch.where(is_row, cu[b:b + at_once, None] + i, 0)
            q = s["q"][row].float().view(row.shape[0], len(i), hkv, group, d).permute(0, 2, 3, 1, 4)
            q = q.reshape(row.shape[0], hkv, group * len(i), d)
            scores = torch.matmul(q, k).mul_(d ** -0.5).view(row.shape[0], hkv, group, len(i), most)
            p = (n - new[b:b + at_once, None] + i)[..., None]
            t = tok[:, None]
            seen = is_tok[:, None] & (t <= p)
            if window:
                seen &= (t > p - window) | (t < sinks)
            scores.masked_fill_(~seen[:, None, None], float("-inf"))
            w = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
            w /= w.sum(dim=-1, keepdim=True)
            o = torch.matmul(w.view(row.shape[0], hkv, group * len(i), most), v)
            o = o.view(row.shape[0], hkv, group, len(i), d).permute(0, 3, 1, 2, 4).reshape(row.shape[0], len(i), hq, d)
            out[row[is_row]] = o[is_row].to(out.dtype)
    return out


# ---------------------------------------------------------------- one pass ----

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import ternary_weight_ptq1_amd as P

        if op == "norm_write":
            q = P.ptq1_kv_write_norm(s["q"], s["k"], s["v"], s["slots"], s["kv"], q_gain=s["q_gain"],
                                     k_gain=s["k_gain"], eps=EPS, positions=s["positions"], cos_sin=s["rope"],
                                     q_dtype=DTYPES[case["q"]])
            return q, s["cache"]["k"], s["cache"]["v"]
        if op == "chunk":
            return P.ptq1_attn_chunk(s["q"], s["kv"], s["table"], s["cu"], s["seq_lens"], window=case["window"],
                                     sinks=case["sinks"], max_q=case["new"],
                                     max_len=min(case["new"] + case["context"], s["table"].shape[1] * case["page"]))
        return P.ptq1_attn_decode_window(s["q"], s["kv"], s["table"], s["seq_lens"], window=case["window"],
                                         sinks=case["sinks"], max_len=case["high"])
    if op == "norm_write":
        return _plain_write(s)
    return _plain_attention(s)


# ------------------------------------------------------- the definitions ----

def _exact_norm_turn(x, gain, positions, table):
    x = x.double()
    x = x / torch.sqrt((x ** 2).sum(dim=2, keepdim=True) / x.shape[2] + EPS) * gain.double()
    if table is not None:
        half = table.shape[1] // 2
        for at in range(half):
            c, sn = table[positions.long(), at].double()[:, None], table[positions.long(), half + at].double()[:, None]
            a, b = x[:, :, at].clone(), x[:, :, half + at].clone()
            x[:, :, at] = a * c - b * sn
            x[:, :, half + at] = a * sn + b * c
    return x


def exact(case, seed):
    s = _inputs(case, seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    cache = s["cache"]
    if case["op"] == "norm_write":
        k, v = cache["k"].double(), cache["v"].double()
        at, off = torch.div(s["slots"], page, rounding_mode="floor"), s["slots"] % page
        k[at, :, off] = _exact_norm_turn(s["k"], s["k_gain"], s["positions"], s["rope"])
        v[at, :, :, off] = s["v"].double()
        return _exact_norm_turn(s["q"], s["q_gain"], s["positions"], s["rope"]), k, v
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    first = 0
    for b, (m, n) in enumerate(zip(s["new"], s["lens"])):
        # the oldest query's window begins here (0: everything is seen)
        lo = max(0, n - m + 1 - case["window"]) if case["window"] else 0
        tok = torch.arange(n, device=DEVICE)
        tok = tok[(tok >= lo) | (tok < case["sinks"])]
        pg, off = s["table"][b, torch.div(tok, page, rounding_mode="floor")].long(), tok % page
        p = torch.arange(n - m, n, device=DEVICE).repeat_interleave(group)
        for h in range(hkv):
            k, v = cache["k"][pg, h, off].double(), cache["v"][pg, h, :, off].double()
            if cache["ks"] is not None:
                k *= cache["ks"][pg, h, off].double()[:, None]
                v *= cache["vs"][pg, h, off].double()[:, None]
            q = s["q"][first:first + m, h * group:(h + 1) * group].reshape(m * group, d).double()
            rows = max(1, (1 << 27) // len(tok))
            for r in range(0, m * group, rows):
                logits = q[r:r + rows] @ k.T.contiguous() / math.sqrt(d)
                at = p[r:r + rows, None]
                away = tok[None] > at
                if case["window"]:
                    away |= (at - tok[None] >= case["window"]) & (tok[None] >= case["sinks"])
                logits[away] = -math.inf
                o = torch.softmax(logits, dim=1) @ v
                i = torch.arange(r, min(m * group, r + rows), device=DEVICE)
                out[first + torch.div(i, group, rounding_mode="floor"), h * group + i % group] = o
        first += m
    return out
