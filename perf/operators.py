"""What is measured of the paged-cache serving operators, and their plain forms.

Three operators serve a chunk of new tokens (or a single new token) of every
sequence of a packed batch, next to keys and values that a paged cache holds:

* rope      per-head RMSNorm (optional) and rotary positions of q and k, interleaved
            or half-split pairs, over the first ``rotary`` elements of a head, with
            frequencies scaled for long contexts;
* append    the same on the way into a paged cache: q to a buffer, k rotated into the
            k pages, v copied into the v pages;
* attention softmax attention of the chunk's queries over the cached keys and values,
            causal or not, over a window or not, with grouped heads.

``listed`` gives the cases, ``draw`` more of the same ranges, ``prepare`` the inputs,
``run`` one pass: through the library's entry points where ``own`` is true, else in
elementary torch operations.  ``exact`` gives the same outputs in 64 bits, ``work`` the
bytes and operations a pass cannot do without.
"""
import math
import random

import torch

own = False

EPS = 1e-6
GRID_H, GRID_W = 24, 42  # latent rows and columns of a frame (1344x768 video)
ROW_PAD = 128            # sequences of a packed batch are padded to this many rows


# ------------------------------------------------------------------ cases

def _case(name, op, **kw):
    c = {"name": name, "op": op, "batch": 1, "chunk_lo": 1, "chunk_hi": 1, "past_lo": 0, "past_hi": 0, "mix": 0,
         "q_heads": 16, "kv_heads": 16, "head_dim": 128, "page": 64, "rotary": 128, "mode": "interleaved",
         "scaling": "none", "factor": 1.0, "grid": False, "norm": True, "causal": True, "window": 0, "lse": False,
         "pad": ROW_PAD}
    c.update(kw)
    return c


def listed():
    return [
        # the next token of 8 requests, far into their contexts: latency counts
        _case("rope_tokens", "rope", batch=8, past_lo=30000, past_hi=120000, mix=1, rotary=64, mode="half",
              scaling="yarn", factor=4.0, norm=False, pad=1),
        # four ragged prompts of 1,024 to 30,000 rows, grouped heads, half of each head rotated
        _case("rope_varlen", "rope", batch=4, chunk_lo=1024, chunk_hi=30000, past_lo=0, past_hi=100000, mix=2,
              q_heads=40, kv_heads=8, rotary=64, mode="half", scaling="yarn", factor=8.0),
        # the long video: 61 latent frames of 24x42 and 400 audio rows, t axis stretched
        _case("rope_long_video", "rope", chunk_lo=61888, chunk_hi=61888, mix=3, scaling="ntk", factor=2.0, grid=True),
        # the next token of 64 requests into the cache: one small launch
        _case("append_tokens", "append", batch=64, past_lo=100, past_hi=16000, mix=4, q_heads=40, kv_heads=8,
              mode="half", scaling="linear", factor=4.0, pad=1),
        # chunks of four streamed videos, pages of 16, positions of the whole video
        _case("append_chunk", "append", batch=4, chunk_lo=1008, chunk_hi=8064, past_lo=1000, past_hi=24000, mix=5,
              q_heads=40, kv_heads=8, page=16, scaling="ntk", factor=2.0, grid=True),
        # one prompt of heads of 64, a quarter of the pages' size odd, part of the head rotated, no norm
        _case("append_head64", "append", chunk_lo=8192, chunk_hi=8192, past_lo=37, past_hi=37, mix=6, head_dim=64,
              q_heads=32, kv_heads=32, page=24, rotary=32, mode="half", norm=False),
        # one request's next token over a short cache: latency counts
        _case("attend_token", "attention", past_lo=2047, past_hi=2047, mix=7, pad=1),
        # the next token of 48 requests over long ragged caches, five queries to a key head
        _case("attend_tokens_grouped", "attention", batch=48, past_lo=1000, past_hi=32000, mix=8, q_heads=40,
              kv_heads=8, pad=1),
        # ragged prompt chunks behind a cached prefix, causal, pages of 16, log-sum-exp asked for
        _case("attend_chunk_causal", "attention", batch=4, chunk_lo=500, chunk_hi=4100, past_lo=0, past_hi=8000,
              mix=9, q_heads=40, kv_heads=8, page=16, lse=True),
        # a streamed video's next 4 latent frames and 100 audio rows over 28 cached frames, all visible
        _case("attend_video_chunk", "attention", chunk_lo=4132, chunk_hi=4132, past_lo=28224, past_hi=28224, mix=10,
              q_heads=40, kv_heads=40, page=128, causal=False),
        # heads of 64 under a sliding window
        _case("attend_window_head64", "attention", batch=2, chunk_lo=2048, chunk_hi=4100, past_lo=8000,
              past_hi=30000, mix=11, head_dim=64, kv_heads=4, page=32, window=4096),
        # heads of 256, odd page size
        _case("attend_head256", "attention", batch=2, chunk_lo=300, chunk_hi=1000, past_lo=1000, past_hi=4000,
              mix=12, head_dim=256, q_heads=8, kv_heads=2, page=40),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))) - 1))))


def _draw_once(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    d = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8, 16])
    c = _case("", op, head_dim=d, kv_heads=kv, q_heads=kv * rng.choice([1, 1, 2, 3, 4, 5, 8]), mix=rng.randrange(10**6),
              page=rng.choice([16, 16, 24, 32, 64, 100, 128, 256]), mode=rng.choice(["interleaved", "half"]),
              norm=rng.random() < 0.6, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
              pad=rng.choice([1, 8, 128]))
    del c["name"]
    if c["scaling"] != "none":
        c["factor"] = rng.choice([2.0, 4.0, 8.0])
    c["rotary"] = rng.choice([d, d, d // 2, d // 4, d - 8])
    c["grid"] = op != "attention" and rng.random() < 0.4
    if rng.random() < 0.4:  # next tokens
        c["batch"] = _logint(rng, 1, 64)
        c["pad"] = 1
    else:
        c["batch"] = rng.choice([1, 2, 3, 4, 8])
        hi = _logint(rng, 2, 8000 if op == "attention" else 30000)
        c["chunk_lo"], c["chunk_hi"] = max(1, hi // rng.choice([1, 2, 16])), hi
    hi = _logint(rng, 0, 32000)
    c["past_lo"], c["past_hi"] = hi // rng.choice([1, 2, 16]), hi
    if op == "attention":
        c["causal"] = rng.random() < 0.7
        c["window"] = rng.choice([0, 0, 0, _logint(rng, 16, 8000)])
        c["lse"] = rng.random() < 0.5
    return c


def draw(rng):
    cost = [work(c) for c in listed()]
    most_bytes, most_flops = max(w["bytes"] for w in cost), max(w["flops"] for w in cost)
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= most_bytes and w["flops"] <= most_flops and _cache_tokens(c) * c["kv_heads"] * \
                c["head_dim"] * 4 <= most_bytes:
            return c


def _lengths(case):
    """Per sequence: rows of the chunk and tokens cached before it."""
    rng = random.Random(case["mix"])
    chunk = [_logint(rng, case["chunk_lo"], case["chunk_hi"]) for _ in range(case["batch"])]
    past = [_logint(rng, case["past_lo"], case["past_hi"]) for _ in range(case["batch"])]
    return chunk, past


def _cache_tokens(case):
    chunk, past = _lengths(case)
    return sum(chunk) + sum(past)


def _sections(rotary):
    side = rotary // 3 // 2 * 2
    return rotary - 2 * side, side, side


# ------------------------------------------------------------------ work

def work(case):
    chunk, past = _lengths(case)
    rows, hq, hk, d = sum(chunk), case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":   # q and k read and written once; norm and rotation ~10 per element
        return {"bytes": 4 * rows * (hq + hk) * d, "flops": 10 * rows * (hq + hk) * d}
    if case["op"] == "append":
        return {"bytes": 4 * rows * (hq + 2 * hk) * d, "flops": 10 * rows * (hq + hk) * d}
    pairs, keys = 0, 0
    for n, before in zip(chunk, past):
        total = n + before
        w = case["window"] or total
        if case["causal"]:
            # query i sits at position before + i and sees min(window, before + i + 1) keys
            full = max(0, min(n, w - 1 - before))  # queries that see everything before them
            pairs += full * before + full * (full + 1) // 2 + (n - full) * w
        else:
            # query i sees total - max(0, before + i - w + 1) keys
            cut = max(0, min(n, w - 1 - before))      # queries that see every key
            m = n - cut
            first = before + cut - w + 1
            pairs += cut * total + m * total - (m * first + m * (m - 1) // 2)
        keys += total - max(0, before - w + 1)
    nbytes = 4 * rows * hq * d + 4 * keys * hk * d + (4 * rows * hq if case["lse"] else 0)
    return {"bytes": nbytes, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """Everything but the frequency tables, from the seed alone."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    chunk, past = _lengths(case)
    pad = case["pad"]
    slots = [-(-n // pad) * pad for n in chunk]
    rows, hq, hk, d, page = sum(slots), case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, dtype=torch.bfloat16, device=dev, generator=g).mul_(std)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    def cumulative(values):
        out = [0]
        for v in values:
            out.append(out[-1] + v)
        return out

    s = {"case": case, "chunk": chunk, "past": past, "first_row": cumulative(slots)[:-1],
         "cu_seqlens": ints(cumulative(chunk)), "cu_seqlens_padded": ints(cumulative(slots)),
         "past_dev": ints(past), "total_dev": ints([a + b for a, b in zip(chunk, past)]),
         "q_out": torch.zeros(rows, hq * d, dtype=torch.bfloat16, device=dev)}
    if case["op"] == "attention":
        s["q"] = normal(rows, hq * d)
        if case["lse"]:
            s["lse"] = torch.zeros(rows, hq, dtype=torch.float32, device=dev)
    else:
        qkv = normal(rows, (hq + 2 * hk) * d)  # one fused projection: q, k and v are column slices
        s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
        s["k_out"] = torch.zeros(rows, hk * d, dtype=torch.bfloat16, device=dev)
        s["q_weight"] = normal(d, std=0.02).add_(1.0) if case["norm"] else None
        s["k_weight"] = normal(d, std=0.02).add_(1.0) if case["norm"] else None
        s["grid_host"] = [((a + b) // (GRID_H * GRID_W), GRID_H, GRID_W) for a, b in zip(chunk, past)]
        s["grid"] = ints(s["grid_host"]) if case["grid"] else None
    if case["op"] != "rope":
        need = [-(-(a + b) // page) for a, b in zip(chunk, past)]
        pages = list(range(sum(need) + 3))
        host.shuffle(pages)  # pages are handed out in the order requests came, not in sequence order
        width = max(need) + 1
        table, at = [], 0
        for n in need:
            table.append(pages[at:at + n] + [-1] * (width - n))
            at += n
        s["block_table"] = ints(table)
        s["k_cache"] = normal(len(pages), page, hk, d)
        s["v_cache"] = normal(len(pages), page, hk, d)
    return s


def _yarn_context(case):
    return 4096  # rows the unscaled frequencies were trained for


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "attention":
        rotary = case["rotary"]
        if own:
            import dit_token_b200 as dit

            def table(n, scaled):
                return dit.dit_rope_frequencies(n, scaling=case["scaling"] if scaled else "none",
                                                factor=case["factor"], original_len=_yarn_context(case))
        else:
            def table(n, scaled):
                return _plain_frequencies(n, case, scaled)
        s["freqs"], s["attn_scale"] = table(rotary, True)
        s["grid_freqs"] = None
        if case["grid"]:  # the time axis is stretched, a frame's rows and columns are not
            t, h, w = _sections(rotary)
            s["grid_freqs"] = torch.cat([table(n, n_is_t)[0] for n, n_is_t in ((t, True), (h, False), (w, False))
                                         if n > 0])
    elif own:
        import dit_token_b200 as dit
        c = case
        nbytes = dit.dit_paged_attention_workspace(
            s["q"].size(0), c["batch"], num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"],
            head_dim=c["head_dim"], max_chunk=max(s["chunk"]), max_kv_len=max(a + b for a, b in zip(s["chunk"], s["past"])))
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attention": _own_attention}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention}[op](state)


def _own_rope(s):
    import dit_token_b200 as dit
    c = s["case"]
    return dit.dit_qk_rope_scaled(
        s["q"], s["k"], s["cu_seqlens"], s["cu_seqlens_padded"], num_q_heads=c["q_heads"], num_k_heads=c["kv_heads"],
        head_dim=c["head_dim"], freqs=s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"], rope_grid=s["grid"],
        grid_freqs=s["grid_freqs"], sections=_sections(c["rotary"]), pos_offset=s["past_dev"],
        attn_scale=s["attn_scale"], eps=EPS, rope_mode=c["mode"], q_out=s["q_out"], k_out=s["k_out"])


def _own_append(s):
    import dit_token_b200 as dit
    c = s["case"]
    q = dit.dit_qkv_rope_append(
        s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["past_dev"], s["cu_seqlens"],
        s["cu_seqlens_padded"], num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"], head_dim=c["head_dim"],
        freqs=s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"], rope_grid=s["grid"],
        grid_freqs=s["grid_freqs"], sections=_sections(c["rotary"]), attn_scale=s["attn_scale"], eps=EPS,
        rope_mode=c["mode"], q_out=s["q_out"])
    return q, s["k_cache"], s["v_cache"]


def _own_attention(s):
    import dit_token_b200 as dit
    c = s["case"]
    out = dit.dit_paged_attention(
        s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["total_dev"], s["cu_seqlens"], s["cu_seqlens_padded"],
        num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"], head_dim=c["head_dim"], causal=c["causal"],
        window=c["window"], max_chunk=max(s["chunk"]), max_kv_len=max(a + b for a, b in zip(s["chunk"], s["past"])),
        out=s["q_out"], lse=s.get("lse"), workspace=s["workspace"])
    return (out, s["lse"]) if c["lse"] else out


# ------------------------------------------------------------------ plain forms

def _plain_frequencies(n, case, scaled):
    """Pair frequencies of ``n`` rotated elements (64 bits) and the factor on cos and sin."""
    theta, scaling, factor = 10000.0, case["scaling"] if scaled else "none", case["factor"]
    j = torch.arange(n // 2, dtype=torch.float64, device="cuda")
    if scaling == "ntk" and n > 2:
        theta = theta * factor ** (n / (n - 2))
    f = theta ** (-2.0 * j / n)
    if scaling == "linear":
        f = f / factor
    if scaling != "yarn":
        return f, 1.0

    def turns_at(turns):  # the pair that makes this many turns over the trained context
        return n * math.log(_yarn_context(case) / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low, high = max(math.floor(turns_at(32.0)), 0), min(math.ceil(turns_at(1.0)), n - 1)
    ramp = ((j - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f / factor * ramp + f * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


def _plain_rotate(x, heads, weight, s, b):
    """RMSNorm and rotation of sequence b's rows: [rows, heads * d] -> fp32 [rows, heads, d]."""
    c = s["case"]
    d, rotary = c["head_dim"], c["rotary"]
    n = s["chunk"][b]
    x = x.float().view(n, heads, d)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    pos = torch.arange(n, dtype=torch.float64, device=x.device) + s["past"][b]
    angle = pos[:, None] * s["freqs"]
    if c["grid"]:
        t, h, w = s["grid_host"][b]
        local = torch.where(pos < t * h * w, pos, pos - t * h * w)
        axes = torch.stack([torch.floor(local / (h * w)), torch.floor(local / w) % h, local % w], 1)
        widths = torch.tensor([v // 2 for v in _sections(rotary)], device=x.device)
        axis = torch.repeat_interleave(torch.arange(3, device=x.device), widths)
        angle = torch.where((pos < t * h * w)[:, None], axes[:, axis] * s["grid_freqs"], local[:, None] * s["freqs"])
    cos = (torch.cos(angle) * s["attn_scale"]).float()[:, None]
    sin = (torch.sin(angle) * s["attn_scale"]).float()[:, None]
    turned, rest = x[..., :rotary], x[..., rotary:]
    if c["mode"] == "half":
        a, z = turned[..., :rotary // 2], turned[..., rotary // 2:]
        turned = torch.cat([a * cos - z * sin, a * sin + z * cos], -1)
    else:
        a, z = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - z * sin, a * sin + z * cos], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_rope(s):
    c = s["case"]
    q_out, k_out = torch.zeros_like(s["q_out"]), torch.zeros_like(s["k_out"])
    for b, (n, r0) in enumerate(zip(s["chunk"], s["first_row"])):
        q_out[r0:r0 + n] = _plain_rotate(s["q"][r0:r0 + n], c["q_heads"], s["q_weight"], s, b).flatten(1).bfloat16()
        k_out[r0:r0 + n] = _plain_rotate(s["k"][r0:r0 + n], c["kv_heads"], s["k_weight"], s, b).flatten(1).bfloat16()
    return q_out, k_out


def _slots(s, b, first, last):
    """Page and place within the page of tokens first .. last - 1 of sequence b."""
    pos = torch.arange(first, last, device="cuda")
    page = s["case"]["page"]
    return s["block_table"][b, pos // page].long(), pos % page


def _plain_append(s):
    c = s["case"]
    q_out = torch.zeros_like(s["q_out"])
    for b, (n, r0, past) in enumerate(zip(s["chunk"], s["first_row"], s["past"])):
        q_out[r0:r0 + n] = _plain_rotate(s["q"][r0:r0 + n], c["q_heads"], s["q_weight"], s, b).flatten(1).bfloat16()
        where = _slots(s, b, past, past + n)
        s["k_cache"][where] = _plain_rotate(s["k"][r0:r0 + n], c["kv_heads"], s["k_weight"], s, b).bfloat16()
        s["v_cache"][where] = s["v"][r0:r0 + n].reshape(n, c["kv_heads"], c["head_dim"])
    return q_out, s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    group = hq // hk
    out = torch.zeros_like(s["q_out"])
    lse = torch.zeros(out.size(0), hq, dtype=torch.float32, device=out.device)
    for b, (n, r0, past) in enumerate(zip(s["chunk"], s["first_row"], s["past"])):
        total = n + past
        where = _slots(s, b, 0, total)
        key = s["k_cache"][where].float().permute(1, 2, 0)    # [hk, d, total]
        value = s["v_cache"][where].float().permute(1, 0, 2)  # [hk, total, d]
        seen = torch.arange(total, device=out.device)
        step = max(1, (1 << 28) // (total * hq))
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][r0 + i:r0 + i + m].float().view(m, hk, group, d).permute(1, 0, 2, 3).reshape(hk, m * group, d)
            score = torch.matmul(q, key).mul_(1.0 / math.sqrt(d)).view(hk, m, group, total)
            pos = torch.arange(past + i, past + i + m, device=out.device)[:, None]
            hidden = torch.zeros(m, total, dtype=torch.bool, device=out.device)
            if c["causal"]:
                hidden |= seen > pos
            if c["window"]:
                hidden |= seen <= pos - c["window"]
            score.masked_fill_(hidden[:, None], -math.inf)
            top = score.amax(-1, keepdim=True)
            score.sub_(top).exp_()
            norm = score.sum(-1, keepdim=True)
            o = torch.matmul(score.view(hk, m * group, total), value).view(hk, m, group, d) / norm
            out[r0 + i:r0 + i + m] = o.permute(1, 0, 2, 3).reshape(m, hq * d).bfloat16()
            lse[r0 + i:r0 + i + m] = (top + torch.log(norm)).permute(1, 0, 2, 3).reshape(m, hq)
    return (out, lse) if c["lse"] else out


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    q = _exact_rotated(s, s["q"], case["q_heads"], s["q_weight"])
    k = _exact_rotated(s, s["k"], case["kv_heads"], s["k_weight"])
    if case["op"] == "rope":
        return q.flatten(1), k.flatten(1)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    for b in range(case["batch"]):
        rows = slice(s["first_row"][b], s["first_row"][b] + s["chunk"][b])
        place = torch.arange(s["past"][b], s["past"][b] + s["chunk"][b], device="cuda")
        page = s["block_table"][b].long()[place // case["page"]]
        k_cache[page, place % case["page"]] = k[rows]
        v_cache[page, place % case["page"]] = s["v"][rows].double().unflatten(1, (case["kv_heads"], -1))
    return q.flatten(1), k_cache, v_cache


def _exact_rates(case, n, stretch):
    rates, gain = [], 1.0
    for j in range(n // 2):
        kind = case["scaling"] if stretch else "none"
        base = 10000.0
        if kind == "ntk" and n > 2:
            base *= math.pow(case["factor"], n / (n - 2.0))
        rate = math.pow(base, -(2.0 * j) / n)
        if kind == "linear":
            rate /= case["factor"]
        if kind == "yarn":
            length = _yarn_context(case)
            start = max(0, math.floor(n / 2 * math.log(length / (64 * math.pi), base)))
            end = min(n - 1, math.ceil(n / 2 * math.log(length / (2 * math.pi), base)))
            part = min(1.0, max(0.0, (j - start) / max(end - start, 0.001)))
            rate = part * (rate / case["factor"]) + (1.0 - part) * rate
            gain = 1.0 + math.log(case["factor"]) / 10.0
        rates.append(rate)
    return rates, gain


def _exact_rotated(s, x, heads, weight):
    case = s["case"]
    d, rotary = case["head_dim"], case["rotary"]
    y = torch.zeros(x.size(0), heads, d, dtype=torch.float64, device="cuda")
    line, gain = _exact_rates(case, rotary, True)
    line = torch.tensor(line, dtype=torch.float64, device="cuda")
    pairs_of = [v // 2 for v in _sections(rotary)]
    per_axis = [torch.tensor(_exact_rates(case, 2 * m, axis == 0)[0], dtype=torch.float64, device="cuda")
                for axis, m in enumerate(pairs_of)]
    for b, n in enumerate(s["chunk"]):
        r0 = s["first_row"][b]
        place = torch.arange(s["past"][b], s["past"][b] + n, device="cuda")
        angle = torch.outer(place.double(), line)
        if case["grid"]:
            t, h, w = s["grid_host"][b]
            inside = place < t * h * w
            p = place[inside]
            coords = (p // (h * w), p // w % h, p % w)
            angle[inside] = torch.cat([torch.outer(v.double(), r) for v, r in zip(coords, per_axis)], 1)
            angle[~inside] = torch.outer((place[~inside] - t * h * w).double(), line)
        turn = torch.polar(torch.full_like(angle, gain), angle)[:, None]
        rows = x[r0:r0 + n].double().unflatten(1, (heads, d))
        if weight is not None:
            rows = rows / torch.sqrt(rows.square().mean(-1, keepdim=True) + EPS) * weight.double()
        head = rows[..., :rotary]
        if case["mode"] == "half":
            z = torch.complex(*head.unflatten(-1, (2, rotary // 2)).unbind(-2)) * turn
            head = torch.cat([z.real, z.imag], -1)
        else:
            head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        y[r0:r0 + n] = torch.cat([head, rows[..., rotary:]], -1)
    return y


def _exact_attention(s):
    case = s["case"]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    rows = s["q"].size(0)
    out = torch.zeros(rows, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, hq, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["chunk"]):
        r0, total = s["first_row"][b], s["past"][b] + s["chunk"][b]
        places = torch.arange(total, device="cuda")
        page = s["block_table"][b].long()[places // case["page"]]
        keys = s["k_cache"][page, places % case["page"]]
        values = s["v_cache"][page, places % case["page"]]
        block = max(1, (1 << 28) // total)
        for i in range(0, n, block):
            at = torch.arange(i, min(i + block, n), device="cuda")
            distance = (at + s["past"][b])[:, None] - places[None]
            allowed = torch.ones_like(distance, dtype=torch.bool)
            if case["causal"]:
                allowed &= distance >= 0
            if case["window"]:
                allowed &= distance < case["window"]
            for h in range(hq):
                kh, vh = keys[:, h // (hq // hk)].double(), values[:, h // (hq // hk)].double()
                logit = s["q"][r0 + at, h * d:(h + 1) * d].double() @ kh.T / math.sqrt(d)
                logit = torch.where(allowed, logit, -math.inf)
                lse[r0 + at, h] = torch.logsumexp(logit, -1)
                out[r0 + at, h] = torch.exp(logit - lse[r0 + at, h][:, None]) @ vh
    out = out.flatten(1)
    return (out, lse) if case["lse"] else out
