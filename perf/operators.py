"""The attention operators around the 8-bit key/value cache, and how they are measured.

Four operators, each in its plain form (elementary torch operations) and as the calls that a
user makes of the library:

* ``rope``: norm of every query and key head and the position rotation, in one pass;
* ``append``: new tokens into pages of 8-bit codes with one magnitude for each page and head
  (and the values of every page that changed, read back);
* ``read``: the values that a stretch of the cache stands for;
* ``attention``: grouped-query attention over that cache, from one token a sequence to prompts.

``own`` selects the side; ``listed``/``draw`` give the cases, ``prepare`` the inputs, ``run`` one
pass, ``work`` the bytes and operations it cannot do without and ``exact`` the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases

def _rope(tokens, q_heads, kv_heads, dim, rotary, interleaved, scaling, far, dtype, **name):
    return {**name, "kind": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "rotary": rotary, "interleaved": interleaved, "scaling": scaling,
            "far": far, "dtype": dtype}


def _cache(kind, batch, new, old, ragged, q_heads, kv_heads, dim, page, window, dtype, layout,
           **name):
    return {**name, "kind": kind, "batch": batch, "new": new, "old": old, "ragged": ragged,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "window": window, "dtype": dtype, "layout": layout}


def listed():
    return [
        # One decode step of one conversation at the library's 2048-wide layers: 16 query heads
        # and 2 key heads of 256, a quarter of each head rotated.  Latency counts.
        _rope(1, 16, 2, 256, 64, False, "none", 200000, "bf16", name="rope-token"),
        # A prompt chunk with a context stretched by frequency ramps, neighbouring pairs rotated.
        _rope(8192, 32, 8, 128, 128, True, "yarn", 130000, "bf16", name="rope-prompt"),
        # One decode step of 16 conversations: every page has earlier tokens.
        _cache("append", 16, 1, 4095, True, 0, 2, 256, 64, 0, "bf16", 1, name="append-step"),
        # Ragged prompts, the pages at both ends of each partly filled.
        _cache("append", 5, 4096, 700, True, 0, 8, 128, 32, 0, "fp16", 2, name="append-prompts"),
        # Reading back a few short sequences (a prefix moved to another cache).
        _cache("read", 3, 400, 100, True, 0, 4, 64, 16, 0, "fp16", 3, name="read-short"),
        # Reading back one long sequence of the 2048-wide model.
        _cache("read", 1, 131072, 0, False, 0, 2, 256, 64, 0, "bf16", 4, name="read-long"),
        # Decode, one conversation, a short context: launch and join latency.
        _cache("attention", 1, 1, 776, False, 16, 2, 256, 64, 0, "bf16", 5, name="attention-token"),
        # Decode, 64 conversations of very different lengths: the cache's bytes.
        _cache("attention", 64, 1, 32767, True, 32, 8, 128, 32, 0, "bf16", 6, name="attention-batch"),
        # Decode, one conversation at the longest context the library's model takes.
        _cache("attention", 1, 1, 262143, False, 16, 2, 256, 64, 0, "bf16", 7, name="attention-long"),
        # Checking two drafts a step: three tokens a sequence, a sliding window, one head a group.
        _cache("attention", 16, 3, 16381, True, 6, 6, 64, 16, 4096, "fp16", 8, name="attention-drafts"),
        # Ragged prompts with earlier context, grouped heads of 128.
        _cache("attention", 5, 3000, 5000, True, 32, 8, 128, 64, 0, "fp16", 9, name="attention-prompts"),
        # The largest: a 4096-token prompt chunk far into a context, 16 heads of 256 over 2.
        _cache("attention", 1, 4096, 28672, False, 16, 2, 256, 64, 0, "bf16", 10, name="attention-chunk"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "rope":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rotary = dim if rng.random() < 0.5 else 2 * rng.randint(0, dim // 2)
        kv_heads = rng.choice([1, 2, 4, 8])
        return _rope(_spread(rng, 1, 8192), kv_heads * rng.randint(1, 8), kv_heads, dim, rotary,
                     rng.random() < 0.5, rng.choice(["none", "linear", "yarn"]),
                     _spread(rng, 10, 1000000), dtype)
    dim, page = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    ragged, layout = rng.random() < 0.7, rng.randint(100, 1 << 30)
    if kind != "attention":
        new = _spread(rng, 1, 4096)
        batch = _spread(rng, 1, max(1, min(200, 16384 // new)))
        return _cache(kind, batch, new, _spread(rng, 1, 2000), ragged, 0, kv_heads, dim, page, 0,
                      dtype, layout)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 16])
    while kv_heads * group > 48:
        kv_heads //= 2
    new = rng.choice([1, 1, rng.randint(2, 8), _spread(rng, 9, 4096)])
    old = _spread(rng, 1, 200000)
    window = 0 if rng.random() < 0.75 else _spread(rng, 16, 8192)
    q_heads = kv_heads * group
    batch = _spread(rng, 1, 100)

    def costs():
        keys = batch * (old + new)
        return max(keys * kv_heads * dim * 2 / 2.0e9, 4 * batch * new * (old + new) * q_heads * dim / 2.0e12,
                   batch * new * (old + new) * q_heads * 4 / 9.0e9)

    while costs() > 1:
        if batch > 1:
            batch = (batch + 1) // 2
        elif old > 2 * new:
            old //= 2
        else:
            new = (new + 1) // 2
    return _cache("attention", batch, new, old, ragged, q_heads, kv_heads, dim, page, window, dtype,
                  layout)


# --------------------------------------------------------------------------- inputs

def _lengths(case):
    """New and old tokens of every sequence: a matter of the case, not of the seed."""
    rs = np.random.RandomState(case["layout"])
    b = case["batch"]
    new, old = np.full(b, case["new"]), np.full(b, case["old"])
    if case["ragged"]:
        new[1:] = rs.randint(1, case["new"] + 1, b - 1)
        old[1:] = rs.randint(0, case["old"] + 1, b - 1)
        if b > 2 and case["new"] > 1:
            new[b // 2] = 0  # a sequence that waits in this step
    return new.astype(np.int64), old.astype(np.int64)


def _frequencies(case):
    """Radians a position, for every rotated pair, in 64 bits."""
    half = case["rotary"] // 2
    f = 10000000.0 ** (-np.arange(half, dtype=np.float64) / max(half, 1))
    if case["scaling"] == "linear":
        f = f / 4.0
    elif case["scaling"] == "yarn":  # published ramp over the turns in the original context
        turns = 32768.0 * f / (2 * np.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / 4.0 * (1 - keep)
    return f


def _rope_factor(case):
    return 0.1 * math.log(4.0) + 1.0 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    kv, dim = case["kv_heads"], case["dim"]
    if case["kind"] == "rope":
        t, q_heads = case["tokens"], case["q_heads"]
        # Queries, keys and values come out of one projection: the two parts are views of its rows.
        rows = (randn(t, q_heads + 2 * kv, dim) * 2).to(dtype)
        first = torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device="cuda")
        return {"case": case, "q": rows[:, :q_heads], "k": rows[:, q_heads:q_heads + kv],
                "positions": (first + torch.arange(t, device="cuda")).to(torch.int32),
                "q_weight": (1 + 0.2 * randn(dim)).to(dtype), "k_weight": (1 + 0.2 * randn(dim)).to(dtype),
                "frequencies": torch.from_numpy(_frequencies(case)).cuda()}
    new, old = _lengths(case)
    page, b = case["page"], case["batch"]
    lengths = new + old
    pages = -(-lengths // page)
    total = int(pages.sum()) + 3
    ids = torch.randperm(total, generator=g, device="cuda")
    row = np.zeros((b, max(1, int(pages.max()))), np.int64)
    start = np.cumsum(pages) - pages
    for i in range(b):
        row[i, :pages[i]] = start[i] + np.arange(pages[i])
    table = ids[torch.from_numpy(row).cuda()].to(torch.int32)
    q_start = np.concatenate([[0], np.cumsum(new)])
    state = {"case": case, "table": table, "tokens": int(new.sum()), "max_new": int(new.max()),
             "max_kv": int(lengths.max()),
             "q_start": torch.from_numpy(q_start).to(torch.int32).cuda(),
             "kv_len": torch.from_numpy(lengths).to(torch.int32).cuda()}

    def filled(spread):
        codes = torch.empty((total, kv, page, dim), dtype=torch.int8, device="cuda")
        amax = torch.empty((total, kv), dtype=torch.float32, device="cuda")
        step = max(1, (1 << 28) // (kv * page * dim))
        for i in range(0, total, step):
            x = randn(min(step, total - i), kv, page, dim) * spread
            a = x.abs().amax((2, 3)).to(dtype).float()
            codes[i:i + step] = (x * 127 / a[:, :, None, None]).round_().clamp_(-127, 127).to(torch.int8)
            amax[i:i + step] = a
        return codes, amax

    # Keys have a few channels that stand out; values differ in size from head to head.
    channels = torch.where(torch.rand(dim, generator=g, device="cuda") < 0.03, 4.0, 1.0)
    heads = torch.exp(0.5 * randn(kv, 1, 1))
    state["k_codes"], state["k_amax"] = filled(channels)
    state["v_codes"], state["v_amax"] = filled(heads)
    if case["kind"] == "append":
        rows = torch.cat([randn(state["tokens"], kv, dim) * channels,
                          randn(state["tokens"], kv, dim) * heads[None, :, :, 0]], 1).to(dtype)
        state["k"], state["v"] = rows[:, :kv], rows[:, kv:]
        # The tokens of every page that the call changes, earlier ones of its first page too.
        changed = np.where(new > 0, new + old % page, 0)
        state["changed"] = int(changed.sum())
        state["changed_start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(changed)])).to(torch.int32).cuda()
    elif case["kind"] == "attention":
        state["q"] = (randn(state["tokens"], case["q_heads"], dim) * 1.5).to(dtype)
        state["scale"] = dim ** -0.5
    return state


# --------------------------------------------------------------------------- plain forms

def _plain_rope(s):
    case, half = s["case"], s["case"]["rotary"] // 2
    angles = s["positions"].double()[:, None] * s["frequencies"]
    cos = (torch.cos(angles).float() * _rope_factor(case))[:, None, :]
    sin = (torch.sin(angles).float() * _rope_factor(case))[:, None, :]

    def one(x, weight):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
        turn, rest = y[..., :2 * half], y[..., 2 * half:]
        if case["interleaved"]:
            a, b = turn[..., 0::2], turn[..., 1::2]
            turn = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = turn[..., :half], turn[..., half:]
            turn = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([turn, rest], -1).to(x.dtype)

    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])


def _places(s, starts, count):
    """For each row of ragged rows that end at their sequences' ends: its sequence and position."""
    rows = torch.arange(count, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), rows, right=True)
    return seq, (rows - starts.long()[seq + 1]) + s["kv_len"].long()[seq]


def _plain_read(s, starts, count, dtype):
    page = s["case"]["page"]
    seq, at = _places(s, starts, count)
    ids = s["table"].long()[seq, at // page]

    def one(codes, amax):
        return (codes[ids, :, at % page].float() * amax[ids][..., None] / 127).to(dtype)

    return one(s["k_codes"], s["k_amax"]), one(s["v_codes"], s["v_amax"])


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    t = s["tokens"]
    seq, at = _places(s, s["q_start"], t)
    first = (at % page == 0) | (torch.arange(t, device="cuda") == s["q_start"].long()[seq])
    run = torch.cumsum(first, 0) - 1  # the page of the call that a token falls into
    most = min(t, t // page + 2 * case["batch"])
    ids = s["table"].long()[seq, at // page]
    page_of = torch.full((most,), -1, dtype=torch.long, device="cuda").scatter_(0, run, ids)
    page_of = torch.where(page_of < 0, page_of[0], page_of)
    fresh = torch.zeros(s["k_amax"].shape[0], dtype=torch.int32, device="cuda")
    fresh = fresh.index_add(0, ids, (at % page == 0).int()) > 0

    def one(x, codes, amax):
        x = x.float()
        had = torch.where(fresh[:, None], torch.zeros_like(amax), amax)
        top = had.index_reduce(0, ids, x.abs().amax(-1), "amax")
        was, now = had[page_of][..., None, None], top[page_of][..., None, None]
        codes[page_of] = torch.where(now > was, codes[page_of].float() * was / now, codes[page_of].float()).round().to(torch.int8)
        now = top[ids][..., None]
        codes[ids, :, at % page] = torch.where(now > 0, x * 127 / now, x * 0).round().to(torch.int8)
        amax[page_of] = top[page_of]

    one(s["k"], s["k_codes"], s["k_amax"])
    one(s["v"], s["v_codes"], s["v_amax"])


def _plain_attention(s):
    case, page, b, n = s["case"], s["case"]["page"], s["case"]["batch"], s["max_new"]
    kv, dim, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
    keys = s["table"].shape[1] * page

    def values(codes, amax):
        x = codes[s["table"].long()].float() * (amax / 127)[s["table"].long()][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(b, kv, keys, dim)

    start, length = s["q_start"].long(), s["kv_len"].long()
    count = start[1:] - start[:-1]
    step = torch.arange(n, device="cuda")
    rows = (start[:-1, None] + step).clamp(max=s["tokens"] - 1)
    q = s["q"].float()[rows].reshape(b, n, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(b, kv, group * n, dim)
    at = (length - count)[:, None] + step
    key = torch.arange(keys, device="cuda")
    seen = (key <= at[..., None]) & (key < length[:, None, None])
    if case["window"]:
        seen &= key > at[..., None] - case["window"]
    scores = (q @ values(s["k_codes"], s["k_amax"]).transpose(-1, -2)).mul_(s["scale"])
    scores = scores.view(b, kv, group, n, keys).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(b, kv, group * n, keys) @ values(s["v_codes"], s["v_amax"])).view(b, kv, group, n, dim)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total))[..., 0]
    seq, place = _places(s, s["q_start"], s["tokens"])
    i = place - (length - count)[seq]
    return (out[seq, :, :, i].reshape(-1, kv * group, dim).to(s["q"].dtype),
            lse[seq, :, :, i].reshape(-1, kv * group))


# --------------------------------------------------------------------------- one pass

def _handles(s):
    """What a program makes once and keeps: the operator's table, the cache's and batch's handles."""
    if "handles" in s:
        return s["handles"]
    import bit_affine_quantized_mlx_gb300 as q4
    case = s["case"]
    if case["kind"] == "rope":
        turns = q4.lily_rope_turns(case["rotary"], 10000000.0, case["scaling"], factor=4.0,
                                   original_len=32768)
        h = (q4.QKNormRope(case["dim"], case["rotary"], q4.to_device(turns), s["q_weight"],
                           s["k_weight"], eps=1e-6, interleaved=case["interleaved"],
                           rope_scale=_rope_factor(case)),
             torch.empty_like(s["q"], memory_format=torch.contiguous_format),
             torch.empty_like(s["k"], memory_format=torch.contiguous_format))
    else:
        cache = q4.KV8Cache(s["k_codes"], s["v_codes"], s["k_amax"], s["v_amax"])
        batch = q4.KV8Batch(s["table"], s["q_start"], s["kv_len"], s["max_new"], s["max_kv"])
        if case["kind"] == "attention":
            ws = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(cache, batch, s["tokens"],
                                                                        case["q_heads"]))
            h = (cache, batch, ws, torch.empty_like(s["q"]),
                 torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda"))
        else:
            count = s["changed"] if case["kind"] == "append" else s["tokens"]
            changed = None
            if case["kind"] == "append":
                changed = q4.KV8Batch(s["table"], s["changed_start"], s["kv_len"],
                                      s["max_new"] + case["page"], s["max_kv"])
            dtype = torch.float32 if case["kind"] == "append" else DTYPES[case["dtype"]]
            shape = (count, case["kv_heads"], case["dim"])
            h = (cache, batch, q4.new_workspace(256), changed,
                 torch.empty(shape, dtype=dtype, device="cuda"),
                 torch.empty(shape, dtype=dtype, device="cuda"))
    s["handles"] = (q4, h)
    return s["handles"]


def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if own:
        q4, h = _handles(s)
        if kind == "rope":
            op, q_out, k_out = h
            q4.lily_qk_norm_rope(op, s["q"], s["k"], s["positions"], q_out, k_out)
            return {"q": q_out, "k": k_out}
        if kind == "attention":
            cache, batch, ws, out, lse = h
            q4.lily_kv8_attention(cache, batch, s["q"], out, s["scale"], lse=lse,
                                  window=case["window"], ws=ws)
            return {"out": out, "lse": lse}
        cache, batch, ws, changed, k_out, v_out = h
        if kind == "append":
            q4.lily_kv8_append(cache, batch, s["k"], s["v"], ws=ws)
            q4.lily_kv8_read(cache, changed, k_out, v_out, ws=ws)
            return {"k": k_out, "v": v_out, "k_amax": s["k_amax"], "v_amax": s["v_amax"]}
        q4.lily_kv8_read(cache, batch, k_out, v_out, ws=ws)
        return {"k": k_out, "v": v_out}
    if kind == "rope":
        q, k = _plain_rope(s)
        return {"q": q, "k": k}
    if kind == "attention":
        out, lse = _plain_attention(s)
        return {"out": out, "lse": lse}
    if kind == "append":
        _plain_append(s)
        k, v = _plain_read(s, s["changed_start"], s["changed"], torch.float32)
        return {"k": k, "v": v, "k_amax": s["k_amax"], "v_amax": s["v_amax"]}
    k, v = _plain_read(s, s["q_start"], s["tokens"], DTYPES[case["dtype"]])
    return {"k": k, "v": v}


# --------------------------------------------------------------------------- work and exact results

def work(case):
    kv, dim = case["kv_heads"], case["dim"]
    if case["kind"] == "rope":
        values = case["tokens"] * (case["q_heads"] + kv) * dim
        return {"bytes": 4 * values + 4 * case["tokens"] + 4 * dim + 4 * case["rotary"], "flops": 10 * values}
    new, old = _lengths(case)
    page = case["page"]
    t, per = int(new.sum()), kv * dim * 2
    if case["kind"] == "read":
        return {"bytes": t * per * 3 + int((-(-(new + old) // page) - old // page).sum()) * kv * 8, "flops": 2 * t * per}
    if case["kind"] == "append":
        changed = int(np.where(new > 0, new + old % page, 0).sum())
        return {"bytes": t * per * 3 + changed * per * 5, "flops": 4 * t * per + 2 * changed * per}
    first = old - (case["window"] - 1) if case["window"] else old * 0
    read = int(np.where(new > 0, new + old - np.maximum(first, 0), 0).sum())
    pairs = 0
    for n, o in zip(new.tolist(), old.tolist()):
        at = np.arange(o + 1, o + n + 1, dtype=np.int64)
        pairs += int((np.minimum(at, case["window"]) if case["window"] else at).sum())
    return {"bytes": read * per + t * case["q_heads"] * (4 * dim + 4),
            "flops": 4 * pairs * case["q_heads"] * dim}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rope":
        half = case["rotary"] // 2
        turn = torch.polar(torch.full((case["tokens"], 1, half), _rope_factor(case), dtype=torch.float64, device="cuda"),
                           (s["positions"].double()[:, None] * s["frequencies"])[:, None])
        out = {}
        for x, w, to in ((s["q"], s["q_weight"], "q"), (s["k"], s["k_weight"], "k")):
            y = x.double() * w.double() / (x.double().square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt()
            if not half:
                out[to] = y
                continue
            head = y[..., :2 * half]
            pair = head.unflatten(-1, (half, 2)) if case["interleaved"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
            pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            head = pair.flatten(-2) if case["interleaved"] else pair.transpose(-1, -2).flatten(-2)
            out[to] = torch.cat([head, y[..., 2 * half:]], -1)
        return out
    new, old = _lengths(case)
    page, table = case["page"], s["table"].cpu().numpy()
    if case["kind"] == "attention":
        group = case["q_heads"] // case["kv_heads"]
        outs, lses, row = [], [], 0
        for b in range(case["batch"]):
            n, length = int(new[b]), int(new[b] + old[b])
            if n == 0:
                continue
            low = max(0, int(old[b]) - case["window"] + 1) // page * page if case["window"] else 0
            ids = torch.from_numpy(table[b, low // page:-(-length // page)].astype(np.int64)).cuda()
            at = torch.arange(int(old[b]), length, device="cuda")[:, None]
            key = torch.arange(low, length, device="cuda")[None]
            hide = key > at
            if case["window"]:
                hide = hide | (at - key >= case["window"])
            o = torch.empty((n, case["q_heads"], case["dim"]), dtype=torch.float64, device="cuda")
            l = torch.empty((n, case["q_heads"]), dtype=torch.float64, device="cuda")
            for h in range(case["kv_heads"]):
                k, v = ((s[x + "_codes"][ids, h].double() * s[x + "_amax"][ids, h].double()[:, None, None] / 127)
                        .flatten(0, 1)[:length - low] for x in "kv")
                for j in range(h * group, (h + 1) * group):
                    score = (s["q"][row:row + n, j].double() @ k.T) * s["scale"]
                    score = score.masked_fill_(hide, -math.inf)
                    l[:, j] = torch.logsumexp(score, -1)
                    o[:, j] = score.sub_(l[:, j, None]).exp_() @ v
            outs.append(o)
            lses.append(l)
            row += n
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    out, rows = {}, np.concatenate([[0], np.cumsum(new)])
    for x in "kv":
        codes, amax = s[x + "_codes"], s[x + "_amax"].double()
        parts = []
        fresh = s[x].double() if case["kind"] == "append" else None
        for b in range(case["batch"]):
            if new[b] == 0:
                continue
            first = int(old[b]) // page
            ids = torch.from_numpy(table[b, first:-(-int(new[b] + old[b]) // page)].astype(np.int64)).cuda()
            q = codes[ids].double()
            if fresh is None:
                part = (q * amax[ids][..., None, None] / 127).transpose(1, 2).flatten(0, 1)
                parts.append(part[int(old[b]) - first * page:][:int(new[b])])
                continue
            had = int(old[b]) - first * page
            x_new = torch.zeros((ids.numel() * page,) + fresh.shape[1:], dtype=torch.float64, device="cuda")
            x_new[had:had + int(new[b])] = fresh[rows[b]:rows[b + 1]]
            x_new = x_new.unflatten(0, (-1, page)).transpose(1, 2)
            was = amax[ids].clone()
            was[1 if had else 0:] = 0
            now = torch.maximum(was, x_new.abs().amax((-1, -2)))
            kept = torch.round(q * was[..., None, None] / now.clamp(min=1e-300)[..., None, None])
            is_old = torch.zeros((ids.numel() * page, 1, 1), dtype=torch.bool, device="cuda")
            is_old[:had] = True
            is_old = is_old.unflatten(0, (-1, page)).transpose(1, 2)
            ratio = x_new * 127 / now.clamp(min=1e-300)[..., None, None]
            part = torch.where(is_old, kept, torch.round(ratio)) * now[..., None, None] / 127
            amax[ids] = now
            parts.append(part.transpose(1, 2).flatten(0, 1)[:had + int(new[b])])
        out[x] = torch.cat(parts)
        if fresh is not None:
            out[x + "_amax"] = amax
    return out
