"""Cases of the decode step's operators around the attention: page plan, norm + rotation, windowed
attention, and the 4-bit cache.

``run`` computes each operator in elementary torch operations, in 32 bits (integers in 64), or, where
``own`` is true, by the calls a program makes of ``stochastic_sparse_decode_gb300``.

The 4-bit cache: [rows][Hkv][d + d/8] bytes; a record holds the d/2 bytes of K's codes (element i in
byte i // 2, the even element in the low half), V's codes, then for K and for V the d/64 pairs (scale,
minimum) in fp16.  Element i stands for minimum_g + scale_g * code_i with g = (i // 8) mod (d / 64).
"""

import math

import numpy as np
import torch

own = False

LLAMA = {"hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"}


def listed():
    return [
        # one decode step of a serving batch: 64 sequences append a token each
        {"name": "plan_step_b64", "op": "plan", "batch": 64, "len_lo": 4096, "len_hi": 32768, "new_lo": 1, "new_hi": 1,
         "page": 64, "pad": 0},
        # 200 prompts admitted at once (some sequences already hold a prefix), token rows padded to a fixed size
        {"name": "plan_prompts_b200", "op": "plan", "batch": 200, "len_lo": 0, "len_hi": 700, "new_lo": 1, "new_hi": 8191,
         "page": 32, "pad": 77},
        # the new token of one sequence, a layer with per-head norms
        {"name": "rope_step_b1", "op": "rope", "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "rot": 128,
         "inter": False, "norm": True, "rows": 32768, "fused": True},
        # a prompt of 8191 tokens, the layer without norms, q, k and v slices of one projection
        {"name": "rope_prompt_8191", "op": "rope", "tokens": 8191, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "rot": 128,
         "inter": False, "norm": False, "rows": 16384, "fused": True},
        # a ragged fp32 batch, d = 64, neighbouring pairs, half of the elements rotated
        {"name": "rope_f32_777", "op": "rope", "tokens": 777, "hq": 16, "hkv": 4, "d": 64, "dtype": "f32", "rot": 32,
         "inter": True, "norm": True, "rows": 4096, "fused": False},
        # one sequence of 32768 tokens, window 4096 behind 4 sinks
        {"name": "window_b1_32k", "op": "window", "batch": 1, "len_lo": 32768, "len_hi": 32768, "window": 4096, "sinks": 4,
         "page": 0, **LLAMA},
        # a ragged serving batch on a paged cache
        {"name": "window_b64_ragged", "op": "window", "batch": 64, "len_lo": 4096, "len_hi": 32768, "window": 4096,
         "sinks": 4, "page": 64, **LLAMA},
        # a small fp32 model: short sequences, many of them shorter than the window
        {"name": "window_f32_b8", "op": "window", "batch": 8, "len_lo": 1, "len_hi": 1024, "window": 300, "sinks": 5,
         "page": 0, "hq": 4, "hkv": 1, "d": 64, "dtype": "f32"},
        # the whole 4-bit cache of one sequence of 32768 tokens
        {"name": "kv4_b1_32k", "op": "kv4", "batch": 1, "len_lo": 32768, "len_hi": 32768, "window": 0, "sinks": 0, "page": 0,
         **LLAMA},
        # the largest: 16 sequences of 32768 tokens
        {"name": "kv4_b16_32k", "op": "kv4", "batch": 16, "len_lo": 32768, "len_hi": 32768, "window": 0, "sinks": 0,
         "page": 64, **LLAMA},
        # a decode step stores 64 tokens' K and V in 4 bits (and reads them back)
        {"name": "store_step_b64", "op": "store", "tokens": 64, "hkv": 8, "d": 128, "dtype": "bf16", "rows": 65536},
        # a prompt of 8191 tokens into the 4-bit cache
        {"name": "store_prompt_8191", "op": "store", "tokens": 8191, "hkv": 8, "d": 128, "dtype": "bf16", "rows": 16384},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "window", "kv4", "store"])
    page = rng.choice([0, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    if op == "plan":
        b = _log(rng, 1, 300)
        hi = _log(rng, 1, max(2, 600_000 // b))
        return {"op": op, "batch": b, "len_lo": 0, "len_hi": _log(rng, 1, 32768), "new_lo": rng.choice([0, 1]), "new_hi": hi,
                "page": page or 32, "pad": rng.randrange(0, 200)}
    if op == "rope":
        t = _log(rng, 1, 8000)
        return {"op": op, "tokens": t, "hq": hkv * g, "hkv": hkv, "d": d, "dtype": dtype,
                "rot": rng.choice([d, d // 2, 16 * rng.randrange(1, d // 16 + 1)]), "inter": rng.random() < 0.4,
                "norm": rng.random() < 0.6, "rows": t + _log(rng, 1, 8000), "fused": rng.random() < 0.5}
    if op == "store":
        t = _log(rng, 1, 8000)
        return {"op": op, "tokens": t, "hkv": hkv, "d": d, "dtype": dtype, "rows": t + _log(rng, 1, 8000)}
    b = _log(rng, 1, 64)
    hi = _log(rng, 1, min(32768, (240_000 if dtype == "bf16" else 120_000) // b))
    lo = rng.choice([1, max(1, hi // 2), hi])
    win = _log(rng, 1, 8192)
    if op == "kv4" and rng.random() < 0.5:
        win = 0
    return {"op": op, "batch": b, "len_lo": lo, "len_hi": hi, "window": win, "sinks": rng.choice([0, 0, 1, 4, 37]) if win else 0,
            "page": page, "hq": hkv * g, "hkv": hkv, "d": d, "dtype": dtype}


# ---------------------------------------------------------------------------- inputs


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda", dtype=torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    s = {"case": case}
    op = case["op"]
    if op == "plan":
        _prepare_plan(s, case, gen)
    elif op == "rope":
        _prepare_rope(s, case, gen)
    elif op == "store":
        _prepare_store(s, case, gen)
    else:
        _prepare_attention(s, case, gen)
    if own:
        _prepare_own(s, case)
    return s


def _prepare_plan(s, case, gen):
    b, ps = case["batch"], case["page"]
    lens, new = _ints(gen, case["len_lo"], case["len_hi"], b), _ints(gen, case["new_lo"], case["new_hi"], b)
    # the step's token count is the program's own: every other sequence complements its neighbour
    mean = case["new_lo"] + case["new_hi"]
    new[1::2] = mean - new[0:b - b % 2:2]
    if b % 2:
        new[-1] = mean // 2
    have = (lens + ps - 1) // ps
    need = (lens + new + ps - 1) // ps - have
    s["max_pages"] = (case["len_hi"] + case["new_hi"]) // ps + 2
    n_have, n_need = int(have.sum()), int(need.sum())
    s["num_pages"] = n_have + n_need + 5
    ids = torch.randperm(s["num_pages"], generator=gen, device="cuda").to(torch.int32)
    j = torch.arange(s["max_pages"], device="cuda")
    held = j[None, :] < have[:, None]
    table = torch.full((b, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
    table[held] = ids[:n_have]
    s["table"], s["free"] = table, ids[n_have:].contiguous()
    s["lens"], s["new"] = lens.to(torch.int32), new.to(torch.int32)
    s["tokens"] = int(new.sum()) + case["pad"]
    t = max(1, s["tokens"])
    s["slots"] = torch.empty(t, dtype=torch.int64, device="cuda")
    s["positions"] = torch.empty(t, dtype=torch.int32, device="cuda")
    s["lens_out"] = torch.empty(b, dtype=torch.int32, device="cuda")
    s["counts"] = torch.empty(2, dtype=torch.int32, device="cuda")


def _prepare_rope(s, case, gen):
    t, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], _torch_dtype(case)
    if case["fused"]:  # slices of one projection's rows
        qkv = torch.randn((t, (hq + 2 * hkv), d), generator=gen, device="cuda").to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"], s["k"], s["v"] = (torch.randn((t, h, d), generator=gen, device="cuda").to(dt) for h in (hq, hkv, hkv))
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt) for _ in range(2))
    s["eps"] = 1e-6
    s["positions"] = _ints(gen, 0, 32767, t).to(torch.int32)
    s["slots"] = torch.randperm(case["rows"], generator=gen, device="cuda")[:t].contiguous()
    half = case["rot"] // 2
    freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(32768, dtype=torch.float64, device="cuda")[:, None] * freq
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)
    s["k_cache"], s["v_cache"] = (torch.randn((case["rows"], hkv, d), generator=gen, device="cuda").to(dt) for _ in range(2))
    s["out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")


def _prepare_store(s, case, gen):
    t, hkv, d, dt = case["tokens"], case["hkv"], case["d"], _torch_dtype(case)
    s["k"], s["v"] = (torch.randn((t, hkv, d), generator=gen, device="cuda").to(dt) for _ in range(2))
    s["slots"] = torch.randperm(case["rows"], generator=gen, device="cuda")[:t].contiguous()
    s["cache"] = torch.zeros((case["rows"], hkv, d + d // 8), dtype=torch.uint8, device="cuda")
    s["k_out"], s["v_out"] = (torch.empty((t, hkv, d), dtype=dt, device="cuda") for _ in range(2))


def _prepare_attention(s, case, gen):
    b, hq, hkv, d, ps, dt = case["batch"], case["hq"], case["hkv"], case["d"], case["page"], _torch_dtype(case)
    lens = _ints(gen, case["len_lo"], case["len_hi"], b)
    s["max_len"] = int(lens.max())
    s["q"] = torch.randn((b, hq, d), generator=gen, device="cuda").to(dt)
    if ps:
        have = (lens + ps - 1) // ps
        n_have = int(have.sum())
        s["max_pages"] = int(have.max()) + 1
        s["num_pages"] = n_have + 3
        ids = torch.randperm(s["num_pages"], generator=gen, device="cuda").to(torch.int32)
        held = torch.arange(s["max_pages"], device="cuda")[None, :] < have[:, None]
        s["table"] = torch.full((b, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
        s["table"][held] = ids[:n_have]
        s["rows"] = s["num_pages"] * ps
    else:
        s["rows"] = int(lens.sum())
    s["lens"] = lens.to(torch.int32)
    s["indptr"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
    # keys and values of a decode layer: normal, with one key in a hundred lined up with a query of its group
    k = torch.randn((s["rows"], hkv, d), generator=gen, device="cuda", dtype=torch.float32)
    heavy = torch.randint(0, s["rows"], (max(1, s["rows"] // 100),), generator=gen, device="cuda")
    qh = s["q"][0, ::hq // hkv].float()
    k[heavy] += 0.5 * math.sqrt(d) * qh / qh.norm(dim=-1, keepdim=True)
    v = torch.randn((s["rows"], hkv, d), generator=gen, device="cuda", dtype=torch.float32)
    if case["op"] == "kv4":
        s["cache"] = torch.cat([torch.cat([_quantise(x)[0] for x in (k, v)], -1),
                                torch.cat([_quantise(x)[1] for x in (k, v)], -1)], -1)
    else:
        s["k"], s["v"] = k.to(dt), v.to(dt)
    s["out"] = torch.empty((b, hq, d), dtype=torch.float32, device="cuda")


def _prepare_own(s, case):
    """The handle that a program keeps from call to call."""
    from stochastic_sparse_decode_gb300.decoder import Decoder

    op = case["op"]
    rows = {"plan": lambda: s["num_pages"] * case["page"], "rope": lambda: case["rows"],
            "store": lambda: case["rows"]}.get(op, lambda: s["rows"])()
    s["dec"] = Decoder(batch=case.get("batch", 1), num_q_heads=case.get("hq", case.get("hkv", 1)),
                       num_kv_heads=case.get("hkv", 1), head_dim=case.get("d", 128), total_tokens=rows,
                       max_len=s.get("max_len", rows), tile=256, S=1, dtype=case.get("dtype", "bf16"))


# ---------------------------------------------------------------------------- one pass


def run(s):
    return {"plan": _run_plan, "rope": _run_rope, "window": _run_window, "kv4": _run_kv4,
            "store": _run_store}[s["case"]["op"]](s)


def _run_plan(s):
    ps = s["case"]["page"]
    if own:
        s["dec"].page_plan(s["lens"], s["new"], s["table"], s["free"], ps, s["slots"], s["positions"], s["lens_out"],
                           s["counts"])
        return s["table"], s["slots"], s["positions"], s["lens_out"], s["counts"]
    lens, new, table, free = s["lens"].long(), s["new"].long(), s["table"], s["free"]
    have = (lens + ps - 1) // ps
    need = (lens + new + ps - 1) // ps - have
    off = need.cumsum(0) - need
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    at = (off[:, None] + j - have[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at], table)
    ends = new.cumsum(0)
    t = torch.arange(s["slots"].numel(), device="cuda")
    b = torch.searchsorted(ends, t, right=True)
    real = b < lens.numel()
    b = b.clamp(max=lens.numel() - 1)
    pos = lens[b] + t - (ends - new)[b]
    page = table[b, torch.where(real, pos // ps, 0)].long()
    slots = torch.where(real, page * ps + pos % ps, -1)
    positions = torch.where(real, pos, 0).to(torch.int32)
    counts = torch.stack([need.sum(), ends[-1]]).to(torch.int32)
    return table, slots, positions, (lens + new).to(torch.int32), counts


def _turn(x, w, s):
    """Norm over the head's elements and rotation of the first ``rot`` of them, in fp32."""
    rot, half, dt = s["case"]["rot"], s["case"]["rot"] // 2, x.dtype
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :half], cs[..., half:]
    y = x.clone()
    if s["case"]["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(dt)


def _run_rope(s):
    if own:
        s["dec"].norm_rope(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["k_cache"], s["v_cache"],
                           q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], interleaved=s["case"]["inter"], out=s["out"])
        return s["out"], s["k_cache"], s["v_cache"]
    s["k_cache"][s["slots"]] = _turn(s["k"], s["kw"], s)
    s["v_cache"][s["slots"]] = s["v"]
    return _turn(s["q"], s["qw"], s), s["k_cache"], s["v_cache"]


def _visible(s):
    """Cache rows [B][N] of each sequence's visible keys, and which of them are keys."""
    c = s["case"]
    lens, n_max = s["lens"].long(), s["max_len"]
    win = c["window"] or n_max
    n_max = min(n_max, win + c["sinks"])
    sinks = lens.clamp(max=c["sinks"])
    lo = torch.maximum(lens - win, sinks)
    j = torch.arange(n_max, device="cuda")[None, :]
    pos = torch.where(j < sinks[:, None], j, lo[:, None] + j - sinks[:, None])
    valid = pos < lens[:, None]
    pos = torch.where(valid, pos, 0)
    if c["page"]:
        rows = torch.gather(s["table"].long(), 1, pos // c["page"]) * c["page"] + pos % c["page"]
    else:
        rows = s["indptr"][:-1, None] + pos
    return torch.where(valid, rows, 0), valid


def _attend(q, k, v, valid):
    """q [B][Hq][d], k and v [B][N][Hkv][d] in fp32."""
    b, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().view(b, hkv, hq // hkv, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    x = x.masked_fill(~valid[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(z > 0, z, 1.0)
    return o.reshape(b, hq, d)


def _run_window(s):
    c = s["case"]
    if own:
        if c["page"]:
            return s["dec"].window_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], c["page"], c["window"], c["sinks"],
                                         out=s["out"])
        return s["dec"].window(s["q"], s["k"], s["v"], s["indptr"], c["window"], c["sinks"], out=s["out"])
    rows, valid = _visible(s)
    return _attend(s["q"], s["k"][rows].float(), s["v"][rows].float(), valid)


def _quantise(x):
    """Codes [..][d / 2] and parameters [..][d / 16] (bytes of the fp16 pairs) of rows x [..][d]."""
    d = x.shape[-1]
    x = x.float().unflatten(-1, (d // 8 // (d // 64), d // 64, 8))  # [..][block pair][group][8]
    lo = x.amin((-3, -1), keepdim=True).to(torch.float16)
    hi = x.amax((-3, -1), keepdim=True)
    scale = ((hi - lo.float()) * (1.0 / 15.0)).to(torch.float16)
    safe = torch.where(scale > 0, scale, 1.0).float()
    n = torch.round((x - lo.float()) / safe).clamp(0, 15)
    n = torch.where(scale > 0, n, 0.0).to(torch.uint8).flatten(-3).unflatten(-1, (d // 2, 2))
    pairs = torch.cat([scale, lo], -1).flatten(-3).contiguous()  # [..][group][scale, minimum]
    return n[..., 0] | (n[..., 1] << 4), pairs.view(torch.uint8)


def _values(codes, pairs):
    """The fp32 values [..][d] of codes [..][d / 2] and parameter bytes."""
    d = codes.shape[-1] * 2
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (d // 8 // (d // 64), d // 64, 8))
    p = pairs.contiguous().view(torch.float16).float().unflatten(-1, (1, d // 64, 1, 2))
    return (p[..., 1] + p[..., 0] * n).flatten(-3)


def _record(rec):
    """K and V in fp32 of 4-bit records [..][d + d / 8]."""
    d = rec.shape[-1] * 8 // 9
    a, b, c = d // 2, d, d + d // 16
    return _values(rec[..., :a], rec[..., b:c]), _values(rec[..., a:b], rec[..., c:])


def _run_kv4(s):
    c = s["case"]
    if own:
        if c["page"]:
            return s["dec"].kv4_paged(s["q"], s["cache"], s["table"], s["lens"], c["page"], c["window"], c["sinks"],
                                      out=s["out"])
        return s["dec"].kv4(s["q"], s["cache"], s["indptr"], c["window"], c["sinks"], out=s["out"])
    rows, valid = _visible(s)
    k, v = _record(s["cache"][rows])
    return _attend(s["q"], k, v, valid)


def _run_store(s):
    if own:
        s["dec"].kv4_append(s["k"], s["v"], s["slots"], s["cache"])
        return s["dec"].kv4_read(s["cache"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    (kc, kp), (vc, vp) = _quantise(s["k"]), _quantise(s["v"])
    s["cache"][s["slots"]] = torch.cat([kc, vc, kp, vp], -1)
    k, v = _record(s["cache"][s["slots"]])
    return k.to(s["k"].dtype), v.to(s["v"].dtype)


# ---------------------------------------------------------------------------- what a pass cannot do without


def _visible_keys(case):
    """Expected visible keys of a case (mean over the lengths' range), all sequences."""
    lens = np.linspace(case["len_lo"], case["len_hi"], 257)
    seen = np.minimum(lens, case["window"] + case["sinks"]) if case["window"] else lens
    return case["batch"] * float(seen.mean())


def work(case):
    op, es = case["op"], 2 if case.get("dtype") == "bf16" else 4
    if op == "plan":
        b, tokens = case["batch"], case["batch"] * (case["new_lo"] + case["new_hi"]) / 2
        return {"bytes": 12 * b + 12 * (tokens + case["pad"]) + 8 * tokens / case["page"], "flops": 0}
    if op == "rope":
        row = case["d"] * es
        return {"bytes": case["tokens"] * (2 * row * (case["hq"] + 2 * case["hkv"]) + 4 * case["rot"] + 12),
                "flops": case["tokens"] * (case["hq"] + case["hkv"]) * (3 * case["rot"] + 4 * case["d"] * case["norm"])}
    if op == "store":  # rows in, records out, records in, rows out
        return {"bytes": case["tokens"] * (case["hkv"] * (4 * case["d"] * es + 2 * (case["d"] + case["d"] // 8)) + 8),
                "flops": case["tokens"] * case["hkv"] * 12 * case["d"]}
    keys, d = _visible_keys(case), case["d"]
    per_key = case["hkv"] * (2 * d * es if op == "window" else d + d // 8)
    return {"bytes": keys * per_key + case["batch"] * case["hq"] * d * (es + 4), "flops": keys * case["hq"] * 4 * d}


# ---------------------------------------------------------------------------- the definitions in 64 bits


def _exact_rows(s, b):
    """Cache rows of the visible keys of sequence b."""
    c, n = s["case"], int(s["lens"][b])
    keep = [i for i in range(n) if not c["window"] or i < c["sinks"] or i >= n - c["window"]]
    pos = torch.tensor(keep, dtype=torch.int64, device="cuda")
    if c["page"]:
        return s["table"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]
    return int(s["indptr"][b]) + pos


def _exact_values(codes, pairs, d):
    i = torch.arange(d, device="cuda")
    n = ((codes.long()[..., i // 2] >> (4 * (i % 2))) & 15).double()
    p = pairs.contiguous().view(torch.float16).double()
    g = (i // 8) % (d // 64)
    return p[..., 2 * g + 1] + p[..., 2 * g] * n


def _exact_attention(s):
    c = s["case"]
    d, hkv = c["d"], c["hkv"]
    out = torch.zeros((c["batch"], c["hq"], d), dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        rows = _exact_rows(s, b)
        if not rows.numel():
            continue
        for g in range(hkv):
            if c["op"] == "kv4":
                r = s["cache"][rows, g]
                k = _exact_values(r[:, :d // 2], r[:, d:d + d // 16], d)
                v = _exact_values(r[:, d // 2:d], r[:, d + d // 16:], d)
            else:
                k, v = s["k"][rows, g].double(), s["v"][rows, g].double()
            heads = slice(g * (c["hq"] // hkv), (g + 1) * (c["hq"] // hkv))
            x = (s["q"][b, heads].double() @ k.T) / math.sqrt(d)
            out[b, heads] = torch.softmax(x, -1) @ v
    return out


def _exact_rope(s):
    c = s["case"]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + s["eps"]) * w.double()
        half = c["rot"] // 2
        cs = s["cos_sin"].double()[s["positions"].long()]
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
            co, si = cs[:, i, None], cs[:, half + i, None]
            y[..., a] = x[..., a] * co - x[..., b] * si
            y[..., b] = x[..., b] * co + x[..., a] * si
        return y

    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[s["slots"]], v[s["slots"]] = one(s["k"], s["kw"]), s["v"].double()
    return one(s["q"], s["qw"]), k, v


def _exact_store(s):
    d = s["case"]["d"]
    group = (np.arange(d) // 8) % (d // 64)

    def one(x):
        x = x.double().cpu().numpy()
        y = np.empty_like(x)
        for g in range(d // 64):
            r = x[..., group == g]
            lo = r.min(-1, keepdims=True).astype(np.float16).astype(np.float64)
            step = ((r.max(-1, keepdims=True) - lo) / 15).astype(np.float16).astype(np.float64)
            n = np.clip(np.rint((r - lo) / np.where(step > 0, step, 1)), 0, 15)
            y[..., group == g] = lo + step * np.where(step > 0, n, 0)
        return y

    return one(s["k"]), one(s["v"])


def _exact_plan(s):
    ps, lens, new = s["case"]["page"], s["lens"].tolist(), s["new"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    slots, positions = np.full(s["slots"].numel(), -1, np.int64), np.zeros(s["slots"].numel(), np.int32)
    taken = t = 0
    for b in range(len(lens)):
        for p in range(lens[b], lens[b] + new[b]):
            if p % ps == 0:
                table[b, p // ps] = free[taken]
                taken += 1
            slots[t], positions[t] = int(table[b, p // ps]) * ps + p % ps, p
            t += 1
    return table, slots, positions, np.array(lens, np.int32) + np.array(new, np.int32), np.array([taken, t], np.int32)


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "store": _exact_store}.get(case["op"], _exact_attention)(s)
