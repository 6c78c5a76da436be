"""Cases of four more operators of the decode step: rotation by several position axes, attention for a
batch that shares a prefix, accumulated attention weights of the cached keys, and eviction by them.

``run`` computes each operator in elementary torch operations, in 32 bits, or, where ``own`` is true, by
the calls a program makes of ``stochastic_sparse_decode_gb300``.
"""

import math

import numpy as np
import torch

own = False

LLAMA = {"hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"}


def listed():
    return [
        # one decode step of 16 sequences of a model for images and text: time, height, width in sections
        {"name": "axes_step_b16", "op": "axes", "tokens": 16, "rot": 128, "kind": "sections", "axes": 3, "inter": False,
         "norm": False, "rows": 32768, "fused": True, **LLAMA},
        # a prompt of 8191 tokens with images in it, the layer with per-head norms, axes in turn from pair to pair
        {"name": "axes_prompt_8191", "op": "axes", "tokens": 8191, "rot": 128, "kind": "turns", "axes": 3, "inter": False,
         "norm": True, "rows": 16384, "fused": True, **LLAMA},
        # rows and columns of an image's 777 patches, fp32, neighbouring pairs, half of the elements rotated
        {"name": "axes_f32_777", "op": "axes", "tokens": 777, "rot": 32, "kind": "own", "axes": 2, "inter": True,
         "norm": True, "rows": 4096, "fused": False, "hq": 16, "hkv": 4, "d": 64, "dtype": "f32"},
        # four answers to one short prompt
        {"name": "shared_b4_1000", "op": "shared", "batch": 4, "prefix": 1000, "len_lo": 1, "len_hi": 64, "page": 0, **LLAMA},
        # sixteen requests behind a system prompt, d = 64, one query head per KV head, odd lengths
        {"name": "shared_b16_8191", "op": "shared", "batch": 16, "prefix": 8191, "len_lo": 0, "len_hi": 700, "page": 0,
         "hq": 8, "hkv": 8, "d": 64, "dtype": "bf16"},
        # the largest: 64 requests over one document of 32768 tokens, paged
        {"name": "shared_b64_32k", "op": "shared", "batch": 64, "prefix": 32768, "len_lo": 1, "len_hi": 512, "page": 64,
         **LLAMA},
        # a small fp32 model
        {"name": "shared_f32_b8", "op": "shared", "batch": 8, "prefix": 1023, "len_lo": 1, "len_hi": 200, "page": 32,
         "hq": 4, "hkv": 1, "d": 64, "dtype": "f32"},
        # one sequence of 32768 tokens after a decode step: every key's weight is added to its score
        {"name": "weights_b1_32k", "op": "weights", "batch": 1, "len_lo": 32768, "len_hi": 32768, "page": 0, **LLAMA},
        # a ragged serving batch on a paged cache
        {"name": "weights_b16_ragged", "op": "weights", "batch": 16, "len_lo": 4096, "len_hi": 32768, "page": 64, **LLAMA},
        # the prompt of one sequence is cut to 1024 keys per head
        {"name": "evict_b1_8192", "op": "evict", "batch": 1, "len_lo": 8192, "len_hi": 8192, "sinks": 4, "recent": 256,
         "budget": 764, "page": 0, **LLAMA},
        # a ragged serving batch, cut into fewer pages
        {"name": "evict_b16_ragged", "op": "evict", "batch": 16, "len_lo": 4096, "len_hi": 32768, "sinks": 4, "recent": 1020,
         "budget": 1024, "page": 64, **LLAMA},
        # a small fp32 model, some sequences shorter than what is kept
        {"name": "evict_f32_b8", "op": "evict", "batch": 8, "len_lo": 1, "len_hi": 1024, "sinks": 5, "recent": 33,
         "budget": 100, "page": 32, "hq": 4, "hkv": 1, "d": 64, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "shared", "weights", "evict"])
    page = rng.choice([0, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    heads = {"hq": hkv * g, "hkv": hkv, "d": d, "dtype": dtype}
    if op == "axes":
        t = _log(rng, 1, 8000 * 48 // max(48, (g + 2) * hkv * (2 if dtype == "f32" else 1)))
        return {"op": op, "tokens": t, "rot": rng.choice([d, d // 2, 16 * rng.randrange(1, d // 16 + 1)]),
                "kind": rng.choice(["sections", "turns", "own"]), "axes": rng.choice([1, 2, 3, 4]),
                "inter": rng.random() < 0.4, "norm": rng.random() < 0.6, "rows": t + _log(rng, 1, 8000),
                "fused": rng.random() < 0.5, **heads}
    if op == "shared":
        b = _log(rng, 1, 64)
        most = min(32768, (1 << 23 if dtype == "bf16" else 1 << 18) // (b * g))
        return {"op": op, "batch": b, "prefix": _log(rng, 1, most), "len_lo": rng.choice([0, 1]),
                "len_hi": _log(rng, 1, 32768 // b), "page": page, **heads}
    b = _log(rng, 1, 32)
    hi = _log(rng, 1, min(32768, (200_000 if dtype == "bf16" else 100_000) // b))
    lo = rng.choice([1, max(1, hi // 2), hi])
    if op == "weights":
        return {"op": op, "batch": b, "len_lo": lo, "len_hi": hi, "page": page, **heads}
    return {"op": op, "batch": b, "len_lo": lo, "len_hi": hi, "sinks": rng.choice([0, 1, 4, 37]),
            "recent": rng.choice([0, _log(rng, 1, 1000)]), "budget": _log(rng, 1, max(2, hi // 2)), "page": page, **heads}


# ---------------------------------------------------------------------------- inputs


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda", dtype=torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 6271 + 5)
    s = {"case": case}
    {"axes": _prepare_axes, "shared": _prepare_shared, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](
        s, case, gen)
    if own:
        _prepare_own(s, case)
    return s


def _pair_axes(case):
    """The axis of each pair: runs of pairs, in turn, or runs whose frequencies begin anew on each axis."""
    half, n = case["rot"] // 2, case["axes"]
    if case["kind"] == "turns":
        return [i % n for i in range(half)]
    return [min(i * n // half, n - 1) for i in range(half)]


def _prepare_axes(s, case, gen):
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
    # the first axis is the time, the others a place within an image
    s["positions"] = torch.stack([_ints(gen, 0, 8191 if a == 0 else 99, t) for a in range(case["axes"])]).to(torch.int32)
    s["slots"] = torch.randperm(case["rows"], generator=gen, device="cuda")[:t].contiguous()
    s["axis"] = _pair_axes(case)
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device="cuda")
    span = half
    if case["kind"] == "own":  # the place of a pair within its axis's run
        starts = torch.tensor([s["axis"].index(a) for a in s["axis"]], device="cuda")
        i, span = i - starts, -(-half // case["axes"])
    freq = 10000.0 ** (-i / span)
    ang = torch.arange(8192, dtype=torch.float64, device="cuda")[:, None] * freq
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)
    s["axis_t"] = torch.tensor(s["axis"], device="cuda")
    s["k_cache"], s["v_cache"] = (torch.randn((case["rows"], hkv, d), generator=gen, device="cuda").to(dt) for _ in range(2))
    s["out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")


def _cache_rows(s, case, gen, lens, most):
    """Pages of sequences of these lengths, or their contiguous rows, in a cache that has room for `most` keys each."""
    b, ps = lens.numel(), case["page"]
    s["lens"] = lens.to(torch.int32)
    s["indptr"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
    if not ps:
        return b * max(1, most)
    have = (lens + ps - 1) // ps
    s["max_pages"] = int(have.max()) + 1
    num_pages = b * (-(-most // ps)) + 3
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    held = torch.arange(s["max_pages"], device="cuda")[None, :] < have[:, None]
    s["table"] = torch.full((b, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
    s["table"][held] = ids[:int(have.sum())]
    return num_pages * ps


def _keys(s, case, gen):
    """Keys of a decode layer: normal, with one in a hundred lined up with a query of its group."""
    hq, hkv, d, rows = case["hq"], case["hkv"], case["d"], s["rows"]
    k = torch.randn((rows, hkv, d), generator=gen, device="cuda", dtype=torch.float32)
    heavy = torch.randint(0, rows, (max(1, rows // 100),), generator=gen, device="cuda")
    qh = s["q"][0, ::hq // hkv].float()
    k[heavy] += 0.5 * math.sqrt(d) * qh / qh.norm(dim=-1, keepdim=True)
    return k.to(_torch_dtype(case))


def _prepare_shared(s, case, gen):
    b, hq, hkv, d, ps, dt = case["batch"], case["hq"], case["hkv"], case["d"], case["page"], _torch_dtype(case)
    lens, prefix = _ints(gen, case["len_lo"], case["len_hi"], b), case["prefix"]
    s["q"] = torch.randn((b, hq, d), generator=gen, device="cuda").to(dt)
    if ps:  # every sequence's table begins with the prefix's pages; a prefix that ends inside a page leaves it whole
        prefix = s["prefix"] = max(ps, prefix // ps * ps)
        shared = prefix // ps
        rows = _cache_rows(s, case, gen, lens, case["len_hi"])
        first = rows // ps
        ids = torch.randperm(first + shared, generator=gen, device="cuda").to(torch.int32)
        own_part = s["table"]
        own_part = torch.where(own_part >= 0, ids[own_part.long().clamp(min=0)], own_part)
        s["table"] = torch.cat([ids[first:].expand(b, shared), own_part], 1).contiguous()
        s["max_pages"] += shared
        s["rows"] = rows + prefix
        s["lens"] = (lens + prefix).to(torch.int32)
        s["max_len"] = int(s["lens"].max())
    else:  # the prefix's rows lie before the sequences' own
        s["prefix"] = prefix
        rows = _cache_rows(s, case, gen, lens, case["len_hi"])
        s["rows"] = prefix + rows
        s["indptr"] += prefix
        s["max_len"] = int(lens.max())
    s["own_lens"] = lens
    s["k"] = _keys(s, case, gen)
    s["v"] = torch.randn((s["rows"], hkv, d), generator=gen, device="cuda", dtype=torch.float32).to(dt)
    s["out"] = torch.empty((b, hq, d), dtype=torch.float32, device="cuda")


def _prepare_weights(s, case, gen):
    b, hq, d, dt = case["batch"], case["hq"], case["d"], _torch_dtype(case)
    lens = _ints(gen, case["len_lo"], case["len_hi"], b)
    s["max_len"] = int(lens.max())
    s["q"] = torch.randn((b, hq, d), generator=gen, device="cuda").to(dt)
    s["rows"] = _cache_rows(s, case, gen, lens, case["len_hi"])
    s["k"] = _keys(s, case, gen)
    # scores of some steps before; the last key is new and starts from nothing
    s["scores"] = torch.rand((case["hkv"], s["rows"]), generator=gen, device="cuda") * (8.0 / max(8, s["max_len"]))
    s["scores_out"] = torch.zeros_like(s["scores"])
    s["decay"], s["fresh"] = 0.97, 1


def _prepare_evict(s, case, gen):
    b, hkv, d, ps, dt = case["batch"], case["hkv"], case["d"], case["page"], _torch_dtype(case)
    lens = _ints(gen, case["len_lo"], case["len_hi"], b)
    s["max_len"] = int(lens.max())
    s["rows"] = _cache_rows(s, case, gen, lens, case["len_hi"])
    s["k"], s["v"] = (torch.randn((s["rows"], hkv, d), generator=gen, device="cuda", dtype=torch.float32).to(dt)
                      for _ in range(2))
    # few keys have most of the weight; a tenth never had any
    scores = torch.rand((hkv, s["rows"]), generator=gen, device="cuda")
    s["scores"] = torch.where(scores < 0.1, 0.0, scores ** 8)
    s["keep"] = case["sinks"] + case["recent"] + case["budget"]
    src = {n: s.get(n) for n in ("lens", "indptr", "table", "max_pages")}
    s["rows_out"] = _cache_rows(s, case, gen, lens.clamp(max=s["keep"]), min(s["keep"], case["len_hi"]))
    s["indptr_out"], s["table_out"] = s["indptr"], s.get("table")
    s.update(src)
    s["k_out"], s["v_out"] = (torch.zeros((s["rows_out"], hkv, d), dtype=dt, device="cuda") for _ in range(2))
    s["scores_out"] = torch.zeros((hkv, s["rows_out"]), dtype=torch.float32, device="cuda")
    s["kept"] = torch.empty((b, hkv, s["keep"]), dtype=torch.int32, device="cuda")
    s["lens_out"] = torch.empty(b, dtype=torch.int32, device="cuda")


def _prepare_own(s, case):
    """The handle that a program keeps from call to call."""
    from stochastic_sparse_decode_gb300.decoder import Decoder

    rows = case["rows"] if case["op"] == "axes" else s["rows"]
    s["dec"] = Decoder(batch=case.get("batch", 1), num_q_heads=case["hq"], num_kv_heads=case["hkv"], head_dim=case["d"],
                       total_tokens=rows, max_len=s.get("max_len", rows), tile=256, S=1, dtype=case["dtype"])


# ---------------------------------------------------------------------------- one pass


def run(s):
    return {"axes": _run_axes, "shared": _run_shared, "weights": _run_weights, "evict": _run_evict}[s["case"]["op"]](s)


def _turn(x, w, s):
    """Norm over the head's elements and rotation of the first ``rot`` of them, in fp32."""
    rot, half, dt = s["case"]["rot"], s["case"]["rot"] // 2, x.dtype
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    pair = torch.arange(half, device="cuda")
    n = s["positions"].long()[s["axis_t"]].T  # [tokens][pairs]
    cos, sin = s["cos_sin"][n, pair][:, None], s["cos_sin"][n, half + pair][:, None]
    y = x.clone()
    if s["case"]["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(dt)


def _run_axes(s):
    if own:
        s["dec"].norm_rope_axes(s["q"], s["k"], s["v"], s["positions"], s["axis"], s["slots"], s["cos_sin"], s["k_cache"],
                                s["v_cache"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                                interleaved=s["case"]["inter"], out=s["out"])
        return s["out"], s["k_cache"], s["v_cache"]
    s["k_cache"][s["slots"]] = _turn(s["k"], s["kw"], s)
    s["v_cache"][s["slots"]] = s["v"]
    return _turn(s["q"], s["qw"], s), s["k_cache"], s["v_cache"]


def _rows(s, n_max, lens=None, first=0, table="table", indptr="indptr"):
    """Cache rows [B][N] of keys first, first + 1, ... of each sequence (of `lens` keys), and which of them there are."""
    lens = s["lens"].long() if lens is None else lens
    pos = first + torch.arange(n_max, device="cuda")[None, :]
    valid = pos < lens[:, None]
    pos = torch.where(valid, pos, 0)
    ps = s["case"]["page"]
    rows = torch.gather(s[table].long(), 1, pos // ps) * ps + pos % ps if ps else s[indptr][:-1, None] + pos
    return torch.where(valid, rows, 0), valid


def _run_shared(s):
    c, prefix = s["case"], s["prefix"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    if own:
        if c["page"]:
            return s["dec"].shared_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], c["page"], prefix, out=s["out"])
        return s["dec"].shared(s["q"], s["k"], s["v"], s["indptr"], 0, prefix, out=s["out"])
    if c["page"]:
        ps = c["page"]
        at = (s["table"][0, :prefix // ps, None].long() * ps + torch.arange(ps, device="cuda")).flatten()
        rows, valid = _rows(s, c["len_hi"], first=prefix)
    else:
        at = torch.arange(prefix, device="cuda")
        rows, valid = _rows(s, c["len_hi"], s["own_lens"])
    q = s["q"].float().view(b, hkv, hq // hkv, d) / math.sqrt(d)
    qs = q.transpose(0, 1).flatten(1, 2)  # the batch's queries of a KV head, [Hkv][B G][d]
    kp, vp = (s[x][at].float().transpose(0, 1) for x in ("k", "v"))  # [Hkv][P][d]
    x0 = torch.matmul(qs, kp.transpose(1, 2)).view(hkv, b, hq // hkv, prefix).transpose(0, 1)
    k, v = s["k"][rows].float().transpose(1, 2), s["v"][rows].float().transpose(1, 2)  # [B][Hkv][N][d]
    v = v.masked_fill(~valid[:, None, :, None], 0.0)
    x1 = torch.matmul(q, k.transpose(2, 3)).masked_fill(~valid[:, None, None, :], -math.inf)
    m = torch.maximum(x0.amax(-1, keepdim=True), x1.amax(-1, keepdim=True))
    e0, e1 = torch.exp(x0 - m), torch.exp(x1 - m)
    z = e0.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True)
    o0 = torch.matmul(e0.transpose(0, 1).flatten(1, 2), vp).view(hkv, b, hq // hkv, d).transpose(0, 1)
    return ((o0 + torch.matmul(e1, v)) / z).reshape(b, hq, d)


def _run_weights(s):
    c = s["case"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    if own:
        if c["page"]:
            return s["dec"].key_weights_paged(s["q"], s["k"], s["table"], s["lens"], c["page"], s["scores"],
                                              out=s["scores_out"], decay=s["decay"], fresh=s["fresh"])
        return s["dec"].key_weights(s["q"], s["k"], s["indptr"], s["scores"], out=s["scores_out"], decay=s["decay"],
                                    fresh=s["fresh"])
    rows, valid = _rows(s, s["max_len"])
    q = s["q"].float().view(b, hkv, hq // hkv, d) / math.sqrt(d)
    x = torch.matmul(q, s["k"][rows].float().permute(0, 2, 3, 1)).masked_fill(~valid[:, None, None, :], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    w = (e / e.sum(-1, keepdim=True)).sum(2).transpose(0, 1)[:, valid]  # [Hkv][keys]
    old = torch.arange(s["max_len"], device="cuda")[None, :] < s["lens"].long()[:, None] - s["fresh"]
    at = rows[valid]
    s["scores_out"][:, at] = torch.where(old[valid], s["decay"] * s["scores"][:, at], 0.0) + w
    return s["scores_out"]


def _run_evict(s):
    c, keep = s["case"], s["keep"]
    if own:
        if c["page"]:
            s["dec"].evict_paged(s["k"], s["v"], s["scores"], s["table"], s["lens"], c["page"], c["sinks"], c["recent"],
                                 c["budget"], s["k_out"], s["v_out"], s["scores_out"], s["table_out"], s["kept"], s["lens_out"])
        else:
            s["dec"].evict(s["k"], s["v"], s["scores"], s["indptr"], c["sinks"], c["recent"], c["budget"], s["k_out"],
                           s["v_out"], s["scores_out"], s["indptr_out"], s["kept"], s["lens_out"])
        return s["k_out"], s["v_out"], s["scores_out"], s["kept"], s["lens_out"]
    hkv, n = c["hkv"], s["max_len"]
    lens = s["lens"].long()[:, None]
    rows, valid = _rows(s, n)
    pos = torch.arange(n, device="cuda")[None, :]
    always = (pos < c["sinks"]) | (pos >= lens - c["recent"])
    sc = s["scores"][:, rows].transpose(0, 1)  # [B][Hkv][N]
    # first what is always kept, then by score (ties: the lowest index), behind all what is no key
    rank = torch.where(always[:, None], math.inf, sc).masked_fill(~valid[:, None], -math.inf)
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)[..., :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]))
    lens_out = torch.minimum(lens, torch.full_like(lens, keep))
    there = torch.arange(keep, device="cuda") < lens_out  # [B][keep]
    kept = torch.where(there[:, None], order, n).sort(-1).values  # in the order of the sequence
    rows_out, _ = _rows(s, keep, lens_out[:, 0], table="table_out", indptr="indptr_out")
    src = torch.gather(rows[:, None].expand(-1, hkv, -1), 2, kept.clamp(max=n - 1))
    h = torch.arange(hkv, device="cuda")[None, :, None].expand(src.shape)
    ok = there[:, None].expand(src.shape)
    to = rows_out[:, None].expand(src.shape)[ok]
    src, h = src[ok], h[ok]
    s["k_out"][to, h], s["v_out"][to, h] = s["k"][src, h], s["v"][src, h]
    s["scores_out"][h, to] = s["scores"][h, src]
    return s["k_out"], s["v_out"], s["scores_out"], torch.where(ok, kept, -1).to(torch.int32), lens_out[:, 0].to(torch.int32)


# ---------------------------------------------------------------------------- what a pass cannot do without


def _mean(lo, hi, f=lambda n: n):
    """Mean of f over lengths spread evenly over [lo, hi]."""
    return float(f(np.linspace(lo, hi, 257)).mean())


def work(case):
    op, es, d, hq, hkv = case["op"], 2 if case["dtype"] == "bf16" else 4, case["d"], case["hq"], case["hkv"]
    if op == "axes":
        return {"bytes": case["tokens"] * (2 * d * es * (hq + 2 * hkv) + 4 * case["rot"] + 4 * case["axes"] + 8),
                "flops": case["tokens"] * (hq + hkv) * (3 * case["rot"] + 4 * d * case["norm"])}
    b = case["batch"]
    if op == "shared":
        prefix = max(case["page"], case["prefix"] // case["page"] * case["page"]) if case["page"] else case["prefix"]
        keys = b * _mean(case["len_lo"], case["len_hi"])
        return {"bytes": (prefix + keys) * hkv * 2 * d * es + b * hq * d * (es + 4), "flops": (b * prefix + keys) * hq * 4 * d}
    keys = b * _mean(case["len_lo"], case["len_hi"])
    if op == "weights":
        return {"bytes": keys * hkv * (d * es + 8) + b * hq * d * es, "flops": keys * hq * 2 * d}
    kept = b * _mean(case["len_lo"], case["len_hi"],
                     lambda n: np.minimum(n, case["sinks"] + case["recent"] + case["budget"]))
    return {"bytes": hkv * (4 * keys + kept * (4 * d * es + 8)), "flops": keys * hkv}


# ---------------------------------------------------------------------------- the definitions in 64 bits


def _exact_axes(s):
    c = s["case"]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + s["eps"]) * w.double()
        half = c["rot"] // 2
        y = x.clone()
        for i, axis in enumerate(_pair_axes(c)):
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + half)
            row = s["cos_sin"].double()[s["positions"][axis].long()]
            co, si = row[:, i, None], row[:, half + i, None]
            y[..., a] = x[..., a] * co - x[..., b] * si
            y[..., b] = x[..., b] * co + x[..., a] * si
        return y

    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[s["slots"]], v[s["slots"]] = one(s["k"], s["kw"]), s["v"].double()
    return one(s["q"], s["qw"]), k, v


def _exact_row(s, b, n, table="table", indptr="indptr"):
    """Cache rows of the first n keys of sequence b."""
    ps, pos = s["case"]["page"], torch.arange(n, device="cuda")
    return s[table][b].long()[pos // ps] * ps + pos % ps if ps else int(s[indptr][b]) + pos


def _exact_shared(s):
    c = s["case"]
    d, g = c["d"], c["hq"] // c["hkv"]
    out = torch.zeros((c["batch"], c["hq"], d), dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        if c["page"]:
            rows = _exact_row(s, b, int(s["lens"][b]))
        else:
            rows = torch.cat([torch.arange(s["prefix"], device="cuda"), _exact_row(s, b, int(s["own_lens"][b]))])
        for h in range(c["hkv"]):
            heads = slice(h * g, (h + 1) * g)
            x = s["q"][b, heads].double() @ s["k"][rows, h].double().T / math.sqrt(d)
            out[b, heads] = torch.softmax(x, -1) @ s["v"][rows, h].double()
    return out


def _exact_weights(s):
    c = s["case"]
    g, out = c["hq"] // c["hkv"], s["scores_out"].double()
    for b in range(c["batch"]):
        n = int(s["lens"][b])
        rows = _exact_row(s, b, n)
        for h in range(c["hkv"]):
            x = s["q"][b, h * g:(h + 1) * g].double() @ s["k"][rows, h].double().T / math.sqrt(c["d"])
            before = s["decay"] * s["scores"][h, rows].double()
            before[max(0, n - s["fresh"]):] = 0
            out[h, rows] = before + torch.softmax(x, -1).sum(0)
    return out


def _exact_evict(s):
    c = s["case"]
    k, v, sc = s["k_out"].double(), s["v_out"].double(), s["scores_out"].double()
    kept = np.full(tuple(s["kept"].shape), -1, np.int32)
    lens_out = np.zeros(c["batch"], np.int32)
    scores = s["scores"].cpu().numpy()
    for b in range(c["batch"]):
        n = int(s["lens"][b])
        rows = _exact_row(s, b, n)
        host = rows.cpu().numpy()
        m = lens_out[b] = min(n, s["keep"])
        to = _exact_row(s, b, m, "table_out", "indptr_out")
        for h in range(c["hkv"]):
            index = np.arange(n)
            middle = index[c["sinks"]:max(c["sinks"], n - c["recent"])]
            best = middle[np.argsort(-scores[h, host[middle]], kind="stable")[:c["budget"]]]
            rest = np.setdiff1d(index, middle)
            chosen = np.sort(np.concatenate([rest, best]))[:m]
            kept[b, h, :m] = chosen
            at = rows[torch.from_numpy(chosen).cuda()]
            k[to, h], v[to, h], sc[h, to] = s["k"][at, h].double(), s["v"][at, h].double(), s["scores"][h, at].double()
    return k, v, sc, kept, lens_out


def exact(case, seed):
    s = prepare(case, seed)
    return {"axes": _exact_axes, "shared": _exact_shared, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)
