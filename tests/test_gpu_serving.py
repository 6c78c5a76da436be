"""The operators around the attention, on the GPU: page plan, norm + rotation, windowed attention, the
4-bit cache, and a run of them together.

Every operator is compared with a plain implementation in 64 bits (integers: exactly).  Tolerances come from
the arithmetic: u is the unit of the sums (fp32 2^-24; sums on the tensor cores are counted at 2^-23, because
they may truncate), a rounding of the output to its type is half a step, torch.finfo(t).eps / 2.
"""

import math

import numpy as np
import pytest
import torch

import stochastic_sparse_decode_gb300 as sd
from stochastic_sparse_decode_gb300.decoder import Decoder, rope_table

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="session", autouse=True)
def built_library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from stochastic_sparse_decode_gb300.build import build

    build()


def _flags(dbg_word):
    return sd.santa_read_device_error(dbg_word)


def _debug():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    dbg = sd.Debug()
    dbg.error_flags = word.data_ptr()
    return dbg, word


# ------------------------------------------------------------------------------ page plan


def _plan_reference(lens, new, table, free, ps, num_pages, max_tokens):
    """The definition, token by token."""
    table = table.copy()
    max_pages = table.shape[1]
    slots, pos = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int32)
    out, taken, placed, flags, row, out_of_pages = [], 0, 0, 0, 0, False
    for b, (n, m) in enumerate(zip(lens.tolist(), new.tolist())):
        rows = max(m, 0)
        first, row = row, row + rows
        need = -(-(n + m) // ps) - -(-n // ps)
        fits = n >= 0 and m >= 0 and -(-(n + m) // ps) <= max_pages and (rows == 0 or row <= max_tokens)
        if fits and need > 0 and (out_of_pages or taken + need > len(free)):
            out_of_pages, fits = True, False
        if not fits:
            flags |= sd.ERR_PAGES
            out.append(max(n, 0))
            continue
        for i in range(need):
            table[b, -(-n // ps) + i] = free[taken + i]
        taken += need
        placed += rows
        out.append(n + m)
        for i in range(m):
            page = int(table[b, (n + i) // ps])
            pos[first + i] = n + i
            if 0 <= page < num_pages:
                slots[first + i] = page * ps + (n + i) % ps
            else:
                flags |= sd.ERR_INDPTR
    return table, slots, pos, np.array(out, np.int32), np.array([taken, placed], np.int32), flags


def _plan_inputs(rng, batch, ps, hi_len, hi_new, spare_pages=4, max_pages=None):
    lens, new = rng.integers(0, hi_len + 1, batch), rng.integers(0, hi_new + 1, batch)
    have = -(-lens // ps)
    need = -(-(lens + new) // ps) - have
    max_pages = max_pages or int((have + need).max(initial=0)) + 1
    num_pages = int(have.sum() + need.sum()) + spare_pages
    ids = rng.permutation(num_pages).astype(np.int32)
    table = np.full((batch, max_pages), -9, np.int32)
    at = 0
    for b in range(batch):
        table[b, :min(have[b], max_pages)] = ids[at:at + have[b]][:max_pages]
        at += have[b]
    return lens.astype(np.int32), new.astype(np.int32), table, ids[at:].copy(), num_pages


def _run_plan(lens, new, table, free, ps, num_pages, max_tokens, stream=None):
    t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    d = [t(lens), t(new), t(table), t(free)]
    slots = torch.full((max_tokens,), 12345, dtype=torch.int64, device="cuda")
    pos = torch.full((max_tokens,), 12345, dtype=torch.int32, device="cuda")
    out = torch.full((len(lens),), 12345, dtype=torch.int32, device="cuda")
    counts = torch.full((2,), 12345, dtype=torch.int32, device="cuda")
    dbg, word = _debug()
    dec = Decoder(1, 1, 1, 64, num_pages * ps, 32, 256, 1, "f32")
    for _ in range(2):  # a repeated call gives the same answer
        dec.page_plan(d[0], d[1], d[2], d[3], ps, slots, pos, out, counts, debug=dbg)
    flags = _flags(word)
    return [x.cpu().numpy() for x in (d[2], slots, pos, out, counts)] + [flags]


def _check_plan(lens, new, table, free, ps, num_pages, max_tokens):
    want = _plan_reference(lens, new, table, free, ps, num_pages, max_tokens)
    got = _run_plan(lens, new, table, free, ps, num_pages, max_tokens)
    for name, a, b in zip(("table", "slots", "positions", "lens", "counts"), got, want):
        assert np.array_equal(a, b), name
    assert got[5] == want[5]
    return want


@pytest.mark.parametrize("batch,ps,hi_len,hi_new", [
    (1, 32, 0, 1), (1, 1, 5, 7), (3, 64, 200, 1), (64, 64, 3000, 1), (255, 7, 30, 40), (256, 32, 0, 100),
    (257, 128, 500, 33), (1000, 16, 100, 3), (5, 32, 100, 20000), (2, 4096, 9000, 9000), (40, 32, 64, 0),
])
def test_page_plan(batch, ps, hi_len, hi_new):
    rng = np.random.default_rng(batch * 1000 + ps)
    lens, new, table, free, num_pages = _plan_inputs(rng, batch, ps, hi_len, hi_new)
    _check_plan(lens, new, table, free, ps, num_pages, int(new.sum()) + 13)
    if int(new.sum()):
        _check_plan(lens, new, table, free, ps, num_pages, int(new.sum()))


def test_page_plan_refuses_sequences_that_do_not_fit():
    rng = np.random.default_rng(3)
    lens, new, table, free, num_pages = _plan_inputs(rng, 300, 32, 200, 100, max_pages=8)
    lens[7], lens[200], new[11], new[299] = -3, -2**31, -1, -2**31
    new[20], lens[30], new[31] = 2**31 - 1, 2**31 - 1, 32 * 8  # beyond the table's row, beyond 32 bits
    total = int(np.maximum(new.astype(np.int64), 0).sum())
    new[20] = 40
    rows = int(np.maximum(new, 0).sum())
    assert total > rows
    for free_n in (len(free), len(free) // 2, 1, 0):
        for tokens in (rows + 5, rows // 2, 1):
            want = _check_plan(lens, new, table, free[:free_n], 32, num_pages, tokens)
            assert want[5] & sd.ERR_PAGES


def test_page_plan_with_more_rows_than_32_bits_asked():
    lens = np.zeros(4, np.int32)
    new = np.array([5, 2**31 - 1, 2**31 - 1, 3], np.int32)
    table = np.full((4, 4), -1, np.int32)
    got = _run_plan(lens, new, table, np.arange(9, dtype=np.int32), 32, 9, 64)
    assert got[4].tolist() == [1, 5] and got[3].tolist() == [5, 0, 0, 0] and got[5] == sd.ERR_PAGES
    assert got[1][:5].tolist() == list(range(5)) and (got[1][5:] == -1).all()


def test_page_plan_flags_bad_page_ids():
    lens, new = np.array([10, 0, 5], np.int32), np.array([3, 4, 2], np.int32)
    table = np.array([[99, -1], [-1, -1], [1, -1]], np.int32)
    want = _check_plan(lens, new, table, np.array([-4], np.int32), 32, 4, 9)
    assert want[5] == sd.ERR_INDPTR and (want[1][:7] == -1).all() and (want[1][7:] >= 0).all()


def test_page_plan_of_no_sequence_pads():
    got = _run_plan(np.zeros(0, np.int32), np.zeros(0, np.int32), np.zeros((0, 3), np.int32), np.zeros(2, np.int32), 32, 4, 7)
    assert (got[1] == -1).all() and (got[2] == 0).all() and got[4].tolist() == [0, 0]


# ------------------------------------------------------------------------------ norm + rotation


def _rope_reference(x, w, eps, cs, rot, inter):
    """(y, bound on |a| + |b| of its pair) in 64 bits; x [T][H][d], cs [T][rot] (cosines, sines)."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    half = rot // 2
    cos, sin = cs[:, None, :half].double(), cs[:, None, half:].double()
    y, mag = x.clone(), x.abs()
    first = slice(0, rot, 2) if inter else slice(0, half)
    second = slice(1, rot, 2) if inter else slice(half, rot)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    mag[..., first] = mag[..., second] = a.abs() + b.abs()
    return y, mag


def _close(got, want, mag, what, u=2.0 ** -24):
    # the sum of squares (its d terms are positive: (8 + 4) u relative after fused multiply-adds in a tree of
    # 8 + 4 levels), root, division, two products and the rotation's two: 24 u of the pair's magnitude
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + 24 * u * mag
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - want).abs() - tol).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hq,hkv,rot,inter,norm,fused", [
    (1, 4, 1, 1.0, False, True, False), (3, 32, 8, 1.0, False, False, True), (17, 8, 8, 0.5, True, True, True),
    (200, 6, 2, 0.75, False, True, True), (33, 5, 5, 0.25, True, False, False), (1000, 32, 4, 1.0, True, True, True),
])
def test_norm_rope(dtype, d, T, hq, hkv, rot, inter, norm, fused):
    dt = DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    if fused:
        qkv = rnd(T, hq + 2 * hkv + 1, d).to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = (rnd(T, h, d).to(dt) for h in (hq, hkv, hkv))
    q[0, 0] *= 1e-3  # eps matters there
    rot = int(rot * d)
    rows = T + 7
    cs = rope_table(5000, rot, 10000.0)
    pos = torch.randint(0, 5000, (T,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(rows, generator=gen, device="cuda")[:T].contiguous()
    slots[T // 2] = -1 if T > 1 else slots[0]  # padding
    qw, kw = ((1 + 0.3 * rnd(d)).to(dt), (1 + 0.3 * rnd(d)).to(dt)) if norm else (None, None)
    kc, vc = rnd(rows, hkv, d).to(dt), rnd(rows, hkv, d).to(dt)
    kc0, vc0 = kc.clone(), vc.clone()
    dec = Decoder(1, hq, hkv, d, rows, rows, 256, 1, dtype)
    dbg, word = _debug()
    out = dec.norm_rope(q, k, v, pos, slots, cs, kc, vc, qw, kw, 1e-5, inter, debug=dbg)
    assert _flags(word) == 0
    want, mag = _rope_reference(q, qw, 1e-5, cs[pos.long()], rot, inter)
    _close(out, want, mag, "q")
    want, mag = _rope_reference(k, kw, 1e-5, cs[pos.long()], rot, inter)
    live = slots >= 0
    _close(kc[slots[live]], want[live], mag[live], "k")
    assert torch.equal(vc[slots[live]], v[live])
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert torch.equal(kc[rest], kc0[rest]) and torch.equal(vc[rest], vc0[rest])


def test_norm_rope_parts_in_place_and_identity_map():
    """q alone in place, k alone, v alone, and no slot map: each like the whole call."""
    T, hq, hkv, d = 9, 4, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((T, h, d), generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    cs = rope_table(64, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    dec = Decoder(1, hq, hkv, d, T, T, 256, 1, "bf16")
    kc, vc = torch.zeros_like(k), torch.zeros_like(v)
    out = dec.norm_rope(q, k, v, pos, None, cs, kc, vc)
    q2, kc2, vc2 = q.clone(), torch.zeros_like(k), torch.zeros_like(v)
    assert dec.norm_rope(q2, None, None, pos, None, cs, None, None, out=q2).data_ptr() == q2.data_ptr()
    dec.norm_rope(None, k, None, pos, None, cs, kc2, None)
    dec.norm_rope(None, None, v, pos, None, cs, None, vc2)
    assert torch.equal(out, q2) and torch.equal(kc, kc2) and torch.equal(vc, vc2) and torch.equal(vc, v)


def test_norm_rope_bad_positions_and_slots_are_flagged():
    T, d = 5, 64
    q = torch.randn((T, 1, d), device="cuda")
    cs = rope_table(10, d)
    pos = torch.tensor([0, -1, 10, 9, 2**31 - 1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 6, 1, -2**40, 2**40], dtype=torch.int64, device="cuda")
    kc, vc = torch.zeros((6, 1, d), device="cuda"), torch.zeros((6, 1, d), device="cuda")
    dec = Decoder(1, 1, 1, d, 6, 6, 256, 1, "f32")
    dbg, word = _debug()
    out = dec.norm_rope(q, q, q, pos, slots, cs, kc, vc, debug=dbg)
    assert _flags(word) == sd.ERR_POSITION | sd.ERR_SLOT
    want, mag = _rope_reference(q, None, 0.0, cs[pos.clamp(0, 9).long()], d, False)
    _close(out, want, mag, "q")
    assert torch.equal(vc[0], q[0]) and torch.equal(vc[1], q[2]) and not vc[2:].any()


def test_norm_rope_keeps_special_values_to_their_pairs():
    """An infinity or NaN reaches its own pair only (no norm), never the elements behind rot_dim or another head."""
    q = torch.randn((2, 3, 64), device="cuda")
    q[0, 1, 3], q[1, 2, 40], q[1, 0, 63] = math.inf, math.nan, math.inf
    cs = rope_table(10, 32)
    pos = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    dec = Decoder(1, 3, 3, 64, 2, 2, 256, 1, "f32")
    out = dec.norm_rope(q, None, None, pos, None, cs, None, None)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 1, 3] = want[0, 1, 19] = want[1, 2, 40] = want[1, 0, 63] = True
    assert torch.equal(bad, want) and out[1, 0, 63] == math.inf


# ------------------------------------------------------------------------------ attention


def _attention_reference(q, k, v, scale, u):
    """Exact output of one KV head's group and its error bound; q [G][d], k, v [n][d] in 64 bits."""
    x = q @ k.T * scale
    m = x.amax(-1, keepdim=True)
    p = torch.softmax(x, -1)
    d, n = k.shape[1], k.shape[0]
    # logit: d products and sums; exponential: its argument's roundings and 4 units of the function; the sums:
    # a chain of at most n / 32 blocks of 32 keys, then parts (64 levels allowed)
    dx = (d + 8) * u * (q.abs() @ k.abs().T) * scale + 4 * u * (x - m).abs() + 8 * u
    chain = (n / 32 + 96) * u
    dz = (p * dx).sum(-1, keepdim=True)
    tol = (p * (dx + dz)) @ v.abs() + 2 * chain * (p @ v.abs())
    return p @ v, tol


def _seen(n, window, sinks):
    return [i for i in range(n) if i < sinks or window == 0 or i >= n - window]


def _make_cache(lens, hkv, d, dt, page, gen, poison):
    """Keys and values of each sequence, laid out contiguously or in shuffled pages amid `poison`."""
    kv = [[torch.randn((n, hkv, d), generator=gen, device="cuda").to(dt) for n in lens] for _ in range(2)]
    B = len(lens)
    if not page:
        rows = sum(lens) + 3
        pools = [torch.full((rows, hkv, d), poison, device="cuda", dtype=dt) for _ in range(2)]
        start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        where = [torch.arange(start[b], start[b + 1], device="cuda") for b in range(B)]
        addr = dict(indptr=torch.from_numpy(start).cuda())
    else:
        have = [-(-n // page) for n in lens]
        num = sum(have) + 2
        rows = num * page
        pools = [torch.full((rows, hkv, d), poison, device="cuda", dtype=dt) for _ in range(2)]
        ids = torch.randperm(num, generator=gen, device="cuda").cpu().numpy()
        table = np.full((B, max(have) + 1), -3, np.int32)
        at, where = 0, []
        for b, n in enumerate(lens):
            table[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
            i = np.arange(n)
            where.append(torch.from_numpy(table[b, i // page].astype(np.int64) * page + i % page).cuda())
        addr = dict(table=torch.from_numpy(table).cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for pool, x in zip(pools, kv):
        for b in range(B):
            pool[where[b]] = x[b]
    return pools, kv, where, addr, rows


def _values64(rec, d):
    """K and V in 64 bits of 4-bit records [..][d + d / 8]."""
    i = torch.arange(d, device=rec.device)
    out = []
    for which in range(2):
        codes = rec[..., which * (d // 2):(which + 1) * (d // 2)].long()
        n = ((codes[..., i // 2] >> (4 * (i % 2))) & 15).double()
        at = d + which * (d // 16)
        p = rec[..., at:at + d // 16].contiguous().view(torch.float16).double()
        g = (i // 8) % (d // 64)
        out.append(p[..., 2 * g + 1] + p[..., 2 * g] * n)
    return out


def _run_attention(kind, dec, q, pools, addr, page, window, sinks, debug=None, out=None):
    if kind == "window":
        if page:
            return dec.window_paged(q, *pools, addr["table"], addr["lens"], page, window, sinks, out=out, debug=debug)
        return dec.window(q, *pools, addr["indptr"], window, sinks, out=out, debug=debug)
    if page:
        return dec.kv4_paged(q, pools[0], addr["table"], addr["lens"], page, window, sinks, out=out, debug=debug)
    return dec.kv4(q, pools[0], addr["indptr"], window, sinks, out=out, debug=debug)


def _attention_case(kind, dtype, d, hkv, g, lens, window, sinks, page, seed=0, poison=math.nan, q_scale=1.0, k_shift=0.0):
    dt = DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pools, kv, where, addr, rows = _make_cache(lens, hkv, d, dt, page, gen, poison)
    if k_shift:
        for b in range(len(lens)):
            kv[0][b] = (kv[0][b].float() + k_shift).to(dt)
            pools[0][where[b]] = kv[0][b]
    q = (torch.randn((len(lens), hkv * g, d), generator=gen, device="cuda") * q_scale).to(dt)
    dec = Decoder(len(lens), hkv * g, hkv, d, rows, max(max(lens), 1), 256, 1, dtype)
    if kind == "kv4":
        cache = torch.full((rows, hkv, d + d // 8), 0xFF, dtype=torch.uint8, device="cuda")  # NaN scales outside
        for b in range(len(lens)):
            if lens[b]:
                dec.kv4_append(kv[0][b], kv[1][b], where[b], cache)
        pools = [cache]
    dbg, word = _debug()
    out = torch.full((len(lens), hkv * g, d), 77.0, device="cuda")
    _run_attention(kind, dec, q, pools, addr, page, window, sinks, dbg, out)
    assert _flags(word) == 0
    return dict(kind=kind, dec=dec, q=q, pools=pools, kv=kv, where=where, addr=addr, page=page, window=window,
                sinks=sinks, lens=lens, out=out, d=d, hkv=hkv, g=g, dtype=dtype)


def _check_attention(c):
    # tensor-core sums may truncate (2^-23); the 4-bit path holds q and the weights in two fp16 parts (2^-22)
    u = {"window": 2.0 ** -23 if c["dtype"] == "bf16" else 2.0 ** -24, "kv4": 2.0 ** -22}[c["kind"]]
    d, worst = c["d"], 0.0
    for b, n in enumerate(c["lens"]):
        keep = torch.tensor(_seen(n, c["window"], c["sinks"]), dtype=torch.int64, device="cuda")
        if not len(keep):
            assert not c["out"][b].any()
            continue
        for h in range(c["hkv"]):
            if c["kind"] == "kv4":
                k, v = _values64(c["pools"][0][c["where"][b][keep], h], d)
            else:
                k, v = (c["kv"][i][b][keep, h].double() for i in range(2))
            heads = slice(h * c["g"], (h + 1) * c["g"])
            want, tol = _attention_reference(c["q"][b, heads].double(), k, v, 1 / math.sqrt(d), u)
            err = (c["out"][b, heads].double() - want).abs()
            assert (err <= tol).all(), (b, h, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
    return worst


CASES = [  # lens, window, sinks
    ([1], 1, 0), ([1, 0, 2, 31, 32, 33], 0, 0), ([64, 65, 100, 0], 7, 0), ([300, 5, 40, 260], 33, 4),
    ([1000, 999], 1, 1), ([129, 700], 128, 500), ([2500], 64, 3), ([4100, 17, 2049], 1000, 36),
    ([33, 34, 96, 97], 64, 1), ([0, 0], 5, 5), ([200] * 20, 10, 2),
]


@pytest.mark.parametrize("kind", ["window", "kv4"])
@pytest.mark.parametrize("dtype,d,hkv,g,page", [
    ("bf16", 128, 2, 4, 0), ("bf16", 64, 1, 8, 32), ("f32", 64, 1, 4, 0), ("f32", 128, 3, 1, 96),
    ("bf16", 128, 1, 7, 64), ("bf16", 64, 4, 3, 0), ("f32", 64, 2, 5, 32), ("f32", 128, 1, 8, 0),
    ("bf16", 128, 8, 1, 0), ("bf16", 128, 3, 2, 32), ("f32", 64, 1, 6, 0),
])
def test_attention(kind, dtype, d, hkv, g, page):
    """Every case with NaN in all rows that no query may see, and NaN pages and unread table entries around."""
    for i, (lens, window, sinks) in enumerate(CASES):
        _check_attention(_attention_case(kind, dtype, d, hkv, g, lens, window, sinks, page, seed=i))


@pytest.mark.parametrize("kind", ["window", "kv4"])
@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf])
def test_masked_keys_do_not_matter(kind, garbage):
    """Keys of the sequence itself that lie outside the window: any content, the same bits."""
    for page in (0, 32):
        c = _attention_case(kind, "bf16", 128, 2, 4, [400, 77], 50, 3, page, seed=5)
        for b, n in enumerate(c["lens"]):
            hide = torch.tensor([i for i in range(n) if i not in _seen(n, 50, 3)], device="cuda")
            for pool in c["pools"]:
                pool[c["where"][b][hide]] = 0xFF if kind == "kv4" else garbage
        again = _run_attention(kind, c["dec"], c["q"], c["pools"], c["addr"], page, 50, 3)
        assert torch.equal(again, c["out"])


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_long_and_many(kind):
    """A long sequence split over the whole GPU, a batch of unequal ones, more sequences than a CTA has threads."""
    _check_attention(_attention_case(kind, "bf16", 128, 1, 4, [40000], 0, 0, 0, seed=1))
    _check_attention(_attention_case(kind, "bf16", 128, 2, 8, [9000, 1, 3000, 0, 12345, 64], 5000, 4, 64, seed=2))
    _check_attention(_attention_case(kind, "f32", 64, 1, 2, [5000, 9000], 0, 0, 32, seed=3))
    rng = np.random.default_rng(4)
    _check_attention(_attention_case(kind, "bf16", 64, 1, 1, rng.integers(0, 50, 1100).tolist(), 20, 2, 32, seed=4))
    # 40 and 128 sequences (two and four scans per warp), with long ones behind the first 32
    _check_attention(_attention_case(kind, "bf16", 128, 2, 4, [3, 0] * 17 + [9000, 1, 0, 5000, 64, 2], 0, 0, 0, seed=5))
    _check_attention(_attention_case(kind, "bf16", 64, 1, 2, rng.integers(0, 900, 128).tolist(), 0, 0, 32, seed=6))


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_many_units_allowed_by_a_large_bound(kind):
    """max_len far beyond the lengths: the count of units is then kept in 64 bits, by another path of the plan."""
    for lens in ([5000, 0, 33, 700], [40], list(range(140))):
        c = _attention_case(kind, "bf16", 128, 2, 4, lens, 600, 3, 0, seed=50)
        p = c["dec"].problem
        big = Decoder(p.batch, 8, 2, 128, p.total_tokens, 2**31 - 1, 256, 1, "bf16")
        c["out"] = _run_attention(kind, big, c["q"], c["pools"], c["addr"], 0, 600, 3)
        _check_attention(c)


@pytest.mark.parametrize("kind", ["window", "kv4"])
@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 4), ("bf16", 128, 8), ("bf16", 64, 2), ("f32", 64, 4), ("f32", 128, 1)])
def test_precision_of_means_over_many_keys(kind, dtype, d, g):
    """The mean of many values is small against each of them, and errors that do not average out show.  Logits
    here are below 8, formed to 8 2^-24 times a few roundings of each product's sum (about 1e-6), exponentials
    to 2^-22, weights in parts of 22 bits or more: relative to the output, whose terms average like the errors,
    2e-6 in all; twice that is allowed."""
    for n in (100, 3000, 30000):
        c = _attention_case(kind, dtype, d, 2, g, [n], 0, 0, 0, seed=n)
        for h in range(2):
            if kind == "kv4":
                k, v = _values64(c["pools"][0][c["where"][0], h], d)
            else:
                k, v = (c["kv"][i][0][:, h].double() for i in range(2))
            want = torch.softmax(c["q"][0, h * g:(h + 1) * g].double() @ k.T / math.sqrt(d), -1) @ v
            err = float((c["out"][0, h * g:(h + 1) * g].double() - want).norm() / want.norm())
            assert err <= 4e-6, (n, h, err)


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_large_logits_and_offsets(kind):
    """Logits of hundreds (weights that underflow) and keys with a common offset."""
    _check_attention(_attention_case(kind, "bf16", 128, 2, 4, [3000, 50], 0, 0, 0, seed=6, q_scale=20.0))
    _check_attention(_attention_case(kind, "f32", 64, 2, 4, [3000, 50], 700, 4, 32, seed=7, q_scale=20.0))
    _check_attention(_attention_case(kind, "bf16", 128, 2, 4, [2000], 0, 0, 0, seed=8, k_shift=3.0))


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_values_of_any_scale(kind):
    """Rows whose values span many powers of two, and rows of one value: the tolerance is relative to them."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    for factor in (1e-4, 1.0, 1e3):
        n, d = 500, 128
        q = torch.randn((1, 4, d), generator=gen, device="cuda").bfloat16()
        k = torch.randn((n, 1, d), generator=gen, device="cuda").bfloat16()
        v = (torch.randn((n, 1, d), generator=gen, device="cuda") * factor
             * torch.exp2(-torch.randint(0, 6, (n, 1, 1), generator=gen, device="cuda").float())).bfloat16()
        v[7] = 0
        v[8] = factor
        dec = Decoder(1, 4, 1, d, n, n, 256, 1, "bf16")
        ind = torch.tensor([0, n], device="cuda")
        if kind == "kv4":
            cache = dec.kv4_cache()
            dec.kv4_append(k, v, None, cache)
            out = dec.kv4(q, cache, ind)
            kk, vv = _values64(cache[:, 0], d)
        else:
            out = dec.window(q, k, v, ind, 0)
            kk, vv = k[:, 0].double(), v[:, 0].double()
        want, tol = _attention_reference(q[0].double(), kk, vv, 1 / math.sqrt(d), 2.0 ** -22)
        assert ((out[0].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_window_of_everything_equals_no_window(kind):
    c = _attention_case(kind, "bf16", 128, 2, 4, [700, 32, 1], 0, 0, 0, seed=9)
    for window, sinks in ((700, 0), (10**9, 7), (2**31 - 1, 2**31 - 1), (1, 2**31 - 1), (1, 699)):
        got = _run_attention(kind, c["dec"], c["q"], c["pools"], c["addr"], 0, window, sinks)
        assert torch.equal(got, c["out"]) or torch.allclose(got, c["out"], rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_paged_equals_contiguous_and_calls_repeat(kind):
    """Bit for bit: the cache's layout and the call's timing do not change the result; the workspace's
    counters are zero again."""
    a = _attention_case(kind, "bf16", 128, 2, 4, [5000, 300, 0, 31], 2000, 4, 0, seed=10)
    dec, where = a["dec"], a["where"]
    page, pages_per = 32, [-(-n // 32) for n in a["lens"]]
    num = sum(pages_per) + 1
    pools = [torch.zeros((num * page, *p.shape[1:]), dtype=p.dtype, device="cuda") for p in a["pools"]]
    table = np.full((4, max(pages_per)), -1, np.int32)
    ids = np.random.default_rng(0).permutation(num)
    at = 0
    for b, n in enumerate(a["lens"]):
        table[b, :pages_per[b]] = ids[at:at + pages_per[b]]
        at += pages_per[b]
        i = np.arange(n)
        rows = torch.from_numpy(table[b, i // page].astype(np.int64) * page + i % page).cuda()
        for pool, src in zip(pools, a["pools"]):
            pool[rows] = src[where[b]]
    pdec = Decoder(4, 8, 2, 128, num * page, 5000, 256, 1, "bf16")
    addr = dict(table=torch.from_numpy(table).cuda(), lens=torch.tensor(a["lens"], dtype=torch.int32, device="cuda"))
    for _ in range(5):
        assert torch.equal(_run_attention(kind, pdec, a["q"], pools, addr, page, 2000, 4), a["out"])
        assert torch.equal(_run_attention(kind, dec, a["q"], a["pools"], a["addr"], 0, 2000, 4), a["out"])
    assert not dec.split_workspace()[:4 * 2 * 4].any()


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_bad_device_data_is_flagged(kind):
    c = _attention_case(kind, "bf16", 128, 1, 2, [100, 64, 200], 0, 0, 0, seed=12)
    dbg, word = _debug()
    ind = c["addr"]["indptr"].clone()
    ind[1] = 10**12
    got = _run_attention(kind, c["dec"], c["q"], c["pools"], dict(indptr=ind), 0, 0, 0, dbg)
    assert _flags(word) == sd.ERR_INDPTR
    assert not got[:2].any()
    # where a head is cut depends on the other sequences' lengths: equal to rounding, not to the bit
    one = dict(c, out=got, lens=[0, 0, 200])
    _check_attention(one)
    p = _attention_case(kind, "bf16", 128, 1, 2, [100, 64, 200], 0, 0, 32, seed=12)
    table = p["addr"]["table"].clone()
    table[0, 1], table[2, 0] = -1, 10**9  # pages dropped: their keys carry no weight
    lens = p["addr"]["lens"].clone()
    lens[1] = -5
    got = _run_attention(kind, p["dec"], p["q"], p["pools"], dict(table=table, lens=lens), 32, 0, 0, dbg)
    assert _flags(word) == sd.ERR_INDPTR
    assert not got[1].any() and torch.isfinite(got).all()
    keep = {0: [i for i in range(100) if i // 32 != 1], 2: [i for i in range(200) if i // 32 != 0]}
    for b, rows in keep.items():
        rows = p["where"][b][torch.tensor(rows, device="cuda")]
        if kind == "kv4":
            k, v = _values64(p["pools"][0][rows, 0], 128)
        else:
            k, v = (x[rows, 0].double() for x in p["pools"])
        want, tol = _attention_reference(p["q"][b].double(), k, v, 1 / math.sqrt(128), 2.0 ** -22)
        assert ((got[b].double() - want).abs() <= tol).all()


# ------------------------------------------------------------------------------ 4-bit cache


def _quantised(x):
    """Record parts by the definition, in numpy single precision: codes [..][d / 2], pairs [..][d / 64][2]."""
    x = x.float().cpu().numpy()
    d = x.shape[-1]
    x = np.clip(np.nan_to_num(x, nan=0.0, posinf=65504, neginf=-65504), -65504, 65504).astype(np.float32)
    g = (np.arange(d) // 8) % (d // 64)
    codes, pairs = np.zeros(x.shape, np.uint8), np.zeros((*x.shape[:-1], d // 64, 2), np.float16)
    for i in range(d // 64):
        r = x[..., g == i]
        lo = r.min(-1).astype(np.float16)
        scale = ((r.max(-1) - lo.astype(np.float32)) * np.float32(1.0 / 15.0)).astype(np.float16)
        s = scale.astype(np.float32)[..., None]
        with np.errstate(all="ignore"):
            n = np.rint((r - lo.astype(np.float32)[..., None]) / s)
        codes[..., g == i] = np.where(s > 0, np.clip(np.nan_to_num(n), 0, 15), 0).astype(np.uint8)
        pairs[..., i, 0], pairs[..., i, 1] = scale, lo
    return codes[..., 0::2] | (codes[..., 1::2] << 4), pairs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hkv,fused", [(1, 1, False), (5, 3, True), (64, 8, True), (1000, 2, False)])
def test_kv4_append_and_read(dtype, d, T, hkv, fused):
    dt = DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T)
    kv = torch.randn((T, 2 * hkv + 1, d), generator=gen, device="cuda").to(dt)
    kv[0, 0] = 0.25  # one value: scale 0
    k, v = kv[:, :hkv], kv[:, hkv:2 * hkv]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    if T > 4:
        v[1, 0] *= 1e-6  # fp16 subnormals
        v[2, 0] *= 3000.0
    rows = T + 5
    slots = torch.randperm(rows, generator=gen, device="cuda")[:T].contiguous()
    if T > 1:
        slots[T - 1] = -1
    dec = Decoder(1, hkv, hkv, d, rows, rows, 256, 1, dtype)
    cache = dec.kv4_cache()
    cache.fill_(0xAB)
    dbg, word = _debug()
    dec.kv4_append(k, v, slots, cache, debug=dbg)
    kr, vr = dec.kv4_read(cache, slots, debug=dbg)
    assert _flags(word) == 0
    live = slots >= 0
    rec = cache[slots[live]]
    for x, got, a, b in ((k, kr, 0, d), (v, vr, d // 2, d + d // 16)):
        codes, pairs = _quantised(x[live])
        assert np.array_equal(rec[..., a:a + d // 2].cpu().numpy(), codes)
        assert np.array_equal(rec[..., b:b + d // 16].contiguous().view(torch.float16).cpu().numpy().reshape(pairs.shape), pairs)
        values = _values64(rec, d)[0 if a == 0 else 1]
        assert torch.equal(got[live], values.to(dt))  # fp32: base + scale * code is exact to half a step
        assert not got[~live].any()
        # half a step of the scale, and the roundings of the minimum (fp16) and of the scale (15 steps of 2^-11)
        scale = torch.from_numpy(pairs[..., 0].astype(np.float64)).cuda()
        lo = torch.from_numpy(np.abs(pairs[..., 1]).astype(np.float64)).cuda()
        g = (torch.arange(d, device="cuda") // 8) % (d // 64)
        tol = scale[..., g] * (0.5 + 16 * 2.0 ** -11) + lo[..., g] * 2.0 ** -10 + 16 * 2.0 ** -24
        assert ((values - x[live].double()).abs() <= tol).all()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert (cache[rest] == 0xAB).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_kv4_ties_between_codes(dtype, d):
    """Values in the middle between two codes, and a unit in the last place beside it: as the division rounds."""
    dt = DT[dtype]
    step = 2.0 ** torch.arange(-6, 6, device="cuda").double()[:, None, None]
    half = torch.arange(d, device="cuda").double() % 31 / 2  # 0, 0.5, .. 15: every group has 0 and 15
    k = (half * step).to(dt).expand(12, 1, d).contiguous()
    v = k.clone()
    near = torch.nextafter(k.float(), torch.full_like(k, 1e9, dtype=torch.float32)) if dt == torch.float32 else k.float()
    v[:] = torch.where((half % 1 == 0.5).expand_as(k), near.to(dt), k)
    dec = Decoder(1, 1, 1, d, 12, 12, 256, 1, dtype)
    cache = dec.kv4_cache()
    dec.kv4_append(k, v, None, cache)
    for x, a, b in ((k, 0, d), (v, d // 2, d + d // 16)):
        codes, pairs = _quantised(x)
        assert np.array_equal(cache[..., a:a + d // 2].cpu().numpy(), codes)
        assert np.array_equal(cache[..., b:b + d // 16].contiguous().view(torch.float16).cpu().numpy().reshape(pairs.shape), pairs)


def test_kv4_special_values_and_slots():
    T, d = 6, 64
    k = torch.randn((T, 1, d), device="cuda")
    v = torch.randn((T, 1, d), device="cuda")
    k[0, 0, 5], k[1, 0, 6], v[2, 0, 7], v[3, 0, 0] = math.nan, math.inf, -math.inf, 1e30
    dec = Decoder(1, 1, 1, d, T, T, 256, 1, "f32")
    cache = dec.kv4_cache()
    dbg, word = _debug()
    dec.kv4_append(k, v, None, cache, debug=dbg)
    assert _flags(word) == sd.ERR_VALUE
    for x, a, b in ((k, 0, d), (v, d // 2, d + d // 16)):
        codes, pairs = _quantised(x)
        assert np.array_equal(cache[..., a:a + d // 2].cpu().numpy(), codes)
        assert np.array_equal(cache[..., b:b + d // 16].contiguous().view(torch.float16).cpu().numpy().reshape(pairs.shape), pairs)
    kr, vr = dec.kv4_read(cache, torch.tensor([T, 2**40, -1, 4], device="cuda"), debug=dbg)
    assert _flags(word) == sd.ERR_SLOT
    assert not kr[:3].any() and kr[3].any() and torch.isfinite(vr).all()
    before = cache.clone()
    dec.kv4_append(k[:2].contiguous(), v[:2].contiguous(), torch.tensor([T, -7], device="cuda"), cache, debug=dbg)
    assert _flags(word) == sd.ERR_SLOT and torch.equal(cache, before)


# ------------------------------------------------------------------------------ together


def _step_state(kind, batch=5, hq=8, hkv=2, d=128, page=32, steps=40):
    """A small serving loop's buffers: prompts of different lengths, then one token per sequence and step."""
    num_pages, max_pages = 64, 12
    dec = Decoder(batch, hq, hkv, d, num_pages * page, max_pages * page, 256, 1, "bf16")
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(dec=dec, page=page, table=torch.full((batch, max_pages), -1, **i32), lens=torch.zeros(batch, **i32),
             cs=rope_table(max_pages * page, d), kw=torch.ones(d, device="cuda").bfloat16() * 1.25, num_pages=num_pages,
             free=torch.from_numpy(np.random.default_rng(0).permutation(num_pages).astype(np.int32)).cuda())
    if kind == "kv4":
        s["cache"] = dec.kv4_cache()
    rows = [torch.full((num_pages * page, hkv, d), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    s["k"], s["v"] = rows
    return s


def _step(kind, s, new, qkv, max_tokens, window, sinks, lens_out, slots, pos, counts):
    dec, (hq, hkv) = s["dec"], (s["dec"].problem.num_q_heads, s["dec"].problem.num_kv_heads)
    dec.page_plan(s["lens"], new, s["table"], s["free"], s["page"], slots, pos, lens_out, counts)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if kind == "kv4":  # rotate into a row per token, then store 4 bits
        kr, vr = torch.empty_like(k, memory_format=torch.contiguous_format), v
        tok = Decoder(1, hq, hkv, dec.problem.head_dim, max_tokens, max_tokens, 256, 1, "bf16")
        qr = tok.norm_rope(q, k, None, pos, None, s["cs"], kr, None, s["kw"], s["kw"])
        dec.kv4_append(kr, vr, slots, s["cache"])
    else:
        qr = dec.norm_rope(q, k, v, pos, slots, s["cs"], s["k"], s["v"], s["kw"], s["kw"])
    return qr


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_a_serving_loop(kind):
    """Prompts are placed, then tokens are decoded one by one: the loop's outputs against the whole history
    held densely in 64 bits (the 4-bit cache's own values for kv4)."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    s = _step_state(kind)
    dec, d, hq, hkv, B = s["dec"], 128, 8, 2, 5
    prompts = [40, 1, 0, 97, 64]
    i32 = dict(dtype=torch.int32, device="cuda")
    free_host = s["free"].cpu().numpy()
    hist = [[] for _ in range(B)]  # (rotated key, value) rows in 64 bits
    window, sinks = 50, 3
    for step in range(6):
        new = prompts if step == 0 else [1] * B
        max_tokens = sum(new) + 3
        qkv = torch.randn((max_tokens, hq + 2 * hkv, d), generator=gen, device="cuda").bfloat16()
        slots, pos = torch.empty(max_tokens, dtype=torch.int64, device="cuda"), torch.empty(max_tokens, **i32)
        lens_out, counts = torch.empty(B, **i32), torch.empty(2, **i32)
        qr = _step(kind, s, torch.tensor(new, **i32), qkv, max_tokens, window, sinks, lens_out, slots, pos, counts)
        s["lens"] = lens_out
        taken = int(counts[0])
        free_host = free_host[taken:]
        s["free"] = torch.from_numpy(free_host.copy()).cuda()
        t = 0
        for b in range(B):
            for i in range(new[b]):
                hist[b].append(int(slots[t]))
                assert int(pos[t]) == len(hist[b]) - 1
                t += 1
        assert (slots[t:] == -1).all()
        if step == 0:
            continue
        out = (dec.kv4_paged(qr[:B].contiguous(), s["cache"], s["table"], s["lens"], s["page"], window, sinks) if kind == "kv4"
               else dec.window_paged(qr[:B].contiguous(), s["k"], s["v"], s["table"], s["lens"], s["page"], window, sinks))
        for b in range(B):
            keep = torch.tensor(_seen(len(hist[b]), window, sinks), device="cuda")
            rows = torch.tensor(hist[b], device="cuda")[keep]
            for h in range(hkv):
                if kind == "kv4":
                    k, v = _values64(s["cache"][rows, h], d)
                else:
                    k, v = s["k"][rows, h].double(), s["v"][rows, h].double()
                heads = slice(4 * h, 4 * h + 4)
                want, tol = _attention_reference(qr[b, heads].double(), k, v, 1 / math.sqrt(d), 2.0 ** -22)
                assert ((out[b, heads].double() - want).abs() <= tol).all()
    assert [len(x) for x in hist] == s["lens"].tolist()
    assert len({r for x in hist for r in x}) == sum(len(x) for x in hist)  # no row twice


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_captured_step_replays_on_new_inputs(kind):
    """Plan, rotation, store and attention in one CUDA graph; replays on other lengths, keys and queries equal
    eager calls bit for bit."""
    B, hq, hkv, d, page = 4, 8, 2, 128, 32
    s = _step_state(kind, batch=B)
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.ones(B, **i32)
    qkv = torch.zeros((B, hq + 2 * hkv, d), device="cuda", dtype=torch.bfloat16)
    slots, pos = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, **i32)
    lens_out, counts = torch.empty(B, **i32), torch.empty(2, **i32)
    out = torch.empty((B, hq, d), device="cuda")
    s["k"].normal_(), s["v"].normal_()
    if kind == "kv4":
        allrows = torch.arange(s["num_pages"] * page, device="cuda")
        s["dec"].kv4_append(s["k"], s["v"], allrows, s["cache"])
    dec = s["dec"]

    def step():
        qr = _step(kind, s, new, qkv, B, 100, 4, lens_out, slots, pos, counts)
        if kind == "kv4":
            dec.kv4_paged(qr, s["cache"], s["table"], lens_out, page, 100, 4, out=out)
        else:
            dec.window_paged(qr, s["k"], s["v"], s["table"], lens_out, page, 100, 4, out=out)

    def load(i):
        g = torch.Generator(device="cuda").manual_seed(i)
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        lens = [(37 * i + 61 * b) % 300 for b in range(B)]
        s["lens"].copy_(torch.tensor(lens, **i32))
        ids = np.random.default_rng(i).permutation(s["num_pages"]).astype(np.int32)
        table, at = np.full(tuple(s["table"].shape), -1, np.int32), 0
        for b, n in enumerate(lens):
            have = -(-n // page)
            table[b, :have] = ids[at:at + have]
            at += have
        s["table"].copy_(torch.from_numpy(table))
        s["free"][:len(ids) - at].copy_(torch.from_numpy(ids[at:]))

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 2, 3):
        load(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, slots, pos, lens_out, s["table"])]
        load(i)
        step()
        for a, b in zip(got, (out, slots, pos, lens_out, s["table"])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_two_streams_with_a_workspace_each(kind):
    cases = [_attention_case(kind, "bf16", 128, 2, 4, [6000, 10, 3000], 0, 0, 0, seed=30 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                outs.append((c, _run_attention(kind, c["dec"], c["q"], c["pools"], c["addr"], 0, 0, 0)))
    torch.cuda.synchronize()
    for c, got in outs:
        assert torch.equal(got, c["out"])


def test_c_entry_points_by_name():
    """The functions that carry the C names give what the Decoder's methods give: a caller's own workspace,
    prepared by santa_split_workspace_init and full of garbage before; no window given to the 4-bit call."""
    c = _attention_case("window", "bf16", 128, 2, 4, [4000, 0, 77], 0, 0, 0, seed=41)
    dec, q, (k, v), ind = c["dec"], c["q"], c["pools"], c["addr"]["indptr"]
    p = dec.problem
    n = 6
    ws = torch.full((sd.split_workspace_size(p),), 0xFF, dtype=torch.uint8, device="cuda")
    sd.santa_split_workspace_init(p, ws)
    out = torch.empty_like(c["out"])
    sd.santa_decode_window(p, sd.Window(100, 3), q, k, v, ind, out, ws)
    assert torch.equal(out, dec.window(q, k, v, ind, 100, 3))
    slots = torch.randperm(p.total_tokens, device="cuda")[:n].contiguous()
    caches = [torch.zeros((p.total_tokens, 2, 144), dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert sd.kv4_size(p) == caches[0].numel()
    x = torch.randn((n, 12, 128), device="cuda").bfloat16()
    sd.santa_kv4_append(p, x[:, 8:10], x[:, 10:], slots, caches[0])
    dec.kv4_append(x[:, 8:10], x[:, 10:], slots, caches[1])
    assert torch.equal(*caches)
    a, b = (torch.empty((n, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sd.santa_kv4_read(p, n, caches[0], slots, a, b)
    assert all(torch.equal(s, t) for s, t in zip((a, b), dec.kv4_read(caches[0], slots)))
    sd.santa_kv4_read(p, n, caches[0], None, None, b)  # rows 0 .. n - 1, V alone
    assert torch.equal(b, dec.kv4_read(caches[0], torch.arange(n, device="cuda"))[1])
    sd.santa_decode_kv4(p, None, q, caches[0], ind, out, ws)
    assert torch.equal(out, dec.kv4(q, caches[0], ind))
    cs, pos = rope_table(50, 64), torch.arange(n, dtype=torch.int32, device="cuda")
    w = torch.rand(128, device="cuda").bfloat16()
    rope = sd.Rope(w.data_ptr(), None, 1e-6, cs.data_ptr(), 50, 64, 0)  # norms of the queries alone
    kc, vc, kd, vd = (torch.zeros_like(k) for _ in range(4))
    qo = torch.empty((n, 8, 128), dtype=torch.bfloat16, device="cuda")
    sd.santa_norm_rope(p, rope, x[:, :8], x[:, 8:10], x[:, 10:], pos, slots, qo, kc, vc)
    assert torch.equal(qo, dec.norm_rope(x[:, :8], x[:, 8:10], x[:, 10:], pos, slots, cs, kd, vd, q_weight=w))
    assert torch.equal(kc, kd) and torch.equal(vc, vd)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, new, table = torch.tensor([3, 40], **i32), torch.tensor([1, 30], **i32), torch.tensor([[5, 0, 0], [2, 3, 0]], **i32)
    free, slot_map, positions = torch.tensor([7, 1], **i32), torch.empty(33, dtype=torch.int64, device="cuda"), torch.empty(33, **i32)
    lens_out, counts = torch.empty(2, **i32), torch.empty(2, **i32)
    sd.santa_page_plan(32, 9, lens, new, table, free, slot_map, positions, lens_out, counts)
    assert counts.tolist() == [1, 31] and table.tolist() == [[5, 0, 0], [2, 3, 7]] and lens_out.tolist() == [4, 70]
    assert slot_map[:3].tolist() == [163, 104, 105] and slot_map[-3:].tolist() == [229, -1, -1]


@pytest.mark.parametrize("kind", ["window", "kv4"])
def test_workspace_before_capture_and_windows_in_range(kind):
    """A Decoder whose first call would be captured is refused (its workspace would only be zeroed by a replay);
    windows beyond 31 bits are refused, not cut; a call on another stream finds the workspace prepared."""
    c = _attention_case(kind, "bf16", 128, 2, 4, [5000, 7], 0, 0, 0, seed=40)
    p = c["dec"].problem
    fresh = Decoder(p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim, p.total_tokens, p.max_len, 256, 1, "bf16")
    out = torch.empty_like(c["out"])
    call = lambda dec, w=0, s=0, **kw: _run_attention(kind, dec, c["q"], c["pools"], c["addr"], 0, w, s, out=out)  # noqa: E731
    with pytest.raises(RuntimeError, match="before a capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            call(fresh)
    torch.cuda.synchronize()
    for w, s in ((-1, 0), (2**31, 0), (0, 2**32 + 5)):
        with pytest.raises(ValueError, match="2\\^31"):
            call(fresh, w, s)
    junk = torch.full((1 << 26,), 7, dtype=torch.uint8, device="cuda")  # what a fresh allocation may hold
    del junk
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    if kind == "window":
        fresh.window(c["q"], *c["pools"], c["addr"]["indptr"], 0, out=out, stream=side)
    else:
        fresh.kv4(c["q"], c["pools"][0], c["addr"]["indptr"], out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, c["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(fresh)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c["out"])


def test_rows_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes (and 2^31 elements of a 4-bit one): the last rows are found."""
    hkv, d = 8, 128
    rows = (1 << 32) // (hkv * 144) + 64
    dec = Decoder(1, hkv, hkv, d, rows, 64, 256, 1, "bf16")
    cache = torch.empty((rows, hkv, 144), dtype=torch.uint8, device="cuda")
    k, v, q = (torch.randn((64, hkv, d), device="cuda").bfloat16() for _ in range(3))
    slots = torch.arange(rows - 64, rows, device="cuda")
    dec.kv4_append(k, v, slots, cache)
    ind = torch.tensor([rows - 64, rows], device="cuda")
    out = dec.kv4(q[:1].contiguous(), cache, ind)
    kc = torch.empty((rows, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    pos = torch.zeros(64, dtype=torch.int32, device="cuda")
    dec.norm_rope(None, k, v, pos, slots, rope_table(4, d), kc, vc)
    assert torch.equal(kc[slots], k) and torch.equal(vc[slots], v)
    win = dec.window(q[:1].contiguous(), kc, vc, ind, 0)
    for h in range(hkv):
        k4, v4 = _values64(cache[slots, h], d)
        for got, (kk, vv) in ((out, (k4, v4)), (win, (k[:, h].double(), v[:, h].double()))):
            want, tol = _attention_reference(q[:1, h].double(), kk, vv, 1 / math.sqrt(d), 2.0 ** -22)
            assert ((got[0, h].double() - want[0]).abs() <= tol[0]).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_plan_and_rotation_in_front_of_the_sampled_decodes(dtype, d):
    """santa_page_plan and santa_norm_rope let their successor start before they have written the page table, the
    queries and the caches that it reads.  Steps queued one behind another, and steps replayed from a graph, equal
    bit for bit the steps with a synchronisation between the calls (paged prop, and the fused and two-kernel prop
    on contiguous rows)."""
    B, hq, hkv, page, max_pages, S, steps = 6, 8, 2, 32, 40, 32, 12
    num_pages, dt = B * max_pages, DT[dtype]
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(60)
    rows = num_pages * page
    dec = Decoder(B, hq, hkv, d, rows, max_pages * page, 256, S, dtype)
    modes = ("paged", "prop", "prop_fused")
    for m in ("prop", "prop_fused"):
        dec.workspace(m)
    cs = rope_table(max_pages * page, d)
    w = (1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(dt)
    lens0 = torch.randint(20, (max_pages - 1) * page, (B,), generator=gen, **i32)
    table0 = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32).reshape(B, max_pages)
    have = (lens0 + page - 1) // page
    free0 = torch.cat([table0[b, int(have[b]):] for b in range(B)])
    for b in range(B):
        table0[b, int(have[b]):] = -5  # what the plan enters is read, not what lay there
    pools0 = [torch.randn((rows, hkv, d), generator=gen, device="cuda").to(dt) for _ in range(2)]
    qkvs = torch.randn((steps, B, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
    U = torch.rand((B, hq), generator=gen, device="cuda") / S * 0.999
    indptr = torch.arange(B + 1, device="cuda") * (max_pages * page)
    new = torch.ones(B, **i32)
    s = dict(lens=lens0.clone(), table=table0.clone(), free=free0.clone(), k=pools0[0].clone(), v=pools0[1].clone(),
             qkv=qkvs[0].clone(), slots=torch.empty(B, dtype=torch.int64, device="cuda"), pos=torch.empty(B, **i32),
             lens_out=torch.empty(B, **i32), counts=torch.empty(2, **i32))
    outs = {m: torch.empty((B, hq, d), device="cuda") for m in modes}
    qr = torch.empty((B, hq, d), dtype=dt, device="cuda")

    def restart():
        for name, t in (("lens", lens0), ("table", table0), ("free", free0), ("k", pools0[0]), ("v", pools0[1])):
            s[name].copy_(t)

    def step(pause):
        x = s["qkv"]
        dec.page_plan(s["lens"], new, s["table"], s["free"], page, s["slots"], s["pos"], s["lens_out"], s["counts"])
        pause()
        dec.norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["pos"], s["slots"], cs, s["k"], s["v"], w, w, out=qr)
        pause()
        dec.prop_paged(qr, s["k"], s["v"], s["table"], s["lens_out"], page, U, out=outs["paged"])
        pause()
        dec.norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["pos"], s["slots"], cs, s["k"], s["v"], out=qr)
        pause()
        dec("prop", qr, s["k"], s["v"], indptr, U, out=outs["prop"])
        pause()
        dec.norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["pos"], s["slots"], cs, s["k"], s["v"], w, None, out=qr)
        pause()
        dec("prop_fused", qr, s["k"], s["v"], indptr, U, out=outs["prop_fused"])
        pause()

    def run(one):
        restart()
        got = []
        for i in range(steps):
            s["qkv"].copy_(qkvs[i])
            one()
            got.append([outs[m].clone() for m in modes] + [qr.clone(), s["slots"].clone(), s["lens_out"].clone()])
            s["free"].copy_(torch.roll(s["free"], -int(s["counts"][0])))  # taken pages go to the end
            s["lens"].copy_(s["lens_out"])
        torch.cuda.synchronize()
        return got

    want = run(lambda: step(torch.cuda.synchronize))
    for a in want:
        assert all(torch.isfinite(x.float()).all() for x in a[:4]) and (a[4] >= 0).all()
    eager = run(lambda: step(lambda: None))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lambda: None)
    replayed = run(graph.replay)
    for a, b, c in zip(want, eager, replayed):
        for x, y, z in zip(a, b, c):
            assert torch.equal(x, y) and torch.equal(x, z)


# ------------------------------------------------------------------------------ README's steps, keys from their tokens


def _readme_step(call):
    """README's code block that makes `call`, comments apart."""
    import os
    import re

    readme = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    blocks = [re.sub(r"#[^\n]*", "", b) for b in re.findall(r"```python\n(.*?)```", open(readme).read(), re.S)]
    found = [b for b in blocks if f"dec.{call}(" in b]
    assert len(found) == 1, (call, len(found))
    return found[0]


@pytest.mark.parametrize("call", ["window_paged", "kv4_paged"])
def test_readme_step_as_written(call):
    """The step that README shows, run as it stands on a cache that earlier steps filled: the new token's row of the
    cache holds its key normalised and rotated to its position (worked out here from the raw key in 64 bits), its
    value, and the output is the attention over those."""
    B, hq, hkv, d, page_size, max_pages = 3, 8, 2, 128, 32, 5
    gen = torch.Generator(device="cuda").manual_seed(70)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = B * max_pages * page_size
    dec = Decoder(B, hq, hkv, d, rows, max_pages * page_size, 256, 1, "bf16")
    lens = [70, 31, 96]
    q0, k0, v0 = rnd(B, hq, d), rnd(B, hkv, d), rnd(B, hkv, d)
    qw, kw = (1 + 0.3 * rnd(d).float()).bfloat16(), (1 + 0.3 * rnd(d).float()).bfloat16()
    table = torch.arange(B * max_pages, **i32).reshape(B, max_pages).flip(0).contiguous()
    k_pool, v_pool, kv4 = rnd(rows, hkv, d), rnd(rows, hkv, d), dec.kv4_cache()
    dec.kv4_append(k_pool, v_pool, None, kv4)
    names = dict(dec=dec, torch=torch, q=q0.clone(), k=k0.clone(), v=v0.clone(), kv_lens=torch.tensor(lens, **i32),
                 new_lens=torch.ones(B, **i32), page_table=table, free_pages=torch.tensor([6, 7, 8, 9], **i32),
                 page_size=page_size, slot_map=torch.empty(B, dtype=torch.int64, device="cuda"),
                 positions=torch.empty(B, **i32), lens_out=torch.empty(B, **i32), counts=torch.empty(2, **i32),
                 cos_sin=rope_table(200, d), k_pool=k_pool, v_pool=v_pool, kv4=kv4, q_weight=qw, k_weight=kw)
    exec(_readme_step(call), names)
    assert names["lens_out"].tolist() == [n + 1 for n in lens]
    cs = names["cos_sin"][torch.tensor(lens, device="cuda")]
    kr, kmag = _rope_reference(k0, kw, 1e-6, cs, d, False)
    qr, qmag = _rope_reference(q0, qw, 1e-6, cs, d, False)
    _close(names["q"], qr, qmag, "q")
    for b, n in enumerate(lens):
        i = np.arange(n + 1)
        where = torch.from_numpy(names["page_table"].cpu().numpy()[b, i // page_size].astype(np.int64) * page_size + i % page_size).cuda()
        for h in range(hkv):
            if call == "kv4_paged":
                k, v = _values64(kv4[where, h], d)
                x, y = kr[b, h].bfloat16().double(), v0[b, h].double()
                # a code is off by half a step of the group's scale at most, and the scale (15 of them) and the minimum by
                # a rounding to fp16 (2^-11); the key, and the extremes of its group, by a step of bf16 (2^-7) before
                for got, want in ((k[-1], x), (v[-1], y)):
                    g = (torch.arange(d, device="cuda") // 8) % (d // 64)
                    lo, hi = (torch.stack([f(want[g == j]) for j in range(d // 64)])[g] for f in (torch.min, torch.max))
                    tol = (hi - lo) / 15 * (0.5 + 2.0 ** -6) + (2.0 ** -7 + 2.0 ** -10) * torch.maximum(lo.abs(), hi.abs())
                    assert ((got - want).abs() <= tol).all(), (b, h)
                keep = slice(None)
            else:
                k, v = k_pool[where, h].double(), v_pool[where, h].double()
                _close(k_pool[where[-1:], h], kr[b, h][None], kmag[b, h][None], "k")
                assert torch.equal(v[-1], v0[b, h].double())
                keep = torch.tensor(_seen(n + 1, 4096, 4), device="cuda")
            heads = slice(4 * h, 4 * h + 4)
            want, tol = _attention_reference(names["q"][b, heads].double(), k[keep], v[keep], 1 / math.sqrt(d), 2.0 ** -22)
            assert ((names["out"][b, heads].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_norm_rope_into_a_row_per_token(dtype, d):
    """Without a slot map a buffer of a row per token takes the rotated keys and the values: as rows of a whole cache."""
    dt, T, hkv = DT[dtype], 21, 3
    k, v = (torch.randn((T, hkv, d), device="cuda").to(dt) for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 5
    dec, cs = Decoder(1, hkv, hkv, d, 50, 50, 256, 1, dtype), rope_table(64, d)
    kc, vc = (torch.zeros((50, hkv, d), dtype=dt, device="cuda") for _ in range(2))
    kt, vt = torch.zeros_like(k), torch.zeros_like(v)
    dec.norm_rope(None, k, v, pos, None, cs, kc, vc)
    dec.norm_rope(None, k, v, pos, None, cs, kt, vt)
    assert torch.equal(kt, kc[:T]) and torch.equal(vt, v) and not kc[T:].any()
    slots = torch.arange(T, device="cuda")
    for bad in (dict(k_cache=kt, v_cache=vc, slot_map=slots), dict(k_cache=kc, v_cache=vt, slot_map=slots),
                dict(k_cache=kt[:-1], v_cache=vt, slot_map=None)):
        with pytest.raises(ValueError, match="_cache: shape"):
            dec.norm_rope(None, k, v, pos, bad["slot_map"], cs, bad["k_cache"], bad["v_cache"])
    few = Decoder(1, hkv, hkv, d, T - 1, T - 1, 256, 1, dtype)  # fewer rows than tokens: rows would be dropped
    with pytest.raises(ValueError, match="k_cache: shape"):
        few.norm_rope(None, k, v, pos, None, cs, kt, vt)


def test_a_step_without_a_token():
    """No new token at all: rotation, store and read back take empty tensors and leave the caches as they are."""
    hq, hkv, d, rows = 4, 2, 64, 32
    dec = Decoder(1, hq, hkv, d, rows, rows, 256, 1, "bf16")
    qkv = torch.empty((0, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    kc, vc = (torch.ones((rows, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv4 = dec.kv4_cache()
    pos, slots = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    cs = rope_table(rows, d)
    assert dec.norm_rope(q, k, v, pos, slots, cs, kc, vc).shape == (0, hq, d)
    assert dec.norm_rope(q, k, v, pos, None, cs, torch.empty_like(k), torch.empty_like(v)).shape == (0, hq, d)
    dec.kv4_append(k, v, slots, kv4)
    assert [tuple(x.shape) for x in dec.kv4_read(kv4, slots)] == [(0, hkv, d)] * 2
    assert (kc == 1).all() and (vc == 1).all() and not kv4.any()


@pytest.mark.parametrize("kind", ["window", "kv4"])
@pytest.mark.parametrize("rows,max_len,page", [(0, 64, 0), (64, 0, 0), (0, 0, 0), (64, 0, 32)])
def test_attention_without_a_key_gives_zeros(kind, rows, max_len, page):
    """A cache of no row, or sequences that may hold no key."""
    dec = Decoder(2, 4, 2, 64, rows, max_len, 256, 1, "bf16")
    q = torch.randn((2, 4, 64), device="cuda").bfloat16()
    pools = [torch.empty((rows, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    addr = dict(indptr=torch.zeros(3, dtype=torch.int64, device="cuda"),
                table=torch.zeros((2, 2), dtype=torch.int32, device="cuda"), lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    out = torch.full((2, 4, 64), 7.0, device="cuda")
    _run_attention(kind, dec, q, [dec.kv4_cache()] if kind == "kv4" else pools, addr, page, 10, 2, out=out)
    assert not out.any()


@pytest.mark.parametrize("name", ["window", "kv4", "norm_rope", "kv4_append", "kv4_read", "page_plan", "prop", "flash",
                                  "exact", "feature_blocked"])
def test_a_refused_call_is_reported_once(name):
    """A call into a capture that another call has invalidated is refused by the launch; the next call, after the
    capture's end, is not (the error that the first one left with the runtime is not its own)."""
    import ctypes

    c = _attention_case("window", "bf16", 128, 2, 4, [300, 40], 0, 0, 0, seed=80, poison=0.0)
    k4 = _attention_case("kv4", "bf16", 128, 2, 4, [300, 40], 0, 0, 0, seed=80)
    dec, q, (k, v), ind = c["dec"], c["q"], c["pools"], c["addr"]["indptr"]
    i32 = dict(dtype=torch.int32, device="cuda")
    n, rows = 5, dec.problem.total_tokens
    U, cs = torch.full((2, 8), 0.3, device="cuda"), rope_table(400, 128)
    x = torch.randn((n, 2, 128), device="cuda").bfloat16()
    pos, slots = torch.arange(n, **i32), torch.arange(n, device="cuda")
    out, new = torch.empty((2, 8, 128), device="cuda"), [torch.empty_like(x) for _ in range(2)]
    plan = [torch.zeros(2, **i32), torch.full((2,), 2, **i32), torch.zeros((2, 3), **i32), torch.tensor([3, 1], **i32)]
    got = [torch.empty(4, dtype=torch.int64, device="cuda"), torch.empty(4, **i32), torch.empty(2, **i32), torch.empty(2, **i32)]
    stream = torch.cuda.Stream()
    on = dict(stream=stream)
    calls = {
        "window": lambda: (dec.window(q, k, v, ind, 50, 3, out=out, **on),),
        "kv4": lambda: (k4["dec"].kv4(q, k4["pools"][0], ind, out=out, **on),),
        "norm_rope": lambda: (dec.norm_rope(None, x, x, pos, None, cs, *new, **on), *new)[1:],
        "kv4_append": lambda: (dec.kv4_append(x, x, slots, k4["pools"][0], **on),),
        "kv4_read": lambda: dec.kv4_read(k4["pools"][0], slots, *new, **on),
        "page_plan": lambda: (dec.page_plan(plan[0], plan[1], plan[2], plan[3], 1, *got, **on), *got)[1:],
        "feature_blocked": lambda: (dec.feature_blocked(k, **on),),
        **{m: lambda m=m: (dec(m, q, k, v, ind, U, out=out, **on),) for m in ("prop", "flash", "exact")},
    }
    call = calls[name]
    dec.workspace("prop"), dec.workspace("flash"), dec.workspace("exact")
    torch.cuda.synchronize()
    want = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    want = [t.clone() for t in want]
    torch.cuda.synchronize()
    driver = ctypes.CDLL("libcuda.so.1")
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(handle, ctypes.c_int(2)) == 0
    assert driver.cuStreamSynchronize(handle) != 0  # not allowed in a capture: invalidates it
    with pytest.raises(sd.SantaError) as refused:
        call()
    assert driver.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0 and not graph.value
    assert refused.value.status == sd.CUDA_ERROR
    again = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again)) and len(want) == len(again)


# ------------------------------------------------------------------------------ prompts through norm + rotation


def _many_rows(tokens, heads, d):
    """Whether a call has enough tokens for the kernels that keep several rows of a lane in flight (prompts)."""
    parts = 1
    while parts < heads and tokens * parts * (d // 8) < 152 * 640:
        parts *= 2
    return 4 * parts <= heads


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hq,hkv,rot,inter,norm,form", [
    (6500, 12, 4, 1.0, False, True, "fused"), (2500, 27, 9, 1.0, False, False, "fused"),
    (2500, 27, 9, 0.5, False, True, "in place"), (6500, 12, 4, 0.25, False, False, "in place"),
    (6500, 12, 4, 0.25, True, False, "fused"), (2500, 27, 9, 0.75, True, True, "in place"),
    (12500, 3, 1, 1.0, False, True, "fused"), (12500, 3, 1, 0.5, True, False, "in place"),
    (2500, 40, 1, 0.75, False, True, "fused"), (6500, 20, 2, 1.0, True, True, "q alone"),
    (9000, 30, 30, 0.5, False, True, "k alone"),
])
def test_norm_rope_of_prompts(dtype, d, T, hq, hkv, rot, inter, norm, form):
    """Both pairings, whole and partial rotations, with and without norms, q in place, one kind alone."""
    dt = DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T + hq)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    assert _many_rows(T, {"q alone": hq, "k alone": hkv}.get(form, hq + 2 * hkv), d)
    if form == "fused":
        qkv = rnd(T, hq + 2 * hkv + 1, d).to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = (rnd(T, h, d).to(dt) for h in (hq, hkv, hkv))
    rot, rows = int(rot * d), T + 9
    cs = rope_table(5000, rot)
    pos = torch.randint(0, 5000, (T,), generator=gen, device="cuda", dtype=torch.int32)
    slots = torch.randperm(rows, generator=gen, device="cuda")[:T].contiguous()
    slots[::7] = -1  # padding
    qw, kw = ((1 + 0.3 * rnd(d)).to(dt), (1 + 0.3 * rnd(d)).to(dt)) if norm else (None, None)
    kc, vc = rnd(rows, hkv, d).to(dt), rnd(rows, hkv, d).to(dt)
    kc0, vc0, q0 = kc.clone(), vc.clone(), q.clone()
    dec = Decoder(1, hq, hkv, d, rows, rows, 256, 1, dtype)
    dbg, word = _debug()
    args = dict(interleaved=inter, eps=1e-5, debug=dbg)
    if form == "q alone":
        out = dec.norm_rope(q, None, None, pos, slots, cs, None, None, qw, kw, **args)
    elif form == "k alone":
        out = dec.norm_rope(None, k, None, pos, slots, cs, kc, None, qw, kw, **args)
    else:
        out = dec.norm_rope(q, k, v, pos, slots, cs, kc, vc, qw, kw, out=q if form == "in place" else None, **args)
    assert _flags(word) == 0
    angles = cs[pos.long()]
    if out is not None:
        want, mag = _rope_reference(q0, qw, 1e-5, angles, rot, inter)
        _close(out, want, mag, "q")
    live = slots >= 0
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    if form != "q alone":
        want, mag = _rope_reference(k, kw, 1e-5, angles, rot, inter)
        _close(kc[slots[live]], want[live], mag[live], "k")
    if not form.endswith("alone"):
        assert torch.equal(vc[slots[live]], v[live])
    else:
        assert torch.equal(vc, vc0)
    if form == "q alone":
        assert torch.equal(kc, kc0)
    assert torch.equal(kc[rest], kc0[rest]) and torch.equal(vc[rest], vc0[rest])


# ------------------------------------------------------------------------------ a loop against the tokens' own history


@pytest.mark.parametrize("kind", ["window", "kv4"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_a_serving_loop_against_raw_tokens(kind, dtype, d):
    """Prompts, then tokens one by one: pages and rows come from the plan's definition, keys and queries from the raw
    tokens, normalised and rotated to their index in 64 bits.  Every row of the history is compared with the cache
    after the last step, and each step's output with the attention over the history (in 4 bits: over what those rows
    stand for).

    The cache holds a rounding of each key, and q of each query, with the half step of its type, in front of which the
    rotation errs by 24 u of a pair; in 4 bits a value is off by half a step of the group's scale and the roundings of
    minimum and scale.  With dk and dq as those a logit is off by dx = |q| dk + dq (|k| + dk), and a weight by a factor
    between exp(-2 max dx) and exp(2 max dx)."""
    dt, B, hq, hkv, page, max_pages, num_pages = DT[dtype], 4, 6, 2, 32, 12, 64
    gen = torch.Generator(device="cuda").manual_seed(90)
    i32 = dict(dtype=torch.int32, device="cuda")
    half = torch.finfo(dt).eps / 2
    dec = Decoder(B, hq, hkv, d, num_pages * page, max_pages * page, 256, 1, dtype)
    cs = rope_table(max_pages * page, d)
    qw, kw = ((1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(dt) for _ in range(2))
    k_pool, v_pool = (torch.full((num_pages * page, hkv, d), math.nan, device="cuda", dtype=dt) for _ in range(2))
    kv4 = dec.kv4_cache().fill_(0xFF)  # NaN scales in every row that is not written
    lens, table = torch.zeros(B, **i32), torch.full((B, max_pages), -1, **i32)
    lens_h, table_h = np.zeros(B, np.int32), np.full((B, max_pages), -1, np.int32)
    free_h = np.random.default_rng(2).permutation(num_pages).astype(np.int32)
    hist = [dict(row=[], k=[], v=[]) for _ in range(B)]
    window, sinks, scale = 45, 3, 1 / math.sqrt(d)

    def record_error(x):
        """How far a 4-bit record of x [..][d] may lie from it."""
        g = (torch.arange(d, device="cuda") // 8) % (d // 64)
        lo, hi = (torch.stack([f(x[..., g == j], -1) for j in range(d // 64)], -1)[..., g] for f in (torch.amin, torch.amax))
        # scale and minimum are rounded to fp16 (2^-11), 15 scales between the extremes
        return (hi - lo) / 15 * (0.5 + 16 * 2.0 ** -11) + 2.0 ** -11 * torch.maximum(lo.abs(), hi.abs()) + 2.0 ** -24

    for step in range(5):
        new = [50, 1, 33, 96] if step == 0 else [1, 1, 0, 1] if step == 2 else [1] * B
        tokens = sum(new) + 2
        qkv = torch.randn((tokens, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        slots, pos = torch.empty(tokens, dtype=torch.int64, device="cuda"), torch.empty(tokens, **i32)
        lens_out, counts = torch.empty(B, **i32), torch.empty(2, **i32)
        dec.page_plan(lens, torch.tensor(new, **i32), table, torch.from_numpy(free_h).cuda(), page, slots, pos, lens_out, counts)
        if kind == "kv4":
            k_rot = k.new_empty(k.shape)
            qr = dec.norm_rope(q, k, None, pos, None, cs, k_rot, None, qw, kw)
            dec.kv4_append(k_rot, v, slots, kv4)
        else:
            qr = dec.norm_rope(q, k, v, pos, slots, cs, k_pool, v_pool, qw, kw)
        table_h, slots_h, pos_h, lens_h, counts_h, flags = _plan_reference(lens_h, np.array(new, np.int32), table_h, free_h,
                                                                           page, num_pages, tokens)
        assert flags == 0
        free_h, lens = free_h[counts_h[0]:], lens_out
        t, last = 0, []
        angles = cs[torch.from_numpy(pos_h).long().cuda()]
        (kr, kmag), (qx, qmag) = (_rope_reference(x, w, 1e-6, angles, d, False) for x, w in ((k, kw), (q, qw)))
        for b in range(B):
            for _ in range(new[b]):
                assert int(pos_h[t]) == len(hist[b]["row"])
                hist[b]["row"].append(int(slots_h[t]))
                hist[b]["k"].append((kr[t], half * kr[t].abs() + 24 * 2.0 ** -24 * kmag[t]))
                hist[b]["v"].append(v[t].double())
                t += 1
            last.append(t - 1)  # the sequence's newest token (step 2: sequence 2 has none, its query is another's)
        if step == 0:
            continue
        at = torch.tensor(last, device="cuda")
        qs = qr[at].contiguous()
        if kind == "kv4":
            out = dec.kv4_paged(qs, kv4, table, lens, page, window, sinks)
        else:
            out = dec.window_paged(qs, k_pool, v_pool, table, lens, page, window, sinks)
        assert lens.tolist() == lens_h.tolist() and torch.equal(table.cpu(), torch.from_numpy(table_h))
        for b in range(B):
            keep = _seen(len(hist[b]["row"]), window, sinks)
            for h in range(hkv):
                if kind == "kv4":
                    kk, vv = _values64(kv4[torch.tensor(hist[b]["row"], device="cuda")[keep], h], d)
                    dk = torch.zeros_like(kk)
                else:
                    kk, dk = (torch.stack([hist[b]["k"][i][j][h] for i in keep]) for j in range(2))
                    vv = torch.stack([hist[b]["v"][i][h] for i in keep])
                heads = slice(3 * h, 3 * h + 3)
                qq = qx[at[b], heads]
                dq = half * qq.abs() + 24 * 2.0 ** -24 * qmag[at[b], heads]
                want, tol = _attention_reference(qq, kk, vv, scale, 2.0 ** -22)
                p = torch.softmax(qq @ kk.T * scale, -1)
                dx = (qq.abs() @ dk.T + dq @ (kk.abs() + dk).T) * scale
                tol = tol + torch.expm1(2 * dx.amax(-1, keepdim=True)) * (p @ vv.abs())
                err = (out[b, heads].double() - want).abs()
                assert (err <= tol).all(), (step, b, h, float((err / tol).max()))
    for b in range(B):
        rows = torch.tensor(hist[b]["row"], device="cuda")
        kk, dk = (torch.stack([x[j] for x in hist[b]["k"]]) for j in range(2))
        vv = torch.stack(hist[b]["v"])
        if kind == "kv4":
            got_k, got_v = _values64(kv4[rows], d)
            assert ((got_v - vv).abs() <= record_error(vv)).all()
            # of the rounded key, whose group's extremes may lie dk further out
            dk = dk + record_error(kk) + 2 / 15 * dk.amax(-1, keepdim=True)
        else:
            got_k = k_pool[rows].double()
            assert torch.equal(v_pool[rows].double(), vv)
        assert ((got_k - kk).abs() <= dk).all()
    used = torch.tensor(sorted({r for x in hist for r in x["row"]}), device="cuda")
    rest = torch.ones(num_pages * page, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert len(used) == sum(len(x["row"]) for x in hist)
    assert (kv4[rest] == 0xFF).all() and k_pool[rest].isnan().all() and v_pool[rest].isnan().all()


@pytest.mark.parametrize("garbage", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 4), ("bf16", 64, 8), ("bf16", 128, 1), ("f32", 64, 2)])
def test_exact_decode_sees_no_row_behind_the_sequence(dtype, d, g, garbage):
    """The block of 32 rows that holds a sequence's last keys goes on into the rows behind it (the next sequence's, or
    those of a cache that is not full): whatever they hold, exact_decode gives the same bits."""
    lens, hkv, dt = [1, 45, 64, 31, 333], 2, DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(100)
    gap = 40  # rows between the sequences: kv_indptr leaves none out, so a sequence of garbage stands there
    starts, at = [], 0
    for n in lens:
        starts += [at, at + n]
        at += n + gap
    rows = at + 5
    k, v = (torch.randn((rows, hkv, d), generator=gen, device="cuda").to(dt) for _ in range(2))
    B = 2 * len(lens)  # every second sequence is a gap
    ind = torch.tensor(starts + [at], device="cuda")
    q = torch.randn((B, hkv * g, d), generator=gen, device="cuda").to(dt)
    dec = Decoder(B, hkv * g, hkv, d, rows, 400, 256, 1, dtype)
    want = dec("exact", q, k, v, ind)
    for i, n in enumerate(lens):
        for x in (k, v):
            x[starts[2 * i + 1]:starts[2 * i + 1] + gap] = garbage
    k[at:], v[at:] = garbage, garbage
    got = dec("exact", q, k, v, ind)
    assert torch.isfinite(want).all() and torch.equal(got[::2], want[::2])
