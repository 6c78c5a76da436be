"""Rotation by several axes, attention over a shared prefix, key weights and eviction, on the GPU, each against a
plain implementation in 64 bits (whole numbers and moved rows: exactly), and a run of them together.

Tolerances as in test_gpu_serving: u is the unit of the sums (fp32 2^-24; on the tensor cores, which may truncate,
2^-23), a rounding of the output to its type is half a step.
"""

import math

import numpy as np
import pytest
import torch

import stochastic_sparse_decode_gb300 as sd
from stochastic_sparse_decode_gb300.decoder import (Decoder, rope_sections, rope_table, rope_table_axes, rope_turns)
from test_gpu_serving import DT, _attention_reference, _close, _debug, _flags, _rope_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session", autouse=True)
def built_library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from stochastic_sparse_decode_gb300.build import build

    build()


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


# ------------------------------------------------------------------------------ rotation by several axes


def _axes_table(cs, pos, axis):
    """The rows of cosines and sines [T][rot] that the tokens turn by."""
    half = cs.shape[1] // 2
    pair = torch.arange(half, device="cuda")
    n = pos.long()[torch.tensor(axis, device="cuda")].T
    return torch.cat([cs[n, pair], cs[n, half + pair]], 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hq,hkv,rot,kind,axes,inter,norm", [
    (1, 4, 1, 1.0, "sections", 3, False, True), (3, 32, 8, 1.0, "turns", 3, False, False), (17, 8, 8, 0.5, "own", 2, True, True),
    (200, 6, 2, 0.75, "turns", 4, False, True), (33, 5, 5, 0.25, "own", 4, True, False), (1000, 32, 4, 1.0, "sections", 3, True, True),
    (2500, 16, 2, 1.0, "one", 1, False, False),
])
def test_norm_rope_axes(dtype, d, T, hq, hkv, rot, kind, axes, inter, norm):
    dt, rot = DT[dtype], int(rot * d)
    half = rot // 2
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    qkv = rnd(T, hq + 2 * hkv + 1, d).to(dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    sections = [half // axes] * (axes - 1) + [half - half // axes * (axes - 1)]
    if axes == 3:  # uneven, and no multiple of four
        sections = [half // 4 + 1, half // 4 + 2, half - 2 * (half // 4) - 3]
    axis = rope_turns(half, axes) if kind == "turns" else rope_sections(sections)
    cs = rope_table_axes(3000, sections) if kind == "own" else rope_table(3000, rot)
    wide = torch.randint(0, 3000, (axes, T + 5), generator=gen, device="cuda", dtype=torch.int32)
    pos = wide[:, :T]  # rows further apart than the tokens
    slots = torch.randperm(T + 7, generator=gen, device="cuda")[:T].contiguous()
    slots[T // 2] = -1 if T > 1 else slots[0]
    qw, kw = ((1 + 0.3 * rnd(d)).to(dt), (1 + 0.3 * rnd(d)).to(dt)) if norm else (None, None)
    kc, vc = rnd(T + 7, hkv, d).to(dt), rnd(T + 7, hkv, d).to(dt)
    kc0, vc0 = kc.clone(), vc.clone()
    dec = Decoder(1, hq, hkv, d, T + 7, T + 7, 256, 1, dtype)
    dbg, word = _debug()
    out = dec.norm_rope_axes(q, k, v, pos, axis, slots, cs, kc, vc, qw, kw, 1e-5, inter, debug=dbg)
    assert _flags(word) == 0
    rows = _axes_table(cs, pos, axis)
    _close(out, *_rope_reference(q, qw, 1e-5, rows, rot, inter), "q")
    want, mag = _rope_reference(k, kw, 1e-5, rows, rot, inter)
    live = slots >= 0
    _close(kc[slots[live]], want[live], mag[live], "k")
    assert torch.equal(vc[slots[live]], v[live])
    rest = torch.ones(T + 7, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert torch.equal(kc[rest], kc0[rest]) and torch.equal(vc[rest], vc0[rest])


@pytest.mark.parametrize("T", [1, 40, 3000])
def test_axes_that_agree_give_norm_rope(T):
    """Text: the same number on every axis, and equal bits."""
    q, k = torch.randn((T, 8, 128), device="cuda").bfloat16(), torch.randn((T, 2, 128), device="cuda").bfloat16()
    pos = torch.randint(0, 100, (T,), device="cuda", dtype=torch.int32)
    cs = rope_table(100, 128)
    dec = Decoder(1, 8, 2, 128, T, T, 256, 1, "bf16")
    kc, kc2 = torch.zeros_like(k), torch.zeros_like(k)
    a = dec.norm_rope(q, k, None, pos, None, cs, kc, None)
    b = dec.norm_rope_axes(q, k, None, pos.expand(3, T).contiguous(), rope_sections((16, 24, 24)), None, cs, kc2, None)
    assert torch.equal(a, b) and torch.equal(kc, kc2)


def test_axes_bad_positions_are_flagged_per_axis():
    T, d = 4, 64
    q = torch.randn((T, 1, d), device="cuda")
    cs, axis = rope_table(10, d), rope_sections((10, 22))
    pos = _ints([[0, -1, 3, 9], [10, 2, 2**31 - 1, 9]])
    dec = Decoder(1, 1, 1, d, T, T, 256, 1, "f32")
    dbg, word = _debug()
    out = dec.norm_rope_axes(q, None, None, pos, axis, None, cs, None, None, debug=dbg)
    assert _flags(word) == sd.ERR_POSITION
    _close(out, *_rope_reference(q, None, 0.0, _axes_table(cs, pos.clamp(0, 9), axis), d, False), "q")
    dec.norm_rope_axes(q[:0], None, None, pos[:, :0], axis, None, cs, None, None)


# ------------------------------------------------------------------------------ shared prefix


def _shared_case(dtype, d, hkv, g, prefix, lens, page=0, seed=0, start=3, poison=math.nan, scale=1.0):
    """A cache with the prefix and the sequences' own rows, all others poisoned; kv: (k, v) rows of each sequence."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 7 * prefix + d)
    dt, B = DT[dtype], len(lens)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    q = rnd(B, hkv * g, d) * scale
    if page:
        shared, have = -(-prefix // page), [-(-(prefix + n) // page) for n in lens]
        # a prefix that ends inside a page: its page is copied for each sequence, as a program would
        whole = prefix // page
        num_pages = whole + sum(h - whole for h in have) + 4 + (shared - whole)
        ids = torch.randperm(num_pages, generator=gen, device="cuda").tolist()
        common, table = ids[:whole], []
        at = whole
        for h in have:
            table.append(common + ids[at:at + h - whole])
            at += h - whole
        width = max([len(r) for r in table] + [shared, 1]) + 1
        if not table[0][whole:] and shared > whole:  # sequence 0's row holds the prefix in any case
            table[0] = table[0] + ids[at:at + 1]
        table = [r + [-1] * (width - len(r)) for r in table]
        where = [torch.tensor([table[b][i // page] * page + i % page for i in range(prefix + lens[b])], device="cuda",
                              dtype=torch.int64) for b in range(B)]
        rows = num_pages * page
        first = torch.tensor([table[0][i // page] * page + i % page for i in range(prefix)], device="cuda", dtype=torch.int64)
        addr = (_ints(table), _ints([prefix + n for n in lens]))
        max_len = prefix + max(lens, default=0)
    else:
        gap = 5  # rows between the prefix and the sequences
        indptr = np.cumsum([start + prefix + gap] + lens)
        first = start + torch.arange(prefix, device="cuda")
        where = [torch.cat([first, torch.arange(indptr[b], indptr[b + 1], device="cuda")]) for b in range(B)]
        rows = int(indptr[-1]) + 40
        addr = _ints(indptr.tolist(), torch.int64)
        max_len = max(lens, default=0)
    k, v = (torch.full((rows, hkv, d), poison, device="cuda").to(dt) for _ in range(2))
    common = torch.zeros(rows, dtype=torch.bool, device="cuda")
    common[first] = True
    pk, pv = rnd(prefix, hkv, d), rnd(prefix, hkv, d)
    for w in where:
        k[w[prefix:]], v[w[prefix:]] = rnd(len(w) - prefix, hkv, d), rnd(len(w) - prefix, hkv, d)
        k[w[:prefix]], v[w[:prefix]] = pk, pv  # (the copies of a page that is not whole)
    k[first], v[first] = pk, pv
    dec = Decoder(B, hkv * g, hkv, d, rows, max_len, 256, 1, dtype)
    c = dict(dec=dec, q=q, k=k, v=v, addr=addr, page=page, prefix=prefix, start=start, where=where, g=g, hkv=hkv, d=d,
             dtype=dtype, lens=lens)
    dbg, word = _debug()
    c["out"] = _run_shared(c, debug=dbg)
    assert _flags(word) == 0
    return c


def _run_shared(c, **kw):
    if c["page"]:
        return c["dec"].shared_paged(c["q"], c["k"], c["v"], *c["addr"], c["page"], c["prefix"], **kw)
    return c["dec"].shared(c["q"], c["k"], c["v"], c["addr"], c["start"], c["prefix"], **kw)


def _check_shared(c, out=None):
    u, d = (2.0 ** -23 if c["dtype"] == "bf16" else 2.0 ** -24), c["d"]
    out = c["out"] if out is None else out
    for b, w in enumerate(c["where"]):
        if not len(w):
            assert not out[b].any()
            continue
        for h in range(c["hkv"]):
            heads = slice(h * c["g"], (h + 1) * c["g"])
            want, tol = _attention_reference(c["q"][b, heads].double(), c["k"][w, h].double(), c["v"][w, h].double(),
                                             1 / math.sqrt(d), u)
            err = (out[b, heads].double() - want).abs()
            assert (err <= tol).all(), (b, h, float((err / tol).max()))


@pytest.mark.parametrize("dtype,d,hkv,g", [("bf16", 128, 2, 4), ("bf16", 64, 1, 8), ("f32", 128, 1, 2), ("f32", 64, 2, 3),
                                           ("bf16", 128, 1, 1), ("bf16", 64, 3, 5)])
@pytest.mark.parametrize("page", [0, 32, 96])
def test_shared(dtype, d, hkv, g, page):
    for i, (prefix, lens) in enumerate([(1, [0]), (31, [1, 0, 40]), (64, [5, 64, 65, 33]), (65, [0, 0]), (127, [200, 1]),
                                        (500, [3] * 20), (1000, [0, 700, 31])]):
        _check_shared(_shared_case(dtype, d, hkv, g, prefix, lens, page, seed=i))


@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 4), ("bf16", 64, 8), ("f32", 64, 4)])
@pytest.mark.parametrize("B", [1, 15, 16, 17, 31, 32, 33, 64, 65, 97, 300])
def test_shared_rows_around_the_tiles(dtype, d, g, B):
    """Query rows on both sides of a tile's 64, 128 and 256, and several tiles."""
    _check_shared(_shared_case(dtype, d, 1, g, 333, [i % 3 for i in range(B)], seed=B))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_shared_over_many_keys(dtype, d):
    """Long stretches per CTA, and items that CTAs share unevenly."""
    _check_shared(_shared_case(dtype, d, 2, 4, 20011, [100, 0, 7], 32, seed=1))
    _check_shared(_shared_case(dtype, d, 1, 2, 30000, [1], seed=2))
    _check_shared(_shared_case(dtype, d, 3, 4, 9001, [2] * 70, seed=3))


@pytest.mark.parametrize("garbage", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 0), ("bf16", 64, 32), ("f32", 64, 0)])
def test_rows_that_no_sequence_sees_do_not_matter(dtype, d, page, garbage):
    a = _shared_case(dtype, d, 2, 2, 101, [7, 0, 50], page, seed=4, poison=garbage)
    b = _shared_case(dtype, d, 2, 2, 101, [7, 0, 50], page, seed=4, poison=0.0)
    assert torch.equal(a["out"], b["out"])
    _check_shared(a)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_shared_large_logits(dtype, d):
    """Logits of hundreds: the running maximum moves by many powers of two from block to block."""
    c = _shared_case(dtype, d, 1, 4, 900, [33, 0, 5], seed=5, scale=30.0)
    c["k"][c["where"][0][700]] *= 4
    c["out"] = _run_shared(c)
    _check_shared(c)
    c["q"].zero_()  # every key alike: a mean
    c["out"] = _run_shared(c)
    _check_shared(c)


@pytest.mark.parametrize("dtype,d,g", [("bf16", 128, 4), ("bf16", 64, 2), ("f32", 64, 4)])
def test_shared_precision_of_means_over_many_keys(dtype, d, g):
    """V = 1 + small, equal logits: a drift of the sums over 30000 keys would show.  A stretch's block sums join O by
    an fp32 fma (1.5 u each at most; at most 470 blocks a stretch), the block's own 64 terms are within 64 u."""
    c = _shared_case(dtype, d, 1, g, 30000, [3], seed=6)
    c["q"].zero_()
    c["v"].copy_((1 + torch.rand(c["v"].shape, device="cuda") * 2.0 ** -4).to(c["v"].dtype))
    got = _run_shared(c)[0, 0].double()
    want = c["v"][c["where"][0], 0].double().mean(0)
    assert ((got - want).abs() <= 2.0 ** -23 * (470 * 1.5 + 64) * want).all()
    # ten times closer than that bound, in the mean: roundings do not all point one way
    assert float(((got - want) / want).abs().mean()) <= 2.0 ** -23 * 77


def test_shared_equals_itself_paged_and_again():
    """Pages of 32 and contiguous rows, calls one after another and on a stream with another Decoder: equal bits."""
    lens, prefix = [40, 0, 300, 9], 640
    a = _shared_case("bf16", 128, 2, 4, prefix, lens, 0, seed=8)
    b = _shared_case("bf16", 128, 2, 4, prefix, lens, 32, seed=8)
    for dst, src in zip(b["where"], a["where"]):
        b["k"][dst], b["v"][dst] = a["k"][src], a["v"][src]
    b["q"].copy_(a["q"])
    first = _run_shared(a)
    for _ in range(5):
        assert torch.equal(_run_shared(a), first)
        assert torch.equal(_run_shared(b), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [_run_shared(b) for _ in range(20)]
    outs += [_run_shared(a) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for x in outs)


def test_shared_without_prefix_is_the_windowed_call_and_without_keys_zeros():
    c = _shared_case("bf16", 128, 2, 4, 0, [100, 0, 33], seed=9)
    _check_shared(c)
    assert torch.equal(c["out"], c["dec"].window(c["q"], c["k"], c["v"], c["addr"], 0))
    c = _shared_case("bf16", 128, 2, 4, 0, [0, 0], seed=10)
    assert not c["out"].any()
    c = _shared_case("f32", 64, 1, 1, 50, [0, 0, 0], seed=11)  # max_len 0: the prefix alone
    _check_shared(c)


def test_shared_bad_device_data_is_flagged():
    c = _shared_case("bf16", 128, 1, 4, 128, [64, 10], 32, seed=12)
    dbg, word = _debug()
    table, lens = c["addr"]
    table[0, 1] = 10**6  # one page of the prefix: its 32 keys are dropped for everyone
    out = _run_shared(c, debug=dbg)
    assert _flags(word) == sd.ERR_INDPTR
    kept = [torch.cat([w[:32], w[64:]]) for w in c["where"]]
    _check_shared({**c, "where": kept}, out)
    table[0, 1] = table[1, 1]
    lens[1] = 100  # fewer than the prefix: no keys of its own
    out = _run_shared(c, debug=dbg)
    assert _flags(word) == 0
    _check_shared({**c, "where": [c["where"][0], c["where"][1][:128]]}, out)
    lens[1] = -5
    out = _run_shared(c, debug=dbg)
    assert _flags(word) == sd.ERR_INDPTR
    _check_shared({**c, "where": [c["where"][0], c["where"][1][:128]]}, out)


def test_shared_captured_and_replayed():
    c = _shared_case("bf16", 128, 2, 4, 700, [40, 3, 90], 32, seed=13)
    d = _shared_case("bf16", 128, 2, 4, 700, [1, 80, 30], 32, seed=14)
    graphs = []
    for x in (c, d):  # a workspace each
        x["static"] = torch.empty_like(x["out"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _run_shared(x, out=x["static"])
        graphs.append(g)
    for x in (c, d):
        x["q"].normal_()
        x["want"] = _run_shared(x)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for x in (c, d):
        assert torch.equal(x["static"], x["want"])
        _check_shared(x, x["static"])


# ------------------------------------------------------------------------------ key weights


def _cache(lens, page, rng, spare=40):
    """(rows of each sequence, rows of the cache, page table or indptr, lens)."""
    if not page:
        indptr = np.cumsum([3] + lens)
        return ([torch.arange(indptr[b], indptr[b + 1], device="cuda") for b in range(len(lens))], int(indptr[-1]) + spare,
                _ints(indptr.tolist(), torch.int64))
    have = [-(-n // page) for n in lens]
    num_pages = sum(have) + 3
    ids = rng.permutation(num_pages)
    table, at = np.full((len(lens), max(have, default=0) + 1), -1, np.int32), 0
    for b, h in enumerate(have):
        table[b, :h] = ids[at:at + h]
        at += h
    rows = [torch.tensor([int(table[b, i // page]) * page + i % page for i in range(n)], device="cuda", dtype=torch.int64)
            for b, n in enumerate(lens)]
    return rows, num_pages * page, _ints(table.tolist())


def _weights_reference(q, k, scale, u):
    """Sum over the group of softmax(q k / sqrt d), and its bound (see _attention_reference; two exponentials, the
    factor's product and division: 16 u)."""
    x = q @ k.T * scale
    p = torch.softmax(x, -1)
    d, n = k.shape[1], k.shape[0]
    dx = (d + 8) * u * (q.abs() @ k.abs().T) * scale + 4 * u * (x - x.amax(-1, keepdim=True)).abs() + 16 * u
    dz = (p * dx).sum(-1, keepdim=True) + (n / 32 + 96) * u
    return p.sum(0), (p * (dx + dz)).sum(0) + 8 * u * p.sum(0)


@pytest.mark.parametrize("dtype,d,hkv,g,page", [("bf16", 128, 2, 4, 0), ("bf16", 64, 1, 8, 32), ("f32", 128, 1, 2, 64),
                                                ("f32", 64, 3, 1, 0), ("bf16", 128, 2, 1, 96)])
def test_key_weights(dtype, d, hkv, g, page):
    rng, dt, u = np.random.default_rng(d + page), DT[dtype], (2.0 ** -23 if dtype == "bf16" else 2.0 ** -24)
    for lens in ([1], [0, 5, 31, 32, 33], [300, 1, 64], [5000, 17], [0, 0], [90] * 30):
        where, rows, addr = _cache(lens, page, rng)
        B = len(lens)
        q, k = torch.randn((B, hkv * g, d), device="cuda").to(dt), torch.full((rows, hkv, d), math.nan, device="cuda").to(dt)
        for w in where:
            k[w] = torch.randn((len(w), hkv, d), device="cuda").to(dt)
        dec = Decoder(B, hkv * g, hkv, d, rows, max(lens), 256, 1, dtype)
        scores = torch.rand((hkv, rows), device="cuda")
        before = scores.clone()
        dbg, word = _debug()

        def call(scores, out=None, decay=1.0, fresh=0):
            if page:
                return dec.key_weights_paged(q, k, addr, _ints(lens), page, scores, out, decay, fresh, debug=dbg)
            return dec.key_weights(q, k, addr, scores, out, decay, fresh, debug=dbg)

        apart = torch.full((hkv, rows), 7.0, device="cuda")
        call(scores, apart, 0.75, 2)
        assert torch.equal(scores, before)
        alone = call(None, torch.zeros((hkv, rows), device="cuda"))
        got = call(scores, None, 0.75, 2)
        assert got.data_ptr() == scores.data_ptr() and _flags(word) == 0
        rest = torch.ones(rows, dtype=torch.bool, device="cuda")
        for b, w in enumerate(where):
            rest[w] = False
            for h in range(hkv):
                if not len(w):
                    continue
                want, tol = _weights_reference(q[b, h * g:(h + 1) * g].double(), k[w, h].double(), 1 / math.sqrt(d), u)
                assert ((alone[h, w].double() - want).abs() <= tol).all()
                old = 0.75 * before[h, w].double()
                old[max(0, len(w) - 2):] = 0
                assert ((got[h, w].double() - old - want).abs() <= tol + 2 * 2.0 ** -24 * (old + want)).all()
                assert abs(float(alone[h, w].double().sum()) - g) <= g * 1e-5  # each head's weights add up to one
        assert torch.equal(got[:, rest], before[:, rest]) and (apart[:, rest] == 7.0).all()
        assert torch.equal(apart[:, ~rest], got[:, ~rest])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_key_weights_between_the_sampled_passes(dtype, d):
    """After pass1: the same bits as the whole call, and pass2 samples as if nothing had come between."""
    lens, hq, hkv = [700, 0, 1300], 8, 2
    where, rows, indptr = _cache(lens, 0, None)
    q, k, v = (torch.randn(s, device="cuda").to(DT[dtype]) for s in ((3, hq, d), (rows, hkv, d), (rows, hkv, d)))
    dec = Decoder(3, hq, hkv, d, rows, max(lens), 256, 64, dtype)
    U = torch.rand((3, hq), device="cuda") / 64
    want = dec.key_weights(q, k, indptr, torch.zeros((hkv, rows), device="cuda"))
    out = dec("prop", q, k, v, indptr, U)
    for _ in range(2):
        dec.pass1(q, k, indptr)
        got = dec.key_weights(None, None, indptr, torch.zeros((hkv, rows), device="cuda"))
        assert torch.equal(got, want)
        assert torch.equal(dec.pass2(v, indptr, U), out)
    assert torch.equal(dec("prop_fused", q, k, v, indptr, U), dec("prop_fused", q, k, v, indptr, U))


def test_key_weights_drop_bad_pages():
    lens, page = [100, 40], 32
    where, rows, table = _cache(lens, page, np.random.default_rng(5))
    q, k = torch.randn((2, 4, 64), device="cuda"), torch.randn((rows, 1, 64), device="cuda")
    table[0, 1] = -7
    dec = Decoder(2, 4, 1, 64, rows, 100, 256, 1, "f32")
    dbg, word = _debug()
    got = dec.key_weights_paged(q, k, table, _ints(lens), page, torch.zeros((1, rows), device="cuda"), debug=dbg)
    assert _flags(word) == sd.ERR_INDPTR
    w = torch.cat([where[0][:32], where[0][64:]])
    want, tol = _weights_reference(q[0].double(), k[w, 0].double(), 1 / 8, 2.0 ** -24)
    assert ((got[0, w].double() - want).abs() <= tol).all() and not got[0, where[0][32:64]].any()


# ------------------------------------------------------------------------------ eviction


def _kept(scores, n, sinks, recent, budget):
    """The definition, on the host: the indices kept of n keys."""
    lo = min(sinks, n)
    hi = max(lo, n - recent)
    order = sorted(range(lo, hi), key=lambda i: (-scores[i] if scores[i] == scores[i] else math.inf, i))
    return sorted(list(range(lo)) + list(range(hi, n)) + order[:budget])


def _evict_case(dtype, d, hkv, lens, sinks, recent, budget, page, scores_of, seed=0, same_pool=False):
    rng, dt = np.random.default_rng(seed), DT[dtype]
    B, keep = len(lens), sinks + recent + budget
    where, rows, addr = _cache(lens, page, rng)
    outs = [min(n, keep) for n in lens]
    to, rows_out, addr_out = _cache(outs, page, rng)
    k, v = (torch.randn((rows, hkv, d), device="cuda").to(dt) for _ in range(2))
    scores = torch.from_numpy(np.stack([scores_of(rng, rows) for _ in range(hkv)]).astype(np.float32)).cuda()
    if same_pool:  # the destination pages behind the source's in one pool
        addr_out = torch.where(addr_out >= 0, addr_out + rows // page, addr_out)
        to, base = [w + rows for w in to], rows
        k, v = (torch.cat([x, torch.zeros((rows_out, hkv, d), device="cuda").to(dt)]) for x in (k, v))
        scores = torch.cat([scores, torch.zeros((hkv, rows_out), device="cuda")], 1).contiguous()
        rows += rows_out
        rows_out, ko, vo = rows, k, v
    else:
        ko, vo = (torch.full((rows_out, hkv, d), 9.0, device="cuda").to(dt) for _ in range(2))
    so = torch.full((hkv, rows_out), 9.0, device="cuda")
    dec = Decoder(B, hkv, hkv, d, rows, max(lens), 256, 1, dtype)
    k0, v0 = k.clone(), v.clone()
    dbg, word = _debug()
    args = (sinks, recent, budget, ko, vo, so, addr_out)
    if page:
        kept, lens_out = dec.evict_paged(k, v, scores, addr, _ints(lens), page, *args, debug=dbg)
    else:
        kept, lens_out = dec.evict(k, v, scores, addr, *args, debug=dbg)
    assert _flags(word) == 0 and lens_out.tolist() == outs
    sh, rest = scores.cpu().numpy(), torch.ones(rows_out, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        rest[to[b]] = False
        for h in range(hkv):
            want = _kept(sh[h, where[b].cpu().numpy()].tolist(), n, sinks, recent, budget)
            assert kept[b, h].tolist() == want + [-1] * (keep - len(want)), (b, h)
            src = where[b][torch.tensor(want, dtype=torch.int64, device="cuda")]
            assert torch.equal(ko[to[b], h], k0[src, h]) and torch.equal(vo[to[b], h], v0[src, h])
            assert torch.equal(so[h, to[b]].view(torch.int32), scores[h, src].view(torch.int32))
    if same_pool:
        assert torch.equal(ko[rest], k0[rest]) and torch.equal(vo[rest], v0[rest])
    else:
        assert (ko[rest] == 9.0).all() and (vo[rest] == 9.0).all()
    assert (so[:, rest] == 9.0).all()


def _spread(rng, n):
    return rng.random(n) ** 8


def _few(rng, n):
    return rng.integers(0, 3, n) / 4


def _signed(rng, n):
    x = rng.standard_normal(n) * 10.0 ** rng.integers(-30, 30, n)
    x[rng.random(n) < 0.05] = np.inf
    x[rng.random(n) < 0.05] = -np.inf
    x[rng.random(n) < 0.05] = 0.0
    x[rng.random(n) < 0.05] = -0.0
    return x


def _with_nan(rng, n):
    x = _signed(rng, n)
    x[rng.random(n) < 0.2] = np.nan
    return x


@pytest.mark.parametrize("scores_of", [_spread, _few, _signed, _with_nan])
@pytest.mark.parametrize("dtype,d,hkv,page", [("bf16", 128, 2, 0), ("bf16", 64, 3, 32), ("f32", 128, 1, 64), ("f32", 64, 2, 0)])
def test_evict(dtype, d, hkv, page, scores_of):
    for i, (lens, sinks, recent, budget) in enumerate([
            ([1], 4, 3, 2), ([0, 7, 40, 33], 4, 3, 2), ([100, 200, 31], 0, 0, 50), ([500, 64], 37, 1, 100), ([300], 0, 64, 0),
            ([300, 2], 5, 0, 0), ([2500, 9], 1, 100, 777), ([64] * 40, 3, 5, 7), ([90, 91], 0, 0, 1), ([0, 0], 1, 1, 1)]):
        _evict_case(dtype, d, hkv, lens, sinks, recent, budget, page, scores_of, seed=i)


@pytest.mark.parametrize("scores_of", [_spread, _few, _with_nan, lambda rng, n: np.full(n, 0.5)])
def test_evict_more_keys_than_are_held(scores_of):
    """Beyond what a CTA holds of the scores (40960) and lists of one bin (8192)."""
    _evict_case("bf16", 64, 1, [70001, 12], 4, 100, 5000, 32, scores_of, seed=1)
    _evict_case("bf16", 64, 1, [45000], 33, 0, 30000, 0, scores_of, seed=2)
    _evict_case("bf16", 64, 1, [20000], 1, 1, 12000, 0, scores_of, seed=3)


def test_evict_within_one_pool():
    _evict_case("bf16", 128, 2, [400, 100, 37], 4, 50, 30, 32, _spread, seed=4, same_pool=True)


def test_evict_of_nothing_kept():
    dec = Decoder(2, 1, 1, 64, 64, 32, 256, 1, "f32")
    k = torch.randn((64, 1, 64), device="cuda")
    out = torch.zeros((8, 1, 64), device="cuda"), torch.zeros((8, 1, 64), device="cuda")
    kept, lens = dec.evict(k, k.clone(), torch.rand((1, 64), device="cuda"), _ints([0, 32, 64], torch.int64), 0, 0, 0, *out,
                           None, _ints([0, 0, 0], torch.int64))
    assert lens.tolist() == [0, 0] and kept.shape == (2, 1, 0) and not out[0].any()


def test_evict_bad_device_data_is_flagged():
    lens, page = [100, 80], 32
    where, rows, table = _cache(lens, page, np.random.default_rng(6))
    k, v = torch.randn((rows, 1, 64), device="cuda"), torch.randn((rows, 1, 64), device="cuda")
    scores = torch.rand((1, rows), device="cuda")
    dec = Decoder(2, 1, 1, 64, rows, 100, 256, 1, "f32")
    dbg, word = _debug()
    ko, vo, so = torch.zeros((128, 1, 64), device="cuda"), torch.zeros((128, 1, 64), device="cuda"), torch.zeros((1, 128), device="cuda")
    run = lambda t, to, n: dec.evict_paged(k, v, scores, t, n, page, 2, 8, 30, ko, vo, so, to, debug=dbg)  # noqa: E731
    to = _ints([[0, 1], [2, 4]])  # page 4 of 4 does not exist: rows 32 .. 39 of sequence 1 are not written
    kept, n = run(table, to, _ints(lens))
    assert _flags(word) == sd.ERR_INDPTR and n.tolist() == [40, 40]
    assert torch.equal(ko[:40, 0], k[where[0][kept[0, 0].long()], 0]) and torch.equal(ko[64:96, 0], k[where[1][kept[1, 0, :32].long()], 0])
    assert not ko[96:].any() and not so[0, 96:].any()
    bad = table.clone()
    bad[0, 1] = 10**6  # a source page: its keys count as lowest, and a row that still comes from it is not written
    kept, n = run(bad, _ints([[0, 1], [2, 3]]), _ints(lens))
    assert _flags(word) == sd.ERR_INDPTR and not any(32 <= i < 64 for i in kept[0, 0].tolist())
    kept, n = run(table, _ints([[0, 1], [2, 3]]), _ints([-1, 200]))
    assert _flags(word) == sd.ERR_INDPTR and n.tolist() == [0, 0] and (kept == -1).all()
    ko.zero_()
    dec.evict_paged(k, v, scores, table, _ints(lens), page, 2, 8, 30, ko, vo, so, _ints([[0, 1], [2, 3]]))
    flat = Decoder(2, 1, 1, 64, rows, 100, 256, 1, "f32")
    ko.zero_()
    kept, n = flat.evict(k, v, scores, _ints([0, 90, 180], torch.int64), 2, 8, 30, ko, vo, so, _ints([0, 39, 500], torch.int64),
                         debug=dbg)  # no room for the first, beyond the cache for the second
    assert _flags(word) == sd.ERR_INDPTR and n.tolist() == [40, 40] and not ko.any()


# ------------------------------------------------------------------------------ together


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_a_run_of_them_together(dtype, d):
    """Requests over one prompt with images: the prompt's and the steps' tokens are rotated by three axes into the
    pages, attended behind the shared prefix, their keys' weights gathered; then each sequence is cut into pages of
    its own, and decoding goes on over what was kept.  Every step against 64 bits on raw tokens."""
    B, hq, hkv, page, prefix, steps = 3, 8, 2, 32, 96, 40
    dt, u = DT[dtype], 2.0 ** -23
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    num_pages, width = 40, 8
    dec = Decoder(B, hq, hkv, d, num_pages * page, width * page, 256, 1, dtype)
    kp, vp = (torch.full((num_pages * page, hkv, d), math.nan, device="cuda").to(dt) for _ in range(2))
    cs, axis = rope_table(512, d), rope_turns(d // 2, 3)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, :prefix // page] = _ints([5, 6, 7])
    free = _ints([i for i in range(num_pages) if i not in (5, 6, 7)])
    # the prompt: a text, a 6 x 10 image, a text
    t = torch.arange(prefix, device="cuda")
    image = (t >= 20) & (t < 80)
    pos = torch.stack([torch.where(image, 20, t), torch.where(image, 20 + (t - 20) // 10, t),
                       torch.where(image, 20 + (t - 20) % 10, t)]).to(torch.int32)
    k, v = rnd(prefix, hkv, d), rnd(prefix, hkv, d)
    rows = torch.cat([torch.arange(32, device="cuda") + 32 * p for p in (5, 6, 7)])
    dec.norm_rope_axes(None, k, v, pos, axis, rows, cs, kp, vp)
    want, _ = _rope_reference(k, None, 0.0, _axes_table(cs, pos, axis), d, False)
    hist = [[(kp[rows, h].double(), v[:, h].double()) for h in range(hkv)] for _ in range(B)]
    assert float((kp[rows].double() - want).abs().max()) < 0.1
    lens = _ints([prefix] * B)
    scores = torch.zeros((hkv, num_pages * page), device="cuda")
    slots, positions = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    lens_out, counts = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    shared = True
    scale = 1 / math.sqrt(d)
    for step in range(steps):
        dec.page_plan(lens, _ints([1] * B), table, free, page, slots, positions, lens_out, counts)
        free = free[int(counts[0]):].contiguous()
        q, k, v = rnd(B, hq, d), rnd(B, hkv, d), rnd(B, hkv, d)
        at = torch.full((3, B), 100 + step, dtype=torch.int32, device="cuda")
        qr = dec.norm_rope_axes(q, k, v, at, axis, slots, cs, kp, vp)
        lens = lens_out.clone()
        if shared:
            out = dec.shared_paged(qr, kp, vp, table, lens, page, prefix)
        else:
            out = dec.window_paged(qr, kp, vp, table, lens, page, 0)
        for b in range(B):
            for h in range(hkv):
                kk, vv = hist[b][h]
                kk, vv = torch.cat([kk, kp[slots[b], h].double()[None]]), torch.cat([vv, v[b, h].double()[None]])
                hist[b][h] = kk, vv
                heads = slice(h * 4, h * 4 + 4)
                want, tol = _attention_reference(qr[b, heads].double(), kk, vv, scale, u)
                assert ((out[b, heads].double() - want).abs() <= tol).all(), (step, b, h)
        # each sequence is cut into pages of its own; the prefix's rows belong to all, so one query's weights decide
        if step == 19:
            fresh = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
            own_scores = dec.key_weights_paged(qr[:1].expand(B, hq, d).contiguous(), kp, table, lens, page,
                                               torch.zeros_like(scores))
            keep = (4, 16, 40)
            need = -(-sum(keep) // page) + 1
            for b in range(B):
                fresh[b, :need] = free[b * need:(b + 1) * need]
            free = free[B * need:].contiguous()
            kept, cut = dec.evict_paged(kp, vp, own_scores, table, lens, page, *keep, kp, vp, scores, fresh)
            assert cut.tolist() == [60] * B
            for b in range(B):
                for h in range(hkv):
                    kk, vv = hist[b][h]
                    rows = torch.tensor([int(table[b, i // page]) * page + i % page for i in range(len(kk))], device="cuda")
                    want = _kept(own_scores[h, rows].tolist(), len(kk), *keep)
                    assert kept[b, h].tolist() == want
                    i = torch.tensor(want, device="cuda")
                    hist[b][h] = kk[i], vv[i]
            # (page_plan counts tokens by pages held; a page less than planned stays with the table)
            table, lens, shared = fresh, cut, False
            for b in range(B):
                held = -(-60 // page)
                free = torch.cat([free, table[b, held:need]]).contiguous()
                table[b, held:] = -1


def _readme_block(call):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    return next(b for b in re.findall(r"```python\n(.*?)```", text, re.S) if call in b)


def test_readme_steps_as_written():
    """README's shared step and its eviction, run as they stand there."""
    B, hq, hkv, d, page_size, prefix_len = 2, 8, 2, 128, 64, 128
    lens, num_pages, width = [1900, 1500], 96, 40
    gen = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    ids = torch.randperm(num_pages, generator=gen, device="cuda").tolist()
    shared, at, table = ids[:2], 2, []
    for n in lens:
        own = -(-n // page_size) - 2
        table.append(shared + ids[at:at + own] + [-1] * (width - 2 - own))
        at += own
    pages_to = [ids[at:at + 21], ids[at + 21:at + 42]]
    where = [torch.tensor([table[b][i // page_size] * page_size + i % page_size for i in range(n)], device="cuda")
             for b, n in enumerate(lens)]
    names = dict(dec=Decoder(B, hq, hkv, d, num_pages * page_size, width * page_size, 256, 1, "bf16"), q=rnd(B, hq, d),
                 k=rnd(B, hkv, d), v=rnd(B, hkv, d), positions3=_ints([[7, 9], [7, 3], [7, 5]]),
                 slot_map=torch.stack([w[-1] for w in where]), cos_sin=rope_table(64, d), k_pool=rnd(num_pages * page_size, hkv, d),
                 v_pool=rnd(num_pages * page_size, hkv, d), page_table=_ints(table), lens_out=_ints(lens), page_size=page_size,
                 prefix_len=prefix_len, rope_sections=rope_sections, scores=torch.zeros((hkv, num_pages * page_size), device="cuda"),
                 scores_to=torch.zeros((hkv, num_pages * page_size), device="cuda"), pages_to=_ints(pages_to))
    raw = {n: names[n].clone() for n in "qkv"}
    exec(_readme_block("shared_paged"), names)
    rows = _axes_table(names["cos_sin"], names["positions3"], rope_sections((16, 24, 24)))
    _close(names["q"], *_rope_reference(raw["q"], None, 0.0, rows, d, False), "q")
    for b, w in enumerate(where):
        for h in range(hkv):
            heads = slice(4 * h, 4 * h + 4)
            want, tol = _attention_reference(names["q"][b, heads].double(), names["k_pool"][w, h].double(),
                                             names["v_pool"][w, h].double(), 1 / math.sqrt(d), 2.0 ** -23)
            assert ((names["out"][b, heads].double() - want).abs() <= tol).all()
    k0, v0 = names["k_pool"].clone(), names["v_pool"].clone()
    exec(_readme_block("evict_paged"), names)
    assert names["lens"].tolist() == [1284, 1284]
    for b, w in enumerate(where):
        to = torch.tensor([pages_to[b][i // page_size] * page_size + i % page_size for i in range(1284)], device="cuda")
        for h in range(hkv):
            want = _kept(names["scores"][h, w].tolist(), lens[b], 4, 256, 1024)
            assert names["kept"][b, h].tolist() == want
            src = w[torch.tensor(want, device="cuda")]
            assert torch.equal(names["k_pool"][to, h], k0[src, h]) and torch.equal(names["v_pool"][to, h], v0[src, h])
            assert torch.equal(names["scores_to"][h, to], names["scores"][h, src])
