"""Refusals of rotation by several axes, shared prefixes, key weights and eviction, on the host: no call here reaches a
kernel launch."""

import copy
import ctypes

import pytest
import torch

A = 1 << 20  # an aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def sd():
    from stochastic_sparse_decode_gb300.build import build

    build()
    import stochastic_sparse_decode_gb300 as sd

    return sd


def _problem(sd, **kw):
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, total_tokens=4096, max_len=2048, tile=256, S=1,
             dtype="bf16")
    a.update(kw)
    return sd.make_problem(**a)


PAGES = dict(page_table=A, kv_lens=A, page_size=32, max_pages=64, num_pages=128)
BAD_PAGES = (dict(page_size=0), dict(page_size=48), dict(max_pages=0), dict(max_pages=63), dict(num_pages=127),
             dict(page_table=None), dict(kv_lens=None), dict(page_table=A + 2))


def _pages(sd, **kw):
    return sd.Pages(*{**PAGES, **kw}.values())


def _axes(sd, axes=3, stride=4, ids=(0, 1, 2), p=None, none=False, rot=128, **kw):
    st = sd.Axes(axes, stride, (ctypes.c_ubyte * 64)(*(list(ids) * 32)[:64]))
    a = dict(n=4, q=2 * A, qs=1024, k=3 * A, ks=256, v=4 * A, vs=256, positions=5 * A, slot_map=6 * A, q_out=7 * A,
             k_cache=8 * A, v_cache=9 * A)
    a.update(kw)
    return sd.lib().santa_norm_rope_axes(ctypes.byref(p or _problem(sd)), ctypes.byref(sd.Rope(None, None, 1e-6, A, 100, rot, 0)),
                                         None if none else ctypes.byref(st), *a.values(), None, None)


def test_norm_rope_axes_refuses(sd):
    for bad in (dict(axes=0), dict(axes=5), dict(axes=2), dict(stride=3), dict(stride=1 << 31), dict(none=True), dict(n=-1),
                dict(positions=None), dict(ks=248), dict(q_out=None), dict(k_cache=8 * A + 8), dict(rot=0)):
        assert _axes(sd, **bad) == sd.INVALID_ARG, bad
    assert _axes(sd, rot=24) == sd.UNSUPPORTED
    assert _axes(sd, n=0, stride=0) == sd.OK
    # axes of pairs behind the last one that turns are not looked at
    assert _axes(sd, axes=1, ids=[0] * 8 + [9] * 56, rot=16, n=0) == sd.OK
    assert _axes(sd, axes=1, ids=[0] * 8 + [9] * 56, rot=32, n=0) == sd.INVALID_ARG


def _shared(sd, p=None, prefix=(100, 0), pages=None, none=False, **kw):
    p = p or _problem(sd)
    a = dict(q=A, k=2 * A, v=3 * A, kv_indptr=4 * A, out=5 * A, ws=6 * A, ws_bytes=sd.shared_workspace_size(_problem(sd)))
    a.update(kw)
    return sd.lib().santa_decode_shared(ctypes.byref(p), None if none else ctypes.byref(sd.Prefix(*prefix)),
                                        None if pages is None else ctypes.byref(pages), *a.values(), None, None)


def test_shared_refuses(sd):
    for bad in (dict(none=True), dict(prefix=(-1, 0)), dict(prefix=(100, -1)), dict(prefix=(100, 3997)), dict(prefix=(4097, 0)),
                dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(kv_indptr=None), dict(ws=None), dict(q=A + 8),
                dict(k=2 * A + 8), dict(v=3 * A + 8), dict(out=5 * A + 4), dict(kv_indptr=4 * A + 4), dict(ws=6 * A + 16),
                dict(p=_problem(sd, num_q_heads=7)), dict(p=_problem(sd, batch=-1)), dict(p=_problem(sd, max_len=-1)),
                dict(prefix=(2049, 0), pages=_pages(sd))):
        assert _shared(sd, **bad) == sd.INVALID_ARG, bad
    for bad in BAD_PAGES:
        assert _shared(sd, pages=_pages(sd, **bad)) == sd.INVALID_ARG, bad
    assert _shared(sd, ws_bytes=sd.shared_workspace_size(_problem(sd)) - 1) == sd.WORKSPACE_TOO_SMALL
    assert _shared(sd, p=_problem(sd, head_dim=32)) == sd.UNSUPPORTED
    assert _shared(sd, p=_problem(sd, num_q_heads=18)) == sd.UNSUPPORTED
    assert _shared(sd, p=_problem(sd, batch=0)) == sd.OK
    # the own keys' counters come first: what santa_split_workspace_init prepares
    assert sd.shared_workspace_size(_problem(sd)) > sd.split_workspace_size(_problem(sd))


def _weights(sd, p=None, pages=None, **kw):
    p = p or _problem(sd)
    a = dict(q=A, k=2 * A, kv_indptr=3 * A, scores=4 * A, scores_out=5 * A, decay=1.0, fresh=1, ws=6 * A,
             ws_bytes=sd.workspace_size(_problem(sd), sd.MODE_PROP))
    a.update(kw)
    return sd.lib().santa_key_weights(ctypes.byref(p), None if pages is None else ctypes.byref(pages), *a.values(), None, None)


def test_key_weights_refuses(sd):
    for bad in (dict(q=None), dict(k=None), dict(kv_indptr=None), dict(scores_out=None), dict(ws=None), dict(decay=-0.5),
                dict(decay=float("nan")), dict(decay=float("inf")), dict(fresh=-1), dict(q=A + 8), dict(k=2 * A + 8),
                dict(kv_indptr=3 * A + 4), dict(scores=4 * A + 2), dict(scores_out=5 * A + 2), dict(ws=6 * A + 16),
                dict(q=None, k=None, pages=_pages(sd)), dict(p=_problem(sd, batch=-1))):
        assert _weights(sd, **bad) == sd.INVALID_ARG, bad
    for bad in BAD_PAGES:
        assert _weights(sd, pages=_pages(sd, **bad)) == sd.INVALID_ARG, bad
    assert _weights(sd, ws_bytes=1000) == sd.WORKSPACE_TOO_SMALL
    assert _weights(sd, p=_problem(sd, num_q_heads=6)) == sd.UNSUPPORTED  # 3 query heads per KV head
    assert _weights(sd, p=_problem(sd, max_len=(1 << 22) + 1)) == sd.UNSUPPORTED
    for nothing in (dict(batch=0), dict(max_len=0), dict(total_tokens=0)):
        assert _weights(sd, p=_problem(sd, **nothing)) == sd.OK


def _evict(sd, p=None, keep=(4, 8, 100), pages=None, pages_out=None, none=False, **kw):
    a = dict(k=A, v=2 * A, scores=3 * A, kv_indptr=4 * A, k_out=5 * A, v_out=6 * A, scores_out=7 * A, rows_out=512,
             indptr_out=8 * A)
    b = dict(kept=9 * A, lens_out=10 * A)
    for d in (a, b):
        d.update({x: kw.pop(x) for x in list(kw) if x in d})
    assert not kw
    return sd.lib().santa_evict(ctypes.byref(p or _problem(sd)), None if none else ctypes.byref(sd.Keep(*keep)),
                                None if pages is None else ctypes.byref(pages), *a.values(),
                                None if pages_out is None else ctypes.byref(pages_out), *b.values(), None, None)


def test_evict_refuses(sd):
    out = sd.Pages(A, None, 32, 4, 16)  # its lengths are not used
    for bad in (dict(none=True), dict(keep=(-1, 0, 0)), dict(keep=(0, -1, 0)), dict(keep=(0, 0, -1)),
                dict(keep=(2**31 - 1, 2**31 - 1, 2**31 - 1)), dict(k=None), dict(v=None), dict(scores=None),
                dict(kv_indptr=None), dict(k_out=None), dict(v_out=None), dict(indptr_out=None), dict(kept=None),
                dict(lens_out=None), dict(rows_out=-1), dict(k_out=6 * A), dict(k_out=2 * A), dict(v_out=A),
                dict(scores_out=3 * A), dict(k=A + 8), dict(v_out=6 * A + 8), dict(scores=3 * A + 2), dict(kept=9 * A + 2),
                dict(lens_out=10 * A + 1), dict(indptr_out=8 * A + 4), dict(p=_problem(sd, batch=-1)),
                dict(pages_out=sd.Pages(A, None, 32, 4, 15)), dict(pages_out=sd.Pages(A, None, 32, 3, 16)),
                dict(pages_out=sd.Pages(None, None, 32, 4, 16)), dict(pages_out=sd.Pages(A, None, 48, 4, 16))):
        assert _evict(sd, **bad) == sd.INVALID_ARG, bad
    for bad in BAD_PAGES:
        assert _evict(sd, pages=_pages(sd, **bad), pages_out=out) == sd.INVALID_ARG, bad
    assert _evict(sd, pages=_pages(sd, kv_lens=10 * A), pages_out=out) == sd.INVALID_ARG  # lengths in place
    assert _evict(sd, p=_problem(sd, head_dim=96)) == sd.UNSUPPORTED
    assert _evict(sd, p=_problem(sd, batch=0), pages_out=out) == sd.OK


def test_decoder_refuses_what_the_calls_would_misread(sd):
    """Nothing lies on a CUDA device here: every call raises before the library is entered."""
    from stochastic_sparse_decode_gb300.decoder import Decoder, rope_sections, rope_table_axes, rope_turns

    dec = Decoder(2, 8, 2, 128, 256, 128, 256, 1, "f32", device="cpu")
    dec = copy.deepcopy(dec)
    q, k = torch.zeros(2, 8, 128), torch.zeros(256, 2, 128)
    indptr, scores = torch.zeros(3, dtype=torch.int64), torch.zeros(2, 256)
    table, lens = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    out, out_at = torch.zeros(64, 2, 128), torch.zeros(3, dtype=torch.int64)
    pos = torch.zeros((3, 2), dtype=torch.int32)
    cs = torch.zeros(10, 128)
    calls = [
        lambda: dec.shared(q, k, k.clone(), indptr, 0, -1), lambda: dec.shared(q, k, k.clone(), indptr, -1, 5),
        lambda: dec.shared(q[:1], k, k.clone(), indptr, 0, 5), lambda: dec.shared(q, k[:, :1], k.clone(), indptr, 0, 5),
        lambda: dec.shared(q, k, k.clone(), indptr[:2], 0, 5), lambda: dec.shared_paged(q, k, k.clone(), table, lens, 60, 5),
        lambda: dec.shared_paged(q, k, k.clone(), table.long(), lens, 64, 5),
        lambda: dec.key_weights(q, None, indptr, scores), lambda: dec.key_weights(q, k, indptr, scores[:1]),
        lambda: dec.key_weights(q, k, indptr, scores, fresh=-1), lambda: dec.key_weights(None, None, indptr, scores),
        lambda: dec.key_weights_paged(None, None, table, lens, 64, scores),
        lambda: dec.evict(k, k.clone(), scores, indptr, -1, 0, 4, out, out.clone(), None, out_at),
        lambda: dec.evict(k, k.clone(), scores, indptr, 1, 0, 4, out, out[:32].clone(), None, out_at),
        lambda: dec.evict(k, k.clone(), scores, indptr, 1, 0, 4, out, out.clone(), torch.zeros(2, 63), out_at),
        lambda: dec.evict(k, k.clone(), scores, indptr, 1, 0, 4, out, out.clone(), None, out_at, kept=torch.zeros(2, 2, 4)),
        lambda: dec.evict_paged(k, k.clone(), scores, table, lens, 64, 1, 0, 4, out[:40], out[:40].clone(), None, table),
        lambda: dec.norm_rope_axes(q, None, None, pos, [0, 1, 3] * 21 + [0], None, cs, None, None),
        lambda: dec.norm_rope_axes(q, None, None, pos, [0] * 32, None, cs, None, None),
        lambda: dec.norm_rope_axes(q, None, None, pos.T, [0] * 64, None, cs, None, None),
        lambda: dec.norm_rope_axes(q, None, None, pos[0], [0] * 64, None, cs, None, None),
        # and, all in order but for the device
        lambda: dec.norm_rope_axes(q, None, None, pos, [0, 1, 2, 0] * 16, None, cs, None, None),
        lambda: dec.evict(k, k.clone(), scores, indptr, 1, 0, 4, out, out.clone(), None, out_at),
    ]
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, sd.SantaError)):
            call()
            pytest.fail(f"call {i} was let through")
    assert rope_sections((2, 0, 3)) == (0, 0, 2, 2, 2) and rope_turns(5, 3) == (0, 1, 2, 0, 1)
    t = rope_table_axes(4, (2, 3), 100.0, device="cpu").double()
    freq = torch.tensor([1.0, 0.1, 1.0, 100 ** (-1 / 3), 100 ** (-2 / 3)], dtype=torch.float64)
    assert torch.allclose(t[3], torch.cat([(3 * freq).cos(), (3 * freq).sin()]), atol=1e-7)
