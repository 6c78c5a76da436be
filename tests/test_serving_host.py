"""Refusals of the operators around the attention, on the host: no call here reaches a kernel launch."""

import ctypes
import os
import re

import pytest
import torch


@pytest.fixture(scope="module")
def sd():
    from stochastic_sparse_decode_gb300.build import build

    build()
    import stochastic_sparse_decode_gb300 as sd

    return sd


A = 1 << 20  # an aligned address that is never dereferenced on the host


def _problem(sd, **kw):
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, total_tokens=4096, max_len=2048, tile=256, S=1,
             dtype="bf16")
    a.update(kw)
    return sd.make_problem(**a)


def _plan(sd, **kw):
    a = dict(batch=3, page_size=32, max_pages=8, num_pages=64, kv_lens=A, new_lens=2 * A, page_table=3 * A,
             free_pages=4 * A, num_free=10, slot_map=5 * A, positions=6 * A, max_tokens=100, lens_out=7 * A,
             counts=8 * A)
    a.update(kw)
    return sd.lib().santa_page_plan(*a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(page_size=0), dict(max_pages=0), dict(num_pages=-1), dict(num_free=-1), dict(max_tokens=-1),
    dict(kv_lens=None), dict(new_lens=None), dict(page_table=None), dict(free_pages=None), dict(slot_map=None),
    dict(positions=None), dict(lens_out=None), dict(counts=None), dict(lens_out=A), dict(lens_out=2 * A),
    dict(slot_map=5 * A + 8), dict(positions=6 * A + 4), dict(kv_lens=A + 2), dict(num_pages=1 << 27),
    dict(max_pages=1 << 27),
])
def test_page_plan_refuses(sd, bad):
    assert _plan(sd, **bad) == sd.INVALID_ARG


def _rope(sd, p=None, r=None, **kw):
    rope = dict(q_weight=None, k_weight=None, eps=1e-6, cos_sin=A, max_pos=100, rot_dim=128, interleaved=0)
    rope.update(r or {})
    a = dict(n=4, q=2 * A, qs=1024, k=3 * A, ks=256, v=4 * A, vs=256, positions=5 * A, slot_map=6 * A, q_out=7 * A,
             k_cache=8 * A, v_cache=9 * A)
    a.update(kw)
    return sd.lib().santa_norm_rope(ctypes.byref(p or _problem(sd)), ctypes.byref(sd.Rope(*rope.values())),
                                    *a.values(), None, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(q=None), dict(q_out=None), dict(k=None), dict(k_cache=None), dict(v=None), dict(v_cache=None),
    dict(positions=None), dict(qs=1023), dict(qs=1028), dict(ks=248), dict(vs=260), dict(q=2 * A + 8),
    dict(k_cache=8 * A + 8), dict(q_out=2 * A, qs=2048), dict(k_cache=3 * A), dict(v_cache=4 * A), dict(v_cache=8 * A),
    dict(slot_map=6 * A + 4),
    dict(r=dict(rot_dim=0)), dict(r=dict(rot_dim=144)), dict(r=dict(max_pos=0)), dict(r=dict(eps=-1.0)),
    dict(r=dict(eps=float("nan"))), dict(r=dict(cos_sin=None)), dict(r=dict(q_weight=A + 2)),
])
def test_norm_rope_refuses(sd, bad):
    assert _rope(sd, **bad) == sd.INVALID_ARG


def test_norm_rope_unsupported_and_nothing_to_do(sd):
    assert _rope(sd, r=dict(rot_dim=24)) == sd.UNSUPPORTED
    assert _rope(sd, p=_problem(sd, head_dim=96)) == sd.UNSUPPORTED
    assert _rope(sd, n=0) == sd.OK
    assert _rope(sd, q=None, q_out=None, k=None, k_cache=None, v=None, v_cache=None) == sd.OK


def _attend(sd, name, p=None, window=(100, 4), pages=None, **kw):
    p = p or _problem(sd)
    n = sd.split_workspace_size(_problem(sd))
    a = dict(q=A, k=2 * A, v=3 * A, kv_indptr=4 * A, out=5 * A, ws=6 * A, ws_bytes=n)
    if name == "santa_decode_kv4":
        a = dict(q=A, kv4=2 * A, kv_indptr=4 * A, out=5 * A, ws=6 * A, ws_bytes=n)
    a.update(kw)
    w = None if window is None else ctypes.byref(sd.Window(*window))
    return getattr(sd.lib(), name)(ctypes.byref(p), w, None if pages is None else ctypes.byref(pages), *a.values(),
                                   None, None)


@pytest.mark.parametrize("name", ["santa_decode_window", "santa_decode_kv4"])
def test_attention_refuses(sd, name):
    f = lambda **kw: _attend(sd, name, **kw)  # noqa: E731
    for bad in (dict(window=(-1, 0)), dict(window=(5, -1)), dict(q=None), dict(out=None), dict(kv_indptr=None),
                dict(ws=None), dict(q=A + 8), dict(out=5 * A + 4), dict(kv_indptr=4 * A + 4), dict(ws=6 * A + 16),
                dict(p=_problem(sd, num_q_heads=7)), dict(p=_problem(sd, batch=-1)), dict(p=_problem(sd, max_len=-1)),
                dict(p=_problem(sd, batch=65536)), dict(p=_problem(sd, total_tokens=1 << 31))):
        assert f(**bad) == sd.INVALID_ARG, bad
    assert f(ws_bytes=100) == sd.WORKSPACE_TOO_SMALL
    assert f(p=_problem(sd, head_dim=32)) == sd.UNSUPPORTED
    assert f(p=_problem(sd, num_q_heads=18)) == sd.UNSUPPORTED  # 9 query heads per KV head
    huge = dict(batch=65535, num_q_heads=8, num_kv_heads=8, max_len=2**31 - 1)
    assert f(p=_problem(sd, **huge)) == sd.UNSUPPORTED  # more blocks than a warp counts
    assert f(p=_problem(sd, batch=0)) == sd.OK
    if name == "santa_decode_window":
        assert f(window=None) == sd.INVALID_ARG
        for bad in (dict(k=None), dict(v=None), dict(k=2 * A + 8), dict(v=3 * A + 8)):
            assert f(**bad) == sd.INVALID_ARG, bad
    else:
        assert f(kv4=None) == sd.INVALID_ARG
        assert f(kv4=2 * A + 8) == sd.INVALID_ARG
    good = dict(page_table=A, kv_lens=A, page_size=32, max_pages=64, num_pages=128)
    for bad in (dict(page_size=0), dict(page_size=48), dict(max_pages=0), dict(max_pages=63), dict(num_pages=127),
                dict(page_table=None), dict(kv_lens=None), dict(page_table=A + 2)):
        assert f(pages=sd.Pages(*{**good, **bad}.values())) == sd.INVALID_ARG, bad


def _store(sd, name, p=None, **kw):
    if name == "santa_kv4_append":
        a = dict(n=4, k=A, ks=256, v=2 * A, vs=256, slot_map=3 * A, kv4=4 * A)
    else:
        a = dict(n=4, kv4=4 * A, slot_map=3 * A, k=A, v=2 * A)
    a.update(kw)
    return getattr(sd.lib(), name)(ctypes.byref(p or _problem(sd)), *a.values(), None, None)


def test_kv4_store_refuses(sd):
    for bad in (dict(n=-1), dict(k=None), dict(v=None), dict(kv4=None), dict(kv4=4 * A + 8), dict(ks=255), dict(vs=252),
                dict(k=A + 8), dict(slot_map=3 * A + 4)):
        assert _store(sd, "santa_kv4_append", **bad) == sd.INVALID_ARG, bad
    for bad in (dict(n=-1), dict(kv4=None), dict(kv4=4 * A + 8), dict(k=A + 8), dict(v=A), dict(k=4 * A),
                dict(slot_map=3 * A + 4)):
        assert _store(sd, "santa_kv4_read", **bad) == sd.INVALID_ARG, bad
    for name in ("santa_kv4_append", "santa_kv4_read"):
        assert _store(sd, name, n=0) == sd.OK
        assert _store(sd, name, p=_problem(sd, head_dim=256)) == sd.UNSUPPORTED
    assert _store(sd, "santa_kv4_read", k=None, v=None) == sd.OK
    assert sd.kv4_size(_problem(sd)) == 4096 * 2 * 144
    assert sd.kv4_size(_problem(sd, head_dim=64)) == 4096 * 2 * 72


def test_split_workspace(sd):
    small, large = (sd.split_workspace_size(_problem(sd, batch=b)) for b in (1, 1000))
    assert small % 256 == 0 and large > small
    n = ctypes.c_size_t(0)
    assert sd.lib().santa_split_workspace_size(ctypes.byref(_problem(sd)), None) == sd.INVALID_ARG
    assert sd.lib().santa_split_workspace_size(ctypes.byref(_problem(sd, num_q_heads=9)), ctypes.byref(n)) == sd.INVALID_ARG
    init = sd.lib().santa_split_workspace_init
    assert init(ctypes.byref(_problem(sd)), None, 1 << 30, None) == sd.INVALID_ARG
    assert init(ctypes.byref(_problem(sd)), A + 8, 1 << 30, None) == sd.INVALID_ARG
    assert init(ctypes.byref(_problem(sd)), A, small - 1, None) == sd.WORKSPACE_TOO_SMALL


def test_decoder_refuses_tensors_the_call_would_misread(sd):
    """On the CPU every tensor is refused: none lies on a CUDA device, and shape and dtype come first."""
    from stochastic_sparse_decode_gb300.decoder import Decoder

    dec = Decoder(2, 8, 2, 128, 4096, 2048, 256, 1, "bf16", device="cpu")
    bf = torch.bfloat16
    q, k = torch.zeros(2, 8, 128, dtype=bf), torch.zeros(4096, 2, 128, dtype=bf)
    out = torch.zeros(2, 8, 128)
    ind = torch.zeros(3, dtype=torch.int64)
    for args, what in (((q.float(), k, k, ind), "out|q:"), ((q, k[:100], k, ind), "k|out"), ((q, k, k, ind.int()), "out|ind")):
        with pytest.raises(ValueError, match=what):
            dec.window(*args, 100, out=out)
    with pytest.raises(ValueError, match="slot_map|k:"):
        dec.kv4_append(k[:4], k[:4], torch.zeros(4, dtype=torch.int32), torch.zeros(1))
    with pytest.raises(ValueError):
        dec.page_plan(ind.int(), ind.int(), ind.int()[None], ind.int(), 33, ind, ind.int(), ind.int(), ind.int()[:2])


def test_kernels_launched_early_read_nothing_by_the_read_only_path():
    """A kernel launched with programmatic dependent launch may start while page plan, norm + rotation or the 4-bit
    read (which let their successor start at once) still write its page table, queries or caches; the read-only
    path is for memory that no one writes while the kernel lives.  The files of such kernels: the streaming pass
    and the fused sampler of prop, and the serving operators."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "stochastic_sparse_decode_gb300",
                        "csrc")
    files = [os.path.join(csrc, f) for f in ("santa_stream.cuh", "santa_sampler.cuh")]
    files += [os.path.join(csrc, "serving", f) for f in sorted(os.listdir(os.path.join(csrc, "serving")))]
    bad = re.compile(r"__ldg\s*\(|ld\.global\.nc|ld\.global\.\w+\.nc|__restrict__")
    for f in files:
        assert not bad.search(re.sub(r"//[^\n]*", "", open(f).read())), f
    common = open(os.path.join(csrc, "santa_common.cuh")).read()
    body = re.search(r"long long key_row\(.*?\n}\n", common, re.S).group(0)  # pass 1's page lookup
    assert not bad.search(body)


def test_norm_rope_of_no_token(sd):
    """A step without a token: empty tensors have no address, the caches do."""
    assert _rope(sd, n=0, q=None, k=None, v=None) == sd.OK
    assert _rope(sd, n=0, q=None, q_out=None, k=None, v=None, positions=None, slot_map=None) == sd.OK
    assert _rope(sd, n=0, r=dict(rot_dim=0)) == sd.INVALID_ARG


def test_kv4_of_nothing_needs_no_cache(sd):
    """As the windowed call: no sequence, or no key, and the cache's address is not asked for (an empty tensor has
    none).  With keys it is."""
    none = _problem(sd, batch=0)
    assert _attend(sd, "santa_decode_window", p=none, k=None, v=None) == sd.OK
    assert _attend(sd, "santa_decode_kv4", p=none, kv4=None) == sd.OK
    assert _attend(sd, "santa_decode_kv4", kv4=None) == sd.INVALID_ARG
    for empty in (dict(total_tokens=0), dict(max_len=0)):  # refused before anything is enqueued, with the cache or not
        assert _attend(sd, "santa_decode_kv4", p=_problem(sd, **empty), kv4=None, ws_bytes=0) == sd.WORKSPACE_TOO_SMALL
        assert _attend(sd, "santa_decode_window", p=_problem(sd, **empty), k=None, v=None, ws_bytes=0) == sd.WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_decoder_can_be_copied_and_pickled(sd, how):
    """A Decoder holds a problem and tensors, and goes where those go (to a worker process, into a checkpoint); the
    copy's calls use the copy's problem."""
    import copy
    import pickle

    from stochastic_sparse_decode_gb300.decoder import Decoder

    dec = Decoder(2, 8, 2, 128, 4096, 2048, 256, 1, "bf16", device="cpu")
    dec.workspace("prop")[0] = 7
    dec._window(5, 1)
    twin = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda x: pickle.loads(pickle.dumps(x))}[how](dec)
    assert all(getattr(twin.problem, f) == getattr(dec.problem, f) for f, _ in dec.problem._fields_)
    assert twin.device == dec.device and int(twin.workspace("prop")[0]) == 7
    assert twin._pref._obj is twin.problem and twin._kv4_shape == dec._kv4_shape
    with pytest.raises(ValueError):  # checked and refused as by the original: nothing lies on a CUDA device
        twin.kv4_append(torch.zeros(4, 2, 128), torch.zeros(4, 2, 128), None, twin.kv4_cache())


def test_profiles_were_taken_on_these_sources(tmp_path, monkeypatch):
    """Every summary under profiles/ states the digest of the kernel sources that it describes, and the digest changes
    with any of their files."""
    import shutil
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, root)
    import bench

    serving = ("kv4_", "window_", "page_plan")
    for f in sorted(os.listdir(os.path.join(root, "profiles"))):
        text = open(os.path.join(root, "profiles", f)).read()
        stated = re.search(r"- source_digest: `([0-9a-f]{16})`", text).group(1)
        assert stated == bench.source_digest(serving=f.startswith(serving)), f
    csrc = os.path.join("stochastic_sparse_decode_gb300", "csrc")
    shutil.copytree(os.path.join(root, csrc), tmp_path / csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = {k: bench.source_digest(serving=k) for k in (False, True)}
    for name, changes in (("serving/santa_split.cuh", {True}), ("serving/santa_kv4_attn.cu", {True}),
                          ("serving/santa_serving.h", {True}), ("santa_launch.h", {True}),
                          ("santa_common.cuh", {False, True}), ("santa_prop.cu", {False})):
        path = tmp_path / csrc / name
        old = path.read_bytes()
        path.write_bytes(old + b"\n")
        assert {k for k in before if bench.source_digest(serving=k) != before[k]} == changes, name
        path.write_bytes(old)
