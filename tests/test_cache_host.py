"""Host-side refusals of the cache's operations and of the tree and page-selecting
decode (no GPU needed): bad shapes, parameters, pointers and workspaces are
turned down before the CUDA runtime is touched.  And the host model that the
GPU tests compare with, on cases worked out by hand."""
import ctypes

import numpy as np
import pytest

import serving_ref as R
from polar_attention_b200 import native as N

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x100000                   # 16-byte aligned, never dereferenced
MIS = 0x100008                 # 8 mod 16
MIS4 = 0x100002                # 2 mod 4
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(N.LIB_PATH):
        from polar_attention_b200 import build
        build.build()
    return N.lib()


def params(**kw):
    p = N.make_params(Hq=8, Hkv=2)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def tree(lib, p=None, q=A, k=A, v=A, mask=A, lens=None, tree=4, kv=A, pages=10, pt=A, mp=4, sl=A,
         n=2, u=A, out=A, neff=None, ws=A, wb=BIG):
    return lib.polar_attn_decode_paged_tree(q, k, v, mask, lens, tree, kv, pages, pt, mp, sl, n, u,
                                            ctypes.byref(p or params()), out, neff, ws, wb, None)


def sparse(lib, p=None, q=A, kv=A, b=A, pages=10, pt=A, mp=4, sl=A, n=2, keep=2, u=A, out=A,
           neff=None, sel=None, ws=A, wb=BIG):
    return lib.polar_attn_decode_paged_sparse(q, kv, b, pages, pt, mp, sl, n, keep, u,
                                              ctypes.byref(p or params()), out, neff, sel, ws, wb,
                                              None)


@pytest.mark.parametrize("call", [tree, sparse])
@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 32, UNSUPPORTED), ("Hkv", 3, INVALID), ("dtype", 1, UNSUPPORTED),
    ("dtype", 5, INVALID), ("logit_scale", -1.0, INVALID), ("alpha", float("inf"), INVALID),
    ("beta", float("nan"), INVALID), ("L_train", 1, INVALID), ("window", -1, INVALID),
    ("window", 64, UNSUPPORTED)])
def test_parameters(lib, call, field, value, code):
    assert call(lib, params(**{field: value})) == code


@pytest.mark.parametrize("call", [tree, sparse])
def test_group_sizes(lib, call):
    assert call(lib, params(Hq=6)) == UNSUPPORTED       # three heads a group
    assert call(lib, params(Hq=32)) == UNSUPPORTED      # sixteen


@pytest.mark.parametrize("kw,code", [
    ({"tree": 0}, INVALID), ({"tree": 65}, UNSUPPORTED), ({"pages": 0}, INVALID),
    ({"pages": 1 << 24}, INVALID), ({"mp": 0}, INVALID), ({"mp": 1 << 26}, INVALID),
    ({"mp": (1 << 25) - 1}, INVALID), ({"n": -1}, INVALID), ({"n": 65536}, INVALID),
    ({"q": None}, INVALID), ({"k": None}, INVALID),
    ({"v": None}, INVALID), ({"mask": None}, INVALID), ({"kv": None}, INVALID),
    ({"pt": None}, INVALID), ({"sl": None}, INVALID), ({"u": None}, INVALID),
    ({"out": None}, INVALID), ({"ws": None}, INVALID), ({"q": MIS}, INVALID), ({"k": MIS}, INVALID),
    ({"v": MIS}, INVALID), ({"mask": 0x100004}, INVALID), ({"lens": MIS4}, INVALID),
    ({"kv": MIS}, INVALID), ({"pt": MIS4}, INVALID), ({"sl": MIS4}, INVALID), ({"u": MIS}, INVALID),
    ({"out": MIS}, INVALID), ({"neff": MIS4}, INVALID), ({"ws": MIS}, INVALID),
    ({"wb": 8}, WORKSPACE), ({"n": 0, "q": None}, OK)])
def test_tree(lib, kw, code):
    assert tree(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    ({"keep": 0}, INVALID), ({"keep": -1}, INVALID), ({"pages": 0}, INVALID), ({"mp": 0}, INVALID),
    ({"n": -1}, INVALID), ({"q": None}, INVALID), ({"b": None}, INVALID), ({"kv": None}, INVALID),
    ({"b": MIS}, INVALID), ({"kv": MIS}, INVALID), ({"sel": MIS4}, INVALID), ({"out": MIS}, INVALID),
    ({"ws": None}, INVALID), ({"wb": 8}, WORKSPACE), ({"n": 0, "b": None}, OK)])
def test_sparse(lib, kw, code):
    assert sparse(lib, **kw) == code


def test_workspace_sizes(lib):
    p = params()
    size = lib.polar_attn_decode_tree_workspace_size
    assert size(2, 4, 4, ctypes.byref(p)) > 0
    assert tree(lib, wb=size(2, 4, 4, ctypes.byref(p)) - 1) == WORKSPACE
    assert size(2, 4, 65, ctypes.byref(p)) == 0
    size = lib.polar_attn_decode_sparse_workspace_size
    assert sparse(lib, wb=size(2, 4, 2, ctypes.byref(p)) - 1) == WORKSPACE
    assert size(2, 4, 0, ctypes.byref(p)) == 0
    c = cache()
    assert lib.polar_attn_cache_workspace_size(ctypes.byref(c), 3) > 0
    assert lib.polar_attn_cache_workspace_size(ctypes.byref(cache(Hkv=0)), 3) == 0


def cache(**kw):
    c = N.Cache(A, A, A, 10, 2, 64, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def reserve(lib, c=None, pt=A, mp=4, sl=A, grow=A, n=2, granted=A, ws=A, wb=BIG):
    return lib.polar_attn_cache_reserve(ctypes.byref(c or cache()), pt, mp, sl, grow, n, granted, ws,
                                        wb, None)


def append(lib, c=None, k=A, v=A, src=4, pick=None, tokens=4, counts=None, pt=A, mp=4, sl=A, n=2):
    return lib.polar_attn_cache_append(ctypes.byref(c or cache()), k, v, src, pick, tokens, counts,
                                       pt, mp, sl, n, None)


def fork(lib, c=None, spt=A, ssl=A, ns=2, rows=A, n=2, pt=A + (1 << 20), sl=A + (1 << 20), mp=4):
    return lib.polar_attn_cache_fork(ctypes.byref(c or cache()), spt, ssl, ns, rows, n, pt, sl, mp,
                                     None)


def free(lib, c=None, pt=A, mp=4, sl=A, keep=None, n=2):
    return lib.polar_attn_cache_free(ctypes.byref(c or cache()), pt, mp, sl, keep, n, None)


def compact(lib, c=None, pt=A, mp=4, sl=A, n=2, used=A, ws=A, wb=BIG):
    return lib.polar_attn_cache_compact(ctypes.byref(c or cache()), pt, mp, sl, n, used, ws, wb, None)


CALLS = [reserve, append, fork, free, compact]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 128, UNSUPPORTED), ("dtype", 1, UNSUPPORTED), ("dtype", 9, INVALID),
    ("Hkv", 0, INVALID), ("num_pages", 0, INVALID), ("num_pages", 1 << 25, INVALID),
    ("kv_pages", None, INVALID), ("kv_pages", MIS, INVALID), ("bounds", MIS, INVALID),
    ("refs", MIS4, INVALID)])
def test_pool(lib, call, field, value, code):
    assert call(lib, cache(**{field: value})) == code


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw", [{"pt": None}, {"sl": None}, {"pt": MIS4}, {"sl": MIS4}, {"mp": 0},
                                {"mp": 1 << 26}, {"n": -1}, {"n": 65536}])
def test_rows(lib, call, kw):
    assert call(lib, **kw) == INVALID


@pytest.mark.parametrize("call", [reserve, fork, free, compact])
def test_references_are_needed(lib, call):
    assert call(lib, cache(refs=None)) == INVALID


@pytest.mark.parametrize("call,kw,code", [
    (reserve, {"grow": None}, INVALID), (reserve, {"granted": None}, INVALID),
    (reserve, {"grow": MIS4}, INVALID), (reserve, {"ws": None}, INVALID),
    (reserve, {"ws": MIS}, INVALID), (reserve, {"wb": 100}, WORKSPACE),
    (append, {"k": None}, INVALID), (append, {"v": MIS}, INVALID), (append, {"tokens": 5}, INVALID),
    (append, {"tokens": -1}, INVALID), (append, {"pick": MIS4}, INVALID),
    (append, {"counts": MIS4}, INVALID), (append, {"tokens": 0, "k": None}, OK),
    (fork, {"rows": None}, INVALID), (fork, {"ns": -1}, INVALID), (fork, {"spt": MIS4}, INVALID),
    (fork, {"pt": A + 16}, INVALID), (fork, {"sl": A + 4}, INVALID), (free, {"keep": MIS4}, INVALID),
    (compact, {"used": None}, INVALID), (compact, {"wb": 8}, WORKSPACE), (reserve, {"n": 0}, OK),
    (append, {"n": 0}, OK), (fork, {"n": 0}, OK), (free, {"n": 0}, OK)])
def test_arguments(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_binding_wants_cuda_tensors():
    import torch
    with pytest.raises(ValueError, match="CUDA"):
        N.PageCache(torch.zeros((2, 2, 1, 64, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="kv_pages"):
        N.PageCache(torch.zeros((2, 2, 1, 32, 64), dtype=torch.bfloat16))


def test_host_model_by_hand():
    """Two rows share a page of ten tokens; both grow; the last keeps it."""
    kv = np.arange(4 * 2 * 64 * 64, dtype=np.float64).reshape(4, 2, 1, 64, 64)
    h = R.HostCache(kv, np.array([2, 0, 1, 0]), np.zeros((4, 1, 2, 64)))
    table, lens = np.array([[0, -1], [0, -1], [2, -1]], np.int32), np.array([10, 10, 64], np.int32)
    got = h.reserve(table, lens, np.array([1, 1, 1]))
    assert got.tolist() == [1, 1, 1]
    assert table.tolist() == [[1, -1], [0, -1], [2, 3]] and h.refs.tolist() == [1, 1, 1, 1]
    assert np.array_equal(h.kv[1, :, :, :10], kv[0, :, :, :10])
    assert np.array_equal(h.kv[1, :, :, 10:], kv[1, :, :, 10:])
    h.free(table, lens, [0, -1, 64])
    assert table.tolist() == [[-1, -1], [0, -1], [2, -1]] and h.refs.tolist() == [1, 0, 1, 0]
    assert h.compact(table, lens) == 2 and table.tolist() == [[-1, -1], [0, -1], [1, -1]]


def test_reference_row_by_hand():
    """One key: the direction is its value, n_eff is 1 and the count is 0."""
    v = np.zeros((1, 64))
    v[0, 3] = 2.0
    out, neff, _, _ = R.mixing_row(v[0], v, v, np.ones(64), 8.0, 0.3, 128, 1.0)
    assert neff == 1.0 and out[3] == 1.0 and abs(out).sum() == 1.0


@pytest.mark.parametrize("name", ["kv_pages", "refs", "bounds"])
def test_a_cache_keeps_its_tensors(name):
    """The calls use the addresses that a cache was built with: a tensor put in a
    cache's place later is turned down, not passed over in silence."""
    c = N.PageCache.__new__(N.PageCache)
    with pytest.raises(AttributeError):
        setattr(c, name, None)


def test_status_string_names_what_is_out_of_range(lib):
    """Code 7 stands for lengths and for the counts of the tree and the cache."""
    text = lib.polar_attn_status_string(7).decode()
    assert all(word in text for word in ("length", "node", "growth", "count", "out of range"))
