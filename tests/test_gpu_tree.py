"""GPU parity of the decode for drafted trees (polar_attn_decode_paged_tree)
against a plain 64-bit reference, and its edge cases."""
import numpy as np
import pytest
import torch

import polar_attention_b200 as pa
import serving_ref as R
from polar_attention_b200 import workloads as W

pytestmark = pytest.mark.gpu

ARGS = dict(s=8.0, alpha=0.3, L=128, beta=1.0)


def random_masks(rng, N, M):
    """Ancestor masks of random trees: a node's parent is an earlier node or none."""
    m = np.zeros((N, M), np.int64)
    for i in range(N):
        words = []
        for t in range(M):
            p = int(rng.integers(-1, t))
            words.append((words[p] if p >= 0 else 0) | 1 << t)
            m[i, t] = words[t] - (1 << 64 if words[t] >> 63 else 0)
    return m


def inputs(lens, M, Hq, Hkv, seed=0, max_pages=None, masks=None):
    lens = np.asarray(lens, np.int64)
    N = len(lens)
    npg = -(-lens // 64)
    max_pages = max_pages or max(1, int(npg.max()))
    P = max(1, int(npg.sum()))
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)

    def unit(*shape):
        x = torch.randn(shape, generator=g)
        return (x / x.norm(dim=-1, keepdim=True)).bfloat16()

    kv = unit(P, 2, Hkv, 64, 64)
    table = np.full((N, max_pages), -1, np.int32)
    perm, o = rng.permutation(P), 0
    for i in range(N):
        table[i, :npg[i]] = perm[o:o + npg[i]]
        o += npg[i]
    x = {"q": unit(N, M, Hq, 64), "k": unit(N, M, Hkv, 64), "v": unit(N, M, Hkv, 64),
         "mask": torch.from_numpy(random_masks(rng, N, M) if masks is None else masks),
         "kv": kv, "table": torch.from_numpy(table), "lens": torch.from_numpy(lens.astype(np.int32)),
         "u": 0.02 * torch.randn((Hq, 64), generator=g)}
    for i in range(N):  # a key near a query, so that some weights stand out
        if lens[i]:
            kv[table[i, 0], 0, :, 0] = x["q"][i, 0, ::Hq // Hkv]
    return x


def cuda(x):
    return {k: t.cuda() for k, t in x.items()}


def call(d, tree_lens=None, **kw):
    a = dict(ARGS, **kw)
    return pa.decode_paged_tree(d["q"], d["k"], d["v"], d["mask"], d["kv"], d["table"], d["lens"],
                                d["u"], tree_lens=tree_lens, **a)


def reference(x, tree_lens, rows=None, **kw):
    """mixing_row for each (sequence, node < tree_lens, head)."""
    a = dict(ARGS, **kw)
    q, k, v, kv = (R.f64(x[n]) for n in ("q", "k", "v", "kv"))
    u, table, lens = R.f64(x["u"]), x["table"].numpy(), x["lens"].numpy()
    N, M, Hq, _ = q.shape
    G = Hq // kv.shape[2]
    refs = {}
    for i in range(N):
        for h in range(Hq):
            ck, cv = R.cached(kv, table[i], h // G, lens[i])
            for t in range(tree_lens[i]):
                if rows is not None and (i, t, h) not in rows:
                    continue
                bits = int(x["mask"][i, t]) & (2 ** 64 - 1)
                js = [j for j in range(tree_lens[i]) if bits >> j & 1]
                refs[i, t, h] = R.mixing_row(q[i, t, h], np.concatenate([ck, k[i, js, h // G]]),
                                             np.concatenate([cv, v[i, js, h // G]]), u[h], a["s"],
                                             a["alpha"], a["L"], a["beta"])
    return refs


def check(x, out, neff, tree_lens, rows=None, what="", **kw):
    refs = reference(x, tree_lens, rows, **kw)
    at = np.array(list(refs))
    R.check_rows(out[at[:, 0], at[:, 1], at[:, 2]], neff[at[:, 0], at[:, 1], at[:, 2]],
                 list(refs.values()), what)


# Columns of a page table.  Above 16 rows per kv head a wide table's call runs on
# the tensor cores' 128-row tiles; up to 16 rows it is split over many CTAs.
WIDE = 5000


# Rows per kv head from one to 512, in and across row tiles.
@pytest.mark.parametrize("max_pages", [13, WIDE])
@pytest.mark.parametrize("G,M", [(1, 1), (4, 1), (2, 3), (8, 1), (4, 3), (2, 8), (1, 17), (4, 8),
                                 (8, 5), (1, 64), (4, 17), (2, 63), (4, 33), (8, 17), (4, 64),
                                 (8, 64)])
def test_small_ragged(cuda_ok, G, M, max_pages):
    """Lengths of zero, one, a page's edge and several splits, with node counts
    from none to all of a padded batch."""
    lens = [0, 1, 63, 64, 65, 130, 700, 0]
    x = inputs(lens, M, 2 * G, 2, seed=G * 100 + M, max_pages=max_pages)
    rng = np.random.default_rng(M)
    tl = rng.integers(0, M + 1, len(lens)).astype(np.int32)
    tl[[0, 5]], tl[7] = M, min(1, M)
    d = cuda(x)
    out, neff = call(d, tree_lens=torch.from_numpy(tl).cuda())
    assert pa.get_status() == 0
    check(x, out, neff, tl, what=f"G={G} M={M}")


def test_all_nodes_without_lens(cuda_ok):
    x = inputs([100, 3], 5, 8, 2, seed=3)
    out, neff = call(cuda(x))
    assert pa.get_status() == 0
    check(x, out, neff, [5, 5])


@pytest.mark.parametrize("M", [1, 2, 4, 5, 23])
def test_long_many_splits(cuda_ok, M):
    """Tens of thousands of cached tokens over many splits, temperature active;
    a sample of rows."""
    x = inputs([40001, 5000], M, 16, 4, seed=5)
    out, neff = call(cuda(x), L=2048)
    assert pa.get_status() == 0
    rng = np.random.default_rng(0)
    rows = {(int(rng.integers(2)), int(rng.integers(M)), int(rng.integers(16)))
            for _ in range(24)} | {(0, M - 1, 15), (1, 0, 0)}
    check(x, out, neff, [M, M], rows, L=2048)


@pytest.mark.parametrize("G,M", [(1, 3), (4, 9), (2, 64)])
def test_many_sequences_few_with_work(cuda_ok, G, M):
    """A padded batch: most sequences have no nodes, some of those that have see
    no cache."""
    rng = np.random.default_rng(14)
    lens, tl = np.zeros(400, np.int64), np.zeros(400, np.int32)
    busy = np.sort(rng.choice(400, 12, replace=False))
    lens[busy], tl[busy] = rng.integers(0, 300, 12), rng.integers(1, M + 1, 12)
    lens[rng.choice(400, 50)] = 130  # cached, without nodes
    x = inputs(lens, M, 2 * G, 2, seed=14, max_pages=40)
    d = cuda(x)
    out = torch.full_like(d["q"], 7.0)
    neff = torch.full(out.shape[:3], 7.0, device="cuda")
    pa.decode_paged_tree(d["q"], d["k"], d["v"], d["mask"], d["kv"], d["table"], d["lens"], d["u"],
                         out, neff, tree_lens=torch.from_numpy(tl).cuda(), **ARGS)
    assert pa.get_status() == 0
    check(x, out, neff, tl)
    behind = torch.arange(M)[None] >= torch.from_numpy(tl)[:, None]
    assert (out[behind.cuda()] == 7).all() and (neff[behind.cuda()] == 7).all()


@pytest.mark.parametrize("max_pages", [5, WIDE])
def test_high_scale(cuda_ok, max_pages):
    """Logits up to 60: weights over a range of 2^170."""
    x = inputs([300, 70], 20, 8, 2, seed=6, max_pages=max_pages)
    out, neff = call(cuda(x), s=60.0)
    check(x, out, neff, [20, 20], s=60.0)


@pytest.mark.parametrize("G,max_pages", [(4, 2), (4, WIDE), (8, WIDE)])
def test_rows_that_see_nothing(cuda_ok, G, max_pages):
    """No cache and an empty mask: zeros; an empty mask over a cache: the cache
    alone; bits past the node count are ignored."""
    masks = np.zeros((3, 4), np.int64)
    masks[1] = [1, 0, 7 << 1, -1]
    masks[2] = -16  # bits 4 and up only
    x = inputs([0, 0, 70], 4, 2 * G, 2, seed=7, masks=masks, max_pages=max_pages)
    out, neff = call(cuda(x))
    assert pa.get_status() == 0
    check(x, out, neff, [4, 4, 4])
    assert not out[0].any() and not neff[0].any() and not out[1, 1].any()


@pytest.mark.parametrize("max_pages", [4, WIDE])
def test_rows_behind_a_sequence_are_left(cuda_ok, max_pages):
    x = inputs([10, 200, 0], 6, 8, 2, seed=8, max_pages=max_pages)
    d = cuda(x)
    tl = torch.tensor([2, 0, 6], dtype=torch.int32).cuda()
    out = torch.full_like(d["q"], 7.0)
    neff = torch.full((3, 6, 8), 7.0, device="cuda")
    pa.decode_paged_tree(d["q"], d["k"], d["v"], d["mask"], d["kv"], d["table"], d["lens"], d["u"],
                         out, neff, tree_lens=tl, **ARGS)
    assert pa.get_status() == 0
    for i, n in enumerate([2, 0, 6]):
        assert (out[i, n:] == 7).all() and (neff[i, n:] == 7).all()
        assert n == 0 or (neff[i, :n] != 7).all()
    check(x, out, neff, [2, 0, 6])


@pytest.mark.parametrize("G,M,max_pages", [(4, 2, 2), (4, 8, 2), (4, 40, 2), (2, 9, WIDE),
                                           (4, 40, WIDE)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_does_not_count(cuda_ok, G, M, max_pages, bad):
    """Stale rows behind the cache's end and behind a sequence's nodes, and a
    drafted node that only some rows see: their values, finite or not, reach
    the rows that see them and no others."""
    lens, tl = [70, 5], [M, M - 1]
    x = inputs(lens, M, 2 * G, 2, seed=9, max_pages=max_pages)
    for i, n in enumerate(lens):
        page = x["table"][i, n // 64]
        x["kv"][page, :, :, n % 64:] = bad
    x["k"][1, M - 1], x["v"][1, M - 1] = bad, bad
    node = M // 2  # seen by its descendants alone
    clean = {k: t.clone() for k, t in x.items()}
    x["k"][0, node] = bad
    x["v"][0, node, :, 3] = bad
    out, neff = call(cuda(x), tree_lens=torch.tensor(tl, dtype=torch.int32).cuda())
    assert pa.get_status() == 0
    sees = [bool(int(x["mask"][0, t]) >> node & 1) for t in range(M)]
    rows = {(0, t, h) for t in range(M) if not sees[t] for h in range(2 * G)} | \
        {(1, t, h) for t in range(tl[1]) for h in range(2 * G)}
    check(clean, out, neff, tl, rows)
    for t in range(M):
        if sees[t]:
            assert not torch.isfinite(out[0, t]).all()


@pytest.mark.parametrize("max_pages", [3, WIDE])
@pytest.mark.parametrize("M", [2, 9, 40])
def test_values_not_finite_reach_their_rows(cuda_ok, M, max_pages):
    """A finite key with a value that is infinite in one column: the rows that
    see it have no direction there, the others do not notice."""
    x = inputs([130], M, 8, 2, seed=10, max_pages=max_pages)
    clean = {k: t.clone() for k, t in x.items()}
    x["v"][0, M - 1, :, 5] = float("inf")
    out, neff = call(cuda(x))
    refs = {(0, t, h) for t in range(M - 1) for h in range(8)}
    check(clean, out, neff, [M], refs)
    assert torch.isnan(out[0, M - 1, :, 5]).all() and torch.isfinite(neff).all()


def test_chain_is_a_chunk(cuda_ok):
    """A chain over the cache computes what the chunked decode does once the
    chain's rows are cached (other splits: both within the tolerance)."""
    C, n = 4, 900
    w = W.small_decode(num_seqs=1, min_len=n, max_len=n, Hq=16, Hkv=4, seed=4, plant=2)
    y = W.decode_inputs(w, "cpu", seqlens=[n])
    q = W.decode_chunk_queries(w, y, C).cuda()
    d = {k: t.cuda() for k, t in y.items() if isinstance(t, torch.Tensor)}
    want, nwant = pa.decode_paged_chunk(q, d["kv_pages"], d["page_table"], d["seqlens"], d["u"])
    pos = torch.arange(n - C, n)
    pages = y["page_table"][0, pos // 64].long()
    k = y["kv_pages"][pages, 0, :, pos % 64][None].cuda().contiguous()
    v = y["kv_pages"][pages, 1, :, pos % 64][None].cuda().contiguous()
    x = {"q": q, "k": k, "v": v, "mask": torch.tensor([[2 ** (t + 1) - 1 for t in range(C)]]),
         "kv": y["kv_pages"], "table": y["page_table"], "lens": y["seqlens"] - C, "u": y["u"]}
    out, neff = call(cuda(x), L=2048)
    assert pa.get_status() == 0
    check(x, out, neff, [C], L=2048)
    check(x, want, nwant, [C], L=2048)


@pytest.mark.parametrize("max_pages", [11, WIDE])
def test_twice_and_captured(cuda_ok, max_pages):
    """The same bits twice, on another stream, and from a replayed graph whose
    lengths, masks and drafts change between replays."""
    x = inputs([700, 64, 3], 12, 16, 4, seed=11, max_pages=max_pages)
    y = inputs([600, 1, 128], 12, 16, 4, seed=12, max_pages=max_pages)
    d = cuda(x)
    a, na = call(d)
    b, nb = call(d)
    assert torch.equal(a, b) and torch.equal(na, nb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, nc = call(d, stream=side)
    side.synchronize()
    assert torch.equal(a, c) and torch.equal(na, nc)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, no = call(d)
    graph.replay()
    assert torch.equal(a, o) and torch.equal(na, no)
    for n in d:
        if n != "u":
            d[n].copy_(y[n])
    graph.replay()
    e, ne = call(d)
    assert torch.equal(e, o) and torch.equal(ne, no)
    assert pa.get_status() == 0
    check({**y, "u": x["u"]}, o, no, [12, 12, 12])


@pytest.mark.parametrize("M,max_pages", [(3, 3), (3, WIDE), (30, WIDE)])
def test_bad_pages_and_lengths_are_reported(cuda_ok, M, max_pages):
    x = inputs([130, 130, 130, 50], M, 8, 2, seed=13, max_pages=max_pages)
    x["table"][1, 1] = 10 ** 6
    d = cuda(x)
    call(d)
    assert pa.get_status() == 4
    for field, value in (("lens", 10 ** 6), ("lens", -1), ("nodes", M + 1), ("nodes", -1)):
        d = cuda(inputs([130, 130, 130, 50], M, 8, 2, seed=13, max_pages=max_pages))
        tl = torch.full((4,), M, dtype=torch.int32).cuda()
        (d["lens"] if field == "lens" else tl)[2] = value
        out = torch.full_like(d["q"], 7.0)
        pa.decode_paged_tree(d["q"], d["k"], d["v"], d["mask"], d["kv"], d["table"], d["lens"],
                             d["u"], out, tree_lens=tl, **ARGS)
        assert pa.get_status() == 7, (field, value)
        assert (out[2] == 7).all() and (out[[0, 1, 3]] != 7).any(-1).all()
    assert pa.get_status() == 0


def test_two_graphs_and_eager_calls(cuda_ok):
    """Two captured graphs replayed at once on two streams, and calls between
    them: each has its own workspace."""
    x = [inputs([5000, 900], M, 16, 4, seed=M, max_pages=500) for M in (4, 30)]
    d = [cuda(t) for t in x]
    want = [call(t) for t in d]
    graphs, got, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for t in d:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(call(t))
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        again = [call(t) for t in d]
    torch.cuda.synchronize()
    assert pa.get_status() == 0
    for w, *others in zip(want, got, again):
        assert all(torch.equal(w[i], o[i]) for o in others for i in (0, 1))


def along(axis, dots, rng):
    """Unit rows with the products `dots` with a unit vector along `axis`."""
    dots = np.asarray(dots, np.float64)
    x = rng.standard_normal((*dots.shape, 64))
    x[..., axis] = 0
    x *= np.sqrt(1 - dots ** 2)[..., None] / np.linalg.norm(x, axis=-1, keepdims=True)
    x[..., axis] = dots
    return torch.from_numpy(x).bfloat16()


@pytest.mark.parametrize("G,M", [(4, 20), (1, 40), (8, 64)])
def test_reference_moves_twice_in_a_page(cuda_ok, G, M):
    """Weights far above a row's first reference, then a page whose first half
    moves the reference by more than 2^24 and whose second half moves it as far
    again: what was summed before has to shrink by both.  At s = 60 a product of
    0.3 is 26 log2 units; with one of the moves lost, the second page would weigh
    half as much as the last keys instead of 2^-26 of them."""
    x = inputs([192, 192, 130], M, 2 * G, 2, seed=15, max_pages=WIDE)
    rng = np.random.default_rng(15)
    x["q"].zero_()
    x["q"][..., 0] = 1
    for i, n in enumerate((192, 192, 130)):
        page = x["table"][i].long()
        dots = np.repeat([-0.6, -0.335, -0.29, 0.0], [64, 64, 32, 32])[:n]
        if i == 1:  # three moves in one page, and back
            dots = np.concatenate([np.full(100, -0.9), np.full(60, -0.3), np.full(31, 0.3), [0.9]])
        keys = along(0, np.broadcast_to(dots, (2, n)), rng)
        values = torch.zeros((2, n, 64), dtype=torch.bfloat16)
        for at, d in enumerate(sorted(set(dots.tolist()))):
            values[:, np.flatnonzero(dots == d), 10 + at] = 1
        for p in range(n):
            x["kv"][page[p // 64], 0, :, p % 64] = keys[:, p]
            x["kv"][page[p // 64], 1, :, p % 64] = values[:, p]
    x["k"] = along(0, np.full(x["k"].shape[:-1], -0.95), rng)
    out, neff = call(cuda(x), s=60.0, L=2048)
    assert pa.get_status() == 0
    check(x, out, neff, [M, M, M], s=60.0, L=2048)


@pytest.mark.parametrize("G,M,lens", [(4, 40, [130, 5]), (8, 9, [130, 5]), (1, 64, [4000, 0])])
def test_rows_add_different_numbers_of_values(cuda_ok, G, M, lens):
    """Drafted values that are not finite in columns of their own, seen by none
    to all of them in the rows of one warp, some of whose lanes have no row: a row
    has no direction in the columns it sees, and only there."""
    x = inputs(lens, M, 2 * G, 2, seed=16, max_pages=WIDE)
    clean = {k: t.clone() for k, t in x.items()}
    odd = list(range(0, M, 3))
    for j in odd:
        x["v"][:, j, :, j % 64] = float("inf")
    out, neff = call(cuda(x))
    assert pa.get_status() == 0
    refs = reference(clean, [M, M], {(i, t, 0) for i in range(2) for t in range(M)})
    for (i, t, h), (want, n, _, tol) in refs.items():
        bits = int(x["mask"][i, t]) & (2 ** 64 - 1)
        seen = [j % 64 for j in odd if bits >> j & 1]
        row = out[i, t, h].float().cpu().numpy()
        assert abs(neff[i, t, h].item() - n) <= tol
        assert np.isnan(row[seen]).all() and np.isfinite(np.delete(row, seen)).all()
        if not seen:
            check(clean, out, neff, [M, M], {(i, t, h)})


@pytest.mark.parametrize("kind", R.ALIKE)
@pytest.mark.parametrize("G,M,max_pages", [(1, 1, 1025), (4, 4, 1025), (4, 16, WIDE), (8, 64, WIDE)])
def test_keys_that_are_alike(cuda_ok, G, M, max_pages, kind):
    """Long caches whose keys are alike: the null floor's spread is not what sums
    of squares lose beside the squared mean.  Values alike, too, so that the
    direction is certain, and a count of the direction's size."""
    lens = [65536, 20011]
    x = inputs(lens, M, G, 1, seed=17, max_pages=max_pages)
    rng = np.random.default_rng(17)
    key = R.at_angle(np.eye(64)[0], 0.1, (), rng)
    x["q"] = torch.from_numpy(R.at_angle(key, 0.77, x["q"].shape[:-1], rng)).bfloat16()
    value = along(1, np.float64(0.3), rng)
    for i, n in enumerate(lens):
        page = x["table"][i, :-(-n // 64)].long()
        keys = torch.full((page.numel() * 64, 64), float("nan"), dtype=torch.bfloat16)
        keys[:n] = R.alike_keys(kind, key, n, rng)
        x["kv"][page, 0, 0] = keys.view(-1, 64, 64)
        x["kv"][page, 1, 0] = value
    x["k"][:] = R.alike_keys("equal", key, 1, rng)[0]
    x["v"][:] = value
    x["u"] = torch.randn(x["u"].shape, generator=torch.Generator().manual_seed(17))
    out, neff = call(cuda(x), L=2048)
    assert pa.get_status() == 0
    rows = {(i, t, h) for i in (0, 1) for t in {0, M // 3, M // 2, M - 1} for h in {0, G - 1}}
    check(x, out, neff, [M, M], rows, L=2048)


@pytest.mark.parametrize("max_pages", [13, WIDE])
@pytest.mark.parametrize("G,M", [(1, 2), (4, 5), (8, 1), (8, 3), (2, 31), (4, 64)])
def test_counts_of_the_directions_size(cuda_ok, G, M, max_pages):
    """Few keys and many, with values alike and u of order one: the outputs' size
    is the count's, so that mean, spread and n_eff are seen in them."""
    lens = [0, 1, 2, 3, 17, 63, 64, 65, 130, 700]
    x = inputs(lens, M, 2 * G, 2, seed=18, max_pages=max_pages)
    rng = np.random.default_rng(18)
    key = R.at_angle(np.eye(64)[0], 0.2, (), rng)
    x["kv"][:, 1] = torch.from_numpy(R.at_angle(key, 0.99, x["kv"][:, 1].shape[:-1], rng)).bfloat16()
    x["v"] = torch.from_numpy(R.at_angle(key, 0.99, x["v"].shape[:-1], rng)).bfloat16()
    near = x["kv"][:, 0].float() + 0.5 * x["kv"][:, 0, :, :1].float()  # a page's keys alike
    x["kv"][:, 0] = (near / near.norm(dim=-1, keepdim=True)).bfloat16()
    x["u"] = torch.from_numpy(rng.choice([-1.0, 1.0], x["u"].shape)).float()
    out, neff = call(cuda(x))
    assert pa.get_status() == 0
    check(x, out, neff, [M] * len(lens), what=f"G={G} M={M}")
