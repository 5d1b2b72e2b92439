"""The paged cache's operations on the GPU against a host model, alone and in
the runs that a serving loop makes of them."""
import numpy as np
import pytest
import torch

import polar_attention_b200 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu

OK, BAD_PAGE, BAD_SEQLEN, BAD_SLOT, NO_PAGES = 0, 4, 7, 8, 9


def unit(rng, *shape):
    x = rng.standard_normal(shape)
    x = torch.from_numpy(x / np.linalg.norm(x, axis=-1, keepdims=True)).bfloat16()
    return x


class Pair:
    """A cache on the GPU and its host model, with one page table."""

    def __init__(self, P, Hkv, rows, max_pages, seed=0):
        self.rng = np.random.default_rng(seed)
        kv = unit(self.rng, P, 2, Hkv, 64, 64)
        b = unit(self.rng, P, Hkv, 2, 64)
        self.dev = pa.PageCache(kv.cuda(), torch.zeros(P, dtype=torch.int32).cuda(), b.cuda())
        self.host = R.HostCache(R.f64(kv), np.zeros(P, np.int64), R.f64(b))
        self.table = np.full((rows, max_pages), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.Hkv = Hkv
        self.up()

    def up(self):
        self.dtable, self.dlens = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()

    def same(self, status=OK):
        assert pa.get_status() == status
        assert np.array_equal(self.dtable.cpu().numpy(), self.table)
        assert np.array_equal(self.dlens.cpu().numpy(), self.lens)
        assert np.array_equal(self.dev.refs.cpu().numpy(), self.host.refs)
        assert np.array_equal(R.f64(self.dev.kv_pages), self.host.kv)
        assert np.array_equal(R.f64(self.dev.bounds), self.host.bounds)

    def reserve(self, grow, status=OK):
        grow = np.asarray(grow, np.int32)
        got = pa.cache_reserve(self.dev, self.dtable, self.dlens, torch.from_numpy(grow).cuda())
        want = self.host.reserve(self.table, self.lens, grow)
        assert np.array_equal(got.cpu().numpy(), want), (got, want)
        self.same(status)
        return want

    def append(self, counts, T=None, pick=None):
        counts = np.asarray(counts, np.int32)
        T = max(1, int(counts.max())) if T is None else T
        k, v = unit(self.rng, 2, len(counts), T, self.Hkv, 64)
        pa.cache_append(self.dev, k.cuda(), v.cuda(), self.dtable, self.dlens,
                        torch.from_numpy(counts).cuda(),
                        None if pick is None else torch.from_numpy(pick).cuda())
        self.host.append(R.f64(k), R.f64(v), self.table, self.lens, counts, pick)
        self.same()

    def grow(self, grow):
        self.append(self.reserve(grow))

    def fork(self, src_rows):
        """The rows become copies of src_rows of the old table; the old rows are freed."""
        src = np.asarray(src_rows, np.int32)
        new, nlens = np.full_like(self.table, -1), np.zeros_like(self.lens)
        dnew, dlens = torch.from_numpy(new).cuda(), torch.from_numpy(nlens).cuda()
        pa.cache_fork(self.dev, self.dtable, self.dlens, torch.from_numpy(src).cuda(), dnew, dlens)
        self.host.fork(self.table, self.lens, src, new, nlens)
        pa.cache_free(self.dev, self.dtable, self.dlens)
        self.host.free(self.table, self.lens)
        self.same()
        self.table, self.lens, self.dtable, self.dlens = new, nlens, dnew, dlens
        self.same()

    def free(self, keep=None):
        pa.cache_free(self.dev, self.dtable, self.dlens, None if keep is None else
                      torch.tensor(keep, dtype=torch.int32).cuda())
        self.host.free(self.table, self.lens, keep)
        self.same()

    def compact(self):
        used = pa.cache_compact(self.dev, self.dtable, self.dlens)
        assert used.item() == self.host.compact(self.table, self.lens)
        self.same()


@pytest.mark.parametrize("Hkv", [1, 2, 3, 4])
def test_growth(cuda_ok, Hkv):
    """Rows of no tokens, one, a page's edge and several pages, grown from every
    offset; rows that do not grow stay as they are."""
    p = Pair(60, Hkv, 6, 20, seed=Hkv)
    p.grow([0, 1, 63, 64, 65, 200])
    p.grow([1, 63, 1, 1, 0, 57])
    p.grow([130, 1, 0, 64, 1, 1])
    p.append([0, 0, 0, 0, 0, 0])


@pytest.mark.parametrize("seed", range(6))
def test_random_life(cuda_ok, seed):
    """Growth, forks, rollbacks and compactions in a random order: every state
    equals the host model's."""
    rng = np.random.default_rng(seed)
    p = Pair(90, 2, 7, 12, seed=seed)
    p.grow(rng.integers(0, 300, 7))
    for _ in range(14):
        op = rng.integers(4)
        if op == 0:
            room = np.minimum(12 * 64 - p.lens, rng.integers(0, 100, 7))
            p.grow(np.where(rng.random(7) < 0.7, room, 0))
        elif op == 1:
            p.fork(rng.integers(0, 7, 7))
        elif op == 2:
            p.free([int(rng.integers(-1, n + 2)) for n in p.lens])
        else:
            p.compact()


def test_shared_tails(cuda_ok):
    """Three rows on one partly filled page: two copy it and the last keeps it;
    with a sharer outside the call all copy; a rollback into a shared full page
    is copied before it is written."""
    p = Pair(40, 2, 4, 8, seed=9)
    p.grow([100, 0, 0, 70])
    p.fork([0, 0, 0, 3])
    refs = p.host.refs[p.table[0, 1]]
    assert refs == 3
    keep = p.table[2, 1]
    p.grow([1, 2, 3, 1])
    assert p.table[2, 1] == keep and len({p.table[i, 1] for i in range(3)}) == 3
    p.fork([2, 2, 2, 3])
    tail = p.table[0, 1]
    p.grow([0, 5, 1, 0])
    assert tail not in (p.table[1, 1], p.table[2, 1])
    p.fork([1, 1, 1, 1])
    p.free([30, 40, 200, 20])  # into the shared first page, at different lengths
    p.grow([1, 1, 1, 1])


def test_many_rows_share_tails(cuda_ok):
    """More rows than one launch plans and copies: forks of few rows, grown."""
    N = 300
    p = Pair(700, 1, N, 3, seed=13)
    p.grow([70, 10, 64] + [0] * (N - 3))
    p.fork(np.arange(N) % 3)
    p.grow(np.arange(N) % 5 % 3)
    p.fork(np.arange(N)[::-1] // 2)
    got = p.reserve(np.ones(N, np.int32))
    assert got.all()
    p.append(got)
    p.fork(np.zeros(N, np.int32))
    p.host.refs[p.host.refs == 0] = 9  # no free page
    p.dev.refs.copy_(torch.from_numpy(p.host.refs.astype(np.int32)))
    assert not p.reserve(np.ones(N, np.int32), status=NO_PAGES).any()


def test_pages_past_32_bits(cuda_ok):
    """The last pages of a pool of more than 2^32 bytes and 2^31 values."""
    P, Hkv, N, T = 70000, 4, 3, 150
    cache = pa.PageCache(torch.zeros((P, 2, Hkv, 64, 64), dtype=torch.bfloat16, device="cuda"),
                         torch.ones(P, dtype=torch.int32, device="cuda"),
                         torch.zeros((P, Hkv, 2, 64), dtype=torch.bfloat16, device="cuda"))
    small = pa.PageCache(torch.zeros((20, 2, Hkv, 64, 64), dtype=torch.bfloat16, device="cuda"),
                         torch.zeros(20, dtype=torch.int32, device="cuda"),
                         torch.zeros((20, Hkv, 2, 64), dtype=torch.bfloat16, device="cuda"))
    cache.refs[P - 20:] = 0
    rng = np.random.default_rng(14)
    k, v = unit(rng, 2, 2 * N, T, Hkv, 64).cuda().unbind(0)
    k, v = k.contiguous(), v.contiguous()
    q = unit(rng, 2 * N, 9, 16, 64).cuda()
    mask = torch.tensor([2 ** (t + 1) - 1 for t in range(9)]).repeat(2 * N, 1).cuda()
    u = torch.zeros((16, 64), device="cuda")

    def run(c, max_pages):
        def rows():
            return (torch.full((2 * N, max_pages), -1, dtype=torch.int32, device="cuda"),
                    torch.zeros(2 * N, dtype=torch.int32, device="cuda"))
        (t0, l0), (t, n) = rows(), rows()
        grow = torch.tensor([T] * N + [0] * N, dtype=torch.int32).cuda()
        got = pa.cache_reserve(c, t0, l0, grow)
        pa.cache_append(c, k, v, t0, l0, got)
        src = (torch.arange(2 * N) % N).int().cuda()
        pa.cache_fork(c, t0, l0, src, t, n)
        pa.cache_free(c, t0, l0)
        got = pa.cache_reserve(c, t, n, torch.full((2 * N,), 2, dtype=torch.int32).cuda())
        pa.cache_append(c, k, v, t, n, got)  # N copies of tails
        def decodes():
            return [*pa.decode_paged_tree(q, k[:, :9].contiguous(), v[:, :9].contiguous(), mask,
                                          c.kv_pages, t, n, u),
                    *pa.decode_paged_sparse(q[:, 0].contiguous(), c.kv_pages, c.bounds, t, n, u, 2)]
        first = decodes()
        top = t.max().item()
        c.refs[:-20] = 0  # the others' pages
        used = pa.cache_compact(c, t, n).item()
        assert used == 4 * N and t.max().item() == used - 1 and (c.refs[used:] == 0).all()
        return first, decodes(), top

    want, wagain, _ = run(small, 3)
    got, again, top = run(cache, 3)
    assert pa.get_status() == OK and top == P - 20 + 4 * N - 1
    for a, b, c, d in zip(want, wagain, got, again):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)


def test_pool_runs_out(cuda_ok):
    """From the first row that cannot be served on, no row is; what was served
    is whole, and a row that needs no page waits with the others."""
    p = Pair(10, 1, 5, 12, seed=2)
    p.grow([64 * 3, 10, 64 * 2, 1, 0])
    got = p.reserve([64, 1, 64 * 3, 1, 1], status=NO_PAGES)
    assert got.tolist() == [64, 1, 0, 0, 0]
    p.reserve([0, 0, 64 * 2, 0, 0])
    p.reserve([0, 0, 0, 0, 1], status=NO_PAGES)
    p.free([0, -1, -1, -1, -1])
    p.reserve([0, 0, 0, 0, 1])


def test_last_sharer_keeps_only_when_all_are_served(cuda_ok):
    """Two sharers, one free page short: the first takes the copy, or, with no
    page at all, none is served and the page stays shared."""
    p = Pair(3, 1, 2, 4, seed=3)
    p.grow([10, 64])
    p.free([-1, 0])
    p.fork([0, 0])
    p.grow([1, 1])
    p = Pair(1, 1, 2, 4, seed=3)
    p.grow([10, 0])
    p.fork([0, 0])
    got = p.reserve([1, 1], status=NO_PAGES)
    assert got.tolist() == [0, 0] and p.host.refs[0] == 2


def test_bad_rows_are_passed_over(cuda_ok):
    """A length or a growth out of range, a tail outside the pool: reported, and
    the other rows are served."""
    p = Pair(20, 1, 4, 3, seed=4)
    p.grow([10, 10, 10, 10])
    for i, (n, g) in enumerate([(10, -1), (10, 64 * 3 - 9), (64 * 3 + 1, 0), (-2, 1)]):
        lens, grow = p.lens.copy(), np.ones(4, np.int32)
        lens[1], grow[1] = n, g
        p.lens[:] = lens
        p.up()
        got = p.reserve(grow, status=BAD_SEQLEN)
        assert got.tolist() == [1, 0, 1, 1]
        p.lens[1] = 10
        p.up()
    p.table[1, 0] = 20
    p.up()
    assert p.reserve([1, 1, 1, 1], status=BAD_PAGE).tolist() == [1, 0, 1, 1]


def test_large_pool_and_many_rows(cuda_ok):
    """Free pages past the first steps of the search; more rows than a block has
    threads."""
    P, N = 40000, 1500
    g = torch.Generator().manual_seed(0)
    kv = torch.zeros((P, 2, 1, 64, 64), dtype=torch.bfloat16, device="cuda")
    refs = (torch.rand(P, generator=g) < 0.8).int().cuda()
    refs[:20000] = 1
    before = refs.cpu().numpy().copy()
    cache = pa.PageCache(kv, refs)
    table = torch.full((N, 2), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    grow = torch.randint(0, 129, (N,), generator=g).int()
    got = pa.cache_reserve(cache, table, lens, grow.cuda())
    assert pa.get_status() == OK and torch.equal(got.cpu(), grow)
    free = np.flatnonzero(before == 0)
    want = np.full((N, 2), -1, np.int32)
    k = 0
    for i, n in enumerate(grow.tolist()):
        for c in range(-(-n // 64)):
            want[i, c] = free[k]
            k += 1
    assert np.array_equal(table.cpu().numpy(), want)
    before[free[:k]] = 1
    assert np.array_equal(cache.refs.cpu().numpy(), before)
    used = pa.cache_compact(cache, table, lens)
    assert pa.get_status() == OK
    n = int((before > 0).sum())
    assert used.item() == n and (cache.refs[:n] > 0).all() and not cache.refs[n:].any()


def test_compaction_moves_what_it_must(cuda_ok):
    """Nothing live, everything live, one page at the end, and pages whose
    numbers of blocks are odd."""
    p = Pair(33, 3, 3, 40, seed=5)
    p.compact()
    p.grow([33 * 64, 0, 0])
    p.compact()
    p.free([64 * 32, -1, -1])
    p.grow([0, 0, 7])
    p.free([0, -1, -1])
    assert p.table[2, 0] == 32
    p.compact()
    assert p.table[2, 0] == 0


def test_compaction_reports_bad_entries(cuda_ok):
    p = Pair(12, 1, 2, 4, seed=6)
    p.grow([64 * 4, 64 * 2])
    p.free([0, -1])
    d = p.dtable.clone()
    for bad in (12, -3, 9):  # outside the pool, and a free page
        p.dtable.copy_(d)
        p.dtable[1, 0] = bad
        cache = pa.PageCache(p.dev.kv_pages.clone(), p.dev.refs.clone())
        pa.cache_compact(cache, p.dtable, p.dlens)
        assert pa.get_status() == BAD_PAGE and p.dtable[1, 0].item() == bad
        assert p.dtable[1, 1].item() < 2


def test_append_picks_and_reports(cuda_ok):
    """Accepted rows by index, the same row twice among them; an index, a count
    or a page out of range is reported and nothing else is lost."""
    p = Pair(20, 2, 3, 4, seed=7)
    p.grow([60, 5, 0])
    pick = np.array([[4, 1, 1, 0, 9], [0, 9, 9, 9, 9], [3, 2, 1, 0, 5]], np.int32)
    got = p.reserve([4, 1, 5])
    p.append(got, T=6, pick=pick)
    k = torch.zeros((3, 6, 2, 64), dtype=torch.bfloat16, device="cuda")
    before = p.dev.kv_pages.clone()
    bad = torch.tensor([[0, 1, 2, 6, -1]] * 3, dtype=torch.int32).cuda()
    pa.cache_append(p.dev, k, k, p.dtable, p.dlens, torch.tensor([4, 0, 5]).int().cuda(), bad)
    assert pa.get_status() == BAD_SLOT
    page = p.dtable[2, 0].long()  # tokens 3 and 4 of row 2 are skipped
    assert not p.dev.kv_pages[page, :, :, :3].any()
    assert torch.equal(p.dev.kv_pages[page, :, :, 3:5], before[page, :, :, 3:5])
    for counts, lens in (([6, 0, 0], None), ([-1, 0, 0], None), ([5, 0, 0], [4, 6, 5]),
                         ([1, 0, 0], [257, 6, 5])):
        before = p.dev.kv_pages.clone()
        dl = p.dlens if lens is None else torch.tensor(lens).int().cuda()
        pa.cache_append(p.dev, k[:, :5].contiguous(), k[:, :5].contiguous(), p.dtable, dl,
                        torch.tensor(counts).int().cuda())
        assert pa.get_status() == BAD_SEQLEN and torch.equal(before, p.dev.kv_pages)
    p.dev.refs[p.dtable[0, 0].long()] = 2  # a page that another entry names
    pa.cache_append(p.dev, k, k, p.dtable, p.dlens, torch.tensor([6, 0, 0]).int().cuda())
    assert pa.get_status() == BAD_PAGE
    assert torch.equal(before[p.dtable[0, 0].long()], p.dev.kv_pages[p.dtable[0, 0].long()])


def test_append_without_references_or_bounds(cuda_ok):
    rng = np.random.default_rng(1)
    kv = unit(rng, 4, 2, 2, 64, 64).cuda()
    k, v = unit(rng, 2, 1, 130, 2, 64).cuda().unbind(0)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32).cuda()
    other = kv[1].clone()
    pa.cache_append(pa.PageCache(kv), k.contiguous(), v.contiguous(), table,
                    torch.tensor([140], dtype=torch.int32).cuda())
    assert pa.get_status() == OK and torch.equal(other, kv[1])
    rows = kv[table[0].long()].permute(1, 0, 3, 2, 4).reshape(2, 192, 2, 64)[:, 10:140]
    assert torch.equal(rows[0], k[0]) and torch.equal(rows[1], v[0])
    with pytest.raises(pa.PolarError):
        pa.cache_free(pa.PageCache(kv), table, torch.tensor([140], dtype=torch.int32).cuda())


def test_bounds_follow_nan_and_signed_zero(cuda_ok):
    p = Pair(4, 1, 1, 2, seed=8)
    p.reserve([3])
    k = torch.zeros((1, 3, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[0, 1, 0, 5], k[0, 2, 0, 6], k[0, 0, 0, 7] = float("nan"), float("inf"), -0.0
    pa.cache_append(p.dev, k, k, p.dtable, p.dlens)
    b = p.dev.bounds[p.dtable[0, 0].long(), 0].float()
    assert torch.isnan(b[:, 5]).all() and b[0, 6] == 0 and b[1, 6] == float("inf")
    assert (b[:, 7] == 0).all() and not b[:, 8:].any()


def test_fork_leaves_rows_and_reports(cuda_ok):
    p = Pair(20, 1, 3, 4, seed=9)
    p.grow([100, 64, 0])
    new, lens = torch.full_like(p.dtable, 77), torch.full_like(p.dlens, 77)
    src = torch.tensor([-1, 2, 0], dtype=torch.int32).cuda()
    pa.cache_fork(p.dev, p.dtable, p.dlens, src, new, lens)
    assert pa.get_status() == OK and lens.tolist() == [77, 0, 100]
    assert (new[:2] == 77).all() and (new[2, 2:] == 77).all()
    pa.cache_fork(p.dev, p.dtable, p.dlens, torch.tensor([3, -1, -1]).int().cuda(), new, lens)
    assert pa.get_status() == BAD_SLOT and lens[0] == 77
    with pytest.raises(pa.PolarError):
        pa.cache_fork(p.dev, p.dtable, p.dlens, src, p.dtable, lens)
    # One table's rows as source and destination, in ranges of their own.
    pa.cache_fork(p.dev, p.dtable[:1], p.dlens[:1], torch.zeros(1).int().cuda(), p.dtable[2:],
                  p.dlens[2:])
    assert pa.get_status() == OK and torch.equal(p.dtable[2, :2], p.dtable[0, :2])


def test_free_reports_a_page_without_references(cuda_ok):
    p = Pair(8, 1, 2, 4, seed=10)
    p.grow([64, 64])
    p.dtable[1, 0] = 5  # free
    pa.cache_free(p.dev, p.dtable, p.dlens)
    assert pa.get_status() == BAD_PAGE
    assert p.dev.refs.tolist() == [0, 1] + [0] * 6 and (p.dtable == -1).all()


def test_speculative_loop(cuda_ok):
    """Prompts, drafted trees, the accepted path appended, in a captured graph
    that is replayed: afterwards the cache decodes as one written at once, and
    the kept bounds select the same pages."""
    Hq, Hkv, N, M, MP = 8, 2, 3, 7, 12
    rng = np.random.default_rng(3)
    p = Pair(40, Hkv, N, MP, seed=11)
    p.grow([70, 300, 5])
    q = unit(rng, N, M, Hq, 64).cuda()
    u = (0.02 * torch.randn((Hq, 64))).cuda()
    mask = torch.tensor([1, 3, 5, 11, 19, 37, 69]).repeat(N, 1).cuda()
    k, v = unit(rng, 2, N, M, Hkv, 64).cuda().unbind(0)
    k, v = k.contiguous(), v.contiguous()
    pick = torch.tensor([[0, 1, 4], [0, 2, 6], [0, 1, 3]], dtype=torch.int32).cuda()
    count = torch.tensor([3, 1, 2], dtype=torch.int32).cuda()
    graph = torch.cuda.CUDAGraph()
    for _ in range(2):  # the kernels are loaded before the capture
        pa.decode_paged_tree(q, k, v, mask, p.dev.kv_pages, p.dtable, p.dlens, u)
        pa.decode_paged_sparse(q[:, 0].contiguous(), p.dev.kv_pages, p.dev.bounds, p.dtable,
                               p.dlens, u, 3)
    with torch.cuda.graph(graph):
        out, neff = pa.decode_paged_tree(q, k, v, mask, p.dev.kv_pages, p.dtable, p.dlens, u)
        granted = pa.cache_reserve(p.dev, p.dtable, p.dlens, count)
        pa.cache_append(p.dev, k, v, p.dtable, p.dlens, granted, pick)
        sel = pa.decode_paged_sparse(q[:, 0].contiguous(), p.dev.kv_pages, p.dev.bounds, p.dtable,
                                     p.dlens, u, 3)
    for _ in range(30):
        k.copy_(unit(rng, N, M, Hkv, 64))
        v.copy_(unit(rng, N, M, Hkv, 64))
        hk, hv = R.f64(k), R.f64(v)
        graph.replay()
        got = p.host.reserve(p.table, p.lens, count.cpu().numpy())
        p.host.append(hk, hv, p.table, p.lens, got, pick.cpu().numpy())
    p.same()
    # The tree's node 1 of the last replay, from its key cached: row 0 accepted
    # nodes 0, 1, 4, so the cache holds node 1's view up to two tokens before its end.
    lens = p.dlens.clone()
    lens[0] -= 1
    want, nwant = pa.decode_paged(q[:, 1].contiguous(), p.dev.kv_pages, p.dtable, lens, u)
    assert ((neff[0, 1] - nwant[0]).abs() / nwant[0]).max() < 1e-4
    whole = pa.decode_paged_sparse(q[:, 0].contiguous(), p.dev.kv_pages,
                                   torch.stack((p.dev.kv_pages[:, 0].amin(2),
                                                p.dev.kv_pages[:, 0].amax(2)), 2).contiguous(),
                                   p.dtable, p.dlens, u, 3)
    # Bounds over stale rows too are wider only on a newest page, which is read anyway.
    assert pa.get_status() == OK and torch.equal(sel[2], whole[2])


def test_beam_steps_on_a_stream(cuda_ok):
    """Beam steps on a stream of their own, no synchronisation between calls."""
    side = torch.cuda.Stream()
    p = Pair(80, 2, 6, 6, seed=12)
    p.grow([90, 90, 90, 130, 10, 64])
    side.wait_stream(torch.cuda.current_stream())
    tables = [(p.dtable, p.dlens), (torch.full_like(p.dtable, -1), torch.zeros_like(p.dlens))]
    srcs = [np.array(s, np.int32) for s in ([0, 0, 1, 3, 3, 5], [5, 4, 3, 2, 1, 0],
                                            [2, 2, 2, 2, 2, 2])]
    dsrc = [torch.from_numpy(s).cuda() for s in srcs]
    ones = torch.ones(6, dtype=torch.int32).cuda()
    ks = [[unit(p.rng, 6, 1, 2, 64) for _ in range(2)] for _ in srcs]
    dks = [[t.cuda() for t in kk] for kk in ks]
    torch.cuda.synchronize()
    for s, kk in zip(dsrc, dks):
        (a, al), (b, bl) = tables
        pa.cache_fork(p.dev, a, al, s, b, bl, stream=side)
        pa.cache_free(p.dev, a, al, stream=side)
        g = pa.cache_reserve(p.dev, b, bl, ones, stream=side)
        pa.cache_append(p.dev, *kk, b, bl, g, stream=side)
        tables.reverse()
    side.synchronize()
    for s, kk in zip(srcs, ks):
        new, nl = np.full_like(p.table, -1), np.zeros_like(p.lens)
        p.host.fork(p.table, p.lens, s, new, nl)
        p.host.free(p.table, p.lens)
        g = p.host.reserve(new, nl, np.ones(6, np.int32))
        p.host.append(R.f64(kk[0]), R.f64(kk[1]), new, nl, g)
        p.table, p.lens = new, nl
    p.dtable, p.dlens = tables[0]
    live = np.arange(6)[None] < -(-p.lens // 64)[:, None]
    p.dtable = torch.where(torch.from_numpy(live).cuda(), p.dtable, -1)
    p.same()


def test_a_shrunk_pool_is_another_cache(cuda_ok):
    """After a compaction the pool's front goes on as a cache of its own; the old
    cache takes no other tensors and still names its own."""
    p = Pair(30, 2, 3, 8, seed=15)
    p.grow([200, 300, 64])
    p.free([0, -1, -1])
    p.compact()
    n = int((p.host.refs > 0).sum()) + 4
    old = p.dev
    with pytest.raises(AttributeError):
        old.refs = old.refs[:n].clone()
    p.dev = pa.PageCache(*(t[:n].clone() for t in (old.kv_pages, old.refs, old.bounds)))
    p.host = R.HostCache(p.host.kv[:n], p.host.refs[:n], p.host.bounds[:n])
    before = [t.clone() for t in (old.kv_pages, old.refs, old.bounds)]
    p.grow([70, 20, 64])
    assert p.reserve([128, 64, 0], status=NO_PAGES).tolist() == [0, 0, 0]
    for a, b in zip(before, (old.kv_pages, old.refs, old.bounds)):
        assert torch.equal(a, b)
