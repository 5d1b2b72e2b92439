"""GPU parity of the page-selecting decode (polar_attn_decode_paged_sparse)."""
import numpy as np
import pytest
import torch

import polar_attention_b200 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu

ARGS = dict(s=8.0, alpha=0.3, L=128, beta=1.0)


def inputs(lens, Hq, Hkv, seed=0, max_pages=None):
    lens = np.asarray(lens, np.int64)
    N = len(lens)
    npg = -(-lens // 64)
    max_pages = max_pages or int(npg.max())
    P = int(npg.sum())
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((P, 2, Hkv, 64, 64), generator=g)
    x[:, 0] += torch.randn((P, Hkv, 1, 64), generator=g)
    kv = (x / x.norm(dim=-1, keepdim=True)).bfloat16()
    q = torch.randn((N, Hq, 64), generator=g)
    table = np.full((N, max_pages), -1, np.int32)
    perm, o = np.random.default_rng(seed).permutation(P), 0
    for i in range(N):
        table[i, :npg[i]] = perm[o:o + npg[i]]
        o += npg[i]
    return {"q": (q / q.norm(dim=-1, keepdim=True)).bfloat16(), "kv": kv,
            "bounds": torch.stack((kv[:, 0].amin(2), kv[:, 0].amax(2)), 2).contiguous(),
            "table": torch.from_numpy(table), "lens": torch.from_numpy(lens.astype(np.int32)),
            "u": 0.02 * torch.randn((Hq, 64), generator=g)}


def cuda(x):
    return {k: t.cuda() for k, t in x.items()}


def call(d, keep, **kw):
    return pa.decode_paged_sparse(d["q"], d["kv"], d["bounds"], d["table"], d["lens"], d["u"],
                                  keep, **dict(ARGS, **kw))


def select(x, i, g, keep):
    """The pages of (sequence i, kv head g), in ascending order."""
    q, b = R.f64(x["q"]), R.f64(x["bounds"])
    n = int(x["lens"][i])
    npg, G = -(-n // 64), q.shape[1] // b.shape[1]
    ids = x["table"].numpy()[i, :npg]
    lo, hi = b[ids, g, 0], b[ids, g, 1]
    with np.errstate(all="ignore"):
        score = np.stack([np.maximum(qh * lo, qh * hi).sum(1) for qh in q[i, g * G:(g + 1) * G]])
        score = score.astype(np.float32).max(0)
    order = sorted(range(npg), key=lambda p: (p != npg - 1, not np.isnan(score[p]),
                                              0 if np.isnan(score[p]) else -score[p], p))
    return sorted(order[:keep])


def check(x, keep, out, neff, sel, seqs=None, **kw):
    a = dict(ARGS, **kw)
    q, kv, u = R.f64(x["q"]), R.f64(x["kv"]), R.f64(x["u"])
    N, Hq, _ = q.shape
    Hkv = kv.shape[2]
    G = Hq // Hkv
    for i in range(N) if seqs is None else seqs:
        n = int(x["lens"][i])
        for g in range(Hkv):
            want = select(x, i, g, keep)
            got = sel[i, g].tolist()
            assert got == want + [-1] * (keep - len(want)), (i, g)
            pos = np.concatenate([np.arange(p * 64, min(n, p * 64 + 64)) for p in want])
            pages = x["table"].numpy()[i, pos // 64]
            refs = [R.mixing_row(q[i, h], kv[pages, 0, g, pos % 64], kv[pages, 1, g, pos % 64],
                                 u[h], a["s"], a["alpha"], a["L"], a["beta"])
                    for h in range(g * G, (g + 1) * G)]
            R.check_rows(out[i, g * G:(g + 1) * G], neff[i, g * G:(g + 1) * G], refs, f"seq {i}")


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("keep", [1, 2, 3, 7, 16, 40])
def test_small_ragged(cuda_ok, G, keep):
    """From one token to many pages; fewer pages than kept, as many, and more."""
    x = inputs([1, 63, 64, 65, 129, 700, 64 * keep, 64 * keep + 1, 2500], 2 * G, 2, seed=G + keep)
    out, neff, sel = call(cuda(x), keep)
    assert pa.get_status() == 0
    check(x, keep, out, neff, sel)


@pytest.mark.parametrize("keep", [1, 100, 513, 1100])
def test_long(cuda_ok, keep):
    """More pages than the selection's block has threads; temperature active."""
    x = inputs([70001, 33000], 8, 2, seed=3)
    out, neff, sel = call(cuda(x), keep, L=2048)
    assert pa.get_status() == 0
    check(x, keep, out, neff, sel, L=2048)


def test_whole_sequence_is_the_plain_decode(cuda_ok):
    x = inputs([100, 640, 1], 16, 4, seed=4)
    d = cuda(x)
    out, neff, sel = call(d, 10)
    want, nwant = pa.decode_paged(d["q"], d["kv"], d["table"], d["lens"], d["u"], **ARGS)
    assert ((neff - nwant).abs() / nwant).max() < 1e-5
    check(x, 10, out, neff, sel)
    check(x, 10, want, nwant, sel)


def test_ties_go_to_the_lower_page(cuda_ok):
    """Equal bounds everywhere, and bounds whose scores are +0 and -0."""
    x = inputs([64 * 30 + 5, 64 * 12], 8, 2, seed=5)
    x["bounds"][:] = x["bounds"][0].clone()
    out, neff, sel = call(cuda(x), 6)
    check(x, 6, out, neff, sel)
    assert sel[0, 0].tolist() == [0, 1, 2, 3, 4, 30]
    x["bounds"][:] = 0.0
    x["bounds"][x["table"][0, 3].item()] = -0.0
    out, neff, sel = call(cuda(x), 4)
    assert sel[0, 0].tolist() == [0, 1, 2, 30] and sel[1, 1].tolist() == [0, 1, 2, 11]


def test_many_ties(cuda_ok):
    """More pages in question than get exact scores one by one; some above them."""
    x = inputs([64 * 500 + 5], 8, 2, seed=11)
    x["bounds"][:] = x["bounds"][0].clone()
    above = [400, 7, 130]
    x["bounds"][x["table"][0, above].long()] *= 2
    for keep in (1, 3, 100, 400):
        out, neff, sel = call(cuda(x), keep)
        assert pa.get_status() == 0
        check(x, keep, out, neff, sel)


def test_scores_closer_than_their_roundings(cuda_ok):
    """Bounds whose large terms cancel: the order is in the small ones, below the
    rounding of an fp32 sum."""
    x = inputs([64 * 300], 2, 2, seed=12)
    x["q"][:], x["bounds"][:] = 0, 0
    x["q"][..., :3] = torch.tensor([1.0, 1.0, 2.0 ** -26]).bfloat16()
    g = torch.Generator().manual_seed(0)
    x["bounds"][..., 0], x["bounds"][..., 1] = 3.0, -3.0
    small = torch.randperm(300, generator=g)[:, None].expand(300, 2)
    x["bounds"][:, :, 1, 2] = (small % 256).bfloat16()  # ties, too
    for keep in (5, 80):
        out, neff, sel = call(cuda(x), keep)
        check(x, keep, out, neff, sel)


def test_longer_than_the_shared_keys(cuda_ok):
    """A sequence whose scores do not fit in shared memory beside a short one."""
    x = inputs([64 * 10500 + 9, 200], 4, 1, seed=13)
    for keep in (3, 300):
        out, neff, sel = call(cuda(x), keep, L=2048)
        assert pa.get_status() == 0
        check(x, keep, out, neff, sel, L=2048)


def test_scores_that_are_not_finite(cuda_ok):
    """A NaN score ranks above every number, an infinite one where it belongs."""
    x = inputs([64 * 20], 8, 2, seed=6)
    t = x["table"][0].tolist()
    x["bounds"][t[7], 0, :, 3] = float("nan")
    x["bounds"][t[9], 0] = torch.tensor([-float("inf"), float("inf")])[:, None].bfloat16()
    x["bounds"][t[2], 1] = torch.tensor([-float("inf"), -float("inf")])[:, None].bfloat16()
    out, neff, sel = call(cuda(x), 3)
    assert pa.get_status() == 0
    check(x, 3, out, neff, sel)
    assert sel[0, 0].tolist() == [7, 9, 19]


@pytest.mark.parametrize("keep", [4, 30, 150])
def test_many_pages_with_scores_that_are_not_finite(cuda_ok, keep):
    """Every score is in question then: all get exact ones."""
    x = inputs([64 * 200 + 1, 64 * 90], 8, 2, seed=14)
    t = x["table"][0].tolist()
    for p in (3, 11, 150):
        x["bounds"][t[p], 0, :, 7] = float("nan")
    for p in (5, 60):
        x["bounds"][t[p]] = torch.tensor([-float("inf"), float("inf")])[:, None].bfloat16()
    out, neff, sel = call(cuda(x), keep)
    assert pa.get_status() == 0
    check(x, keep, out, neff, sel)


def test_stale_rows_do_not_count(cuda_ok):
    x = inputs([64 * 9 + 10], 8, 2, seed=7)
    clean = {k: t.clone() for k, t in x.items()}
    x["kv"][x["table"][0, 9].item(), :, :, 10:] = float("nan")
    out, neff, sel = call(cuda(x), 4)
    check(clean, 4, out, neff, sel)


def test_twice_captured_and_on_a_stream(cuda_ok):
    x, y = inputs([5000, 300], 16, 4, seed=8), inputs([4994, 310], 16, 4, seed=9)
    d = cuda(x)
    a = call(d, 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = call(d, 9, stream=side)
    side.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = call(d, 9)
    graph.replay()
    assert all(torch.equal(s, t) for s, t in zip(a, c))
    for n in d:
        d[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert pa.get_status() == 0
    check(y, 9, *c)


def test_bad_pages_and_lengths_are_reported(cuda_ok):
    x = inputs([700, 700], 8, 2, seed=10)
    d = cuda(x)
    d["table"][0, 10] = -5  # the newest page, always read
    call(d, 3)
    assert pa.get_status() == 4
    for n in (0, -3, 64 * 11 + 1):
        d = cuda(x)
        d["lens"][0] = n
        out = torch.full_like(d["q"], 7.0)
        sel = torch.full((2, 2, 3), 7, dtype=torch.int32, device="cuda")
        pa.decode_paged_sparse(d["q"], d["kv"], d["bounds"], d["table"], d["lens"], d["u"], 3, out,
                               selected=sel, **ARGS)
        assert pa.get_status() == 7
        assert (out[0] == 7).all() and (sel[0] == 7).all() and (out[1] != 7).any()


@pytest.mark.parametrize("kind", R.ALIKE)
@pytest.mark.parametrize("Hq,keep", [(1, 40), (4, 513), (8, 1100)])
def test_keys_that_are_alike(cuda_ok, Hq, keep, kind):
    """Keys and values alike over many selected pages: the null floor's spread is
    not what sums of squares lose beside the squared mean."""
    n = 70001
    x = inputs([n], Hq, 1, seed=15)
    rng = np.random.default_rng(15)
    key = R.at_angle(np.eye(64)[0], 0.1, (), rng)
    x["q"] = torch.from_numpy(R.at_angle(key, 0.77, (1, Hq), rng)).bfloat16()
    page = x["table"][0].long()
    keys = torch.zeros((page.numel() * 64, 64), dtype=torch.bfloat16)
    keys[:n] = R.alike_keys(kind, key, n, rng)
    keys[n:] = keys[n - 1]
    x["kv"][page, 0, 0] = keys.view(-1, 64, 64)
    x["kv"][page, 1, 0] = x["kv"][0, 1, 0, 0].clone()
    x["bounds"] = torch.stack((x["kv"][:, 0].amin(2), x["kv"][:, 0].amax(2)), 2).contiguous()
    x["u"] = torch.randn(x["u"].shape, generator=torch.Generator().manual_seed(15))
    out, neff, sel = call(cuda(x), keep, L=2048)
    assert pa.get_status() == 0
    check(x, keep, out, neff, sel, L=2048)


def test_row_is_that_of_the_selected_pages(cuda_ok):
    """The plain decode over tables of the selected pages gives the same rows: n is
    the number of selected positions, not the sequence's."""
    x = inputs([64 * 90 + 7, 64 * 40, 64 * 300 + 64], 8, 2, seed=16)
    d, keep = cuda(x), 20
    out, neff, sel = call(d, keep)
    for g in range(2):
        table = d["table"].gather(1, sel[:, g].long())
        lens = (keep - 1) * 64 + (d["lens"] - 1) % 64 + 1
        want, nwant = pa.decode_paged(d["q"], d["kv"], table.contiguous(), lens.int(), d["u"], **ARGS)
        heads = slice(4 * g, 4 * g + 4)
        for i in range(3):  # both against 64 bits, over the same pages
            keys, values = R.cached(R.f64(x["kv"]), table[i].cpu().numpy(), g, int(lens[i]))
            refs = [R.mixing_row(R.f64(x["q"])[i, h], keys, values, R.f64(x["u"])[h], **ARGS)
                    for h in range(4 * g, 4 * g + 4)]
            R.check_rows(out[i, heads], neff[i, heads], refs)
            R.check_rows(want[i, heads], nwant[i, heads], refs)
    assert pa.get_status() == 0


@pytest.mark.parametrize("G,keep", [(1, 3), (4, 8), (8, 20)])
def test_counts_of_the_directions_size(cuda_ok, G, keep):
    """Values alike and u of order one: mean, spread and n_eff are seen in the
    outputs, from one key to all of the selected pages."""
    x = inputs([1, 2, 17, 64, 65, 700, 64 * keep, 3000], 2 * G, 2, seed=17)
    rng = np.random.default_rng(17)
    key = R.at_angle(np.eye(64)[0], 0.2, (), rng)
    x["kv"][:, 1] = torch.from_numpy(R.at_angle(key, 0.99, x["kv"][:, 1].shape[:-1], rng)).bfloat16()
    x["u"] = torch.from_numpy(rng.choice([-1.0, 1.0], x["u"].shape)).float()
    out, neff, sel = call(cuda(x), keep)
    assert pa.get_status() == 0
    check(x, keep, out, neff, sel)
