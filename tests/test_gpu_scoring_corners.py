"""The scoring operators where their definitions are easily lost: values that are not finite side by side, ranges of fp32,
heads with outliers, blocks of several tiles, row pointers out of order."""
import numpy as np
import pytest
import torch

from tests import test_gpu_label_logprobs as head_ops
from tests import test_gpu_logprobs as score_ops
from tests import test_gpu_q4 as q4_ops
from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


# ---------------------------------------------------------------- rows of scores
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("L", [3, 100, 5000, 40_000, 400_000])
def test_rows_with_nan_beside_infinity(dtype, L):
    """A NaN spoils a row whatever else it holds, in the same vector, block or part as an infinity or far from it; rows
    with infinities alone keep lse = +inf."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L)
    places = [(0, 1), (1, 0), (0, L - 1), (L - 1, 0), (L // 2, L // 2 + 1), (L // 3, 2 * L // 3)]
    z = rng.normal(0, 3, (len(places) + 4, L)).astype(np.float32)
    for b, (n, i) in enumerate(places):
        z[b, i], z[b, n] = INF, NAN
    n = len(places)
    z[n, 0], z[n, 2] = INF, INF                                 # two infinities and no NaN
    z[n + 1, 1] = INF
    z[n + 2] = np.where(np.arange(L) == 1, NAN, -INF)
    z[n + 3] = np.where(np.arange(L) == 1, INF, -INF)
    rowptr = np.arange(len(z) + 1, dtype=np.int32)
    cols = np.full(len(z), 2, np.int32)
    cols[3] = cols[2] = 1
    Z = score_ops.on_gpu(z, dtype)
    logp, lse, H, idx, top = score_ops.scored(elmo, Z, rowptr, cols, 2)
    spoiled = np.r_[0:n, n + 2]
    assert np.isnan(lse[spoiled]).all() and np.isnan(H).all()
    assert np.isnan(logp[spoiled]).all()
    assert (lse[[n, n + 1, n + 3]] == INF).all()
    assert np.isnan(logp[n]) and logp[n + 1] == -INF and logp[n + 3] == -INF
    best = np.where(np.isnan(z), -INF, z)
    first = np.argmax(best, 1)
    assert (idx[:, 0] == np.where(best.max(1) > -INF, first, -1)).all()
    # the gradient of a spoiled row is NaN, that of a row whose lse is infinite zero
    dZ = torch.empty_like(Z)
    up = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    elmo.elmo_score_logprobs_backward(Z, up(rowptr), up(cols), up(lse), None, torch.ones(len(z), device="cuda"), None, None, dZ)
    dz = dZ.float().cpu().numpy()
    assert np.isnan(dz[spoiled]).all() and (dz[[n, n + 1, n + 3]] == 0).all()


@pytest.mark.parametrize("op", ["scores", "head"])
def test_bad_row_pointers_write_their_own_entries_only(op):
    """Row pointers that lie outside [0, nnz) or run backwards: entries of the rows that remain are right, all others and
    what lies around the array are left as they were."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(0)
    L, d, nnz, guard = 500, 64, 6, 64
    cols = np.array([499, 3, 250, 7, 7, 0], np.int32)
    W, h = head_ops.head_of(elmo, rng.normal(0, 0.1, (L, d)), "bf16")
    X = head_ops.bf16(rng.normal(0, 1, (3, d)))
    z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
    Z = torch.from_numpy(z.astype(np.float32)).cuda()
    want = z - np.log(np.exp(z).sum(1, keepdims=True))
    work = torch.empty(elmo.elmo_score_logprobs_workspace_bytes(3, L, 2), dtype=torch.uint8, device="cuda")
    for ptr in ([-3, 2, 1, 99], [9, 8, 7, 6], [0, 2**31 - 1, -2**31, 2], [2, 4, 4, 5], [6, 6, 0, 3]):
        whole = torch.full((nnz + 2 * guard,), 55.0, device="cuda")
        out = (whole[guard:guard + nnz], *head_ops.buffers(3, 0, 2)[1:])
        lists = torch.tensor(ptr, dtype=torch.int32).cuda(), torch.from_numpy(cols).cuda()
        if op == "scores":
            elmo.elmo_score_logprobs(Z, *lists, *out, work)
        else:
            elmo.elmo_label_logprobs(h, X, *lists, *out)
            elmo.elmo_sync_status(h)
        got = whole.cpu().numpy()
        assert (got[:guard] == 55).all() and (got[guard + nnz:] == 55).all(), ptr
        rows = [(max(ptr[b], 0), min(ptr[b + 1], nnz)) for b in range(3)]
        for e in range(nnz):
            owners = [b for b, (e0, e1) in enumerate(rows) if e0 <= e < e1]
            if not owners:
                assert got[guard + e] == 55, (ptr, e)
            else:                                               # an entry of two rows has either one's
                assert min(abs(got[guard + e] - want[b, cols[e]]) for b in owners) < 1e-4, (ptr, e)
    h.close()


# ---------------------------------------------------------------- heads
@pytest.mark.parametrize("grid,d", [("bf16", 128), ("bf16", 832), ("e5m2", 128), ("e5m2", 832)])
@pytest.mark.parametrize("L", [2000, 60_000])
def test_weights_of_nan_beside_infinity(grid, d, L):
    """A NaN score spoils the statistics beside an infinite one too; the list goes by the scores that are numbers."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + d)
    w = rng.normal(0, 0.02, (L, d))
    x = np.abs(rng.normal(0, 1, (3, d))) + 0.1
    rowptr, cols = np.array([0, 2, 4, 6], np.int32), np.array([7, 1, 7, 2, 7, 3], np.int32)
    for infinite, spoiled in ((7, 9), (9, 7), (7, L - 1), (L - 1, 7)):
        ww = w.copy()
        ww[infinite, 3], ww[spoiled, 0] = INF, NAN
        W, h = head_ops.head_of(elmo, ww, grid)
        logp, lse, H, idx, top = head_ops.run(elmo, h, head_ops.bf16(x), rowptr, cols, 3)
        assert np.isnan(lse).all() and np.isnan(H).all() and np.isnan(logp).all()
        z = head_ops.bf16(x).double().cpu().numpy() @ np.where(np.isnan(ww), 0, W.double().cpu().numpy()).T
        z[:, spoiled] = -INF
        assert np.array_equal(idx, np.argsort(-z, 1, kind="stable")[:, :3]) and (idx[:, 0] == infinite).all()
        h.close()


@pytest.mark.parametrize("d", [128, 832])
@pytest.mark.parametrize("L,k", [(2000, 3), (2000, 0), (20_000, 3)])
def test_infinite_weights_of_an_e5m2_head(d, L, k):
    """An infinite weight makes an infinite score, whatever the two 8-bit numbers that a query's element becomes are."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + d)
    w = rng.normal(0, 0.02, (L, d))
    B = 6
    x = rng.normal(0, 1, (B, d))
    x[:, 5] = [1.0, 1.0078125, 1.0703125, -1.0, -1.0703125, 0.0]  # the second number zero, of the same and of the other sign
    rowptr, cols = np.arange(0, 2 * B + 1, 2).astype(np.int32), np.tile(np.array([7, 1], np.int32), B)
    X = head_ops.bf16(x)
    for value in (INF, -INF):
        ww = w.copy()
        ww[7, 5] = value
        W, h = head_ops.head_of(elmo, ww, "e5m2")
        logp, lse, H, idx, top = head_ops.run(elmo, h, X, rowptr, cols, k)
        with np.errstate(invalid="ignore"):
            z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
        assert np.isnan(lse[5]) and np.isnan(H[5]) and np.isnan(logp[10:]).all()      # 0 times infinity
        for b in range(5):
            if z[b, 7] == INF:
                assert lse[b] == INF and np.isnan(H[b]) and np.isnan(logp[2 * b]) and logp[2 * b + 1] == -INF
            else:
                assert z[b, 7] == -INF
                rest = np.delete(z[b], 7)
                m = rest.max()
                want = m + np.log(np.exp(rest - m).sum())
                p = np.exp(rest - want)
                assert abs(lse[b] - want) < 1e-4 and abs(H[b] + (p * (rest - want)).sum()) < 1e-3
                assert logp[2 * b] == -INF and abs(logp[2 * b + 1] - (z[b, 1] - want)) < 1e-4
        if k:
            order = np.argsort(-np.where(np.isnan(z), -INF, z), 1, kind="stable")[:, :k]
            assert np.array_equal(idx, order)
        h.close()


@pytest.mark.parametrize("L", [3000, 20_000])
def test_lists_where_sums_leave_the_range(L):
    """Scores that are ordinary numbers, but whose fp32 sums pass through an infinity: the list is still that of the
    exact scores."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L)
    d, k = 128, 5
    w = rng.normal(0, 1, (L, d)) * 2.0**88
    for at, lift in ((77, 1.25), (L - 5, 1.125)):               # -2^129 half way, then 2^127 and 2^126 in all
        w[at, :64], w[at, 64:] = -2.0**96, lift * 2.0**96
    W, h = head_ops.head_of(elmo, w, "bf16")
    X = head_ops.bf16(np.full((2, d), 2.0**27))
    idx = head_ops.run(elmo, h, X, np.zeros(3, np.int32), np.zeros(0, np.int32), k)[3]
    z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
    assert z.max() < 3e38
    assert np.array_equal(idx, np.argsort(-z, 1, kind="stable")[:, :k]) and (idx[:, :2] == [77, L - 5]).all()
    h.close()


@pytest.mark.parametrize("grid,L,d", [("bf16", 3000, 768), ("bf16", 20_000, 512), ("bf16", 3000, 1024), ("e4m3", 3000, 768),
                                      ("e4m3", 20_000, 768), ("e5m2", 3000, 1024)])
def test_products_that_the_tensor_cores_cut_off(grid, L, d):
    """Tensor-core sums cut every product at 2^-25 of the largest addend: one label whose score is made of one large and
    many small products just below that, and one that the small ones lower, as far apart as this can put them the wrong
    way round."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(d)
    instructions = d // 16
    big, x_small, w_small = 256.0, 1.75 * 2.0**-15, 0.140625     # their product is 0.984 2^-25 of the large one
    lift = 1.5 * instructions * 2.0**-21 * big                  # of twice as much that the cuts may add up to
    w = rng.normal(0, 0.02, (L, d))
    a, b = L - 7, 40
    w[a], w[b] = w_small, -w_small
    w[[a, b], 0] = big
    w[a, 1], w[b, 1] = 0, np.float32(lift * 2.0**9)
    x = np.full((2, d), x_small)
    x[:, 0], x[:, 1] = 1, 2.0**-9
    W, h = head_ops.head_of(elmo, w, grid)
    X = head_ops.bf16(x)
    z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
    assert z[0, a] > z[0, b] and np.argmax(z[0]) == a
    idx = head_ops.run(elmo, h, X, np.zeros(3, np.int32), np.zeros(0, np.int32), 2)[3]
    one = head_ops.run(elmo, h, X, np.zeros(3, np.int32), np.zeros(0, np.int32), 1)[3]
    assert (idx == [a, b]).all() and (one == a).all()
    h.close()


@pytest.mark.parametrize("grid,L,d", [("bf16", 3000, 768), ("bf16", 20_000, 1024), ("e4m3", 20_000, 768), ("e5m2", 3000, 1024)])
@pytest.mark.parametrize("place", [0, 16, 100, 384, 640, 700])
def test_products_cut_off_from_the_large_one_on(grid, L, d, place):
    """The same with the large product anywhere in the sum: what comes before it is not cut, and the bound, which counts
    an element of the query for the instructions from its own on, still covers what comes after."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(d + place)
    instructions = (d - place) // 16
    big, x_small, w_small = 256.0, 1.75 * 2.0**-15, 0.140625
    lift = 1.9 * instructions * 2.0**-21 * big
    w = rng.normal(0, 0.02, (L, d))
    a, b = L - 7, 40
    w[a], w[b] = 0, 0
    w[a, place:], w[b, place:] = w_small, -w_small
    w[[a, b], place] = big
    at = place + 1
    w[a, at], w[b, at] = 0, np.float32(lift * 2.0**9)
    x = np.full((2, d), x_small)
    x[:, place], x[:, at] = 1, 2.0**-9
    W, h = head_ops.head_of(elmo, w, grid)
    X = head_ops.bf16(x)
    z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
    order = np.argsort(-z, 1, kind="stable")[:, :2]             # a first, but for what the grid makes of the lift
    assert set(order[0]) == {a, b}
    one = head_ops.run(elmo, h, X, np.zeros(3, np.int32), np.zeros(0, np.int32), 1)[3]
    assert (one == order[:, :1]).all()
    h.close()


@pytest.mark.parametrize("grid,L", [("e4m3", 100_003), ("bf16", 60_001), ("e5m2", 40_000)])
def test_long_lists_of_the_widest_heads(grid, L):
    """Many labels within the bound of the last listed one: 4096 weights a label, 64 best."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    d, B, k = 4096, 16, 64
    g = torch.Generator(device="cuda").manual_seed(L)
    W = (torch.randn(L, d, generator=g, device="cuda") * 0.02).to(head_ops.GRIDS[grid])
    X = torch.randn(B, d, generator=g, device="cuda").to(torch.bfloat16)
    h = elmo.elmo_init_head(W, grid)
    idx = head_ops.run(elmo, h, X, np.zeros(B + 1, np.int32), np.zeros(0, np.int32), k)[3]
    Z = torch.cat([X.double() @ W[a:a + 20_000].double().T for a in range(0, L, 20_000)], 1)
    assert np.array_equal(idx, torch.topk(Z, k, 1)[1].int().cpu().numpy())
    h.close()


@pytest.mark.parametrize("grid", ["bf16", "e4m3", "e5m2"])
def test_small_queries(grid):
    """Queries down to the smallest magnitudes beside ordinary ones: statistics and lists of each."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(17)
    L, d, k = 20_011, 128, 5
    W, h = head_ops.head_of(elmo, rng.normal(0, 4, (L, d)), grid)
    x = rng.normal(0, 1, (7, d)) * 2.0 ** np.array([0, -45, -55, -70, -90, -110, -118])[:, None]
    X = head_ops.bf16(x)
    rowptr, cols = head_ops.lists(rng, 7, L, 3)
    head_ops.check(head_ops.run(elmo, h, X, rowptr, cols, k), X.double().cpu().numpy(), W.double().cpu().numpy(), grid,
                   rowptr, cols, k)
    h.close()


@pytest.mark.parametrize("grid,outlier", [("e4m3", 448.0), ("bf16", 1e4), ("e5m2", 57344.0)])
def test_one_weight_far_above_the_others(grid, outlier):
    """The bound of the list goes with the largest weight of the head: one outlier sends the queries to the exact path."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(23)
    L, d, B, k = 60_000, 768, 5, 5
    w = rng.normal(0, 0.02, (L, d))
    w[41_234, 5] = outlier
    W, h = head_ops.head_of(elmo, w, grid)
    x = rng.normal(0, 1, (B, d))
    x[2, 5] = 0                                                 # the outlier's label is an ordinary one of this query
    X = head_ops.bf16(x)
    z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
    idx = head_ops.run(elmo, h, X, np.zeros(B + 1, np.int32), np.zeros(0, np.int32), k)[3]
    assert np.array_equal(idx, np.argsort(-z, 1, kind="stable")[:, :k])
    h.close()


@pytest.mark.parametrize("grid,L,d,pairs", [("bf16", 600_011, 64, 2), ("e4m3", 600_011, 64, 2), ("e4m3", 1_100_003, 64, 4),
                                            ("bf16", 1_048_577, 128, 4), ("e5m2", 1_060_001, 832, 2)])
def test_blocks_of_several_tiles(grid, L, d, pairs):
    """Heads and batches so large that a block's maximum stands for several half tiles (4096 queries x L / 64 tiles, or
    / 128 of wide heads, of maxima pass 256 MB): the best labels are found wherever they lie, in the last, partial blocks
    of every stream among others."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    B, k = 4096, 8
    g = torch.Generator(device="cuda").manual_seed(L)
    W = torch.randn(L, d, generator=g, device="cuda") * 0.02
    W[-700:] *= 1.6                                             # many of the best are among the last labels,
    W[::1009] *= 1.5                                            # the others spread over all places in a block
    W = W.to(head_ops.GRIDS[grid])
    X = torch.randn(B, d, generator=g, device="cuda").to(torch.bfloat16)
    rng = np.random.default_rng(L)
    rowptr, cols = head_ops.lists(rng, B, L, 1)
    h = elmo.elmo_init_head(W, grid)
    logp, lse, H, idx, top = head_ops.run(elmo, h, X, rowptr, cols, k)
    pick = np.r_[0, 1, 127, 128, 300:310, 2047, 2048, 4000:4004, B - 2, B - 1]
    Z = torch.cat([X[torch.from_numpy(pick).cuda()].double() @ W[a:a + 100_000].double().T for a in range(0, L, 100_000)], 1)
    want = torch.logsumexp(Z, 1)
    p = torch.exp(Z - want[:, None])
    wH = -(p * (Z - want[:, None])).sum(1)
    steps = (1 if grid == "bf16" else 2) * -(-d * (2 if grid == "bf16" else 1) // 128) * 4
    dz = steps * 2.0**-22 * float((X[:200].double().abs() @ W[-2000:].double().abs().T).max()) * 1.2
    assert np.abs(lse[pick] - want.cpu().numpy()).max() < dz + 2e-5
    assert np.abs(H[pick] - wH.cpu().numpy()).max() < 4 * dz + 1e-4
    wt, wi = torch.topk(Z, k, 1)
    assert np.array_equal(idx[pick], wi.int().cpu().numpy())
    assert (wi >= L - 700).sum() > 20 and (wi < L - 700).sum() > 20
    assert np.abs(top[pick] - (wt - want[:, None]).cpu().numpy()).max() < dz + 2e-5
    for i, b in enumerate(pick):
        at = (Z[i, torch.from_numpy(cols[rowptr[b]:rowptr[b + 1]]).long().cuda()] - want[i]).cpu().numpy()
        assert (np.abs(logp[rowptr[b]:rowptr[b + 1]] - at) < dz + 2e-5).all(), b
    h.close()


def test_classes_of_their_own_in_the_profile():
    """The launches of elmo_label_logprobs are told apart from the top-k prediction's."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(13)
    W, h = head_ops.head_of(elmo, rng.normal(0, 0.02, (20_000, 128)), "e4m3")
    X = head_ops.bf16(rng.normal(0, 1, (5, 128)))
    idx, sc = torch.empty(5, 3, dtype=torch.int32, device="cuda"), torch.empty(5, 3, device="cuda")
    read = lambda: {c: elmo.elmo_profile_read(h, c)[1] for c in elmo.KERNEL_CLASSES}   # noqa: E731
    elmo.elmo_topk_predict(h, X, 3, 20_000, idx, sc)
    head_ops.run(elmo, h, X, np.zeros(6, np.int32), np.zeros(0, np.int32), 3)
    elmo.elmo_profile_enable(h, True)
    elmo.elmo_topk_predict(h, X, 3, 20_000, idx, sc)
    alone = read()
    elmo.elmo_profile_reset(h)
    elmo.elmo_topk_predict(h, X, 3, 20_000, idx, sc)
    head_ops.run(elmo, h, X, np.zeros(6, np.int32), np.zeros(0, np.int32), 3)
    both = read()
    assert both["topk_score"] == alone["topk_score"] and both["topk_merge"] == alone["topk_merge"]
    assert both["prep"] == alone["prep"] + 1
    assert both["logprob_score"] > 0 and both["logprob_join"] > 0
    assert alone["logprob_score"] == alone["logprob_join"] == 0
    h.close()


# ---------------------------------------------------------------- 4-bit copies
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("L,B", [(300, 1), (300, 9), (300, 30), (40_011, 2), (80_003, 8)])
def test_scores_of_large_scales(group, L, B):
    """Scales up to the largest that packing makes: scores that fp32 holds come out, and only the others are infinite."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + B + group)
    d = 256
    u = rng.integers(0, 16, (L, d)).astype(np.uint8)
    s = q4_ops.bf16_of(rng.uniform(1, 2, (L, d // group)) * 2.0 ** rng.integers(85, 122, (L, 1)))
    s[5:40] = q4_ops.bf16_of(np.abs(rng.normal(0, 0.01, (35, d // group))))   # ordinary labels among them
    x = q4_ops.bf16_of(rng.normal(0, 1, (B, d)) * 2.0 ** rng.integers(-20, 2, (B, 1)))
    Z = torch.full((B, L + 3), 123.0, device="cuda")
    elmo.elmo_q4_scores(torch.from_numpy(q4_ops.nibbles(u)).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(),
                        torch.from_numpy(x).to(torch.bfloat16).cuda(), Z[:, :L])
    z, mag = q4_ops.scored(u, s, x, group)
    got = Z.double().cpu().numpy()
    assert (got[:, L:] == 123.0).all()
    got, most = got[:, :L], float(np.finfo(np.float32).max)
    bound = q4_ops.tolerance(d, group) * mag + np.abs(z) * 2.0**-24
    holds = np.abs(z) + bound < most
    assert (np.abs(np.where(holds, got, 0) - np.where(holds, z, 0)) <= bound)[holds].all()
    over = np.abs(z) - bound > most * (1 + 2.0**-24)
    assert (got[over] == np.sign(z[over]) * INF).all()
    scaled = np.abs(z) * 2.0 ** (14 - np.floor(np.log2(np.abs(x).max(1))))[:, None]
    assert (scaled > most)[holds].mean() > 0.1                  # with each query's largest element in [2^14, 2^15)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("L,d,B", [(80_003, 128, 8), (75_776, 192, 1), (76_001, 256, 5)])
def test_scores_with_two_label_blocks_a_warp(group, L, d, B):
    """Few queries and labels for every SM twice over: all labels of the last, partial tiles among the others."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    if d % group:
        d += 64
    rng = np.random.default_rng(L + group)
    u = rng.integers(0, 16, (L, d)).astype(np.uint8)
    s = q4_ops.bf16_of(np.abs(rng.normal(0, 0.01, (L, d // group))))
    x = q4_ops.bf16_of(rng.normal(0, 1, (B, d)))
    Z = torch.full((B, L + 1), 123.0, device="cuda")
    elmo.elmo_q4_scores(torch.from_numpy(q4_ops.nibbles(u)).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(),
                        torch.from_numpy(x).to(torch.bfloat16).cuda(), Z[:, :L])
    z, mag = q4_ops.scored(u, s, x, group)
    got = Z.double().cpu().numpy()
    assert (got[:, L:] == 123.0).all()
    assert (np.abs(got[:, :L] - z) <= q4_ops.tolerance(d, group) * mag + np.abs(z) * 2.0**-24).all()
