"""Log probabilities of labels straight from the head, against the definition in 64 bits; and the operators together:
a 4-bit copy, its scores, their statistics and gradient."""
import numpy as np
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

GRIDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
E = 2.0**-24


def head_of(elmo, w, grid):
    W = torch.from_numpy(np.asarray(w, dtype=np.float32)).to(GRIDS[grid]).cuda()
    return W, elmo.elmo_init_head(W, grid)


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).cuda()


def lists(rng, B, L, lam):
    rowptr = np.zeros(B + 1, np.int32)
    rowptr[1:] = np.cumsum(rng.poisson(lam, B))
    return rowptr, rng.integers(0, L, rowptr[-1]).astype(np.int32)


def buffers(B, nnz, k):
    return (torch.full((nnz,), 5.0, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda"),
            torch.full((B, k), -7, dtype=torch.int32, device="cuda"), torch.empty(B, k, device="cuda"))


def run(elmo, h, X, rowptr, cols, k, stream=None):
    out = buffers(X.shape[0], len(cols), k)
    elmo.elmo_label_logprobs(h, X, torch.from_numpy(rowptr).cuda(), torch.from_numpy(cols).cuda(), *out, stream)
    elmo.elmo_sync_status(h)
    return [o.cpu().numpy() for o in out]


def slack(x, w, p, d, grid):
    """How far lse and entropy of a query may be off: its tensor-core scores (2^-22 of the magnitudes summed an
    instruction; in 8-bit heads also what two 8-bit numbers leave of x, 2^-14 of at least 224 after scaling, so at most
    2^-21 of the query's largest magnitude an element), then the fp32 sums: a term's 2.5 |d| E and 2^-22, chains of 8 and 2 additions, two per tile of a range
    (each may rescale), the ranges joined in 64 bits."""
    fp8 = grid != "bf16"
    steps = (2 if fp8 else 1) * -(-x.size * (1 if fp8 else 2) // 128) * 4
    mag = np.abs(w) @ np.abs(x)
    dz = (steps * 2.0**-22 * mag + (2.0**-21 * np.abs(x).max() * np.abs(w).sum(1) if fp8 else 0)).max()
    nt = 2 * (-(-w.shape[0] // 64) // 100 + 2)               # at least 100 ranges where there are as many tiles
    D, D2, R = -(p * d).sum(), (p * d * d).sum(), min(200.0, -d.min())
    chain = 2.0**-22 * (2 + nt) + (12 + 2 * nt) * E + 5 * R * E
    es = 2.5 * D * E + chain
    # lse moves by at most dz; H = lse - E[z] by at most dz (1 + 1) + |cov| <= 2 dz (1 + D')
    spread = np.sqrt(max(0.0, D2 - D * D))
    return es + dz, es * (1 + D) + 2.5 * D2 * E + D * (chain + 3 * E) + 2 * dz * (1 + spread)


def check(got, x, w, grid, rowptr, cols, k):
    logp, lse, H, idx, top = (g.astype(np.float64) for g in got)
    for b in range(x.shape[0]):
        z = w @ x[b]
        m = z.max()
        d = z - m
        p = np.exp(d)
        s = p.sum()
        p /= s
        on = p > 0
        es, eH = slack(x[b], w, p[on], d[on], grid)
        want = m + np.log(s)
        assert abs(lse[b] - want) <= es + E * abs(want), (b, lse[b] - want, es)
        wH = np.log(s) - (p[on] * d[on]).sum()
        assert abs(H[b] - wH) <= eH + E * wH, (b, H[b] - wH, eH)
        at = z[cols[rowptr[b]:rowptr[b + 1]]] - m - np.log(s)
        assert (np.abs(logp[rowptr[b]:rowptr[b + 1]] - at) <= es + E * np.abs(at)).all(), b
        best = np.lexsort((np.arange(len(z)), -z))[:k]
        assert np.array_equal(idx[b], best), (b, idx[b], best, z[best], z[idx[b].astype(int)])
        assert (np.abs(top[b] - (d[best] - np.log(s))) <= es + E * np.abs(d[best] - np.log(s))).all(), b


@pytest.mark.parametrize("grid,L,d,B,k,lam", [
    ("bf16", 1, 64, 1, 1, 1), ("e4m3", 63, 64, 3, 5, 4), ("e5m2", 1000, 128, 130, 10, 2), ("bf16", 4099, 768, 33, 64, 5),
    ("e4m3", 20_011, 768, 257, 5, 9), ("e4m3", 5000, 704, 5, 16, 0), ("bf16", 3000, 1024, 40, 5, 3),
    ("e4m3", 3001, 4096, 130, 64, 1), ("e5m2", 700, 832, 2, 64, 2), ("e4m3", 60_000, 320, 1, 1, 50),
    ("bf16", 16_384, 64, 20, 64, 3), ("e4m3", 16_385, 64, 20, 64, 3), ("bf16", 60_001, 192, 4, 0, 3), ("e5m2", 20_000, 768, 128, 6, 1), ("bf16", 129, 4096, 7, 9, 2)])
def test_matches_64_bits(grid, L, d, B, k, lam):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + d + B)
    W, h = head_of(elmo, rng.normal(0, 0.02, (L, d)), grid)
    X = bf16(rng.normal(0, 1, (B, d)) * 2.0 ** rng.integers(-3, 4, (B, 1)))
    rowptr, cols = lists(rng, B, L, lam)
    got = run(elmo, h, X, rowptr, cols, k)
    check(got, X.double().cpu().numpy(), W.double().cpu().numpy(), grid, rowptr, cols, k)
    again = run(elmo, h, X, rowptr, cols, k)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))
    h.close()


@pytest.mark.parametrize("grid", list(GRIDS))
@pytest.mark.parametrize("d", [256, 896])
def test_odd_queries(grid, d):
    """Zero queries, outliers, mixed, tiny and large magnitudes."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(d)
    L, B, k = 3000, 7, 5
    W, h = head_of(elmo, rng.normal(0, 0.02, (L, d)), grid)
    x = rng.normal(0, 1, (B, d))
    x[0] = 0
    x[1, 5] = 300.0                                             # one coordinate far above the others
    x[2] *= 2.0 ** rng.integers(-12, 1, d)
    x[3] *= 2.0**-90
    x[4] = np.where(np.arange(d) == 9, 1, 0)
    x[5] *= 100
    X = bf16(x)
    rowptr, cols = lists(rng, B, L, 5)
    check(run(elmo, h, X, rowptr, cols, k), X.double().cpu().numpy(), W.double().cpu().numpy(), grid, rowptr, cols, k)
    h.close()


@pytest.mark.parametrize("grid,L,d", [("e4m3", 300_001, 128), ("bf16", 3001, 832), ("e5m2", 40_000, 64)])
def test_padded_batches(grid, L, d):
    """Queries of zeros among the others, and queries that belong to nobody's list."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L)
    B, k = 130, 7
    W, h = head_of(elmo, rng.normal(0, 0.02, (L, d)), grid)
    x = rng.normal(0, 1, (B, d))
    x[5:], x[129] = 0, x[0]
    X = bf16(x)
    rowptr = np.concatenate([np.arange(6), np.full(B - 5, 5)]).astype(np.int32)
    cols = rng.integers(0, L, 5).astype(np.int32)
    got = run(elmo, h, X, rowptr, cols, k)
    keep = [0, 1, 4, 5, 77, 129]
    xs, w = X.double().cpu().numpy()[keep], W.double().cpu().numpy()
    ptr = np.array([0, 1, 2, 3, 3, 3, 3], np.int32)
    check([got[0][[0, 1, 4]], *(g[keep] for g in got[1:])], xs, w, grid, ptr, cols[[0, 1, 4]], k)
    assert (got[3][5:129] == np.arange(k)).all()
    h.close()


@pytest.mark.parametrize("grid", ["bf16", "e4m3"])
def test_scores_of_any_size(grid):
    """Scores of 1e30 and more, all of one sign: nothing but them counts, however few labels the last tile has."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(3)
    for L in (65, 5000):
        w = np.abs(rng.normal(0, 0.02, (L, 128))) + 0.02
        W, h = head_of(elmo, w, grid)
        X = bf16(np.array([[-1.0], [1.0]]) * (np.abs(rng.normal(0, 1, (2, 128))) + 0.5) * 2.0**110)
        rowptr, cols = np.array([0, 1, 2], np.int32), np.array([3, L - 1], np.int32)
        logp, lse, H, idx, top = run(elmo, h, X, rowptr, cols, 3)
        z = X.double().cpu().numpy() @ W.double().cpu().numpy().T
        assert np.array_equal(idx, np.argsort(-z, 1, kind="stable")[:, :3])
        assert np.abs(lse / z.max(1) - 1).max() < 1e-5 and (H == 0).all()
        assert np.array_equal(top[:, 0] == 0, [True, True]) or np.abs(top[:, 0] / z.max(1)).max() < 1e-5
        h.close()


@pytest.mark.parametrize("kind", ["zeros", "few values", "best repeated", "two apart"])
@pytest.mark.parametrize("grid,d", [("e4m3", 128), ("bf16", 832)])
def test_ties_go_to_the_lower_label(grid, d, kind):
    """Heads whose best scores tie: more ties than a range keeps, and pairs that fp32 sums cannot tell apart."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(7)
    L, B, k = 9000, 3, 10
    w = rng.normal(0, 0.02, (L, d))
    x = rng.normal(0, 1, (B, d))
    if kind == "zeros":
        w[:] = 0
    elif kind == "few values":
        w = rng.integers(-1, 2, (L, 1)) * 0.125 * np.ones((1, d))
    else:
        x[:] = np.abs(x)
        w[rng.permutation(L)[:200]] = 0.25
        if kind == "two apart":                                 # one element one step up: about 2^-13 of the score
            w[5000, 0] = 0.28125
    W, h = head_of(elmo, w, grid)
    X = bf16(x)
    rowptr, cols = lists(rng, B, L, 2)
    check(run(elmo, h, X, rowptr, cols, k), X.double().cpu().numpy(), W.double().cpu().numpy(), grid, rowptr, cols, k)
    h.close()


@pytest.mark.parametrize("grid", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("L,B,k", [(32767, 3, 1), (32768, 3, 1), (32771, 1, 1), (65537, 2, 2), (65537, 4, 2), (66000, 1, 2)])
def test_all_labels_tied_but_one(grid, L, B, k):
    """Every list comes from the exact path, with many label segments a query and with few: labels that all tie, and one
    above them that lies in a segment's last place, in the head's, or is the lowest."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + B)
    d = 128
    x = np.abs(rng.normal(0, 1, (B, d))) + 0.1
    for above in (None, 0, L * 5 // 296 - 1, L - 1):
        w = np.full((L, d), 0.5)
        if above is not None:
            w[above] = 0.5625                                   # one step of E4M3 above
            if grid == "e5m2":
                w[above] = 0.625
        W, h = head_of(elmo, w, grid)
        logp, lse, H, idx, top = run(elmo, h, bf16(x), np.zeros(B + 1, np.int32), np.zeros(0, np.int32), k)
        want = ([] if above is None else [above]) + [i for i in range(k + 1) if i != above]
        assert (idx == np.array(want[:k])).all(), (above, idx)
        h.close()


@pytest.mark.parametrize("d", [128, 832])
def test_values_that_are_not_finite(d):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(11)
    L, B = 2000, 4
    w = rng.normal(0, 0.02, (L, d))
    x = np.abs(rng.normal(0, 1, (B, d))) + 0.1
    rowptr, cols = np.array([0, 2, 4, 6, 8], np.int32), np.array([7, 1, 7, 2, 7, 3, 7, 4], np.int32)
    # a query with NaN, one with infinity: theirs alone are NaN and empty
    bad = x.copy()
    bad[1, 3], bad[2, 4] = np.nan, np.inf
    W, h = head_of(elmo, w, "bf16")
    logp, lse, H, idx, top = run(elmo, h, bf16(bad), rowptr, cols, 3)
    assert np.isnan(lse[1:3]).all() and np.isnan(H[1:3]).all() and np.isnan(logp[2:6]).all()
    assert (idx[1:3] == -1).all() and (top[1:3] == -np.inf).all()
    good = run(elmo, h, bf16(x), rowptr, cols, 3)
    for a, b, n in zip((logp, lse, H, idx, top), good, (2, 1, 1, 1, 1)):
        assert np.array_equal(a[:n], b[:n]) and np.array_equal(a[-n:], b[-n:])
    h.close()
    # a label of -infinity is masked, one of +infinity takes all, one of NaN spoils the sums but not the order
    for value, where in ((-np.inf, "masked"), (np.inf, "all"), (np.nan, "nan")):
        ww = w.copy()
        ww[7, 0] = value
        W, h = head_of(elmo, ww, "bf16")
        logp, lse, H, idx, top = run(elmo, h, bf16(x), rowptr, cols, 3)
        z = bf16(x).double().cpu().numpy() @ bf16(w).double().cpu().numpy().T
        z[:, 7] = -np.inf
        best = np.argsort(-z, 1, kind="stable")[:, :3]
        if where == "masked":
            assert np.array_equal(idx, best) and (logp[::2] == -np.inf).all()
            m = z.max(1)
            want = m + np.log(np.exp(z - m[:, None]).sum(1))
            assert np.abs(lse - want).max() < 1e-4 and np.isfinite(H).all() and np.isfinite(top).all()
        elif where == "all":
            assert (lse == np.inf).all() and np.isnan(H).all() and (idx[:, 0] == 7).all()
            assert np.array_equal(idx[:, 1:], best[:, :2]) and (logp[1::2] == -np.inf).all() and np.isnan(logp[::2]).all()
        else:
            assert np.isnan(lse).all() and np.isnan(H).all() and np.isnan(logp).all() and np.array_equal(idx, best)
        h.close()


def test_labels_out_of_range_set_the_status():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(1)
    W, h = head_of(elmo, rng.normal(0, 0.02, (300, 64)), "e4m3")
    X = bf16(rng.normal(0, 1, (2, 64)))
    out = buffers(2, 4, 2)
    rp, cs = torch.tensor([0, 2, 4], dtype=torch.int32).cuda(), torch.tensor([299, 300, 3, 0], dtype=torch.int32).cuda()
    elmo.elmo_label_logprobs(h, X, rp, cs, *out)
    with pytest.raises(elmo.ElmoError) as e:
        elmo.elmo_sync_status(h)
    assert e.value.status == 6 and "entry 1" in str(e.value)
    assert out[0].isnan().tolist() == [False, True, False, False]
    for bad in ([-3, 2, 1], [4, 2, 2**31 - 1]):
        elmo.elmo_label_logprobs(h, X, torch.tensor(bad, dtype=torch.int32).cuda(), cs % 300, *out)
        elmo.elmo_sync_status(h)
    h.close()


@pytest.mark.parametrize("grid,L,d,B", [("e4m3", 1_000_003, 768, 300), ("bf16", 400_000, 768, 5), ("e5m2", 300_001, 1024, 20)])
def test_large_heads(grid, L, d, B):
    """Whole ranges of a real head, against 64-bit products on the device; agreement with the top-k prediction."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    g = torch.Generator(device="cuda").manual_seed(3)
    W = (torch.randn(L, d, generator=g, device="cuda") * 0.02).to(GRIDS[grid])
    X = torch.randn(B, d, generator=g, device="cuda").to(torch.bfloat16)
    rng = np.random.default_rng(8)
    rowptr, cols = lists(rng, B, L, 9)
    h = elmo.elmo_init_head(W, grid)
    k = 10
    logp, lse, H, idx, top = run(elmo, h, X, rowptr, cols, k)
    Z = torch.cat([X.double() @ W[a:a + 50_000].double().T for a in range(0, L, 50_000)], 1)
    want = torch.logsumexp(Z, 1)
    p = torch.exp(Z - want[:, None])
    wH = -(p * (Z - want[:, None])).sum(1)
    # scores within 2^-22 of the magnitudes an instruction, as in slack(); sums well inside
    steps = (1 if grid == "bf16" else 2) * -(-d * (2 if grid == "bf16" else 1) // 128) * 4
    dz = steps * 2.0**-22 * float((X.double().abs() @ W[:2000].double().abs().T).max()) * 1.2
    assert np.abs(lse - want.cpu().numpy()).max() < dz + 2e-5
    assert np.abs(H - wH.cpu().numpy()).max() < 4 * dz + 1e-4
    wt, wi = torch.topk(Z, k, 1)
    assert np.array_equal(idx, wi.int().cpu().numpy())
    assert np.abs(top - (wt - want[:, None]).cpu().numpy()).max() < dz + 2e-5
    row = torch.from_numpy(np.repeat(np.arange(B), np.diff(rowptr))).cuda()
    at = Z[row, torch.from_numpy(cols).long().cuda()] - want[row]
    assert np.abs(logp - at.cpu().numpy()).max() < dz + 2e-5
    ti, ts = torch.empty(B, k, dtype=torch.int32, device="cuda"), torch.empty(B, k, device="cuda")
    elmo.elmo_topk_predict(h, X, k, 131072, ti, ts)
    assert (ti.cpu().numpy() == idx).mean() > 0.999             # apart from scores that fp32 cannot tell apart
    h.close()


def test_captured_then_the_workspace_grows():
    """A captured call replays correctly after a larger call on the same head has taken a larger workspace."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(12)
    W, h = head_of(elmo, rng.normal(0, 0.02, (5000, 128)), "e4m3")
    X, big = bf16(rng.normal(0, 1, (3, 128))), bf16(rng.normal(0, 1, (600, 128)))
    rowptr, cols = lists(rng, 3, 5000, 4)
    rp, cs = torch.from_numpy(rowptr).cuda(), torch.from_numpy(cols).cuda()
    out = buffers(3, len(cols), 5)
    elmo.elmo_label_logprobs(h, X, rp, cs, *out)
    torch.cuda.synchronize()
    first = [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        elmo.elmo_label_logprobs(h, X, rp, cs, *out)
    held = elmo.elmo_head_workspace_bytes(h)
    run(elmo, h, big, np.zeros(601, np.int32), np.zeros(0, np.int32), 64)
    assert elmo.elmo_head_workspace_bytes(h) > held
    fill = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device="cuda")   # what a freed buffer's place would hold
    for _ in range(2):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    side = torch.cuda.Stream()
    for o in out:
        o.zero_()
    torch.cuda.synchronize()
    elmo.elmo_label_logprobs(h, X, rp, cs, *out, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    del graph, fill
    h.close()


def test_leaves_the_prediction_as_it_was():
    """The top-k prediction's own counters and results survive a call in between."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(13)
    W, h = head_of(elmo, np.zeros((4000, 128)), "e4m3")           # every row ties: none is certified
    X = bf16(rng.normal(0, 1, (5, 128)))
    idx, sc = torch.empty(5, 3, dtype=torch.int32, device="cuda"), torch.empty(5, 3, device="cuda")
    elmo.elmo_topk_predict(h, X, 3, 4000, idx, sc)
    before = elmo.elmo_topk_uncertified_rows(h, 5, 3)
    n = elmo.elmo_launch_count(h)
    run(elmo, h, X, np.zeros(6, np.int32), np.zeros(0, np.int32), 3)
    assert elmo.elmo_launch_count(h) == n + 4                   # operands, scores, join, exact path
    assert elmo.elmo_topk_uncertified_rows(h, 5, 3) == before == 5
    h.close()


def test_refusals():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    W, h = head_of(elmo, np.zeros((100, 64)), "e4m3")
    X, rp, cs = bf16(np.zeros((2, 64))), torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(4, dtype=torch.int32).cuda()
    out = buffers(2, 4, 2)
    elmo.elmo_label_logprobs(h, X, rp, cs, *out)
    for bad in [(bf16(np.zeros((2, 128))), rp, cs), (X.float(), rp, cs), (X, rp[:2], cs), (X, rp, cs.long()),
                (X, rp, cs[:3]), (X.cpu(), rp, cs)]:
        with pytest.raises((ValueError, TypeError)):
            elmo.elmo_label_logprobs(h, *bad, *out)
    with pytest.raises(elmo.ElmoError, match="k = 65"):
        elmo.elmo_label_logprobs(h, X, rp, cs, *buffers(2, 4, 65))
    part = elmo.elmo_init_head_shard(W, 128, 500, "e4m3")
    with pytest.raises(elmo.ElmoError) as e:
        elmo.elmo_label_logprobs(part, X, rp, cs, *out)
    assert e.value.status == 5
    part.close()
    h.close()


@pytest.mark.parametrize("grid", list(GRIDS))
def test_the_operators_together(grid):
    """Serving from a 4-bit copy: pack, scores, statistics, gradient; the same statistics straight from a head of what
    the copy stands for."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(21)
    L, d, B, k, group = 7003, 768, 6, 10, 64
    W, full = head_of(elmo, rng.normal(0, 0.02, (L, d)), grid)
    X = bf16(rng.normal(0, 1, (B, d)))
    rowptr, cols = lists(rng, B, L, 6)
    codes = torch.empty(L, d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(L, d // group, dtype=torch.bfloat16, device="cuda")
    # scales that are powers of two: the copy's values are bf16 numbers, so that a bf16 head holds it exactly
    elmo.elmo_q4_pack(W, grid, group, codes, scales)
    scales.copy_(torch.exp2(torch.floor(torch.log2(scales.float()))))
    back = torch.empty(L, d, dtype=torch.bfloat16, device="cuda")
    elmo.elmo_q4_unpack(codes, scales, back)
    Z = torch.empty(B, L, device="cuda")
    elmo.elmo_q4_scores(codes, scales, X, Z)
    up = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    a, b = buffers(B, len(cols), k), buffers(B, len(cols), k)
    work = torch.empty(elmo.elmo_score_logprobs_workspace_bytes(B, L, k), dtype=torch.uint8, device="cuda")
    elmo.elmo_score_logprobs(Z, up(rowptr), up(cols), *a, work)
    h = elmo.elmo_init_head(back, "bf16")
    elmo.elmo_label_logprobs(h, X, up(rowptr), up(cols), *b)
    elmo.elmo_sync_status(h)
    x, w = X.double().cpu().numpy(), back.double().cpu().numpy()
    check([t.cpu().numpy() for t in b], x, w, "bf16", rowptr, cols, k)
    for s, t, name in zip(a, b, ("logp", "lse", "entropy", "idx", "top")):
        if name == "idx":
            assert (s == t).float().mean() > 0.98               # apart from scores that fp32 cannot tell apart
        else:
            assert (s - t).abs().max() < 2e-4, name             # 48 instructions of 2^-22 of about 10, twice
    g = torch.ones(len(cols), device="cuda") / B
    dZ = torch.empty_like(Z)
    elmo.elmo_score_logprobs_backward(Z, up(rowptr), up(cols), a[1], a[2], g, None, None, dZ)
    z = x @ w.T
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want = -p * (np.diff(rowptr) / B)[:, None]
    np.add.at(want, (np.repeat(np.arange(B), np.diff(rowptr)), cols), 1 / B)
    assert np.abs(dZ.cpu().numpy() - want).max() < 1e-5
    h.close()
    full.close()
