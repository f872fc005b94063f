"""Log probabilities of labels from rows of scores, and their gradient, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
E = 2.0**-24                      # half a step of fp32, relative


def lists(rng, B, L, lam):
    counts = rng.poisson(lam, B)
    rowptr = np.zeros(B + 1, np.int32)
    rowptr[1:] = np.cumsum(counts)
    return rowptr, rng.integers(0, L, rowptr[-1]).astype(np.int32)


def on_gpu(z, dtype, pad=0, start=0):
    """Scores with rows `pad` elements apart, the first `start` elements past an allocation's start; nan around them."""
    B, L = z.shape
    buf = torch.full((start + B * (L + pad) + 64,), float("nan"), dtype=TYPES[dtype], device="cuda")
    Z = torch.as_strided(buf, (B, L), (L + pad, 1), start)
    Z.copy_(torch.from_numpy(z.astype(np.float32)))
    return Z


def scored(elmo, Z, rowptr, cols, k, stream=None):
    B, L = Z.shape
    out = (torch.full((len(cols),), 55.0, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda"),
           torch.full((B, k), -7, dtype=torch.int32, device="cuda"), torch.empty(B, k, device="cuda"))
    work = torch.full((elmo.elmo_score_logprobs_workspace_bytes(B, L, k),), 0xFF, dtype=torch.uint8, device="cuda")
    elmo.elmo_score_logprobs(Z, torch.from_numpy(rowptr).cuda(), torch.from_numpy(cols).cuda(), *out, work, stream)
    return [o.cpu().numpy() for o in out]


def expected(z, rowptr, cols, k):
    """The definition in 64 bits, and how far off fp32 sums of a row may be (see slack)."""
    B, L = z.shape
    z = z.astype(np.float64)
    lse, H, slack_s, slack_H, most, logs = (np.zeros(B) for _ in range(6))   # log p = (z - most) - logs
    idx, top = np.full((B, k), -1, np.int32), np.full((B, k), -np.inf)
    for b in range(B):
        m = z[b].max()
        if m == -np.inf:
            lse[b] = -np.inf
        else:
            d = z[b] - m
            p = np.exp(d)
            s = p.sum()
            p /= s
            on = p > 0
            lse[b], most[b], logs[b] = m + np.log(s), m, np.log(s)
            H[b] = np.log(s) - (p[on] * d[on]).sum()
            slack_s[b], slack_H[b] = slack(p[on], d[on], L)
        order = np.lexsort((np.arange(L), -z[b]))[:k]
        order = order[z[b][order] > -np.inf]
        idx[b, :len(order)] = order
        top[b, :len(order)] = z[b][order] - most[b] - logs[b]
    row = np.repeat(np.arange(B), np.diff(rowptr))
    at = z[row, cols]
    logp = np.where(at == -np.inf, -np.inf, at - most[row] - logs[row])
    return logp, lse, H, idx, top, slack_s, slack_H, row


def slack(p, d, L):
    """Bounds on the errors of log s and H from the kernel's fp32 arithmetic.  A term e^d carries the rounding of d, of
    d log2(e) and of that constant (2.5 |d| E) and 2^-22 of ex2; a thread's sums are chains of 8 additions, 2 more, one
    per block of its warp (nb, each also a rescaling by such a term if the maximum moved: the moves add up to at most the
    range of d), 5 across lanes, 8 across warps (rescaled once more).  t's terms have one rounding more."""
    nb = -(-L // 8192) + 1
    D, D2, R = -(p * d).sum(), (p * d * d).sum(), min(200.0, -d.min())
    chain = 2.0**-22 * (2 + nb) + (25 + 2 * nb) * E + 5 * R * E
    es = 2.5 * D * E + chain
    return es, es * (1 + D) + 2.5 * D2 * E + D * (chain + 3 * E)


def check(got, z, rowptr, cols, k):
    logp, lse, H, idx, top, es, eH, row = expected(z, rowptr, cols, k)
    g_logp, g_lse, g_H, g_idx, g_top = got
    near = lambda a, b, tol: np.array_equal(np.isinf(a), np.isinf(b)) and np.all(   # noqa: E731
        (a == b) | (np.abs(np.where(np.isinf(a), 0, a.astype(np.float64)) - np.where(np.isinf(b), 0, b)) <= tol))
    assert near(g_lse, lse, es + E * np.where(np.isinf(lse), 0, np.abs(lse)))
    assert near(g_H, H, eH + E * H)
    assert near(g_logp, logp, es[row] + E * np.where(np.isinf(logp), 0, np.abs(logp)))
    assert np.array_equal(g_idx, idx)
    assert near(g_top, top, es[:, None] + E * np.where(np.isinf(top), 0, np.abs(top)))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,L,pad,start,k,lam", [
    (1, 1, 0, 0, 1, 1), (3, 2, 1, 3, 2, 2), (5, 7, 0, 1, 7, 1), (2, 64, 0, 0, 64, 0), (4, 1023, 2, 5, 5, 3),
    (2, 1024, 0, 0, 64, 9), (9, 1025, 7, 7, 10, 2), (33, 4099, 2, 0, 64, 5), (2, 33_000, 0, 0, 5, 40),
    (1, 33_001, 0, 1, 1, 300), (70, 40_007, 1, 2, 64, 3), (700, 33_800, 0, 0, 3, 1), (2, 200_003, 6, 0, 0, 2)])
def test_scores_match_64_bits(dtype, B, L, pad, start, k, lam):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + B)
    Z = on_gpu(rng.normal(0, 3, (B, L)), dtype, pad, start)
    rowptr, cols = lists(rng, B, L, lam)
    check(scored(elmo, Z, rowptr, cols, k), Z.float().cpu().numpy(), rowptr, cols, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("L", [3000, 50_000, 400_000])
@pytest.mark.parametrize("kind", ["equal", "steps", "up", "down", "blocks", "masked", "nearly", "lowest", "zeros"])
def test_orders_ties_and_masks(dtype, L, kind):
    """Rows made to be awkward for the selection and for the running maximum."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L)
    B = 3
    z = {"equal": lambda: np.full((B, L), 1.5),
         "steps": lambda: rng.integers(0, 4, (B, L)).astype(float),
         "up": lambda: np.sort(rng.normal(0, 20, (B, L)), 1),
         "down": lambda: -np.sort(rng.normal(0, 20, (B, L)), 1),
         "blocks": lambda: np.repeat(rng.normal(0, 5, (B, -(-L // 100))), 100, 1)[:, :L],     # runs of equal scores
         "masked": lambda: np.where(rng.random((B, L)) < 0.9, -np.inf, rng.normal(0, 3, (B, L))),
         "nearly": lambda: np.where(np.arange(L) % 1700 == 1699, rng.normal(0, 3, (B, L)), -np.inf),
         "lowest": lambda: np.where(rng.random((B, L)) < 0.5, -3.3e38, rng.normal(0, 3, (B, L))),
         "zeros": lambda: np.where(rng.random((B, L)) < 0.5, -0.0, 0.0)}[kind]()
    z[1] = {"masked": -np.inf, "lowest": -3.3e38}.get(kind, z[1])
    Z = on_gpu(z, dtype, 1)
    rowptr, cols = lists(rng, B, L, 5)
    for k in (1, 5, 64):
        check(scored(elmo, Z, rowptr, cols, k), Z.float().cpu().numpy(), rowptr, cols, k)


@pytest.mark.parametrize("L", [100, 40_000])
def test_rows_with_nan_and_infinity(L):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L)
    z = rng.normal(0, 3, (5, L)).astype(np.float32)
    z[0, 17], z[1, 18], z[2, :], z[3, 20] = np.nan, np.inf, np.nan, -np.inf
    rowptr = np.array([0, 2, 4, 5, 7, 8], np.int32)
    cols = np.array([17, 3, 18, 3, 0, 20, 3, 3], np.int32)
    logp, lse, H, idx, top = scored(elmo, on_gpu(z, "fp32"), rowptr, cols, 5)
    assert np.isnan(lse[[0, 2]]).all() and lse[1] == np.inf and np.isfinite(lse[[3, 4]]).all()
    assert np.isnan(H[:3]).all() and np.isfinite(H[3:]).all()
    assert np.isnan(logp[[0, 1, 2, 4]]).all() and logp[3] == -np.inf and logp[5] == -np.inf and np.isfinite(logp[6:]).all()
    best = np.argsort(-np.where(np.isnan(z), -np.inf, z), 1, kind="stable")[:, :5]
    assert np.array_equal(idx[[0, 1, 3, 4]], best[[0, 1, 3, 4]]) and (idx[2] == -1).all()
    assert np.isnan(top[0]).all() and np.isnan(top[1, 0]) and (top[1, 1:] == -np.inf).all()
    check([logp[5:], lse[3:], H[3:], idx[3:], top[3:]], z[3:], np.array([0, 2, 3], np.int32), cols[5:], 5)


def test_given_labels_out_of_range_and_bad_row_pointers():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(0)
    z = rng.normal(0, 1, (3, 500)).astype(np.float32)
    cols = np.array([499, 500, -1, 2**31 - 1, 7, 7], np.int32)
    logp, lse, H, idx, top = scored(elmo, on_gpu(z, "fp32"), np.array([0, 5, 5, 6], np.int32), cols, 2)
    assert np.isnan(logp[1:4]).all() and np.isfinite(logp[[0, 4, 5]]).all()
    for bad in ([-3, 2, 1, 99], [9, 8, 7, 6], [0, 2**31 - 1, -2**31, 2]):
        logp = scored(elmo, on_gpu(z, "fp32"), np.array(bad, np.int32), cols, 2)[0]
        assert len(logp) == 6                                    # entries of no row are left, nothing else is touched


def test_long_matrices_take_64_bit_offsets():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(4)
    B, L, pitch = 3, 70_001, 1_300_000_001
    buf = torch.empty(2 * pitch + L, dtype=torch.bfloat16, device="cuda")
    Z = torch.as_strided(buf, (B, L), (pitch, 1))
    Z.copy_(torch.from_numpy(rng.normal(0, 3, (B, L)).astype(np.float32)))
    z = Z.float().cpu().numpy()
    rowptr, cols = lists(rng, B, L, 6)
    got = scored(elmo, Z, rowptr, cols, 7)
    check(got, z, rowptr, cols, 7)
    g = torch.ones(len(cols), device="cuda")
    elmo.elmo_score_logprobs_backward(Z, torch.from_numpy(rowptr).cuda(), torch.from_numpy(cols).cuda(),
                                      torch.from_numpy(got[1]).cuda(), None, g, None, None, Z)
    check_grad(Z.float().cpu().numpy(), z, rowptr, cols, got[1], None, np.ones(len(cols)), None, None, "bf16")


# ---------------------------------------------------------------- the gradient
def expected_grad(z, rowptr, cols, lse, H, g, gl, gH):
    """The formula in 64 bits at the given lse and H, and the error that fp32 arithmetic may make."""
    B, L = z.shape
    out, tol = np.zeros((B, L)), np.zeros((B, L))
    for b in range(B):
        if np.isinf(lse[b]):
            continue
        c, gi = cols[rowptr[b]:rowptr[b + 1]], g[rowptr[b]:rowptr[b + 1]].astype(np.float64)
        ok = (c >= 0) & (c < L)
        c, gi = c[ok], gi[ok]
        d = np.maximum(z[b].astype(np.float64) - lse[b], -200)
        p = np.exp(d)
        cH, h = (float(gH[b]), float(H[b])) if gH is not None else (0.0, 0.0)
        c0 = (float(gl[b]) if gl is not None else 0.0) - gi.sum()
        out[b] = p * (c0 - cH * (d + h))
        # p: 2.5 |d| E and 2^-22; the factor: c0 - cH h rounded once, the fma and d's rounding; the product
        tol[b] = p * ((2.5 * np.abs(d) * E + 2.0**-22 + 2 * E) * np.abs(c0 - cH * (d + h))
                      + 2 * E * (np.abs(c0) + np.abs(cH * h) + np.abs(cH * d)))
        np.add.at(out[b], c, gi)
        mag = np.zeros(L)
        np.add.at(mag, c, np.abs(gi))
        n = np.zeros(L)
        np.add.at(n, c, 1)
        tol[b] += (n + 1) * E * (mag + np.abs(out[b]))
    return out, tol + 2.0**-126


def check_grad(got, z, rowptr, cols, lse, H, g, gl, gH, dtype):
    want, tol = expected_grad(z, rowptr, cols, lse, H, g, gl, gH)
    step = E if dtype == "fp32" else 2.0**-8
    assert (np.abs(got - want) <= tol * 1.01 + step * np.abs(want)).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,L,pad,dpad,start,lam,place", [
    (1, 1, 0, 0, 0, 1, False), (3, 7, 1, 1, 1, 4, True), (5, 1025, 2, 0, 3, 30, False), (2, 4096, 0, 0, 0, 3, True),
    (33, 4099, 2, 5, 1, 5, False), (4, 40_011, 8, 8, 0, 600, True), (2, 300, 0, 0, 0, 3000, False)])
def test_gradient_matches_the_formula(dtype, B, L, pad, dpad, start, lam, place):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(B + L)
    z = rng.normal(0, 3, (B, L))
    if B > 2:
        z[rng.random((B, L)) < 0.3] = -np.inf
        z[1] = -np.inf
    Z = on_gpu(z, dtype, pad, start)
    z = Z.float().cpu().numpy()
    rowptr, cols = lists(rng, B, L, lam)
    if B > 2:
        cols[::7] = L + 3
    g, gl, gH = (rng.normal(0, 1, n).astype(np.float32) for n in (len(cols), B, B))
    lse, H = scored(elmo, Z, rowptr, np.clip(cols, 0, L - 1), 0)[1:3]
    up = lambda a: None if a is None else torch.from_numpy(a).cuda()   # noqa: E731
    for grads in ((g, gl, gH), (g, None, None), (None, gl, None), (None, None, gH)):
        Zi = on_gpu(z, dtype, pad, start)
        dZ = Zi if place else on_gpu(np.zeros((B, L)), dtype, dpad, 2)
        elmo.elmo_score_logprobs_backward(Zi, up(rowptr), up(cols), up(lse), up(H), *(up(a) for a in grads), dZ)
        check_grad(dZ.double().cpu().numpy(), z, rowptr, cols, lse, H, g if grads[0] is not None else 0 * g, grads[1],
                   grads[2], dtype)
        whole = dZ.untyped_storage()
        whole = torch.tensor([], dtype=Z.dtype, device="cuda").set_(whole)
        assert whole.isnan().sum() == whole.numel() - B * L       # what lies between the rows is left as it was


def test_gradient_matches_differences():
    """d/dz of a weighted sum of the operator's own outputs, by central differences in 64 bits."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(9)
    B, L = 2, 37
    z = rng.normal(0, 2, (B, L)).astype(np.float32)
    rowptr, cols = np.array([0, 3, 5], np.int32), np.array([4, 4, 36, 0, 12], np.int32)
    g, gl, gH = (rng.normal(0, 1, n).astype(np.float32) for n in (5, B, B))

    def value(zz):
        logp, lse, H = expected(zz, rowptr, cols, 0)[:3]
        return (logp * g).sum() + (lse * gl).sum() + (H * gH).sum()

    lse, H = scored(elmo, on_gpu(z, "fp32"), rowptr, cols, 0)[1:3]
    up = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    dZ = torch.empty(B, L, device="cuda")
    elmo.elmo_score_logprobs_backward(up(z), up(rowptr), up(cols), up(lse), up(H), up(g), up(gl), up(gH), dZ)
    h = 1e-5
    for b in range(B):
        for l in range(L):
            zp, zm = z.astype(np.float64), z.astype(np.float64)
            zp[b, l] += h
            zm[b, l] -= h
            assert abs(float(dZ[b, l]) - (value(zp) - value(zm)) / (2 * h)) < 2e-6    # h^2, 1e-16 / h, and fp32


def test_gradient_of_a_label_given_often_is_the_sum_in_order():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(2)
    L, n = 5000, 2000
    cols = np.full(n, 4321, np.int32)
    cols[::3] = 17
    g = (rng.normal(0, 1, n) * 10.0 ** rng.integers(-3, 4, n)).astype(np.float32)
    rowptr = np.array([0, n], np.int32)
    Z = torch.full((1, L), -1e30, device="cuda")                  # p = 0 but at label 0
    Z[0, 0] = 0
    up = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    outs = []
    for _ in range(3):
        dZ = torch.empty(1, L, device="cuda")
        elmo.elmo_score_logprobs_backward(Z, up(rowptr), up(cols), torch.zeros(1, device="cuda"), None, up(g), None, None, dZ)
        outs.append(dZ.cpu().numpy())
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])
    for l in (17, 4321):
        want = np.float32(0)
        for v in g[cols == l]:
            want = np.float32(want + v)
        assert outs[0][0, l] == want


# ---------------------------------------------------------------- use
def test_captured_replayed_and_on_another_stream():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(6)
    B, L, k = 6, 50_001, 5
    Z = on_gpu(rng.normal(0, 3, (B, L)), "bf16", 3)
    rowptr, cols = lists(rng, B, L, 4)
    up = lambda a: torch.from_numpy(a).cuda()   # noqa: E731
    rp, cs = up(rowptr), up(cols)
    out = (torch.empty(len(cols), device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda"),
           torch.empty(B, k, dtype=torch.int32, device="cuda"), torch.empty(B, k, device="cuda"))
    work = torch.empty(elmo.elmo_score_logprobs_workspace_bytes(B, L, k), dtype=torch.uint8, device="cuda")
    g = torch.ones(len(cols), device="cuda")
    dZ = torch.empty(B, L, dtype=torch.bfloat16, device="cuda")

    def both(stream=None):
        elmo.elmo_score_logprobs(Z, rp, cs, *out, work, stream)
        elmo.elmo_score_logprobs_backward(Z, rp, cs, out[1], out[2], g, None, out[1], dZ, stream)

    both()
    torch.cuda.synchronize()
    first = [o.clone() for o in (*out, dZ)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for how in ("replay", "replay", "stream"):
        for o in (*out, dZ, work):
            o.zero_()
        torch.cuda.synchronize()
        if how == "replay":
            graph.replay()
        else:
            both(torch.cuda.Stream())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (*out, dZ)))


def test_refusals():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    f = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    i = lambda *s: f(*s, dt=torch.int32)   # noqa: E731
    work = f(elmo.elmo_score_logprobs_workspace_bytes(3, 100, 2), dt=torch.uint8)
    good = dict(Z=f(3, 100), rowptr=i(4), cols=i(5), logp=f(5), lse=f(3), entropy=f(3), top_idx=i(3, 2), top_logp=f(3, 2),
                workspace=work)
    elmo.elmo_score_logprobs(**good)
    for bad in [dict(Z=f(3, 100, dt=torch.float16)), dict(Z=f(100, 3).T), dict(rowptr=i(3)), dict(cols=f(5)),
                dict(logp=f(4)), dict(lse=f(4)), dict(top_idx=i(3, 3)), dict(top_idx=None), dict(entropy=f(3).cpu()),
                dict(Z=f(1, 100).expand(3, 100)), dict(workspace=work.float())]:
        with pytest.raises((ValueError, TypeError)):
            elmo.elmo_score_logprobs(**{**good, **bad})
    with pytest.raises(elmo.ElmoError, match="workspace"):
        elmo.elmo_score_logprobs(**{**good, "workspace": work[:-1]})
    with pytest.raises(elmo.ElmoError, match="k = 65"):
        elmo.elmo_score_logprobs(**{**good, "top_idx": i(3, 65), "top_logp": f(3, 65)})
    with pytest.raises(elmo.ElmoError, match="entropy"):
        elmo.elmo_score_logprobs_backward(good["Z"], good["rowptr"], good["cols"], f(3), None, None, None, f(3), f(3, 100))
