"""4-bit copies of a head: codes and scales bit by bit, the values read back, and the scores of a few queries, each
against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

GRIDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def bf16_of(a):
    """fp32 -> the nearest bf16 value (ties to even), as float64."""
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def packed(w, group):
    """(u, s) of weights w [L, d] (float64 of values on their grid) by the definition."""
    w32 = w.astype(np.float32).reshape(w.shape[0], -1, group)
    with np.errstate(all="ignore"):
        m = np.abs(w32).max(2)
        s = bf16_of(m / np.float32(7))
        s[~np.isfinite(m)] = np.nan
        by = s.astype(np.float32)[:, :, None]
        q = np.where(by > 0, np.rint(w32 / by), 0)
    u = np.clip(np.nan_to_num(q, nan=0.0), -8, 7) + 8
    return u.reshape(w.shape).astype(np.uint8), s


def nibbles(u):
    return u[:, 0::2] | (u[:, 1::2] << 4)


def make(elmo, w, grid, group):
    L, d = w.shape
    W = torch.from_numpy(w.astype(np.float32)).to(GRIDS[grid]).cuda()
    codes = torch.full((L, d // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((L, d // group), 7.0, dtype=torch.bfloat16, device="cuda")
    elmo.elmo_q4_pack(W, grid, group, codes, scales)
    return W.double().cpu().numpy(), codes, scales


@pytest.mark.parametrize("grid", list(GRIDS))
@pytest.mark.parametrize("L,d,group", [(1, 64, 32), (3, 64, 64), (257, 128, 128), (1001, 768, 64), (5, 4096, 32)])
def test_pack_is_the_definition(grid, L, d, group):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + d)
    w = rng.normal(0, 0.02, (L, d))
    w[0, :group] = 0                                            # a group of zeros
    W, codes, scales = make(elmo, w, grid, group)
    u, s = packed(W, group)
    assert np.array_equal(codes.cpu().numpy(), nibbles(u))
    assert np.array_equal(scales.double().cpu().numpy(), s)
    back = torch.empty(L, d, dtype=torch.bfloat16, device="cuda")
    elmo.elmo_q4_unpack(codes, scales, back)
    want = bf16_of((u.astype(np.float32) - 8) * np.repeat(s, group, 1).astype(np.float32))
    assert np.array_equal(back.double().cpu().numpy(), want)


def test_pack_exact_ties_go_to_even():
    """w / s = k + 1/2 exactly: every magnitude 3.5, 7 * 3.5 / 7 ... with s = 1/2, and every significand of s."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    group, rows = 32, []
    for m in range(128):                                        # s = (1 + m / 128) 2^-7
        s = (1 + m / 128) * 2.0**-7
        ks = np.array([k / 2 for k in range(-13, 14)] + [7, -7, 0.25, -0.25, 7])
        rows.append(np.concatenate([ks * s, ks * s])[:64])      # two groups, only halves that bf16 holds survive
    w = bf16_of(np.array([np.resize(r, 64) for r in rows]))
    W, codes, scales = make(elmo, w, "bf16", group)
    u, s = packed(W, group)
    t = W.reshape(128, 2, 32) / s[:, :, None]
    assert (np.abs(t - np.floor(t) - 0.5) == 0).sum() > 500     # the ties are there
    assert np.array_equal(codes.cpu().numpy(), nibbles(u))


def test_pack_odd_values():
    """Subnormal groups (the scale's rounding is coarse: the clamp works), NaN and infinities, the largest weights."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(3)
    w = rng.normal(0, 1, (8, 64))
    w[0] *= 2.0**-130
    w[1] = rng.integers(-9, 10, 64) * 2.0**-133                 # multiples of the smallest subnormal
    w[2] *= 2.0**125
    w[3, 5], w[4, 40] = np.nan, np.inf
    w[5] *= 2.0**-100 * 7
    w = bf16_of(w)
    W, codes, scales = make(elmo, w, "bf16", 32)
    u, s = packed(W, 32)
    assert np.array_equal(codes.cpu().numpy(), nibbles(u))
    got = scales.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(s)) and np.isnan(s).sum() == 2
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(s))


def scored(u, s, x, group):
    """(scores, sums of magnitudes) in 64 bits."""
    w = (u.astype(np.float64) - 8) * np.repeat(s, group, 1)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def tolerance(d, group):
    # per group: group / 16 accumulating instructions, each off by at most 2^-22 of the magnitudes summed so far;
    # then one fp32 fma a group and two products with powers of two (exact)
    return group / 16 * 2.0**-22 + (d // group + 1) * 2.0**-24


@pytest.mark.parametrize("L,d,group,B,pad", [
    (1, 64, 32, 1, 0), (130, 64, 64, 3, 1), (1000, 128, 128, 9, 0), (257, 192, 32, 8, 5), (257, 192, 64, 31, 0),
    (4099, 768, 64, 33, 0), (4099, 768, 128, 2, 3), (300, 1024, 128, 17, 0), (129, 4096, 32, 5, 0),
    (77, 4096, 128, 40, 2), (40_011, 768, 64, 1, 0), (40_011, 320, 32, 4, 0)])
def test_scores_match_64_bits(L, d, group, B, pad):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(L + d + B)
    u = rng.integers(0, 16, (L, d)).astype(np.uint8)
    s = bf16_of(np.abs(rng.normal(0, 0.01, (L, d // group))))
    x = bf16_of(rng.normal(0, 1, (B, d)))
    codes = torch.from_numpy(nibbles(u)).cuda()
    scales = torch.from_numpy(s).to(torch.bfloat16).cuda()
    X = torch.from_numpy(x).to(torch.bfloat16).cuda()
    Z = torch.full((B, L + pad), 123.0, device="cuda")
    elmo.elmo_q4_scores(codes, scales, X, Z[:, :L])
    z, mag = scored(u, s, x, group)
    got = Z.double().cpu().numpy()
    assert (got[:, L:] == 123.0).all()                          # the pitch stays as it was
    assert (np.abs(got[:, :L] - z) <= tolerance(d, group) * mag + np.abs(z) * 2.0**-24).all()
    again = torch.empty(B, L, device="cuda")
    elmo.elmo_q4_scores(codes, scales, X, again)
    assert torch.equal(again, Z[:, :L])                         # the same bits whatever the pitch


def test_scores_of_odd_queries():
    """Queries of zeros, of very large, very small and very mixed magnitudes, with infinities and NaN; NaN scales."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(1)
    L, d, group = 500, 256, 64
    u = rng.integers(0, 16, (L, d)).astype(np.uint8)
    s = bf16_of(np.abs(rng.normal(0, 0.01, (L, d // group))))
    s[7, 2] = np.nan
    x = rng.normal(0, 1, (8, d))
    x[0] = 0
    x[1] *= 2.0**120
    x[2] *= 2.0**-120
    x[3] *= 2.0 ** rng.integers(-40, 1, d)
    x[4, 17] = np.inf
    x[5, 3] = np.nan
    x[6] = rng.integers(-1, 2, d) * 2.0**-133
    x = bf16_of(x)
    Z = torch.empty(8, L, device="cuda")
    elmo.elmo_q4_scores(torch.from_numpy(nibbles(u)).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(),
                        torch.from_numpy(x).to(torch.bfloat16).cuda(), Z)
    got = Z.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        z, mag = scored(u, s, x, group)
    assert np.isnan(got[:, 7]).all()
    rest = np.arange(L) != 7
    inf = u[:, 17] != 8                                         # 0 times infinity is NaN
    assert np.array_equal(got[4, rest & inf], z[4, rest & inf]) and np.isnan(got[4, rest & ~inf]).all()
    assert np.isnan(got[5]).all()
    for b in (0, 1, 2, 3, 6, 7):
        # fp16 at a largest magnitude of 2^14 at least: a step of 2^-24, half of it 2^-39 of the largest
        coarse = 2.0**-39 * np.abs(x[b]).max() * np.abs((u.astype(np.float64) - 8) * np.repeat(s, group, 1)).sum(1)
        bound = tolerance(d, group) * mag[b] + np.abs(z[b]) * 2.0**-24 + coarse + 2.0**-149
        assert (np.abs(got[b] - z[b]) <= bound)[rest].all(), b


def test_large_copies_take_64_bit_offsets():
    """B * ldz and L * d pass 2^31: the last rows of codes, scales and scores are the right ones."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    L, d, group, B = 9_000_001, 512, 128, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 256, (L, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(L, d // group, generator=g, device="cuda") * 0.01).to(torch.bfloat16)
    X = torch.randn(B, d, generator=g, device="cuda").to(torch.bfloat16)
    pitch = 1_100_000_000
    buf = torch.empty(2 * pitch + L, device="cuda")
    Z = torch.as_strided(buf, (B, L), (pitch, 1))
    elmo.elmo_q4_scores(codes, scales, X, Z)
    at = torch.tensor([0, 1, 4_194_303, 4_194_304, 8_388_608, L - 129, L - 2, L - 1], device="cuda")
    c = codes[at].cpu().numpy()
    u = np.empty((len(at), d), np.uint8)
    u[:, 0::2], u[:, 1::2] = c & 15, c >> 4
    z, mag = scored(u, scales[at].double().cpu().numpy(), X.double().cpu().numpy(), group)
    got = Z[:, at].double().cpu().numpy()
    assert (np.abs(got - z) <= tolerance(d, group) * mag + np.abs(z) * 2.0**-24).all()
    W = torch.empty(L, d, dtype=torch.bfloat16, device="cuda")
    elmo.elmo_q4_unpack(codes, scales, W)
    want = bf16_of((u.astype(np.float32) - 8) * np.repeat(scales[at].float().cpu().numpy(), group, 1))
    assert np.array_equal(W[at].double().cpu().numpy(), want)


def test_captured_and_on_another_stream():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    g = torch.Generator(device="cuda").manual_seed(5)
    W = (torch.randn(3001, 128, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    X = torch.randn(5, 128, generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.empty(3001, 64, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3001, 4, dtype=torch.bfloat16, device="cuda")
    Z, Z2 = torch.empty(5, 3001, device="cuda"), torch.empty(5, 3001, device="cuda")
    elmo.elmo_q4_pack(W, "bf16", 32, codes, scales)
    elmo.elmo_q4_scores(codes, scales, X, Z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        elmo.elmo_q4_pack(W, "bf16", 32, codes, scales)
        elmo.elmo_q4_scores(codes, scales, X, Z2)
    codes.zero_(), scales.zero_(), Z2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Z, Z2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Z2.zero_()
    side.wait_stream(torch.cuda.current_stream())
    elmo.elmo_q4_scores(codes, scales, X, Z2, stream=side)
    side.synchronize()
    assert torch.equal(Z, Z2)


def test_refusals():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    dev = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    codes, scales, X, Z = dev(10, 32, dt=torch.uint8), dev(10, 2), dev(3, 64), dev(3, 10, dt=torch.float32)
    elmo.elmo_q4_scores(codes, scales, X, Z)
    for bad in [(codes, scales, dev(3, 128), Z), (codes, scales, X, dev(3, 11, dt=torch.float32)),
                (codes, scales, X, dev(10, 3, dt=torch.float32).T), (codes, dev(9, 2), X, Z),
                (codes, scales, dev(3, 64, dt=torch.float32), Z), (codes, scales, X, dev(3, 10)),
                (codes, scales, X, dev(1, 10, dt=torch.float32).expand(3, 10)),
                (codes, scales, dev(64, 3).T, Z), (codes.cpu(), scales, X, Z)]:
        with pytest.raises((ValueError, TypeError)):
            elmo.elmo_q4_scores(*bad)
    for codes_, scales_ in [(dev(10, 32, dt=torch.uint8), dev(10, 4)), (dev(10, 48, dt=torch.uint8), dev(10, 3))]:
        d = 2 * codes_.shape[1]
        with pytest.raises(elmo.ElmoError) as e:                # groups of 16; d = 96
            elmo.elmo_q4_scores(codes_, scales_, dev(3, d), Z)
        assert e.value.status == 1
    with pytest.raises(ValueError):
        elmo.elmo_q4_pack(dev(10, 64), "e4m3", 32, codes, scales)
