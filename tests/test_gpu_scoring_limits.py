"""The scoring operators at the largest batch, without lists, and with calls that overlap on two streams."""
import numpy as np
import pytest
import torch

from tests import test_gpu_label_logprobs as head_ops
from tests import test_gpu_logprobs as score_ops
from tests import test_gpu_q4 as q4_ops
from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu

MOST = 4096                                                     # queries of one call
NONE = np.zeros(0, np.int32)


@pytest.mark.parametrize("group", [32, 64])
def test_most_queries_of_a_4_bit_copy(group):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(1)
    L, d = 301, 128
    u = rng.integers(0, 16, (L, d)).astype(np.uint8)
    s = q4_ops.bf16_of(np.abs(rng.normal(0, 0.01, (L, d // group))))
    x = q4_ops.bf16_of(rng.normal(0, 1, (MOST, d)))
    Z = torch.full((MOST + 1, L), 123.0, device="cuda")
    elmo.elmo_q4_scores(torch.from_numpy(q4_ops.nibbles(u)).cuda(), torch.from_numpy(s).to(torch.bfloat16).cuda(),
                        torch.from_numpy(x).to(torch.bfloat16).cuda(), Z[:MOST])
    z, mag = q4_ops.scored(u, s, x, group)
    got = Z.double().cpu().numpy()
    assert (np.abs(got[:MOST] - z) <= q4_ops.tolerance(d, group) * mag + np.abs(z) * 2.0**-24).all()
    assert (got[MOST] == 123.0).all()                           # a row behind the last stays as it was


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("L", [130, 40_007])
def test_most_rows_of_scores(dtype, L):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(2)
    Z = score_ops.on_gpu(rng.normal(0, 3, (MOST, L)).astype(np.float32), dtype)
    rowptr, cols = score_ops.lists(rng, MOST, L, 1)
    got = score_ops.scored(elmo, Z, rowptr, cols, 2)
    pick = np.r_[0:8, 2040:2056, MOST - 8:MOST]                 # whole rows of some queries, at each end and inside
    at = np.concatenate([np.arange(rowptr[b], rowptr[b + 1]) for b in pick]).astype(int)
    part = np.r_[0, np.cumsum(np.diff(rowptr)[pick])].astype(np.int32)
    z = Z[torch.from_numpy(pick).cuda()].float().cpu().numpy()
    score_ops.check([got[0][at]] + [g[pick] for g in got[1:]], z, part, cols[at], 2)


@pytest.mark.parametrize("grid", ["bf16", "e4m3"])
def test_most_queries_of_a_head(grid):
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(3)
    L, d, k = 500, 64, 3
    W, h = head_ops.head_of(elmo, rng.normal(0, 0.05, (L, d)), grid)
    X = head_ops.bf16(rng.normal(0, 1, (MOST, d)))
    rowptr, cols = head_ops.lists(rng, MOST, L, 1)
    got = head_ops.run(elmo, h, X, rowptr, cols, k)
    head_ops.check(got, X.double().cpu().numpy(), W.double().cpu().numpy(), grid, rowptr, cols, k)
    h.close()


def test_without_labels_and_lists():
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(4)
    B, L = 3, 5001
    Z = torch.from_numpy(rng.normal(0, 1, (B, L)).astype(np.float32)).cuda()
    rowptr = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    logp, lse, H = torch.empty(0, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    work = torch.empty(elmo.elmo_score_logprobs_workspace_bytes(B, L, 0), dtype=torch.uint8, device="cuda")
    elmo.elmo_score_logprobs(Z, rowptr, none, logp, lse, H, None, None, work)
    _, want, wantH, _, _, es, eH, _ = score_ops.expected(Z.cpu().numpy(), np.zeros(B + 1, np.int32), NONE, 0)
    assert (np.abs(lse.cpu().numpy() - want) <= es + 2.0**-24 * np.abs(want)).all()
    assert (np.abs(H.cpu().numpy() - wantH) <= eH + 2.0**-24 * wantH).all()
    dZ = torch.full_like(Z, 5.0)
    elmo.elmo_score_logprobs_backward(Z, rowptr, none, lse, None, None, None, None, dZ)
    assert (dZ == 0).all()                                      # no gradient comes in, none goes out


def test_calls_that_overlap():
    """Two streams, each with its own workspace or head, many calls in flight: the bits of calls made one by one."""
    need_gpu()
    import precision_label_chunk_b200 as elmo
    rng = np.random.default_rng(5)
    L, d, B, k = 60_001, 256, 6, 5
    sides = []
    for grid in ("bf16", "e4m3"):
        W, h = head_ops.head_of(elmo, rng.normal(0, 0.05, (L, d)), grid)
        codes = torch.empty(L, d // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(L, d // 64, dtype=torch.bfloat16, device="cuda")
        elmo.elmo_q4_pack(W, grid, 64, codes, scales)
        rowptr, cols = (torch.from_numpy(a).cuda() for a in head_ops.lists(rng, B, L, 4))
        nnz = cols.numel()
        work = torch.empty(elmo.elmo_score_logprobs_workspace_bytes(B, L, k), dtype=torch.uint8, device="cuda")
        sides.append((W, h, codes, scales, head_ops.bf16(rng.normal(0, 1, (B, d))), rowptr, cols, nnz, work))

    def outputs(nnz):
        return (torch.empty(B, L, device="cuda"), head_ops.buffers(B, nnz, k), head_ops.buffers(B, nnz, k),
                torch.empty(B, L, device="cuda"))

    def call(side, out, stream):
        _, h, codes, scales, X, rowptr, cols, _, work = side
        Z, a, b, dZ = out
        elmo.elmo_q4_scores(codes, scales, X, Z, stream)
        elmo.elmo_score_logprobs(Z, rowptr, cols, *a, work, stream)
        elmo.elmo_score_logprobs_backward(Z, rowptr, cols, a[1], a[2], a[0], a[1], a[2], dZ, stream)
        elmo.elmo_label_logprobs(h, X, rowptr, cols, *b, stream)

    flat = lambda out: [out[0], *out[1], *out[2], out[3]]       # noqa: E731
    alone = []
    for s in sides:
        out = outputs(s[7])
        call(s, out, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in flat(out)])
    streams = [torch.cuda.Stream() for _ in sides]
    outs = [[outputs(s[7]) for _ in range(4)] for s in sides]
    torch.cuda.synchronize()
    for i in range(4):
        for s, st, o in zip(sides, streams, outs):
            call(s, o[i], st)
    torch.cuda.synchronize()
    for want, o in zip(alone, outs):
        for out in o:
            assert all(torch.equal(a, b) for a, b in zip(want, flat(out)))
    for s in sides:
        elmo.elmo_sync_status(s[1])
        s[1].close()
