"""rssm_copy_rows and rssm_compact_rows against the definitions, and a serving run that uses
them with prefill, decode, verify and flush, against the token-by-token fp64 recurrences."""
import numpy as np
import pytest
import torch

from gpu_common import DEV, to64
from hybrid_ssm_decode_replayssm_b200 import rssm
from prefill_common import KINDS, TOL, Layer, i32, scaled

pytestmark = pytest.mark.gpu

FMTS = [rssm.RSSM_READ_FP32, rssm.RSSM_READ_FP8_E4M3_ROW, rssm.RSSM_READ_NVFP4]


def steps(L, n, seed, pending=0):
    """n decode calls on every row (the reference too), then `pending` drafts left open."""
    for j in range(n):
        toks = L.tokens(L.batch, seed * 100 + j)
        y = torch.empty((L.batch, L.H, L.R), device=DEV)
        L.layer.decode_step([t.to(DEV) for t in toks], y)
        want = []
        for r in range(L.batch):
            L.state[r], o = L.ref_run(L.state[r], [t[r:r + 1] for t in toks])
            want.append(o[0])
        if L.layer.desc.read_fmt == rssm.RSSM_READ_FP32:
            assert scaled(to64(y), np.stack(want)) <= TOL
    if pending:
        d = [t.to(DEV).reshape((L.batch, pending) + t.shape[1:]) for t in L.tokens(L.batch * pending, seed + 5)]
        L.layer.verify(pending, d, torch.empty((L.batch, pending, L.H, L.R), device=DEV))


def flushed(L):
    """Every row's state with its window folded in, without changing the layer: by export and import."""
    blob = L.layer.export_state()
    L.layer.flush()
    rows = L.rows()
    L.layer.import_state(blob)
    return rows


def read_copy(L, r):
    codes, scales = L.layer.read_copy_views()
    if L.layer.desc.branching:
        r = int(L.layer.get_slots()[r])
    return codes[r].clone(), scales[r].clone()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("kind", KINDS)
def test_copy_between_layers(kind, fmt):
    src = Layer(kind, batch=5, heads=2, read_fmt=fmt, seed=1)
    dst = Layer(kind, batch=7, heads=2, read_fmt=fmt, seed=2)
    steps(src, 11, 1)                                   # window 8: one fold, three entries
    steps(dst, 3, 2)
    want, old = flushed(src), flushed(dst)
    books, mine = src.layer.get_bookkeeping().cpu(), dst.layer.get_bookkeeping().cpu()
    d, s = [6, 0, 3, 2], [1, 1, 4, -1]
    dst.layer.copy_rows(src.layer, i32(d), i32(s))
    assert dst.layer.get_status() == 0
    now, got = dst.layer.get_bookkeeping().cpu(), flushed(dst)
    for r in range(7):
        if r not in d:
            assert torch.equal(now[:, r], mine[:, r]) and (got[r] == old[r]).all()
        elif s[d.index(r)] < 0:
            assert now[:, r].tolist() == [0, 0, 0, 0] and (got[r] == 0).all()
        else:
            p = s[d.index(r)]
            assert torch.equal(now[:, r], books[:, p]) and (got[r] == want[p]).all()
            if fmt != rssm.RSSM_READ_FP32:
                for a, b in zip(read_copy(dst, r), read_copy(src, p)):
                    assert torch.equal(a, b)
    if fmt != rssm.RSSM_READ_FP32:
        assert all(int(t.float().abs().max()) == 0 for t in read_copy(dst, 2))
    for r, p in zip(d, s):
        dst.state[r] = 0 if p < 0 else src.state[p]
    steps(dst, 9, 3)                                    # and decoding goes on from there, through a fold


@pytest.mark.parametrize("branching", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_fork_and_empty_in_one_layer(kind, branching):
    L = Layer(kind, batch=6, heads=2, branching=branching)
    steps(L, 5, 1)
    d, s = [1, 2, 5, 4, 3], [0, 0, -1, 4, 0]
    L.layer.copy_rows(L.layer, i32(d), i32(s))
    assert L.layer.get_status() == 0
    for r, p in zip(d, s):
        L.state[r] = 0 if p < 0 else L.state[p]
    if branching:
        slots = L.layer.get_slots().cpu().tolist()
        assert slots[0] == slots[1] == slots[2] == slots[3] and len(set(slots)) == 3
    steps(L, 12, 2)                                     # the forks part, folds included
    assert scaled(flushed(L), L.state) <= TOL


@pytest.mark.parametrize("kinds", [(True, True), (True, False), (False, True)])
def test_copy_between_branching_layers(kinds):
    """The rows copied to get slots of their own; rows that shared the old ones keep them."""
    src = Layer("gdn", batch=4, heads=2, branching=kinds[0], seed=1)
    dst = Layer("gdn", batch=5, heads=2, branching=kinds[1], seed=2)
    steps(src, 8, 1)                                    # a fold that no launch has adopted yet
    steps(dst, 8, 2)
    if kinds[1]:
        dst.layer.branch(i32([0, 0, 0, 3, 3]))
        for r, p in ((1, 0), (2, 0), (4, 3)):
            dst.state[r] = dst.state[p]
    d, s = [0, 3, 1], [2, 2, -1]
    dst.layer.copy_rows(src.layer, i32(d), i32(s))
    for r, p in zip(d, s):
        dst.state[r] = 0 if p < 0 else src.state[p]
    assert dst.layer.get_status() == 0
    steps(dst, 10, 3)
    assert scaled(flushed(dst), dst.state) <= TOL


@pytest.mark.parametrize("branching", [False, True])
def test_refused_pairs(branching):
    L = Layer("mamba2", batch=8, heads=2, branching=branching)
    steps(L, 3, 1)
    before, books = flushed(L), L.layer.get_bookkeeping().cpu()
    # row 1 twice; row 2 is read by the pair that writes 3; out of range; a row onto itself
    d, s = [1, 1, 2, 3, 8, 4, 5, 6], [0, 0, 0, 2, 0, 9, -2, 6]
    L.layer.copy_rows(L.layer, i32(d), i32(s))
    assert L.layer.get_status(clear=True) == rssm.RSSM_STATUS_STATE
    got = flushed(L)
    for r in range(8):
        assert (got[r] == before[2 if r == 3 else r]).all(), r
    assert torch.equal(L.layer.get_bookkeeping().cpu()[1:3], books[1:3])
    L.layer.copy_rows(L.layer, i32([6]), i32([6]))
    assert L.layer.get_status() == 0
    # a source with open drafts
    drafts = [t.to(DEV).reshape((8, 2) + t.shape[1:]) for t in L.tokens(16, 4)]
    L.layer.verify(2, drafts, torch.empty((8, 2, L.H, L.R), device=DEV))
    L.layer.rollback(i32([0, 2, 2, 2, 2, 2, 2, 2]))
    L.layer.verify(1, [t[:, :1].contiguous() for t in drafts], torch.empty((8, 1, L.H, L.R), device=DEV))
    L.layer.copy_rows(L.layer, i32([1]), i32([0]))
    assert L.layer.get_status(clear=True) == rssm.RSSM_STATUS_STATE


@pytest.mark.parametrize("live", [[1, 0, 1, 0, 0, 1, 1, 0, 1], [0] * 9, [1] * 9, [0] * 8 + [1], [1] * 4 + [0] * 5])
@pytest.mark.parametrize("kind,branching,fmt,pending", [
    ("gdn", False, FMTS[0], 0), ("mamba2", False, FMTS[1], 2), ("kda", False, FMTS[2], 0),
    ("mamba2", True, FMTS[0], 0), ("gdn", True, FMTS[1], 3)])
def test_compact(kind, branching, fmt, pending, live):
    L = Layer(kind, batch=9, heads=2, read_fmt=fmt, branching=branching)
    steps(L, 10, 1, pending)
    books = L.layer.get_bookkeeping().cpu()
    rows = L.rows()
    new_row, n_live = L.layer.compact_rows(i32(live))
    assert L.layer.get_status() == 0
    n = sum(live)
    holes = [b for b in range(n) if not live[b]]
    movers = [b for b in range(n, 9) if live[b]]
    want = [b if live[b] else -1 for b in range(9)]
    for h, m in zip(holes, movers):
        want[m] = h
    assert new_row.cpu().tolist() == want and int(n_live) == n
    came = {want[b]: b for b in range(9) if live[b]}
    now, got = L.layer.get_bookkeeping().cpu(), L.rows()
    for r in range(9):
        p = came.get(r, r) if r < n else r
        assert torch.equal(now[:, r], books[:, p]) and (got[r] == rows[p]).all()
    L.state = np.stack([L.state[came.get(r, r) if r < n else r] for r in range(9)])
    if pending:
        L.layer.rollback(i32([pending] * 9))
    steps(L, 10, 2)
    if fmt == FMTS[0]:
        assert scaled(flushed(L), L.state) <= TOL


def test_many_rows():
    """More rows and pairs than one pass of the planners holds (1024 threads)."""
    B = 2500
    L = Layer("mamba2", batch=B, heads=1, dstate=64, window=2, max_draft=1, branching=True)
    tag = torch.arange(B, device=DEV, dtype=torch.float32)
    L.layer.ckpt[:B] = tag[:, None, None, None]
    live = [int(b % 3 != 1) for b in range(B)]
    new_row, n_live = L.layer.compact_rows(i32(live))
    n = sum(live)
    holes, movers = [b for b in range(n) if not live[b]], [b for b in range(n, B) if live[b]]
    want = list(range(n))
    for h, m in zip(holes, movers):
        want[h] = m
    assert int(n_live) == n and L.rows()[:n, 0, 0, 0].astype(int).tolist() == want
    # 1100 rows emptied, the others copied onto 1100 more
    d = list(range(0, 1100)) + list(range(1200, 2300))
    s = [-1] * 1100 + list(range(1100, 1200)) * 11
    at = L.rows()[:, 0, 0, 0]
    L.layer.copy_rows(L.layer, i32(d), i32(s))
    assert L.layer.get_status() == 0
    for r, p in zip(d, s):
        at[r] = at[p] if p >= 0 else 0
    assert (L.rows()[:, 0, 0, 0] == at).all()


def test_stream_and_captured_graph():
    src, dst, eager = (Layer("gdn", batch=4, heads=2, seed=s) for s in (1, 2, 2))
    d, s = i32([0, 3]), i32([2, 1])
    live = i32([0, 1, 0, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager.layer.copy_rows(src.layer, d, s, stream=side)
    eager.layer.compact_rows(live, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dst.layer.copy_rows(src.layer, d, s)
        new_row, n_live = dst.layer.compact_rows(live)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dst.layer.ckpt, eager.layer.ckpt) and new_row.tolist() == [-1, 1, -1, 0] and int(n_live) == 2


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("branching", [False, True])
def test_serving_run(kind, branching):
    """Prompts come in, one is reused as a prefix, sequences decode, speculate and end, the batch
    is packed, a second turn goes on from the states: every output against the fp64 recurrence."""
    L = Layer(kind, batch=6, heads=2, branching=branching)
    pool = Layer(kind, batch=2, heads=2, seed=5)

    def prefill(M, lens, rows, fresh, seed):
        toks = M.tokens(sum(lens), seed)
        out = torch.zeros((sum(lens), M.H, M.R), device=DEV)
        off = [sum(lens[:i]) for i in range(len(lens) + 1)]
        M.layer.prefill([t.to(DEV) for t in toks], i32(off), out, rows=i32(rows), fresh=i32(fresh))
        for i, r in enumerate(rows):
            S, o = M.ref_run(M.state[r] * (not fresh[i]), [t[off[i]:off[i + 1]] for t in toks])
            assert scaled(to64(out[off[i]:off[i + 1]]), o) <= TOL
            M.state[r] = S

    prefill(pool, [50], [1], [1], 1)                                  # the shared prefix
    L.layer.copy_rows(pool.layer, i32([0, 1, 2]), i32([1, 1, 1]))
    for r in range(3):
        L.state[r] = pool.state[1]
    prefill(L, [9, 20, 1, 70, 3, 2], [0, 1, 2, 3, 4, 5], [0, 0, 0, 1, 1, 1], 2)
    steps(L, 6, 3)
    drafts = L.tokens(6 * 3, 4)                                        # a speculative round, all taken
    d = [t.reshape((6, 3) + t.shape[1:]) for t in drafts]
    y = torch.empty((6, 3, L.H, L.R), device=DEV)
    L.layer.verify(3, [t.to(DEV) for t in d], y)
    for r in range(6):
        L.state[r], o = L.ref_run(L.state[r], [t[r] for t in d])
        assert scaled(to64(y[r]), o) <= TOL
    L.layer.rollback(i32([0] * 6))
    new_row, n_live = L.layer.compact_rows(i32([0, 1, 0, 1, 0, 1]))    # three sequences end
    assert new_row.tolist() == [-1, 1, -1, 0, -1, 2] and int(n_live) == 3
    L.state[0], L.state[2] = L.state[3], L.state[5]
    L.layer.copy_rows(L.layer, i32([3, 4, 5]), i32([-1, -1, -1]))
    L.state[3:] = 0
    steps(L, 4, 5)
    L.layer.flush(i32([1, 1, 0, 0, 0, 0]))                             # a second turn for rows 0 and 1
    prefill(L, [65, 130], [1, 0], [0, 0], 6)
    steps(L, 9, 7)
    assert L.layer.get_status() == 0
    assert scaled(flushed(L), L.state) <= TOL
