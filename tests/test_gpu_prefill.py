"""rssm_prefill against the token-by-token fp64 recurrences: ragged lengths, every layer
kind and input type, strides, read copies, branching, refusals, graphs and streams."""
import ctypes as C

import numpy as np
import pytest
import torch

from gpu_common import DEV, to64
from hybrid_ssm_decode_replayssm_b200 import rssm
from oracle import codecs
from prefill_common import KINDS, TOL, Layer, i32, offsets_of, scaled

pytestmark = pytest.mark.gpu


def run(L, lens, rows, fresh, seed=1, first=0, behind=0, tol=TOL, toks=None, what=""):
    """One prefill call checked whole: outputs, states, rows and outputs left alone, pointers."""
    off = offsets_of(lens, first)
    T = off[-1] + behind
    toks = L.tokens(T, seed) if toks is None else toks
    dev = [t.to(DEV) for t in toks]
    for a, b in [(0, first), (off[-1], T)]:           # nothing reads the tokens outside
        for t in dev:
            t[a:b] = float("nan")
    out = torch.full((T, L.H, L.R), -77.0, device=DEV)
    before = L.rows()
    books = L.layer.get_bookkeeping().cpu()
    L.layer.prefill(dev, i32(off), out, rows=i32(rows), fresh=i32(fresh))
    assert L.layer.get_status() == 0
    got, after = to64(out), L.rows()
    assert (got[:first] == -77).all() and (got[off[-1]:] == -77).all()
    worst = 0.0
    for i, r in enumerate(rows):
        S0 = np.zeros_like(L.state[r]) if fresh[i] else L.state[r]
        S, o = L.ref_run(S0, [t[off[i]:off[i + 1]] for t in toks])
        e = max(scaled(got[off[i]:off[i + 1]], o), scaled(after[r], S))
        assert e <= tol, f"{what} sequence {i} of {lens[i]} tokens: {e:.3e} > {tol:.1e}"
        worst = max(worst, e)
        L.state[r] = S
    rest = [r for r in range(L.batch) if r not in rows]
    assert (after[rest] == before[rest]).all()
    now = L.layer.get_bookkeeping().cpu()
    for i, r in enumerate(rows):
        touched = bool(fresh[i] or lens[i])
        assert now[1, r] == 0 and now[2, r] == 0 and now[3, r] == books[3, r] + touched
    return worst


LENS = {"one": [1], "tiny": [0, 1, 2, 3], "around 16": [15, 16, 17, 0], "around 64": [63, 64, 65],
        "around 128": [127, 128, 129], "long and short": [1, 517, 7]}


@pytest.mark.parametrize("lens", list(LENS), ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_ragged(kind, dtype, lens):
    n = LENS[lens]
    L = Layer(kind, batch=len(n) + 2, heads=3, dtype=dtype, out_scale=0.7)
    rows = list(range(len(n) + 1, 1, -1))
    run(L, n, rows, [i % 2 for i in range(len(n))], first=2, behind=3)
    run(L, n[::-1], rows, [0] * len(n), seed=2, what="continued")


@pytest.mark.parametrize("heads,groups,dstate", [(1, 1, 64), (6, 2, 64), (6, 3, 128), (16, 1, 128)])
def test_mamba2_groups(heads, groups, dstate):
    for dtype in ("bf16", "f32"):
        L = Layer("mamba2", batch=3, heads=heads, groups=groups, dstate=dstate, dtype=dtype)
        run(L, [70, 0, 33], [2, 0, 1], [1, 1, 0])


@pytest.mark.parametrize("kind", KINDS)
def test_default_rows_and_long(kind):
    L = Layer(kind, batch=2, heads=2)
    toks = L.tokens(1100, 5)
    out = torch.zeros((1100, L.H, L.R), device=DEV)
    L.layer.prefill([t.to(DEV) for t in toks], i32([0, 1100]), out)
    S, o = L.ref_run(L.state[0], toks)
    assert scaled(to64(out), o) <= TOL and scaled(L.rows()[0], S) <= TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_token_strides(kind, dtype):
    """Inputs that are slices of one wider projection give the packed inputs' results."""
    L, M = (Layer(kind, batch=2, heads=4, dtype=dtype) for _ in range(2))
    toks = [t.to(DEV) for t in L.tokens(90, 3)]
    wide = []
    for i, t in enumerate(toks):
        w = torch.full((90, t[0].numel() + 16 * (i + 1)), float("nan"), dtype=t.dtype, device=DEV)
        at = 8 * (i + 1) if t.dtype == torch.bfloat16 else 4 * (i + 1)
        w[:, at:at + t[0].numel()] = t.reshape(90, -1)
        wide.append(w[:, at:at + t[0].numel()].unflatten(1, t.shape[1:]) if t.dim() == 3 else w[:, at:at + t.shape[1]])
    outs = [torch.zeros((90, L.H, L.R), device=DEV) for _ in range(2)]
    L.layer.prefill(toks, i32([0, 50, 90]), outs[0])
    M.layer.prefill(wide, i32([0, 50, 90]), outs[1])
    assert torch.equal(outs[0], outs[1]) and torch.equal(L.layer.ckpt, M.layer.ckpt)


@pytest.mark.parametrize("fmt", [rssm.RSSM_READ_FP8_E4M3_ROW, rssm.RSSM_READ_NVFP4])
@pytest.mark.parametrize("kind", KINDS)
def test_read_copy_of_the_rows_written(kind, fmt):
    for dstate in (64, 128) if kind == "mamba2" else (128,):
        L = Layer(kind, batch=4, heads=2, dstate=dstate, read_fmt=fmt)
        run(L, [40, 0, 90], [3, 0, 1], [0, 1, 1])
        codes, scales = (t.clone() for t in L.layer.read_copy_views())
        L.layer.quantize_read_copy()
        for got, want in zip((codes, scales), L.layer.read_copy_views()):
            assert torch.equal(got, want)
    assert int(codes[0].max()) == 0            # the emptied row
    ck = L.layer.ckpt.cpu().numpy()[1, 0]
    if fmt == rssm.RSSM_READ_FP8_E4M3_ROW:
        want, _ = codecs.fp8_row_quantize(ck)
        assert (codes[1, 0].cpu().numpy() == want).all()


@pytest.mark.parametrize("kind", KINDS)
def test_extreme_gates_and_zero_keys(kind):
    """Gates of 0, of almost 0 and of 1, steps of 0, keys of zeros: no NaN, and the formula's values."""
    for dtype in ("bf16", "f32"):
        L = Layer(kind, batch=2, heads=2, dtype=dtype)
        toks = L.tokens(150, 9)
        gate = toks[3]
        if kind == "mamba2":
            gate[10] = 0.0                      # dt = 0: nothing happens
            gate[20:24] = 300.0                 # dt A down to -4800: the state is forgotten
            gate[70:135] = 0.001
            toks[0][20:24] *= 1e-3
        else:
            gate[10] = 0.0
            gate[20:24] = 1e-30
            gate[70:135] = 1.0
            gate[60:62] = 1e-4
            toks[4][30] = 0.0
            toks[4][31] = 1.0
        toks[1][40] = 0.0
        # gates of 1 keep an error for 65 tokens instead of 14: (65 / 14) TOL
        run(L, [149, 1], [1, 0], [0, 0], tol=5 * TOL, toks=toks)


@pytest.mark.parametrize("kind", ["gdn", "kda"])
def test_extreme_gates_in_chunks(kind):
    """The same in sequences that run in chunks of 64 (every place in and between their blocks of
    sixteen tokens), with channels of their own for KDA."""
    L = Layer(kind, batch=2, heads=2)
    toks = L.tokens(350, 19)
    gate, b = toks[3], toks[4]
    g = torch.Generator().manual_seed(5)
    if kind == "kda":
        gate[torch.rand(gate.shape, generator=g) < 0.02] = 0.0
        gate[torch.rand(gate.shape, generator=g) < 0.02] = 1e-30
        gate[:, :, 5] = 1.0
    gate[[0, 15, 16, 31, 64, 80, 127, 200]] = 0.0
    gate[[7, 47, 48, 90, 91, 128, 250]] = 1e-30
    gate[160:190] = 1e-4
    b[[33, 100]] = 0.0
    b[[34, 101]] = 1.0
    toks[1][[40, 129]] = 0.0
    # KDA's channel 5 never forgets by its gate, only by the keys: its values stay below sqrt(350)
    # of one token's, the errors of 350 tokens on it a factor 350 / 14 of TOL's on one of 128
    # channels of a row, so (350 / 14) / sqrt(128) TOL on its root mean square
    run(L, [201, 149], [1, 0], [0, 0], tol=3 * TOL, toks=toks)


@pytest.mark.parametrize("kind", KINDS)
def test_fresh_rows_do_not_read_what_was_there(kind):
    L = Layer(kind, batch=3, heads=2)
    L.layer.ckpt[1] = float("nan")
    L.state[1] = 0
    run(L, [30, 5], [1, 2], [1, 0])


@pytest.mark.parametrize("kind", KINDS)
def test_refused_sequences_are_left_alone(kind):
    L = Layer(kind, batch=6, heads=2)
    toks = [t.to(DEV) for t in L.tokens(40, 4)]
    one = [t[:6].contiguous() for t in toks]
    y = torch.empty((6, L.H, L.R), device=DEV)
    L.layer.decode_step(one, y)                          # every row has a window now
    L.layer.flush(i32([1, 0, 1, 1, 1, 1]))               # row 1 keeps it
    base = L.layer.ckpt.clone()

    def call(off, rows, fresh=None):
        out = torch.full((40, L.H, L.R), -77.0, device=DEV)
        books = L.layer.get_bookkeeping()
        L.layer.prefill(toks, i32(off), out, rows=i32(rows), fresh=None if fresh is None else i32(fresh))
        bits = L.layer.get_status(clear=True)
        return bits, out, [r for r in range(6) if not torch.equal(L.layer.ckpt[r], base[r])], \
            (L.layer.get_bookkeeping() - books).abs().sum(0).cpu().tolist()

    bits, out, changed, moved = call([0, 8, 20, 40], [1, 7, -1])           # window; out of range twice
    assert bits == rssm.RSSM_STATUS_STATE and changed == [] and (out == -77).all() and sum(moved) == 0
    bits, out, changed, moved = call([0, 8, 8, 40], [2, 2, 3])             # row 2 twice, row 3 once
    assert bits == rssm.RSSM_STATUS_STATE and changed == [3]
    assert (out[:8] == -77).all() and (out[8:] != -77).all()
    for off in ([0, 8, 4, 40], [-1, 8, 20, 40], [0, 8, 20, 41]):
        base.copy_(L.layer.ckpt)
        bits, out, changed, moved = call(off, [0, 2, 3])
        assert bits == rssm.RSSM_STATUS_STATE and changed == [] and (out == -77).all() and sum(moved) == 0
    bits, out, changed, moved = call([0, 8, 20, 40], [1, 2, 3], [1, 0, 0])  # fresh: the window is dropped
    assert bits == 0 and changed == [1, 2, 3] and moved[1] > 0


@pytest.mark.parametrize("kind", KINDS)
def test_branching_rows_that_share_a_state(kind):
    L = Layer(kind, batch=4, heads=2, branching=True)
    run(L, [33], [0], [1])
    L.layer.branch(i32([0, 0, 0, 3]))
    L.state[1] = L.state[2] = L.state[0]
    run(L, [20, 70], [1, 3], [0, 0], seed=7)             # row 1 goes on, rows 0 and 2 keep the prefix
    run(L, [5, 5, 5, 5], [2, 1, 0, 3], [0, 1, 0, 0], seed=8)
    slots = L.layer.get_slots().cpu().tolist()
    assert len(set(slots)) == 4
    toks = [t.to(DEV) for t in L.tokens(4, 11)]
    y = torch.empty((4, L.H, L.R), device=DEV)
    L.layer.decode_step(toks, y)
    for r in range(4):
        _, o = L.ref_run(L.state[r], [t[r:r + 1].cpu() for t in toks])
        assert scaled(to64(y[r:r + 1]), o) <= TOL


@pytest.mark.parametrize("kind", KINDS)
def test_stream_and_captured_graph(kind):
    """A captured call replayed on new inputs in the same buffers gives the eager results."""
    L, M = (Layer(kind, batch=3, heads=2) for _ in range(2))
    toks = [t.to(DEV) for t in L.tokens(100, 3)]
    off, rows = i32([0, 64, 100]), i32([2, 0])
    outs = [torch.zeros((100, L.H, L.R), device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.layer.prefill(toks, off, outs[0], rows=rows, stream=side)       # an eager call on another stream
    side.synchronize()
    M.layer.prefill(toks, off, outs[1], rows=rows)
    assert torch.equal(*outs) and torch.equal(L.layer.ckpt, M.layer.ckpt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.layer.prefill(toks, off, outs[0], rows=rows)
    for seed in (21, 22):
        for t, new in zip(toks, L.tokens(100, seed)):
            t.copy_(new)
        off[1] = 30 + seed
        graph.replay()
        M.layer.prefill(toks, off, outs[1], rows=rows)
        torch.cuda.synchronize()
        assert torch.equal(*outs) and torch.equal(L.layer.ckpt, M.layer.ckpt)
    assert L.layer.get_status() == 0


def test_the_same_call_twice_gives_the_same_bits():
    for kind in KINDS:
        res = []
        for _ in range(2):
            L = Layer(kind, batch=5, heads=4)
            toks = [t.to(DEV) for t in L.tokens(700, 3)]
            out = torch.zeros((700, L.H, L.R), device=DEV)
            L.layer.prefill(toks, i32([0, 100, 101, 400, 650, 700]), out)
            res.append((out, L.layer.ckpt))
        assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


@pytest.mark.parametrize("kind", KINDS)
def test_many_items_of_all_lengths(kind):
    """More (sequence, head) items than SMs, short and long sequences, empty and refused ones in
    one call: the persistent kernels take several items each."""
    heads = 16
    lens = [70, 1, 0, 300, 41, 40, 129, 64, 65, 25, 24, 256, 3, 128, 0, 90]
    n = len(lens)
    L = Layer(kind, batch=n + 3, heads=heads, groups=2 if kind == "mamba2" else 1)
    rows = list(range(n))[::-1]
    fresh = [i % 3 == 0 for i in range(n)]
    toks = L.tokens(sum(lens), 17)
    off = offsets_of(lens)
    out = torch.full((off[-1], heads, L.R), -77.0, device=DEV)
    rows[3] = rows[9] = n + 1                              # a long and a short one name one row
    L.layer.prefill([t.to(DEV) for t in toks], i32(off), out, rows=i32(rows), fresh=i32([int(f) for f in fresh]))
    assert L.layer.get_status(clear=True) == rssm.RSSM_STATUS_STATE
    got, after = to64(out), L.rows()
    for i, r in enumerate(rows):
        o = got[off[i]:off[i + 1]]
        if i in (3, 9):
            assert (o == -77).all()
            continue
        S, want = L.ref_run(L.state[r] * (not fresh[i]), [t[off[i]:off[i + 1]] for t in toks])
        assert max(scaled(o, want), scaled(after[r], S)) <= TOL, (i, lens[i])
    for r in (n, n + 1, n + 2):
        assert (after[r] == L.state[r]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_outputs_of_one_sequence_do_not_depend_on_the_others(kind):
    """A long sequence alone and in a batch gives the same bits (a short call may go by another
    kernel, so the sequence is long enough for either)."""
    L, M = (Layer(kind, batch=4, heads=4) for _ in range(2))
    toks = [t.to(DEV) for t in L.tokens(700, 3)]
    one = torch.zeros((400, 4, L.R), device=DEV)
    L.layer.prefill([t[100:500].contiguous() for t in toks], i32([0, 400]), one, rows=i32([2]))
    all_ = torch.zeros((700, 4, L.R), device=DEV)
    M.layer.prefill(toks, i32([0, 100, 500, 510, 700]), all_, rows=i32([0, 2, 1, 3]))
    assert torch.equal(one, all_[100:500]) and torch.equal(L.layer.ckpt[2], M.layer.ckpt[2])


@pytest.mark.parametrize("kind", KINDS)
def test_a_wait_that_runs_out_ends_the_call(kind):
    """The armed self-test: a chunked kernel's wait gives up, the status says TIMEOUT, and after a
    reset the layer works again."""
    L = Layer(kind, batch=2, heads=80)                     # more items than SMs
    toks = [t.to(DEV) for t in L.tokens(600, 3)]
    out = torch.zeros((600, 80, L.R), device=DEV)
    lib = rssm.lib()
    rssm.check(lib.rssm_set_wait_limit(L.layer.handle, 2_000_000))     # about a millisecond
    rssm.check(lib.rssm_arm_timeout_test(L.layer.handle))
    L.layer.prefill(toks, i32([0, 300, 600]), out)
    assert L.layer.get_status(clear=True) & rssm.RSSM_STATUS_TIMEOUT
    rssm.check(lib.rssm_set_wait_limit(L.layer.handle, 0))
    L.layer.reset()
    L.layer.ckpt.copy_(L.h0.to(DEV))
    run(L, [150, 70], [0, 1], [0, 0])


@pytest.mark.parametrize("kind,branching", [("gdn", False), ("mamba2", True)])
def test_more_sequences_than_planner_threads(kind, branching):
    n = 1300
    L = Layer(kind, batch=n + 5, heads=1, dstate=64, branching=branching)
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 5, n).tolist()
    lens[700], lens[1200], lens[3] = 150, 70, 41
    fresh = rng.integers(0, 2, n).tolist()
    rows = rng.permutation(n + 5)[:n].tolist()
    run(L, lens, rows, fresh, first=1, behind=1)


@pytest.mark.parametrize("kind", KINDS)
def test_the_scan_beside_chunks_waits_for_the_plan(kind):
    """Beside a chunked kernel the short sequences' kernel takes the plan only once the planner says
    that it is written; in the armed self-test it does not, and the wait ends with TIMEOUT and
    the short sequences' rows and outputs as they were."""
    L = Layer(kind, batch=4, heads=2)
    toks = [t.to(DEV) for t in L.tokens(340, 3)]
    out = torch.full((340, 2, L.R), -77.0, device=DEV)
    lib, off, rows = rssm.lib(), i32([0, 20, 320, 340]), i32([3, 0, 2])
    rssm.check(lib.rssm_set_wait_limit(L.layer.handle, 2_000_000))     # about a millisecond
    rssm.check(lib.rssm_arm_timeout_test(L.layer.handle))
    L.layer.prefill(toks, off, out, rows=rows)
    assert L.layer.get_status(clear=True) & rssm.RSSM_STATUS_TIMEOUT
    assert (out[:20] == -77).all() and (out[320:] == -77).all()
    assert (L.layer.ckpt[2:].cpu() == L.h0[2:]).all()
    rssm.check(lib.rssm_set_wait_limit(L.layer.handle, 0))
    L.layer.reset()
    L.layer.ckpt.copy_(L.h0.to(DEV))
    run(L, [20, 300, 20], [3, 0, 2], [0, 0, 0])


@pytest.mark.parametrize("kind", KINDS)
def test_one_workspace_for_many_calls(kind):
    """Calls of other plans, one behind the other in one workspace that nobody clears: the bits of
    calls with workspaces of their own."""
    L, M = (Layer(kind, batch=6, heads=3) for _ in range(2))
    plans = [([10, 300, 20, 0], [5, 0, 2, 1]), ([250, 3, 5, 120], [1, 2, 3, 0]), ([2, 200], [4, 3]),
             ([40, 39, 38, 37, 36, 35], [0, 1, 2, 3, 4, 5]), ([1, 2, 3], [2, 1, 0])]
    lib = rssm.lib()
    size = C.c_size_t()
    need = 0
    for lens, _ in plans:
        rssm.check(lib.rssm_prefill_workspace_size(L.layer.handle, len(lens), sum(lens), C.byref(size)))
        need = max(need, size.value)
    work = torch.full((need,), 0x5E, dtype=torch.uint8, device=DEV)
    calls = []
    for i, (lens, rows) in enumerate(plans * 4):
        toks = [t.to(DEV) for t in L.tokens(sum(lens), i)]
        a, b = (torch.zeros((sum(lens), 3, L.R), device=DEV) for _ in range(2))
        calls.append((toks, i32(offsets_of(lens)), i32(rows), a, b))
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    for toks, off, rows, a, _ in calls:
        ptrs = (C.c_void_p * 5)(*[t.data_ptr() for t in toks])
        rssm.check(lib.rssm_prefill(L.layer.handle, rows.numel(), a.shape[0], off.data_ptr(), rows.data_ptr(), None,
                                    ptrs, None, a.data_ptr(), work.data_ptr(), need, stream))
    for toks, off, rows, _, b in calls:
        M.layer.prefill(toks, off, b, rows=rows)
        torch.cuda.synchronize()
    assert L.layer.get_status() == 0 and M.layer.get_status() == 0
    for *_, a, b in calls:
        assert torch.equal(a, b)
    assert torch.equal(L.layer.ckpt, M.layer.ckpt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("step", [1e4, 1e9, 1e12, 1e30])
def test_mamba2_steps_that_forget_everything(dtype, step):
    """A huge dt (of a token without x) empties the state; the decays between the tokens behind it
    keep their precision."""
    L = Layer("mamba2", batch=2, heads=4, dtype=dtype)
    toks = L.tokens(300, 23)
    for t in (50, 128, 270):
        toks[3][t] = step
        toks[0][t] = 0.0
    run(L, [200, 100], [1, 0], [0, 0], toks=toks)


@pytest.mark.parametrize("kind,least", [("gdn", 41), ("kda", 97)])
def test_the_smallest_workspace(kind, least):
    """Sequences just long enough for chunks need the whole workspace; nothing behind it is written."""
    lens = [least] * 7 + [1, 0, 64 * 3 + 1, least - 1]
    L = Layer(kind, batch=len(lens), heads=3)
    T, size, lib = sum(lens), C.c_size_t(), rssm.lib()
    rssm.check(lib.rssm_prefill_workspace_size(L.layer.handle, len(lens), T, C.byref(size)))
    work = torch.full((size.value + 65536,), 0x3C, dtype=torch.uint8, device=DEV)
    toks, off = L.tokens(T, 3), offsets_of(lens)
    dev, out, doff = [t.to(DEV) for t in toks], torch.zeros((T, 3, L.R), device=DEV), i32(off)
    ptrs = (C.c_void_p * 5)(*[t.data_ptr() for t in dev])
    rssm.check(lib.rssm_prefill(L.layer.handle, len(lens), T, doff.data_ptr(), None, None, ptrs, None, out.data_ptr(),
                                work.data_ptr(), size.value, torch.cuda.current_stream().cuda_stream))
    assert L.layer.get_status() == 0 and (work[size.value:] == 0x3C).all()
    got, after = to64(out), L.rows()
    for i in range(len(lens)):
        S, o = L.ref_run(L.state[i], [t[off[i]:off[i + 1]] for t in toks])
        assert max(scaled(got[off[i]:off[i + 1]], o), scaled(after[i], S)) <= TOL, i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_slices_of_a_longer_run_of_tokens(kind, dtype):
    """Inputs that begin at an odd token of a longer tensor (on a layer of three heads their dt,
    alpha and beta are on no 16 bytes) give the bits of copies of their own, in the scan and in chunks."""
    for T in (60, 330):
        L, M = (Layer(kind, batch=3, heads=3, dtype=dtype) for _ in range(2))
        long = [t.to(DEV) for t in L.tokens(T + 5, 3)]
        part = [t[5:] for t in long]
        assert any(t.data_ptr() % 16 for t in part)
        outs = [torch.zeros((T, 3, L.R), device=DEV) for _ in range(2)]
        off = i32([0, T // 2 + 1, T])
        L.layer.prefill(part, off, outs[0])
        M.layer.prefill([t.clone() for t in part], off, outs[1])
        assert torch.equal(*outs) and torch.equal(L.layer.ckpt, M.layer.ckpt)


# ---------------------------------------------- forms of the chunked kernels
# A call of more than 192 tokens runs a layer's sequences of more than 96 tokens in chunks, whatever
# its kind.  The launches tell: plan, (GDN, KDA: T of every chunk,) chunks, scan, (read copies).
CHUNK_LAUNCHES = {"mamba2": 3, "gdn": 4, "kda": 4}


def launches_of(call):
    before = rssm.lib().rssm_launch_count()
    call()
    return rssm.lib().rssm_launch_count() - before


@pytest.mark.parametrize("kind", KINDS)
def test_token_strides_in_chunks(kind):
    L, M = (Layer(kind, batch=3, heads=4) for _ in range(2))
    T = 360
    toks = [t.to(DEV) for t in L.tokens(T, 3)]
    wide = []
    for i, t in enumerate(toks):
        w = torch.full((T, t[0].numel() + 16 * (i + 1)), float("nan"), dtype=t.dtype, device=DEV)
        at = 8 * (i + 1) if t.dtype == torch.bfloat16 else 4 * (i + 1)
        w[:, at:at + t[0].numel()] = t.reshape(T, -1)
        wide.append(w[:, at:at + t[0].numel()].unflatten(1, t.shape[1:]) if t.dim() == 3 else w[:, at:at + t.shape[1]])
    outs = [torch.zeros((T, L.H, L.R), device=DEV) for _ in range(2)]
    off = i32([0, 201, 350, T])
    L.layer.prefill(toks, off, outs[0])
    n = launches_of(lambda: M.layer.prefill(wide, off, outs[1]))
    assert n == CHUNK_LAUNCHES[kind]
    assert torch.equal(outs[0], outs[1]) and torch.equal(L.layer.ckpt, M.layer.ckpt)
    S, o = L.ref_run(L.state[0], [t[:201].cpu() for t in toks])
    assert scaled(to64(outs[1][:201]), o) <= TOL and scaled(M.rows()[0], S) <= TOL


@pytest.mark.parametrize("branching", [False, True])
@pytest.mark.parametrize("fmt", [rssm.RSSM_READ_FP8_E4M3_ROW, rssm.RSSM_READ_NVFP4])
@pytest.mark.parametrize("kind", KINDS)
def test_read_copies_behind_chunks(kind, fmt, branching):
    for dstate in (64, 128) if kind == "mamba2" else (128,):
        L = Layer(kind, batch=5, heads=2, dstate=dstate, read_fmt=fmt, branching=branching)
        L.layer.quantize_read_copy()
        n = launches_of(lambda: run(L, [140, 0, 201, 7], [3, 0, 1, 4], [0, 1, 1, 0]))
        assert n >= CHUNK_LAUNCHES[kind] + 1
        codes, scales = (t.clone() for t in L.layer.read_copy_views())
        slots = L.layer.get_slots().tolist() if branching else list(range(5))
        assert int(codes[slots[0]].max()) == 0            # the emptied row
        L.layer.quantize_read_copy()
        for got, want in zip((codes, scales), L.layer.read_copy_views()):
            for r in slots:
                assert torch.equal(got[r], want[r])
        if fmt == rssm.RSSM_READ_FP8_E4M3_ROW:
            want, _ = codecs.fp8_row_quantize(L.layer.ckpt.cpu().numpy()[slots[1], 0])
            assert (codes[slots[1], 0].cpu().numpy() == want).all()


@pytest.mark.parametrize("kind", KINDS)
def test_fresh_rows_in_chunks_do_not_read_what_was_there(kind):
    L = Layer(kind, batch=4, heads=2)
    L.layer.ckpt[1] = float("nan")
    L.layer.ckpt[3] = float("inf")
    L.state[1] = L.state[3] = 0
    run(L, [130, 5, 200], [1, 2, 3], [1, 0, 1])


@pytest.mark.parametrize("kind", KINDS)
def test_branching_rows_that_share_a_state_in_chunks(kind):
    L = Layer(kind, batch=4, heads=2, branching=True)
    run(L, [233], [0], [1])
    L.layer.branch(i32([0, 0, 0, 3]))
    L.state[1] = L.state[2] = L.state[0]
    run(L, [120, 150], [1, 3], [0, 0], seed=7)            # row 1 goes on, rows 0 and 2 keep the prefix
    run(L, [100, 99, 20, 130], [2, 1, 0, 3], [0, 1, 0, 0], seed=8)
    assert len(set(L.layer.get_slots().cpu().tolist())) == 4


@pytest.mark.parametrize("kind", KINDS)
def test_captured_chunks(kind):
    """A captured call whose offsets then move across the lengths at which a sequence changes its
    kernel (40 and 96 tokens): the eager results, call after call, also when it is replayed at once
    behind itself and the eager calls stand on another stream."""
    L, M = (Layer(kind, batch=4, heads=2) for _ in range(2))
    T = 400
    toks = [t.to(DEV) for t in L.tokens(T, 3)]
    off, rows = i32([0, 201, 360, T]), i32([2, 0, 3])
    outs = [torch.zeros((T, L.H, L.R), device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.layer.prefill(toks, off, outs[0], rows=rows, stream=side)
    side.synchronize()
    M.layer.prefill(toks, off, outs[1], rows=rows)
    assert torch.equal(*outs) and torch.equal(L.layer.ckpt, M.layer.ckpt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = launches_of(lambda: L.layer.prefill(toks, off, outs[0], rows=rows))
    assert n == CHUNK_LAUNCHES[kind]
    for seed, at in enumerate([(0, 40, 80, T), (0, 41, 82, 179), (0, 96, 192, 390), (10, 107, 204, 300), (0, 1, 1, T),
                               (0, 300, 350, 380), (0, 30, 60, 90)]):
        for t, new in zip(toks, L.tokens(T, 30 + seed)):
            t.copy_(new)
        off.copy_(i32(list(at)))
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        with torch.cuda.stream(side):
            for _ in range(2):
                M.layer.prefill(toks, off, outs[1], rows=rows)
        torch.cuda.synchronize()
        assert torch.equal(*outs) and torch.equal(L.layer.ckpt, M.layer.ckpt), at
    assert L.layer.get_status() == 0 and M.layer.get_status() == 0


@pytest.mark.parametrize("heads", [8, 24])
@pytest.mark.parametrize("kind", KINDS)
def test_long_fp32_prompts_beside_short_ones(kind, heads):
    """fp32 prompts of more than 512 tokens in a batch (by half as many state rows per CTA as the
    others while they are few): the values, and the bits that each has alone in a call."""
    lens = [600, 30, 520, 1, 0, 512, 513, 64, 5, 40, 41, 3]
    L, M = (Layer(kind, batch=len(lens), heads=heads, dtype="f32") for _ in range(2))
    off, toks = offsets_of(lens), L.tokens(sum(lens), 5)
    dev = [t.to(DEV) for t in toks]
    out = torch.zeros((off[-1], heads, L.R), device=DEV)
    L.layer.prefill(dev, i32(off), out)
    assert L.layer.get_status() == 0
    got, after = to64(out), L.rows()
    for i, n in enumerate(lens):
        at = slice(off[i], off[i + 1])
        one = torch.zeros((n, heads, L.R), device=DEV)
        M.layer.prefill([t[at].clone() for t in dev], i32([0, n]), one, rows=i32([i]))
        assert torch.equal(one, out[at]) and torch.equal(M.layer.ckpt[i], L.layer.ckpt[i]), n
        if i in (0, 1, 6):
            S, o = L.ref_run(L.state[i], [t[at] for t in toks])
            assert max(scaled(got[at], o), scaled(after[i], S)) <= TOL, n


@pytest.mark.parametrize("kind", KINDS)
def test_two_layers_on_two_streams(kind):
    """Calls of two layers at once, short and long, give the bits of the same calls in turn."""
    Ls = [[Layer(kind, batch=3, heads=24, seed=s) for s in (1, 2)] for _ in range(2)]
    toks = [[t.to(DEV) for t in Ls[0][0].tokens(500, 40 + s)] for s in range(2)]
    offs = [i32([0, 300, 330, 500]), i32([0, 20, 480, 500])]
    outs = [[torch.zeros((500, 24, Ls[0][0].R), device=DEV) for _ in range(2)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in range(2):
            Ls[0][s].layer.prefill(toks[s], offs[s], outs[0][s], stream=streams[s])
    torch.cuda.synchronize()
    for s in range(2):
        for _ in range(5):
            Ls[1][s].layer.prefill(toks[s], offs[s], outs[1][s])
            torch.cuda.synchronize()
        assert torch.equal(outs[0][s], outs[1][s]) and torch.equal(Ls[0][s].layer.ckpt, Ls[1][s].layer.ckpt)
        assert Ls[0][s].layer.get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
def test_tokens_past_31_bits(kind, dtype):
    """Sequences behind a place that 31 bits of elements do not reach (nothing before it is read)."""
    L, M = (Layer(kind, batch=3, heads=64, groups=2, dtype=dtype) for _ in range(2))
    first = (1 << 31) // (64 * L.R) + 1000
    T = first + 260
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("needs 80 GB")
    part = [t.to(DEV) for t in L.tokens(260, 3)]
    far = [torch.empty((T,) + t.shape[1:], dtype=t.dtype, device=DEV) for t in part]
    for f, t in zip(far, part):
        f[first:] = t
    out, want = (torch.zeros((n, 64, L.R), device=DEV) for n in (T, 260))
    L.layer.prefill(far, i32([first, first + 150, first + 170, T]), out)
    M.layer.prefill(part, i32([0, 150, 170, 260]), want)
    assert L.layer.get_status() == 0 and torch.equal(L.layer.ckpt, M.layer.ckpt)
    assert torch.equal(out[first:], want) and int(torch.count_nonzero(out[first - 100:first])) == 0
