"""Host-side checks of rssm_prefill, rssm_copy_rows and rssm_compact_rows: every refusal
returns its code before anything is enqueued (no GPU used)."""
import ctypes as C
import random

import pytest
import torch

from hybrid_ssm_decode_replayssm_b200 import rssm

FAKE = 1 << 20      # a device address that the refused calls never read


def _handle(kind=rssm.RSSM_GDN, params=True, **kw):
    base = dict(batch=4, nheads=8, headdim=128, dstate=128, window=16, max_draft=4, in_dtype=rssm.RSSM_BF16)
    if kind == rssm.RSSM_MAMBA2:
        base.update(headdim=64, ngroups=2)
    base.update(kw)
    h = C.c_void_p()
    d = rssm.make_desc(kind, **base)
    rc = FAKE if base.get("read_fmt") else None
    assert rssm.lib().rssm_create(C.byref(d), FAKE, FAKE, rc, FAKE, C.byref(h)) == rssm.RSSM_OK
    if params:
        assert rssm.lib().rssm_set_params(h, FAKE, FAKE) == rssm.RSSM_OK
    return h


def _prefill(h, n_seq=2, T=64, off=FAKE, rows=FAKE, fresh=None, ins=None, strides=None, out=FAKE, work=FAKE,
             nbytes=1 << 20, n_in=5):
    arr = None if ins == "null" else (C.c_void_p * 5)(*(ins or [FAKE] * n_in))
    st = None if strides is None else (C.c_int64 * 5)(*strides)
    return rssm.lib().rssm_prefill(h, n_seq, T, off, rows, fresh, arr, st, out, work, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(n_seq=0), dict(n_seq=5), dict(n_seq=-1), dict(T=-1), dict(off=None), dict(ins="null"),
    dict(ins=[FAKE, None, FAKE, FAKE, FAKE]), dict(ins=[FAKE, FAKE + 8, FAKE, FAKE, FAKE]), dict(out=None),
    dict(out=FAKE + 4), dict(out=FAKE + 16), dict(work=None), dict(work=FAKE + 16), dict(nbytes=0),
    dict(strides=[1023, 1024, 1024, 8, 8]), dict(strides=[1024, 1025, 1024, 8, 8]),
    dict(strides=[1024, 1024, 0, 8, 8]), dict(strides=[1024, 1024, 1024, 7, 8]), dict(strides=[-1024, 1024, 1024, 8, 8]),
])
def test_prefill_arguments(kw):
    h = _handle()
    before = rssm.lib().rssm_launch_count()
    assert _prefill(h, **kw) == rssm.RSSM_ERR_INVALID_ARG
    assert rssm.lib().rssm_last_error_string() and rssm.lib().rssm_launch_count() == before
    rssm.lib().rssm_destroy(h)


@pytest.mark.parametrize("kind,dtype,free", [
    (rssm.RSSM_MAMBA2, rssm.RSSM_BF16, {3: 2}), (rssm.RSSM_MAMBA2, rssm.RSSM_F32, {3: 4}),
    (rssm.RSSM_GDN, rssm.RSSM_BF16, {3: 4, 4: 4}), (rssm.RSSM_KDA, rssm.RSSM_BF16, {4: 4})])
def test_prefill_alignment_of_each_input(kind, dtype, free):
    """Inputs with one value per head may begin at any element, the others on 16 bytes.  (The calls
    that pass this check fail at the next, the workspace's size.)"""
    h = _handle(kind, in_dtype=dtype)
    for i in range(4 if kind == rssm.RSSM_MAMBA2 else 5):
        for off in (1, 2, 4, 8):
            ins = [FAKE] * 5
            ins[i] += off
            assert _prefill(h, ins=ins, nbytes=0) == rssm.RSSM_ERR_INVALID_ARG
            text = rssm.lib().rssm_last_error_string().decode()
            taken = i in free and off % free[i] == 0
            assert ("workspace" if taken else f"in[{i}]") in text, (i, off, text)
    rssm.lib().rssm_destroy(h)


def test_prefill_needs_a_handle_and_parameters():
    assert _prefill(None) == rssm.RSSM_ERR_INVALID_ARG
    h = _handle(rssm.RSSM_MAMBA2, params=False)
    for T in (0, 64):
        assert _prefill(h, T=T) == rssm.RSSM_ERR_STATE
    rssm.lib().rssm_destroy(h)


def test_prefill_workspace_size():
    h = _handle()
    n = C.c_size_t()
    size = rssm.lib().rssm_prefill_workspace_size
    assert size(h, 4, 1000, C.byref(n)) == rssm.RSSM_OK and n.value > 0
    assert _prefill(h, n_seq=4, T=1000, nbytes=n.value - 1) == rssm.RSSM_ERR_INVALID_ARG
    for bad in ((None, 1, 1), (h, 0, 1), (h, 5, 1), (h, 1, -1)):
        assert size(*bad, C.byref(n)) == rssm.RSSM_ERR_INVALID_ARG
    assert size(h, 1, 1, None) == rssm.RSSM_ERR_INVALID_ARG
    rssm.lib().rssm_destroy(h)


def _work_size(h, n_seq, n_tokens):
    n = C.c_size_t()
    assert rssm.lib().rssm_prefill_workspace_size(h, n_seq, n_tokens, C.byref(n)) == rssm.RSSM_OK
    return n.value


RECORD = {rssm.RSSM_GDN: (26 * 1024, 41), rssm.RSSM_KDA: (48 * 1024, 97)}   # bytes per chunk and head, shortest in chunks


@pytest.mark.parametrize("kind", list(RECORD))
def test_prefill_workspace_of_many_short_turns(kind):
    """The workspace is what the header says: chunks that the tokens allow, not one per sequence."""
    each, least = RECORD[kind]
    h = _handle(kind, batch=256, nheads=32)
    plan = lambda n: 32 * n + 4 * 256 + 1536   # noqa: E731
    for n_seq, T in ((256, 256), (256, 193), (200, 400), (256, 5000), (3, 5000), (1, 8192)):
        got = _work_size(h, n_seq, T)
        chunks = T // 64 + min(n_seq, T // least)
        assert each * 32 * chunks < got <= each * 32 * chunks + plan(n_seq), (n_seq, T)
    assert _work_size(h, 256, 192) <= plan(256)
    rssm.lib().rssm_destroy(h)
    for kw in (dict(kind=kind, in_dtype=rssm.RSSM_F32), dict(kind=rssm.RSSM_MAMBA2)):
        h = _handle(batch=256, nheads=32, **kw)
        assert _work_size(h, 256, 100000) <= plan(256)
        rssm.lib().rssm_destroy(h)


@pytest.mark.parametrize("kind", list(RECORD))
def test_prefill_workspace_holds_every_batch(kind):
    """Whatever the lengths: the chunks of the long sequences fit."""
    each, least = RECORD[kind]
    h = _handle(kind, batch=64, nheads=1)
    r = random.Random(3)
    for case in range(400):
        n = r.randrange(1, 65)
        top = r.choice((least, least + 1, 2 * least, 64 * 3 + 1, 700))
        lens = [r.choice((0, 1, least - 1, least, 65, 129, r.randrange(top + 1))) for _ in range(n)]
        if case % 4 == 0:
            lens = [least] * n
        T = sum(lens)
        if T > 192:
            used = sum(-(-x // 64) for x in lens if x >= least)
            assert used * each <= _work_size(h, n, T) - (32 * n + 4 * 64 + 1024), (lens,)
    rssm.lib().rssm_destroy(h)


@pytest.mark.parametrize("kw", [
    dict(nheads=4), dict(window=8), dict(max_draft=2), dict(in_dtype=rssm.RSSM_F32), dict(read_fmt=rssm.RSSM_READ_NVFP4),
    dict(kind=rssm.RSSM_KDA), dict(kind=rssm.RSSM_MAMBA2)])
def test_copy_rows_between_layers_that_differ(kw):
    a, b = _handle(), _handle(**kw)
    assert rssm.lib().rssm_copy_rows(a, b, 1, FAKE, FAKE, None) == rssm.RSSM_ERR_INVALID_ARG
    assert rssm.lib().rssm_copy_rows(b, a, 1, FAKE, FAKE, None) == rssm.RSSM_ERR_INVALID_ARG
    for h in (a, b):
        rssm.lib().rssm_destroy(h)


def test_row_move_arguments():
    L, h = rssm.lib(), _handle()
    bad = [(None, h, 1, FAKE, FAKE), (h, None, 1, FAKE, FAKE), (h, h, 0, FAKE, FAKE), (h, h, 5, FAKE, FAKE),
           (h, h, 1, None, FAKE), (h, h, 1, FAKE, None)]
    for args in bad:
        assert L.rssm_copy_rows(*args, None) == rssm.RSSM_ERR_INVALID_ARG
    for args in [(None, FAKE, FAKE, FAKE), (h, None, FAKE, FAKE), (h, FAKE, None, FAKE), (h, FAKE, FAKE, None),
                 (h, FAKE, FAKE, FAKE + 256), (h, FAKE, FAKE + 256, FAKE)]:
        assert L.rssm_compact_rows(*args, None) == rssm.RSSM_ERR_INVALID_ARG
    L.rssm_destroy(h)


class _Bare(rssm.ReplayLayer):
    """A layer's Python checks without a GPU: host tensors, and no call reaches the library."""

    def __init__(self, kind=rssm.RSSM_GDN):
        self.desc = rssm.make_desc(kind, 4, 2, 128, 128)
        self.ckpt = torch.zeros(4, 2, 128, 128)
        self.handle = None


def _ok(T=6):
    t = torch.bfloat16
    return [torch.zeros(T, 2, 128, dtype=t), torch.zeros(T, 2, 128, dtype=t), torch.zeros(T, 2, 128, dtype=t),
            torch.zeros(T, 2), torch.zeros(T, 2)]


@pytest.mark.parametrize("change", [
    lambda i, o, r: (i[:4], o, r), lambda i, o, r: ([i[0].float()] + i[1:], o, r),
    lambda i, o, r: ([i[0][:5]] + i[1:], o, r), lambda i, o, r: ([i[0].transpose(1, 2).contiguous().transpose(1, 2)] + i[1:], o, r),
    lambda i, o, r: (i, o.bfloat16(), r), lambda i, o, r: (i, o[:, :1], r), lambda i, o, r: (i, o[:, :, :64], r),
    lambda i, o, r: (i, o, r.long()), lambda i, o, r: (i, o, r[:1]), lambda i, o, r: (i, o.transpose(1, 2), r)])
def test_python_prefill_checks(change):
    off = torch.tensor([0, 2, 6], dtype=torch.int32)
    ins, out, rows = change(_ok(), torch.zeros(6, 2, 128), torch.tensor([0, 1], dtype=torch.int32))
    with pytest.raises(ValueError):
        _Bare().prefill(ins, off, out, rows=rows)


def test_python_row_checks():
    L = _Bare()
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: L.copy_rows(L, i, i[:2]), lambda: L.copy_rows(L, i.long(), i), lambda: L.compact_rows(i[:3]),
                 lambda: L.compact_rows(i.bool()), lambda: L.copy_rows(L, [0], [1])):
        with pytest.raises((ValueError, AttributeError)):
            call()
