"""The prefill scans and the row moves of the replay layers, as cases to be timed.

Two groups of operators, each in a plain form (elementary torch operations) and
through ``rssm.ReplayLayer``:

* prefill: a ragged batch of prompts runs through a layer's recurrence (gated
  delta rule, its per-channel form, or the Mamba-2 scan), starting from the
  checkpoints of the rows it is assigned to (or from zero) and leaving the final
  states there, with an output for every token;
* rows: sequences' states (checkpoint, read copy, window, pointers) copied from
  one layer's rows to another's, and the live rows of a batch moved together.
"""
import math
import random

import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few short chat turns arriving together, appended to running sequences
        dict(name="gdn short turns", op="gdn", heads=32, seqs=8, tokens=150, skew=0.6, fresh=0.0, rows=16, dtype="bf16", mix=1),
        # one long document read into a fresh row
        dict(name="gdn one long prompt", op="gdn", heads=32, seqs=1, tokens=8192, skew=0.0, fresh=1.0, rows=4, dtype="bf16", mix=2),
        # a prefill batch of ragged prompts, some of them continuing a row
        dict(name="gdn ragged batch", op="gdn", heads=32, seqs=11, tokens=20011, skew=0.8, fresh=0.7, rows=16, dtype="bf16", mix=3),
        # the fp32 parity layer with prompts of a few tokens
        dict(name="mamba2 fp32 short turns", op="mamba2", heads=8, groups=1, dstate=64, seqs=4, tokens=93, skew=0.5, fresh=0.5, rows=4, dtype="f32", mix=4),
        # one long document read into a fresh row of the serving layer
        dict(name="mamba2 one long prompt", op="mamba2", heads=128, groups=8, dstate=128, seqs=1, tokens=8192, skew=0.0, fresh=1.0, rows=4, dtype="bf16", mix=5),
        # a prefill batch of ragged prompts on the serving layer
        dict(name="mamba2 ragged batch", op="mamba2", heads=128, groups=8, dstate=128, seqs=9, tokens=15013, skew=0.8, fresh=0.7, rows=16, dtype="bf16", mix=6),
        # a few short turns on a layer with one gate per channel, fp32 inputs
        dict(name="kda fp32 short turns", op="kda", heads=8, seqs=5, tokens=77, skew=0.6, fresh=0.4, rows=8, dtype="f32", mix=7),
        # ragged prompts on a layer with one gate per channel
        dict(name="kda ragged batch", op="kda", heads=32, seqs=7, tokens=6007, skew=0.8, fresh=0.7, rows=8, dtype="bf16", mix=8),
        # three cached prefixes copied into the decode batch
        dict(name="copy 3 rows gdn", op="copy", kind="gdn", heads=32, rows=32, pairs=3, fp8=False, mix=9),
        # half a serving batch moves to a smaller layer, with its read copy
        dict(name="copy 96 rows mamba2 fp8", op="copy", kind="mamba2", heads=128, groups=8, dstate=128, rows=128, pairs=96, fp8=True, mix=10),
        # a small batch closes the gaps left by sequences that ended
        dict(name="compact 32 rows gdn", op="compact", kind="gdn", heads=32, rows=32, live=0.7, fp8=False, mix=11),
        # the serving batch closes its gaps
        dict(name="compact 256 rows mamba2", op="compact", kind="mamba2", heads=128, groups=8, dstate=128, rows=256, live=0.6, fp8=False, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gdn", "gdn", "mamba2", "mamba2", "kda", "copy", "compact"))
    mix = rng.randrange(1 << 20)
    if op in ("copy", "compact"):
        kind = rng.choice(("gdn", "mamba2", "kda"))
        c = dict(op=op, kind=kind, fp8=rng.random() < 0.4, mix=mix)
        if kind == "mamba2":
            c["groups"] = rng.choice((1, 2, 8))
            c["heads"] = c["groups"] * rng.choice((1, 3, 8, 16))
            c["dstate"] = rng.choice((64, 128))
            c["rows"] = _log(rng, 3, 200)
        else:
            c["heads"] = rng.choice((1, 5, 16, 32))
            c["rows"] = _log(rng, 3, 150)
        if op == "copy":
            c["pairs"] = max(1, min(c["rows"] * 3 // 4, _log(rng, 1, 100)))
        else:
            c["live"] = round(rng.uniform(0.2, 0.95), 3)
        return c
    seqs = _log(rng, 1, 24)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    top = {"gdn": 16000, "mamba2": 12000, "kda": 5000}[op] // (4 if dtype == "f32" else 1)
    c = dict(op=op, seqs=seqs, tokens=max(seqs, _log(rng, 1, top)), skew=round(rng.uniform(0.0, 0.8), 3),
             fresh=round(rng.uniform(0.0, 1.0), 3), rows=seqs + rng.randrange(0, 6), dtype=dtype, mix=mix)
    if op == "mamba2":
        c["groups"] = rng.choice((1, 2, 4, 8))
        c["heads"] = c["groups"] * rng.choice((2, 5, 8, 16))
        c["dstate"] = rng.choice((64, 128))
    else:
        c["heads"] = rng.choice((3, 8, 16, 32))
    return c


def _lengths(case):
    """Prompt lengths that add up to the case's tokens; with skew a few of them hold most."""
    r = random.Random(case["mix"])
    w = [math.exp(2.0 * case["skew"] * r.gauss(0.0, 1.0)) for _ in range(case["seqs"])]
    cut, acc, tot = [0], 0.0, sum(w)
    for x in w:
        acc += x
        cut.append(int(round(case["tokens"] * acc / tot)))
    return [b - a for a, b in zip(cut, cut[1:])]


def _layer(case):
    """(kind, heads, groups, rows R and columns C of a state, input dtype)"""
    kind = case.get("kind", case["op"])
    m2 = kind == "mamba2"
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    return kind, case["heads"], case.get("groups", 1), 64 if m2 else 128, case.get("dstate", 128), dt


WINDOW, DRAFT = 16, 4
CAP = WINDOW + DRAFT


def _rings(kind, B, H, G, R, C, dt):
    """The ring regions of a layer of B rows: [B, outer, entries, width]"""
    f = torch.float32
    if kind == "mamba2":
        return [((B, H, CAP, R), dt), ((B, G, CAP, C), dt), ((B, H, CAP, 1), f)]
    if kind == "kda":
        return [((B, H, CAP, C), dt), ((B, H, CAP, R), dt), ((B, H, CAP, C), f), ((B, H, CAP, 1), f),
                ((B, 2 * H, CAP, R // 2), f)]
    return [((B, H, CAP, C), dt), ((B, 2 * H, CAP, R // 2), dt), ((B, H, CAP, 1), f), ((B, H, CAP, 1), f),
            ((B, 2 * H, CAP, R // 2), f)]


# ---------------------------------------------------------------- prepare
def _randn(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _state(case, rows, g, full):
    """A layer of `rows` rows: its buffers as tensors, and (own) the layer bound to them."""
    kind, H, G, R, C, dt = _layer(case)
    std = 0.1 if kind == "mamba2" else 0.05
    s = {"ckpt": _randn(g, (rows, H, R, C), std)}
    if kind == "mamba2":
        s["A"] = -torch.exp(torch.rand(H, generator=g, device=DEV) * math.log(16.0))
        s["D"] = _randn(g, (H,))
    if full:
        meta = torch.zeros((4, rows), dtype=torch.int32, device=DEV)
        meta[0] = torch.randint(0, CAP, (rows,), generator=g, device=DEV, dtype=torch.int32)
        meta[1] = torch.randint(0, WINDOW, (rows,), generator=g, device=DEV, dtype=torch.int32)
        meta[3] = torch.randint(0, 50, (rows,), generator=g, device=DEV, dtype=torch.int32)
        rings = [_randn(g, shape).to(t) for shape, t in _rings(kind, rows, H, G, R, C, dt)]
        if case["fp8"]:
            s["codes"] = _randn(g, (rows, H, R, C), 100.0).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["scales"] = _randn(g, (rows, H, R)).abs() * 0.001
    if own:
        from hybrid_ssm_decode_replayssm_b200 import rssm
        desc = rssm.make_desc({"mamba2": rssm.RSSM_MAMBA2, "gdn": rssm.RSSM_GDN, "kda": rssm.RSSM_KDA}[kind], rows, H,
                              R, C, ngroups=G, window=WINDOW, max_draft=DRAFT,
                              in_dtype=rssm.RSSM_F32 if dt == torch.float32 else rssm.RSSM_BF16,
                              read_fmt=rssm.RSSM_READ_FP8_E4M3_ROW if case.get("fp8") else rssm.RSSM_READ_FP32)
        layer = s["layer"] = rssm.ReplayLayer(desc, s["ckpt"], s.get("A"), s.get("D"))
        if full:
            at = layer.layout
            views = []
            for off, (shape, t) in zip(at.buf_off, _rings(kind, rows, H, G, R, C, dt)):
                n = math.prod(shape) * t.itemsize
                views.append(layer.buf[off:off + n].view(t).view(shape))
            for v, r in zip(views, rings):
                v.copy_(r)
            rings = views
            # start, len, pending, flushes follow one another in meta, equally far apart
            ptrs = layer.meta.view(torch.int32).as_strided((4, rows), ((at.meta_len_off - at.meta_start_off) // 4, 1))
            meta = ptrs.copy_(meta)
            if case["fp8"]:
                codes, scales = layer.read_copy_views()
                codes = codes.view(torch.float8_e4m3fn)
                codes.copy_(s["codes"])
                scales.copy_(s["scales"])
                s["codes"], s["scales"] = codes, scales
    if full:
        s["rings"], s["meta"] = rings, meta
    return s


def _inputs(case, g):
    kind, H, G, R, C, dt = _layer(case)
    T = case["tokens"]
    if kind == "mamba2":
        x, B, Cm = _randn(g, (T, H, R)).to(dt), _randn(g, (T, G, C)).to(dt), _randn(g, (T, G, C)).to(dt)
        step = torch.log1p(torch.exp(_randn(g, (T, H), 0.5) - 1.0)).to(dt)
        return [x, B, Cm, step]
    q, k = (torch.empty((T, H, C), device=DEV, dtype=dt) for _ in range(2))
    for t in (q, k):
        n = _randn(g, (T, H, C))
        t.copy_(n / n.square().sum(-1, keepdim=True).sqrt())
    v = _randn(g, (T, H, R)).to(dt)
    z = _randn(g, (T, H, C) if kind == "kda" else (T, H))
    alpha = torch.exp(-0.1 * torch.log1p(torch.exp(z)))
    beta = torch.sigmoid(_randn(g, (T, H)))
    return [q, k, v, alpha, beta]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = random.Random(case["mix"] + 1)
    op, rows = case["op"], case["rows"]
    if op == "copy":
        n = case["pairs"]
        return {"case": case, "src": _state(case, rows, g, True), "dst": _state(case, max(n, rows * 3 // 4), g, True),
                "src_rows": torch.tensor([r.randrange(rows) for _ in range(n)], dtype=torch.int32, device=DEV),
                "dst_rows": torch.tensor(r.sample(range(max(n, rows * 3 // 4)), n), dtype=torch.int32, device=DEV)}
    if op == "compact":
        live = [int(r.random() < case["live"]) for _ in range(rows)]
        return {"case": case, "at": _state(case, rows, g, True), "live": torch.tensor(live, dtype=torch.int32, device=DEV)}
    lens = _lengths(case)
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    kind, H, G, R, C, dt = _layer(case)
    s = {"case": case, "at": _state(case, rows, g, False), "in": _inputs(case, g), "lens": lens,
         "rows": torch.tensor(r.sample(range(rows), len(lens)), dtype=torch.int32, device=DEV),
         "fresh": torch.tensor([int(r.random() < case["fresh"]) for _ in lens], dtype=torch.int32, device=DEV),
         "offsets": torch.tensor(off, dtype=torch.int32, device=DEV),
         "out": torch.zeros((case["tokens"], H, R), device=DEV)}
    return s


# -------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if op == "copy":
        if own:
            state["dst"]["layer"].copy_rows(state["src"]["layer"], state["dst_rows"], state["src_rows"])
        else:
            _move(state["dst"], state["src"], state["dst_rows"].long(), state["src_rows"].long())
        return _buffers(state["dst"])
    if op == "compact":
        if own:
            new_row, n_live = state["at"]["layer"].compact_rows(state["live"])
        else:
            new_row, n_live = _compact(state)
        return {"new_row": new_row, "n_live": n_live, **_buffers(state["at"])}
    if own:
        state["at"]["layer"].prefill(state["in"], state["offsets"], state["out"], rows=state["rows"],
                                     fresh=state["fresh"])
    else:
        _prefill(state)
    return {"out": state["out"], "ckpt": state["at"]["ckpt"]}


def _buffers(s):
    return {k: s[k] for k in ("ckpt", "codes", "scales", "rings", "meta") if k in s}


# ------------------------------------------------- plain forms: row moves
def _move(dst, src, d, s):
    """Rows s of src to rows d of dst: states whole, of each ring the entries in use."""
    for key in ("ckpt", "scales"):
        if key in dst:
            dst[key][d] = src[key][s]
    if "codes" in dst:
        dst["codes"].view(torch.uint8)[d] = src["codes"].view(torch.uint8)[s]
    start, n = src["meta"][0][s], src["meta"][1][s]
    place = torch.arange(CAP, device=DEV)
    used = (place - start[:, None]) % CAP < n[:, None]
    for x, y in zip(dst["rings"], src["rings"]):
        x[d] = torch.where(used[:, None, :, None], y[s], x[d])
    for x, y in zip(dst["meta"], src["meta"]):
        x[d] = y[s]


def _compact(state):
    """The live rows behind the first n_live take the places of the dead rows among those."""
    live = state["live"] != 0
    at = torch.arange(live.numel(), device=DEV)
    n_live = live.sum()
    holes, movers = torch.nonzero(~live & (at < n_live))[:, 0], torch.nonzero(live & (at >= n_live))[:, 0]
    new_row = torch.where(live, at, -1)
    new_row[movers] = holes
    _move(state["at"], state["at"], holes, movers)
    return new_row.to(torch.int32), n_live.to(torch.int32).reshape(1)


# -------------------------------------------------- plain forms: prefill
def _padded(x, lens, c):
    """[tokens, heads, ...] -> fp32 [seqs, heads, chunks, c, ...], zeros behind each sequence."""
    chunks = max(1, -(-max(lens) // c))
    y = torch.zeros((len(lens), chunks * c) + tuple(x.shape[1:]), device=DEV)
    at = 0
    for i, n in enumerate(lens):
        y[i, :n] = x[at:at + n]
        at += n
    return y.view((len(lens), chunks, c) + tuple(x.shape[1:])).movedim(3, 1).contiguous()


def _unpadded(out, y, lens):
    """[seqs, heads, chunks, c, rows] into out [tokens, heads, rows]"""
    y = y.movedim(1, 3).flatten(1, 2)
    at = 0
    for i, n in enumerate(lens):
        out[at:at + n] = y[i, :n]
        at += n


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A, by forward substitution over the rows."""
    T = torch.eye(A.shape[-1], device=DEV).expand(A.shape).clone()
    for i in range(1, A.shape[-1]):
        T[..., i, :i] = -(A[..., i, None, :i] @ T[..., :i, :i])[..., 0, :]
    return T


def _prefill(s):
    """Chunk by chunk: within a chunk products of all its tokens, between chunks the state."""
    kind, H, G, R, C, dt = _layer(s["case"])
    lens, rows, ckpt = s["lens"], s["rows"].long(), s["at"]["ckpt"]
    S = torch.where(s["fresh"][:, None, None, None] != 0, 0.0, ckpt[rows])
    c = 16 if kind == "kda" else 64
    i = torch.arange(c, device=DEV)
    low, strict = i[:, None] >= i, i[:, None] > i
    if kind == "mamba2":
        x, B, Cm, step = (_padded(t, lens, c) for t in s["in"])
        heads = torch.arange(H, device=DEV) // (H // G)
        a = (step.double() * s["at"]["A"].double()[:, None, None]).cumsum(-1)
        seg = torch.where(low, a[..., :, None] - a[..., None, :], NEG).exp().float()
        M = seg * (Cm @ B.transpose(-1, -2))[:, heads] * step[..., None, :]
        y = M @ x + s["at"]["D"][:, None, None, None] * x
        tail = (step * (a[..., -1:] - a).exp().float())[..., None] * x
        lead, whole = a.exp().float()[..., None], a[..., -1].exp().float()
        for j in range(x.shape[2]):
            y[:, :, j] += lead[:, :, j] * (Cm[:, heads, j] @ S.transpose(-1, -2))
            S = whole[:, :, j, None, None] * S + tail[:, :, j].transpose(-1, -2) @ B[:, heads, j]
        _unpadded(s["out"], y, lens)
        ckpt[rows] = S
        return
    q, k, v, alpha, beta = s["in"]
    q, k, v, a, beta = (_padded(t, lens, c) for t in (q, k, v, alpha.log(), beta))
    a = a.double().cumsum(3)
    if kind == "kda":
        seg = torch.where(low[..., None], a[:, :, :, :, None] - a[:, :, :, None], NEG).exp().float() * k[:, :, :, None]
        KK = (seg * k[:, :, :, :, None]).sum(-1)
        M = (seg * q[:, :, :, :, None]).sum(-1)
        lead, whole, tail = a.exp().float(), a[:, :, :, -1:].exp().float(), (a[:, :, :, -1:] - a).exp().float()
    else:
        seg = torch.where(low, a[..., :, None] - a[..., None, :], NEG).exp().float()
        KK, M = seg * (k @ k.transpose(-1, -2)), seg * (q @ k.transpose(-1, -2))
        lead, whole, tail = a.exp().float()[..., None], a[..., -1:, None].exp().float(), (a[..., -1:] - a).exp().float()[..., None]
    T = _inverse(torch.where(strict, beta[..., None] * KK, 0.0))
    kl, ql, kt, o = k * lead, q * lead, k * tail, torch.empty_like(v)
    for j in range(q.shape[2]):
        St = S.transpose(-1, -2)
        w = T[:, :, j] @ (beta[:, :, j, :, None] * (v[:, :, j] - kl[:, :, j] @ St))
        o[:, :, j] = ql[:, :, j] @ St + M[:, :, j] @ w
        S = whole[:, :, j] * S + w.transpose(-1, -2) @ kt[:, :, j]
    _unpadded(s["out"], o, lens)
    ckpt[rows] = S


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """Token by token (prefill) and row by row (moves) from the definitions, in 64 bits."""
    kind, H, G, R, C, dt = _layer(case)
    s = prepare(case, seed)
    if case["op"] in ("copy", "compact"):
        return _exact_rows(case, s)
    lens, rows = s["lens"], s["rows"].tolist()
    ckpt = s["at"]["ckpt"].double()
    # sequences by falling length: at step t those longer than t are the first ones
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    first = [int(o) for o in s["offsets"][:-1].tolist()]
    S = torch.stack([torch.zeros_like(ckpt[0]) if s["fresh"][i] else ckpt[rows[i]] for i in order])
    out = torch.zeros(s["out"].shape, device=DEV, dtype=torch.float64)
    begin = torch.tensor([first[i] for i in order], device=DEV)
    alive = len(order)
    for t in range(max(lens)):
        while lens[order[alive - 1]] <= t:
            alive -= 1
        at = begin[:alive] + t
        h = S[:alive]
        if kind == "mamba2":
            x, B, Cm, step = (z[at].double() for z in s["in"])
            B, Cm = B.repeat_interleave(H // G, 1), Cm.repeat_interleave(H // G, 1)
            h.mul_(torch.exp(step * s["at"]["A"].double())[..., None, None])
            h.add_((step[..., None] * x)[..., None] * B[:, :, None, :])
            out[at] = (h @ Cm[..., None])[..., 0] + s["at"]["D"].double()[:, None] * x
        else:
            q, k, v, alpha, beta = (z[at].double() for z in s["in"])
            h.mul_(alpha[:, :, None, :] if kind == "kda" else alpha[..., None, None])
            w = beta[..., None] * (v - (h @ k[..., None])[..., 0])
            h.add_(w[..., None] * k[:, :, None, :])
            out[at] = (h @ q[..., None])[..., 0]
    for j, i in enumerate(order):
        ckpt[rows[i]] = S[j]
    return {"out": out, "ckpt": ckpt}


def _exact_rows(case, s):
    if case["op"] == "copy":
        dst, src = s["dst"], s["src"]
        pairs = list(zip(s["dst_rows"].tolist(), s["src_rows"].tolist()))
        told = {}
    else:
        dst = src = s["at"]
        live = s["live"].tolist()
        n = sum(live)
        holes = [b for b in range(n) if not live[b]]
        movers = [b for b in range(n, len(live)) if live[b]]
        pairs = list(zip(holes, movers))
        to = dict(zip(movers, holes))
        told = {"new_row": torch.tensor([to.get(b, b) if live[b] else -1 for b in range(len(live))], dtype=torch.int32),
                "n_live": torch.tensor([n], dtype=torch.int32)}
    start, used = src["meta"][0].tolist(), src["meta"][1].tolist()
    for d, b in pairs:
        for key in ("ckpt", "scales"):
            if key in dst:
                dst[key][d].copy_(src[key][b])
        if "codes" in dst:
            dst["codes"].view(torch.uint8)[d].copy_(src["codes"].view(torch.uint8)[b])
        for e in range(used[b]):
            for x, y in zip(dst["rings"], src["rings"]):
                x[d][:, (start[b] + e) % CAP].copy_(y[b][:, (start[b] + e) % CAP])
        for x, y in zip(dst["meta"], src["meta"]):
            x[d].copy_(y[b])
    wide = {k: dst[k].float().double() for k in ("scales", "codes") if k in dst}
    return {**told, "ckpt": dst["ckpt"].double(), **wide, "rings": [r.double() for r in dst["rings"]],
            "meta": list(dst["meta"])}


# ------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; the recurrence's own multiply-adds."""
    kind, H, G, R, C, dt = _layer(case)
    word = 2 if dt == torch.bfloat16 else 4
    row = 4 * H * R * C + (H * R * (C + 4) if case.get("fp8") else 0)
    ring = sum(math.prod(shape[1:]) * t.itemsize for shape, t in _rings(kind, 1, H, G, R, C, dt))
    if case["op"] in ("copy", "compact"):
        if case["op"] == "copy":
            moved = case["pairs"]
        else:
            r = random.Random(case["mix"] + 1)
            live = [int(r.random() < case["live"]) for _ in range(case["rows"])]
            moved = sum(live[sum(live):])
        return {"bytes": 2 * moved * (row + ring * (WINDOW - 1) / 2 / CAP) + 12 * case["rows"], "flops": 0}
    T, n = case["tokens"], case["seqs"]
    if kind == "mamba2":
        per = word * (H * R + 2 * G * C + H) + 4 * H * R
        flops = H * (4 * R * C + 3 * R)
    else:
        per = word * H * (2 * C + R) + 4 * H * (C if kind == "kda" else 1) + 4 * H + 4 * H * R
        flops = H * (6 * R * C)
    return {"bytes": T * per + row * n * (2 - case["fresh"]), "flops": T * flops}
