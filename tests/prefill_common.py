"""Ragged prompts, layers and the token-by-token fp64 reference of the prefill tests."""
import numpy as np
import torch

from gpu_common import DEV, to64
from hybrid_ssm_decode_replayssm_b200 import rssm
from oracle import gdn as og
from oracle import kda as ok
from oracle import mamba2 as om

KINDS = ("mamba2", "gdn", "kda")
CODE = {"mamba2": rssm.RSSM_MAMBA2, "gdn": rssm.RSSM_GDN, "kda": rssm.RSSM_KDA}

# Outputs are fp32 sums of products of fp32 values.  One step of a recurrence rounds each
# state element a few times (2^-24 relative each) and a dot over 128 of them less than
# 8 * 2^-24 of their root sum of squares; gates of exp(-0.1 softplus(z)) forget with a time
# constant of about 14 tokens, so an error is at most some 14 * 8 * 2^-24 = 6.7e-6 of the
# result's scale.  Three times that is the bound on |got - want| / (|want| + rms(want)).
TOL = 2e-5


class Layer:
    """A layer with random checkpoints and its numbers on the host."""

    def __init__(self, kind, batch, heads=2, groups=1, dstate=128, dtype="bf16", seed=0, branching=False,
                 read_fmt=rssm.RSSM_READ_FP32, window=8, max_draft=4, out_scale=1.0, auto_flush=True):
        g = torch.Generator().manual_seed(1000 + seed)
        self.kind, self.H, self.G, self.batch = kind, heads, groups, batch
        self.R, self.C = (64, dstate) if kind == "mamba2" else (128, 128)
        self.scale = 1.0 if kind == "mamba2" else out_scale
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        gp = torch.Generator().manual_seed(7)          # one layer's parameters, whatever the batch
        self.A = -torch.exp(torch.rand(heads, generator=gp) * np.log(16.0))
        self.D = torch.randn(heads, generator=gp)
        slots = 2 * batch if branching else batch
        self.h0 = torch.randn((batch, heads, self.R, self.C), generator=g) * 0.1
        ckpt = torch.zeros((slots, heads, self.R, self.C), device=DEV)
        ckpt[:batch] = self.h0.to(DEV)
        self.dA, self.dD = self.A.to(DEV), self.D.to(DEV)
        desc = rssm.make_desc(CODE[kind], batch, heads, self.R, self.C, ngroups=groups, window=window,
                              max_draft=max_draft, in_dtype=rssm.RSSM_BF16 if dtype == "bf16" else rssm.RSSM_F32,
                              read_fmt=read_fmt, branching=branching, out_scale=out_scale, auto_flush=auto_flush)
        self.layer = rssm.ReplayLayer(desc, ckpt, self.dA, self.dD)
        self.state = self.h0.double().numpy().copy()   # the reference's state of every row

    def tokens(self, T, seed):
        """Packed inputs [T, ...] on the host."""
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        H, R, C, dt = self.H, self.R, self.C, self.dtype
        if self.kind == "mamba2":
            step = torch.nn.functional.softplus(0.5 * rn(T, H) - 1.0)
            return [rn(T, H, R).to(dt), rn(T, self.G, C).to(dt), rn(T, self.G, C).to(dt), step.to(dt)]
        q, k = (torch.nn.functional.normalize(rn(T, H, C), dim=-1).to(dt) for _ in range(2))
        z = rn(T, H, C) if self.kind == "kda" else rn(T, H)
        return [q, k, rn(T, H, R).to(dt), torch.exp(-0.1 * torch.nn.functional.softplus(z)), torch.sigmoid(rn(T, H))]

    def ref_run(self, state, toks):
        """fp64 (final state [H,R,C], outputs [n,H,R]) of one sequence's tokens."""
        S, outs = state[None].copy(), []
        t64 = [to64(t) for t in toks]
        for i in range(toks[0].shape[0]):
            at = [t[i][None] for t in t64]
            if self.kind == "mamba2":
                S, o = om.step(S, *at, to64(self.A), to64(self.D))
            else:
                S, o = (og if self.kind == "gdn" else ok).step(S, *at, self.scale)
            outs.append(o[0])
        return S[0], np.stack(outs) if outs else np.zeros((0, self.H, self.R))

    def rows(self):
        return to64(self.layer.checkpoint_rows())


def offsets_of(lens, first=0):
    off = [first]
    for n in lens:
        off.append(off[-1] + n)
    return off


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def scaled(got, want):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    rms = np.sqrt(np.mean(want ** 2)) if want.size else 0.0
    return float(np.max(np.abs(got - want) / (np.abs(want) + rms + 1e-30))) if want.size else 0.0
