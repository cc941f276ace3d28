"""Plain 64-bit form of the masked attention (nvkv_score_mod) for the tests,
with a bound of how far a kernel's bf16 output may be from it, and small
random caches written by the oracle."""
from __future__ import annotations

from dataclasses import dataclass, field

import numpy as np
import torch

import oracle
import nvfp4_quantized_kv_b200 as nv

LOG2E = 1.4426950408889634


@dataclass
class Mod:
    cap: float = 0.0
    window: int = 0
    slopes: list | None = None      # per query head
    prefix: list | None = None      # per sequence
    starts: list | None = None      # decode: per sequence; prefill: per row

    def device(self, dev):
        t = lambda v, d: None if v is None else torch.tensor(v, dtype=d, device=dev)
        return nv.ScoreMod(self.cap, self.window, t(self.slopes, torch.float32),
                           t(self.prefix, torch.int32), t(self.starts, torch.int32))


def visible(p, kv_len, start, window, prefix):
    """Keys a query at position p sees, as a list, by the definition (one key
    at a time)."""
    out = []
    for j in range(kv_len):
        causal = j <= p
        ahead = p < j < prefix and p < prefix
        near = not window or (p - j < window and j - p < window)
        if p >= 0 and j >= start and (causal or ahead) and near:
            out.append(j)
    return out


def interval(p, kv_len, start, window, prefix):
    """The same set as an interval (vectorised over nothing; used for long
    sequences)."""
    if p < 0:
        return 0, 0
    lo = max(0, start, p - window + 1 if window else 0)
    hi = p + 1
    if prefix > p:
        hi = min(prefix, p + window) if window else prefix
    return lo, min(hi, kv_len)


def bits(x):
    t = torch.as_tensor(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


@dataclass
class Case:
    """A random cache of ragged sequences (written by the oracle) and its
    dequantised rows khat[b], vhat[b]: float64 [kv_len][Hkv][D]."""
    Hq: int
    Hkv: int
    D: int
    lens: list
    n: list                       # query rows of each sequence
    seed: int = 0
    k8: bool = False
    q_gain: float = 1.0
    fill: int = 0xA5
    pool: np.ndarray = field(init=False)

    def __post_init__(self):
        rng = np.random.default_rng([self.seed, self.D, self.Hq])
        pages = [(l + 15) // 16 for l in self.lens]
        self.num_pages = sum(pages) + 3
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.max_pages = max(1, max(pages))
        self.pt = np.full((len(self.lens), self.max_pages), -1, np.int32)
        at = 0
        for b, m in enumerate(pages):
            self.pt[b, :m] = perm[at:at + m]
            at += m
        total = sum(self.lens)
        loud = np.where(np.arange(self.D) % 61 == 5, 8.0, 1.0)
        k = bits(rng.standard_normal((total, self.Hkv, self.D)) * loud)
        v = bits(rng.standard_normal((total, self.Hkv, self.D)))
        cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        lens = np.array(self.lens, np.int32)
        pb = oracle.k8v4_page_bytes(self.Hkv, self.D) if self.k8 else oracle.page_bytes(self.Hkv, self.D)
        self.pool = np.full(self.num_pages * pb, self.fill, np.uint8)
        if total:
            f = oracle.append_k8v4 if self.k8 else oracle.append
            f(self.pool, self.Hkv, self.D, self.pt, lens, k, v, cu)
        self.khat, self.vhat = [], []
        for b, l in enumerate(self.lens):
            kb, vb = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
            if l == 0:
                z = np.zeros((0, self.Hkv, self.D))
                self.khat.append(z)
                self.vhat.append(z)
                continue
            self.vhat.append(oracle.qdq_rows(np.ascontiguousarray(vb)))
            if self.k8:
                kr = np.zeros(kb.shape)
                for i in range(l):
                    for h in range(self.Hkv):
                        codes, sc = oracle.k8_quantize_row(kb[i, h])
                        kr[i, h] = [oracle.k8_dequant(int(c), sc) for c in codes]
                self.khat.append(kr)
            else:
                self.khat.append(oracle.qdq_rows(np.ascontiguousarray(kb)))
        self.q = bits(rng.standard_normal((sum(self.n), self.Hq, self.D)) * self.q_gain)
        self.cu = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)

    # ---- device side
    def device(self, dev="cuda"):
        dev = torch.device(dev)
        fmt = "k8v4" if self.k8 else "nvfp4"
        self.cache = nv.Cache(torch.from_numpy(self.pool.copy()).to(dev), self.num_pages, self.Hkv,
                              self.D, fmt)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.seqs = nv.Seqs(torch.from_numpy(self.pt).to(dev),
                            torch.tensor(self.lens, dtype=torch.int32, device=dev),
                            self.max_pages * 16, self.err)
        self.q_dev = torch.from_numpy(self.q.view(np.int16)).to(dev).view(torch.bfloat16)
        self.cu_dev = torch.from_numpy(self.cu).to(dev)
        return self

    # ---- reference
    def q64(self):
        return torch.from_numpy((self.q.astype(np.uint32) << 16).view(np.float32).astype(np.float64))

    def reference(self, mod: Mod, scale: float, decode: bool, slack: str):
        """(out, bound): float64 [rows][Hq][D].  slack names the kernel's
        arithmetic ("fp32", "f16 weights" or "f16 scores")."""
        G = self.Hq // self.Hkv
        q = self.q64()
        out = torch.zeros(sum(self.n), self.Hq, self.D, dtype=torch.float64)
        tol = torch.zeros_like(out)
        for b, l in enumerate(self.lens):
            if self.n[b] == 0:
                continue
            j = torch.arange(l)
            rng = []
            for i in range(self.n[b]):
                p = l - self.n[b] + i
                st = 0 if mod.starts is None else mod.starts[b if decode else self.cu[b] + i]
                rng.append((p,) + interval(p, l, st, mod.window, mod.prefix[b] if mod.prefix else 0))
            r = torch.tensor(rng)
            seen = (j >= r[:, 1:2]) & (j < r[:, 2:3])
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            for h in range(self.Hkv):
                k = torch.from_numpy(np.ascontiguousarray(self.khat[b][:, h]))
                v = torch.from_numpy(np.ascontiguousarray(self.vhat[b][:, h]))
                for g in range(G):
                    hq = h * G + g
                    o, t = attend(q[rows, hq], k, v, seen, r[:, 0], j, scale, mod.cap,
                                  mod.slopes[hq] if mod.slopes else 0.0, slack)
                    out[rows, hq], tol[rows, hq] = o, t
        return out, tol


def attend(q, k, v, seen, p, j, scale, cap, slope, slack):
    x0 = q @ k.t() * scale
    x = cap * torch.tanh(x0 / cap) if cap else x0
    dist = (p[:, None] - j).abs().double()
    slope = float(np.float32(slope))
    x = x - slope * dist
    x = torch.where(seen, x, -torch.inf)
    top = x.amax(1, keepdim=True) if x.shape[1] else torch.full((x.shape[0], 1), -torch.inf)
    some = torch.isfinite(top)
    top = torch.where(some, top, 0.0)
    w = torch.where(seen, torch.exp(x - top), 0.0)
    total = w.sum(1, keepdim=True)
    w = w / torch.where(total > 0, total, 1.0)
    o = w @ v
    # How far a score may be off, in natural-log units.  Exact products of
    # codes and scales, fp32 sums of D terms (at most D roundings of partial
    # sums no larger than sum |q k|): eps_s * sum |q k|; q as f16 adds 2^-11
    # (one rounding of each element), and so does q * scale in fp32 (2^-24).
    absqk = q.abs() @ k.abs().t() * abs(scale)
    eps = (k.shape[1] + 4) * 2.0 ** -24 + (2.0 ** -11 if slack == "f16 scores" else 1e-6)
    off = absqk * eps
    if cap:
        # the cap itself is good to 2^-18 of its result
        off = torch.minimum(off, torch.full_like(off, 2 * cap)) + x.abs() * 2.0 ** -18
    if slope:
        # slope * log2e rounded once, the product with the distance rounded,
        # the sum rounded: 3 roundings of 2^-24 of the bias
        off = off + 3 * 2.0 ** -24 * abs(slope) * dist
    # the running maximum is subtracted in fp32 base-2 units, exp2 is good to
    # 2^-22, the weight is rounded to f16 (2^-11; below 2^-14 absolutely, at
    # most 2^-25 of a weight of at least 2^-8, the lazy maximum)
    span = torch.where(seen, (top - x), 0.0)
    rel = off + (off.amax(1, keepdim=True) if off.shape[1] else 0) + 2.0 ** -21 + 2.0 ** -23 * span
    sub = torch.zeros_like(w)
    if slack != "fp32":
        rel = rel + 2.0 ** -11
        sub = torch.where(seen, 2.0 ** -25 * 2.0 ** 8 / torch.where(total > 0, total, 1.0), 0.0)
    if slack == "f16 scores":
        # the exponent x - m is rounded to f16 before the exponential: 2^-11
        # of its size in base 2, which is at most 8 above and `span` below
        rel = rel + 2.0 ** -11 * torch.maximum(span, torch.full_like(span, 8 * 0.6931))+ 2.0 ** -11
    rel = torch.expm1(rel.clamp(max=30.0))
    dev = torch.zeros_like(o)
    wr = w * rel + sub
    for c0 in range(0, v.shape[1], 32):  # sum_j wr |v_j - o|, 32 channels at a time
        dv = (v[None, :, c0:c0 + 32] - o[:, None, c0:c0 + 32]).abs()
        dev[:, c0:c0 + 32] = (wr[:, :, None] * dv).sum(1)
    # fp32 sums over the keys and the splits, then one rounding to bf16 (2^-8)
    tol = dev * 1.01 + 2.0 ** -18 * (w @ v.abs())
    tol = tol + 2.0 ** -8 * (o.abs() + tol) + 1e-30
    return o, tol


def run_decode(case: Case, mod: Mod, T: int, scale: float, splits: int = 0):
    ws = torch.full((nv.nvkv_decode_workspace_bytes(len(case.lens), T, case.Hq, case.Hkv, case.D, splits),),
                    0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((sum(case.n), case.Hq, case.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    m = mod.device("cuda")
    nv.nvkv_decode_attn_mod(case.cache, case.seqs, case.q_dev, T, case.Hq, scale, m, splits, ws, out)
    torch.cuda.synchronize()
    return out


def run_prefill(case: Case, mod: Mod, scale: float, splits: int = 0):
    total = sum(case.n)
    size = nv.nvkv_prefill_workspace_bytes(total, case.Hq, case.D, splits)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
    out = torch.full((total, case.Hq, case.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    m = mod.device("cuda")
    nv.nvkv_prefill_attn_mod(case.cache, case.seqs, case.q_dev, case.cu_dev, total, max(case.n),
                             case.Hq, scale, m, splits, ws, out)
    torch.cuda.synchronize()
    return out


def assert_within(out: torch.Tensor, ref, tol, what):
    got = out.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - ref).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float(((got - ref).abs() / tol).max()):.3f}")
