"""The several-axis append, the masked attention and the row read as one layer
runs them: an image prompt in one chunk, then decode and verify steps, each
checked against a 64-bit form of the whole run; and the plain calls' results
beside them."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv
import oracle

from mod_ref import assert_within, attend, bits, interval

pytestmark = pytest.mark.gpu


def f64(b):
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Layer:
    """One sequence of a layer: what was appended, in 64 bits, and its cache.
    The 64-bit form attends to the values that the 4-bit format holds for the
    rotated rows (the oracle's rotation and quantisation)."""

    def __init__(self, Hq, Hkv, D, rotary, cap, window, prefix, pages=40):
        self.Hq, self.Hkv, self.D, self.r = Hq, Hkv, D, rotary
        self.cap, self.window, self.prefix = cap, window, prefix
        self.rng = np.random.default_rng(D + Hq)
        dev = self.dev = torch.device("cuda")
        self.cache = nv.Cache.allocate(pages, Hkv, D, dev, fill=0x7F)
        self.pt = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()[None].to(dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.len = 0
        self.kv_lens = torch.zeros(1, dtype=torch.int32, device=dev)
        self.seqs = nv.Seqs(self.pt, self.kv_lens, pages * 16, self.err)
        self.table = np.ascontiguousarray(oracle.rope_table(pages * 16, rotary, 1e6, 1.0), np.float32)
        self.cs = torch.from_numpy(self.table).to(dev)
        half = rotary // 2
        self.axis = [0 if i < half // 4 else 1 + (i - half // 4) % 2 for i in range(half)]
        self.k, self.v = np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))
        self.mod = nv.ScoreMod(softcap=cap, window=window,
                               prefix_lens=torch.tensor([prefix], dtype=torch.int32, device=dev))

    def append(self, n, positions):
        bf = lambda x: torch.from_numpy(x.view(np.int16)).to(self.dev).view(torch.bfloat16)
        k, v, q = (bits(self.rng.standard_normal((n, h, self.D))) for h in (self.Hkv, self.Hkv, self.Hq))
        self.len += n
        self.kv_lens.fill_(self.len)
        cu = torch.tensor([0, n], dtype=torch.int32, device=self.dev)
        q_dev = bf(q)
        nv.nvkv_append_rope_axes(self.cache, self.seqs, bf(k), bf(v), cu, n, n, self.cs, self.r,
                                 torch.from_numpy(positions.astype(np.int32)).to(self.dev), self.axis, q_dev, q_dev)
        # the oracle: rotate in its stated float order, quantise, dequantise
        half = self.r // 2
        kh = np.zeros((n, self.Hkv, self.D))
        for i in range(n):
            cs = self.table[positions[np.array(self.axis), i], np.arange(half)]
            for h in range(self.Hkv):
                row = oracle.rope_rotate_f32(k[i, h], self.r, cs)
                for g in range(self.D // 16):
                    codes, sc = oracle.quantize_group_f32(row[16 * g:16 * g + 16])
                    kh[i, h, 16 * g:16 * g + 16] = [oracle.dequant(int(c), int(sc)) for c in codes]
        self.k = np.concatenate([self.k, kh])
        self.v = np.concatenate([self.v, oracle.qdq_rows(np.ascontiguousarray(v))])
        return q_dev, cu

    def want(self, q_dev, n, slack):
        q = q_dev.double().cpu()
        p = torch.arange(self.len - n, self.len)
        r = torch.tensor([interval(int(i), self.len, 0, self.window, self.prefix) for i in p])
        j = torch.arange(self.len)
        seen = (j >= r[:, :1]) & (j < r[:, 1:])
        out = torch.zeros(n, self.Hq, self.D, dtype=torch.float64)
        tol = torch.zeros_like(out)
        G = self.Hq // self.Hkv
        for hq in range(self.Hq):
            k, v = (torch.from_numpy(np.ascontiguousarray(t[:, hq // G])) for t in (self.k, self.v))
            out[:, hq], tol[:, hq] = attend(q[:, hq], k, v, seen, p, j, self.D ** -0.5, self.cap, 0.0, slack)
        return out, tol

    def read(self, start, n):
        k = torch.empty((n, self.Hkv, self.D), dtype=torch.bfloat16, device=self.dev)
        v = torch.empty_like(k)
        nv.nvkv_read_rows(self.cache, self.seqs, torch.tensor([start], dtype=torch.int32, device=self.dev),
                          torch.tensor([0, n], dtype=torch.int32, device=self.dev), n, n, k, v)
        return k.double().cpu().numpy(), v.double().cpu().numpy()


@pytest.mark.parametrize("Hq,Hkv,D,rotary", [(24, 4, 256, 256), (8, 2, 128, 64)])
def test_image_prompt_then_steps(Hq, Hkv, D, rotary):
    lay = Layer(Hq, Hkv, D, rotary, cap=30.0, window=90, prefix=96)
    # a picture of 12 x 8 tokens (two-way), then 41 text tokens
    i = np.arange(137)
    pos = np.stack([np.where(i < 96, 0, i - 84), np.where(i < 96, i // 8, i - 84), np.where(i < 96, i % 8, i - 84)])
    q, cu = lay.append(137, pos)
    out = torch.empty_like(q)
    ws = torch.empty(nv.nvkv_prefill_workspace_bytes(137, Hq, D, 0), dtype=torch.uint8, device="cuda")
    nv.nvkv_prefill_attn_mod(lay.cache, lay.seqs, q, cu, 137, 137, Hq, D ** -0.5, lay.mod, 0, ws, out)
    torch.cuda.synchronize()
    assert_within(out, *lay.want(q, 137, "f16 scores"), "prompt")
    # decode steps of 1, then verify steps of 3 and 6 tokens
    for T in (1, 1, 3, 1, 6):
        at = lay.len - 84 + np.arange(T)
        q, _ = lay.append(T, np.stack([at] * 3))
        out = torch.empty_like(q)
        ws = torch.empty(nv.nvkv_decode_workspace_bytes(1, T, Hq, Hkv, D, 0), dtype=torch.uint8, device="cuda")
        nv.nvkv_decode_attn_mod(lay.cache, lay.seqs, q, T, Hq, D ** -0.5, lay.mod, 0, ws, out)
        torch.cuda.synchronize()
        assert_within(out, *lay.want(q, T, "f16 scores"), f"step of {T} at {lay.len}")
    assert int(lay.err.item()) == 0
    k, v = lay.read(0, lay.len)
    assert np.array_equal(k, lay.k) and np.array_equal(v, lay.v)
    k, v = lay.read(17, 100)
    assert np.array_equal(k, lay.k[17:117]) and np.array_equal(v, lay.v[17:117])


def test_a_step_captured_and_replayed():
    """Append, attention and read of a step in one graph: replayed with new
    rows at new lengths it gives what direct calls give."""
    Hq, Hkv, D = 24, 4, 256
    dev = torch.device("cuda")
    pages = 16
    g = torch.Generator(device=dev).manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()
    cs = torch.empty((pages * 16, 128, 2), device=dev)
    nv.nvkv_rope_table(cs, 256, 1e6, 1.0)
    k, v, q = rnd(2, Hkv, D), rnd(2, Hkv, D), rnd(2, Hq, D)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    starts = torch.zeros(2, dtype=torch.int32, device=dev)
    pos = torch.zeros((3, 2), dtype=torch.int32, device=dev)
    lens = torch.tensor([40, 7], dtype=torch.int32, device=dev)
    mod = nv.ScoreMod(softcap=25.0, window=33)
    ws = torch.empty(nv.nvkv_decode_workspace_bytes(2, 1, Hq, Hkv, D, 0), dtype=torch.uint8, device=dev)
    caches = [nv.Cache.allocate(2 * pages, Hkv, D, dev, fill=0) for _ in range(2)]
    pt = torch.arange(2 * pages, dtype=torch.int32, device=dev).view(2, pages)
    bufs = [{n: torch.zeros(s, dtype=torch.bfloat16, device=dev) for n, s in
             (("q", (2, Hq, D)), ("o", (2, Hq, D)), ("k", (2, Hkv, D)), ("v", (2, Hkv, D)))} for _ in range(2)]

    def step(cache, b):
        s = nv.Seqs(pt, lens, pages * 16)
        nv.nvkv_append_rope_axes(cache, s, k, v, cu, 2, 1, cs, 256, pos, [i % 3 for i in range(128)], q, b["q"])
        nv.nvkv_decode_attn_mod(cache, s, b["q"], 1, Hq, D ** -0.5, mod, 0, ws, b["o"])
        nv.nvkv_read_rows(cache, s, starts, cu, 2, 1, b["k"], b["v"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(caches[1], bufs[1])
    torch.cuda.current_stream().wait_stream(s)
    caches[1].pool.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], bufs[0])
    caches[0].pool.zero_()
    for it in range(20):
        k.copy_(rnd(2, Hkv, D))
        v.copy_(rnd(2, Hkv, D))
        q.copy_(rnd(2, Hq, D))
        lens += 1
        pos.copy_((lens - 1)[None].expand(3, 2))
        starts.copy_(lens - 1)
        graph.replay()
        step(caches[1], bufs[1])
        torch.cuda.synchronize()
        assert torch.equal(caches[0].pool, caches[1].pool)
        for n in bufs[0]:
            assert torch.equal(bufs[0][n], bufs[1][n]), n


def test_two_streams_at_once():
    """Two layers' steps on two streams, each with its own cache and
    workspace, give what they give one after the other."""
    dev = torch.device("cuda")
    Hq, Hkv, D = 24, 4, 256
    L = 900
    sets = []
    for i in range(2):
        g = torch.Generator(device=dev).manual_seed(20 + i)
        cache = nv.Cache.allocate(60, Hkv, D, dev, fill=0)
        seqs = nv.Seqs(torch.arange(60, dtype=torch.int32, device=dev)[None],
                       torch.tensor([L], dtype=torch.int32, device=dev), 960)
        kv = [torch.randn((L, Hkv, D), generator=g, device=dev).bfloat16() for _ in range(2)]
        nv.nvkv_append(cache, seqs, kv[0], kv[1], torch.tensor([0, L], dtype=torch.int32, device=dev), L, L)
        T = (1, 4)[i]
        q = torch.randn((T, Hq, D), generator=g, device=dev).bfloat16()
        ws = torch.empty(nv.nvkv_decode_workspace_bytes(1, T, Hq, Hkv, D, 0), dtype=torch.uint8, device=dev)
        sets.append((cache, seqs, q, T, nv.ScoreMod(softcap=20.0, window=500 * (i + 1)), ws))
    run = lambda s, out, stream=None: nv.nvkv_decode_attn_mod(s[0], s[1], s[2], s[3], Hq, D ** -0.5, s[4], 0, s[5],
                                                              out, stream=stream)
    want = [torch.empty_like(s[2]) for s in sets]
    for s, w in zip(sets, want):
        run(s, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = [torch.empty_like(s[2]) for s in sets]
        torch.cuda.synchronize()
        for s, o, st in zip(sets, got, streams):
            run(s, o, st)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_score_mod_attributes_may_change():
    """A call takes the ScoreMod's attributes as they are then."""
    dev = torch.device("cuda")
    L, Hq, Hkv, D = 100, 8, 2, 128
    cache = nv.Cache.allocate(8, Hkv, D, dev, fill=0)
    seqs = nv.Seqs(torch.arange(8, dtype=torch.int32, device=dev)[None],
                   torch.tensor([L], dtype=torch.int32, device=dev), 128)
    kv = [torch.randn((L, Hkv, D), device=dev).bfloat16() for _ in range(2)]
    nv.nvkv_append(cache, seqs, kv[0], kv[1], torch.tensor([0, L], dtype=torch.int32, device=dev), L, L)
    q = torch.randn((1, Hq, D), device=dev).bfloat16()
    ws = torch.empty(nv.nvkv_decode_workspace_bytes(1, 1, Hq, Hkv, D, 0), dtype=torch.uint8, device=dev)

    def run(mod):
        out = torch.empty_like(q)
        nv.nvkv_decode_attn_mod(cache, seqs, q, 1, Hq, D ** -0.5, mod, 0, ws, out)
        return out

    mod = nv.ScoreMod(window=10)
    a = run(mod)
    mod.window, mod.key_starts = 0, torch.tensor([90], dtype=torch.int32, device=dev)
    assert torch.equal(run(mod), a)
    mod.key_starts = torch.zeros(0, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="key_starts"):
        run(mod)
    mod.key_starts = torch.zeros(1, dtype=torch.int64, device=dev)
    with pytest.raises(TypeError, match="key_starts"):
        run(mod)


@pytest.mark.parametrize("kind", ["decode", "verify", "prefill", "prefill split"])
def test_back_to_back_calls_see_what_the_kernel_before_wrote(kind):
    """The attention kernels may be set up while the kernel before them ends:
    lengths, queries and rows written just before a call, by kernels that take
    their time, and a workspace still being merged, are waited for."""
    dev = torch.device("cuda")
    Hq, Hkv, D, L = 24, 4, 256, 2000
    g = torch.Generator(device=dev).manual_seed(11)
    cache = nv.Cache.allocate(130, Hkv, D, dev, fill=0)
    lens = torch.tensor([L], dtype=torch.int32, device=dev)
    seqs = nv.Seqs(torch.arange(128, dtype=torch.int32, device=dev)[None], lens, 2048)
    kv = [torch.randn((L, Hkv, D), generator=g, device=dev).bfloat16() for _ in range(2)]
    nv.nvkv_append(cache, seqs, kv[0], kv[1], torch.tensor([0, L], dtype=torch.int32, device=dev), L, L)
    n = {"decode": 1, "verify": 4, "prefill": 100, "prefill split": 100}[kind]
    size = max(nv.nvkv_decode_workspace_bytes(1, min(n, 16), Hq, Hkv, D, 0),
               nv.nvkv_prefill_workspace_bytes(n, Hq, D, 4))
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    q, cu = torch.zeros((n, Hq, D), dtype=torch.bfloat16, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    mod = nv.ScoreMod(softcap=20.0, window=700)
    busy = torch.randn((4096, 4096), generator=g, device=dev)
    steps = [(L - 50 * i, torch.randn((n, Hq, D), generator=g, device=dev).bfloat16()) for i in range(12)]
    cu_new = torch.tensor([0, n], dtype=torch.int32, device=dev)

    def call(out):
        if n <= 16:
            nv.nvkv_decode_attn_mod(cache, seqs, q, n, Hq, 1 / 16, mod, 0, ws, out)
        else:
            nv.nvkv_prefill_attn_mod(cache, seqs, q, cu, n, n, Hq, 1 / 16, mod, 4 if "split" in kind else 1, ws, out)

    def run(wait):
        outs = []
        for length, query in steps:
            q.fill_(float("nan"))
            lens.zero_()
            cu.zero_()
            out = torch.full_like(q, float("nan"))
            torch.cuda.synchronize()
            x = busy @ busy  # keeps the stream busy before the values arrive
            q.copy_(query + (x[0, 0] * 0).bfloat16())
            cu.copy_(cu_new)
            lens.fill_(length)
            if wait:
                torch.cuda.synchronize()
            call(out)
            outs.append(out)
            again = torch.empty_like(out)  # the workspace is still being merged
            call(again)
            torch.cuda.synchronize()
            assert torch.equal(again, out)
        return outs

    for a, b in zip(run(True), run(False)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_append_and_read_back_to_back():
    """Rows appended, read and appended over again, call after call without a
    wait in between, are those of each call."""
    dev = torch.device("cuda")
    Hq, Hkv, D, n = 24, 4, 256, 600
    g = torch.Generator(device=dev).manual_seed(12)
    cache = nv.Cache.allocate(40, Hkv, D, dev, fill=0)
    seqs = nv.Seqs(torch.arange(40, dtype=torch.int32, device=dev)[None],
                   torch.tensor([n], dtype=torch.int32, device=dev), 640)
    cs = torch.empty((640, 128, 2), device=dev)
    nv.nvkv_rope_table(cs, 256, 1e6, 1.0)
    pos = torch.arange(n, dtype=torch.int32, device=dev)[None].expand(2, n).contiguous()
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    axis = [i & 1 for i in range(128)]
    rows = [[torch.randn((n, h, D), generator=g, device=dev).bfloat16() for h in (Hkv, Hkv, Hq)] for _ in range(20)]

    def run(wait):
        outs = [[torch.empty_like(t) for t in r] for r in rows]
        torch.cuda.synchronize()
        for (k, v, q), (ko, vo, qo) in zip(rows, outs):
            nv.nvkv_append_rope_axes(cache, seqs, k, v, cu, n, n, cs, 256, pos, axis, q, qo)
            if wait:
                torch.cuda.synchronize()
            nv.nvkv_read_rows(cache, seqs, zero, cu, n, n, ko, vo)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    for a, b in zip(run(True), run(False)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
