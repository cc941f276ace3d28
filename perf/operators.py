"""The serving operators around a 4-bit paged KV cache, as cases to measure.

Four operators, as an inference engine runs them on each attention layer:

  decode    attention of the newest 1..6 tokens of every sequence over its
            cached keys, with the scores capped by a tanh, a bias that falls
            with distance, a sliding window, a document start or a prefix
            that is visible in both directions
  prefill   the same for a chunk of new tokens
  append    rotary positions with several axes (time, height, width) for the
            new K rows and queries, K and V quantised into the cache, and the
            new rows read back from it
  read      cached rows read back as bf16

The cache is the paged NVFP4 pool: a page holds 16 token slots of every
kv-head; inside a page's kv-head block of 18*D bytes lie K codes [16][D/2] |
K scales [16][D/16] | V codes [D][8] | V scales [D/16][16], two E2M1 codes a
byte (low nibble first) and one E4M3 scale for 16 elements along head_dim.

``run`` computes each operator in elementary fp32 torch operations, or calls
the package where ``own`` is true.  ``exact`` computes the definitions in 64
bits, apart from ``run``.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# --------------------------------------------------------------------- cases
def _attn(name, op, heads, d, ctx, new, cap=0.0, window=0, alibi=False, doc=0, prefix=0):
    """ctx: cached tokens before the step, one number per sequence ("a,b,c")
    or "COUNTxLOW-HIGH" (that many, spread over the range); new: query tokens
    of each sequence, in the same notation."""
    hq, hkv = heads
    return {"name": name, "op": op, "hq": hq, "hkv": hkv, "d": d, "ctx": ctx, "new": new, "cap": cap,
            "window": window, "alibi": alibi, "doc": doc, "prefix": prefix}


def listed():
    return [
        # one user's first answer tokens on a small model: latency is all
        _attn("decode_one_user", "decode", (8, 2), 128, "4096", "1", cap=30.0),
        # a busy server's step on a sliding-window layer, ragged contexts
        _attn("decode_batch_window", "decode", (24, 4), 256, "64x2048-16384", "1", cap=50.0, window=4096),
        # three agentic sessions with very long contexts on a capped global layer
        _attn("decode_long_cap", "decode", (24, 4), 256, "330000,420000,470000", "1", cap=50.0),
        # speculative verify (3 drafts + 1) with a distance bias instead of positions
        _attn("verify_distance_bias", "decode", (24, 4), 256, "2x32768-32768", "4", alibi=True),
        # an image prompt seen in both directions, then its question, on a small model
        _attn("prefill_image_prefix", "prefill", (8, 2), 128, "0", "731", prefix=576),
        # chunks of several users on a sliding-window layer
        _attn("prefill_window", "prefill", (24, 4), 256, "7001,333,0,16000", "512,301,777,65", cap=50.0, window=1024),
        # a packed row of documents that must not see one another
        _attn("prefill_documents", "prefill", (24, 4), 256, "8192", "2048", doc=1500),
        # a long prompt's chunk on a capped global layer
        _attn("prefill_long_cap", "prefill", (24, 4), 256, "65536", "2048", cap=50.0),
        # one decode step of a batch: one row for each sequence
        {"name": "append_step", "op": "append", "hq": 24, "hkv": 4, "d": 256, "ctx": "64x2048-16384", "new": "1",
         "rotary": 256, "axes": 3, "grid": 0},
        # a chunk of picture tokens (32 columns wide), partial rotary width
        _append("append_pictures", (24, 4), 256, "4099", "2048", rotary=128, axes=3, grid=32),
        # a short prompt's rows taken out of the cache again
        {"name": "read_prompt", "op": "read", "hkv": 2, "d": 128, "ctx": "1001", "skip": 7},
        # several users' prefixes read for another cache or another machine
        {"name": "read_prefixes", "op": "read", "hkv": 4, "d": 256, "ctx": "30000,40000,1,60001", "skip": 0},
    ]


def _append(name, heads, d, ctx, new, rotary, axes, grid):
    return {"name": name, "op": "append", "hq": heads[0], "hkv": heads[1], "d": d, "ctx": ctx, "new": new,
            "rotary": rotary, "axes": axes, "grid": grid}


def _log(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "read"])
    hq, hkv, d = rng.choice([(8, 2, 128), (24, 4, 256), (16, 4, 128), (16, 2, 256), (4, 4, 256)])
    if op in ("decode", "prefill"):
        batch = _log(rng, 1, 64 if op == "decode" else 6)
        if op == "decode":
            high = _log(rng, 2, min(470000, 1200000 // batch))
            ctx, new = "%dx%d-%d" % (batch, _log(rng, 1, high), high), str(rng.choice([1, 1, 1, 2, 4, 6]))
        else:
            chunk = _log(rng, 1, 2048 // batch)
            high = _log(rng, 1, 65536 // batch)
            ctx = "%dx%d-%d" % (batch, rng.randrange(0, high + 1), high)
            new = "%dx%d-%d" % (batch, _log(rng, 1, chunk), chunk)
        c = _attn("", op, (hq, hkv), d, ctx, new, cap=rng.choice([0.0, 20.0, 30.0, 50.0]),
                  window=rng.choice([0, 0, _log(rng, 16, 8192)]), alibi=rng.random() < 0.3,
                  doc=rng.choice([0, 0, _log(rng, 64, 8192)]), prefix=rng.choice([0, 0, _log(rng, 16, 2048)]))
    elif op == "append":
        batch = _log(rng, 1, 64)
        high, chunk = _log(rng, 1, 65536 // batch), _log(rng, 1, 4096 // batch)
        c = _append("", (hq, hkv), d, "%dx%d-%d" % (batch, rng.randrange(0, high + 1), high),
                    "%dx%d-%d" % (batch, _log(rng, 1, chunk), chunk), rotary=rng.choice([d, d // 2, 64]),
                    axes=rng.choice([2, 3, 3]), grid=rng.choice([0, 16, 32, 50]))
    else:
        batch = _log(rng, 1, 16)
        high = _log(rng, 1, 120000 // batch)
        c = {"op": "read", "hkv": hkv, "d": d, "ctx": "%dx%d-%d" % (batch, _log(rng, 1, high), high),
             "skip": rng.randrange(0, min(100, high))}
    c.pop("name", None)
    return c


def _numbers(text, count=None):
    """The numbers that a case's text stands for."""
    if "x" in text:
        n, ends = text.split("x")
        low, high = (int(v) for v in ends.split("-"))
        low, high = min(low, high), max(low, high)
        # spread evenly, in an order that mixes short and long
        return [low + (high - low) * (i * 7919 % int(n)) // max(1, int(n) - 1) for i in range(int(n))]
    v = [int(t) for t in text.split(",")]
    return v * count if count and len(v) == 1 else v


def _sizes(case):
    ctx = _numbers(case["ctx"])
    new = _numbers(case["new"], len(ctx)) if "new" in case else [0] * len(ctx)
    return ctx, new


def _ranges(case):
    """(first visible key, one past the last) of every query row, as int64
    arrays over all rows, by the definition; rows in sequence order."""
    ctx, new = _sizes(case)
    lo, hi = [], []
    for c, n in zip(ctx, new):
        p = np.arange(c, c + n, dtype=np.int64)
        low, high = np.zeros(n, np.int64), p + 1
        if case["doc"]:
            # a decode call has one document start for each sequence
            low = np.maximum(low, (p if case["op"] == "prefill" else p[:1]) // case["doc"] * case["doc"])
        if case["window"]:
            low = np.maximum(low, p - case["window"] + 1)
        pre = min(case["prefix"], c + n)
        reach = np.minimum(pre - p, case["window"]) if case["window"] else pre - p
        high = np.where(pre > p, p + reach, high)
        lo.append(low)
        hi.append(np.maximum(low, np.minimum(high, c + n)))
    return lo, hi


def work(case):
    ctx, new = _sizes(case)
    hkv, d = case["hkv"], case["d"]
    cached = hkv * d * 9 // 8  # bytes of one token's K and V in the cache
    if case["op"] in ("decode", "prefill"):
        lo, hi = _ranges(case)
        keys = sum(int(h.max() - low.min()) for low, h in zip(lo, hi) if (h > low).any())
        pairs = sum(int((h - low).sum()) for low, h in zip(lo, hi))
        return {"bytes": keys * cached + 4 * sum(new) * case["hq"] * d, "flops": 4 * d * case["hq"] * pairs}
    if case["op"] == "append":
        n = sum(new)
        rows = max(1, len(set(_axis_positions(case).reshape(-1).tolist())))
        # K, V and q in, rotated q and the rows read back out, the cache written; a table row for each position
        return {"bytes": n * (8 * hkv * d + cached + 4 * case["hq"] * d + 4 * case["axes"]) + rows * case["rotary"] * 4,
                "flops": n * (6 * (hkv + case["hq"]) * case["rotary"] + 4 * hkv * d)}
    n = sum(max(0, c - case["skip"]) for c in ctx)
    return {"bytes": n * (cached + 4 * hkv * d), "flops": n * 2 * hkv * d}


# -------------------------------------------------------------------- inputs
def _axis_positions(case):
    """int32 [axes][rows]: the positions of the new rows on every axis.  Text
    rows stand at the same place on every axis; picture rows share the time
    and count rows and columns of a grid."""
    ctx, new = _sizes(case)
    out = []
    for c, n in zip(ctx, new):
        i = np.arange(n)
        p = np.tile(c + i, (case["axes"], 1))
        if case["grid"]:
            p[0] = c
            p[1] = c + i // case["grid"]
            if case["axes"] > 2:
                p[2] = c + i % case["grid"]
        out.append(p)
    return np.concatenate(out, 1).astype(np.int32)


def _axis_of_pair(case):
    """Which axis turns which pair: time gets a quarter, the others share the rest."""
    half, axes = case["rotary"] // 2, case["axes"]
    first = half // 4
    return [0] * first + [1 + i * (axes - 1) // (half - first) for i in range(half - first)]


def _codes(x, s):
    """E2M1 codes (sign << 3 | magnitude) of x under the scales s: nearest,
    ties to the even code; a scale of 0 and a magnitude of 0 give code 0."""
    a = x.abs()
    m = torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    for mid, even_below in ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        m += (a > mid * s) if even_below else (a >= mid * s)
    m = torch.where(s > 0, m, torch.zeros_like(m))
    return m | (((x < 0) & (m > 0)).to(torch.uint8) << 3)


def _scales(x):
    """E4M3 scales (as float8) of groups of 16 along the last axis."""
    amax = x.unflatten(-1, (-1, PAGE)).abs().amax(-1)
    return (amax / 6).clamp(max=448).to(torch.float8_e4m3fn)


def _make_pool(g, num_pages, hkv, d, device):
    """A pool of quantised normal values; four K channels stand out, as they do in trained models."""
    pool = torch.empty((num_pages, hkv, 18 * d), dtype=torch.uint8, device=device)
    loud = torch.ones(d, device=device)
    loud[torch.randperm(d, generator=g, device=device)[:4]] = 10
    for p0 in range(0, num_pages, 4096):
        n = min(4096, num_pages - p0)
        parts = []
        for kind in "kv":
            x = torch.randn((n, hkv, PAGE, d), generator=g, device=device)
            x = (x * loud if kind == "k" else x).bfloat16().float()
            sc = _scales(x)
            code = _codes(x, sc.float().repeat_interleave(PAGE, -1))
            if kind == "k":
                parts += [code[..., 0::2] | (code[..., 1::2] << 4), sc.view(torch.uint8)]
            else:
                code = code.transpose(-1, -2)
                parts += [code[..., 0::2] | (code[..., 1::2] << 4), sc.view(torch.uint8).transpose(-1, -2)]
        pool[p0:p0 + n] = torch.cat([t.reshape(n, hkv, -1) for t in parts], -1)
    return pool.view(-1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    ctx, new = _sizes(case)
    hkv, d = case["hkv"], case["d"]
    lens = [c + n for c, n in zip(ctx, new)]
    pages = [-(-n // PAGE) for n in lens]
    num_pages, most = sum(pages) + 1, max(pages)
    s = {"case": case, "lens": lens, "new": new, "num_pages": num_pages}
    s["pool"] = _make_pool(g, num_pages, hkv, d, dev)
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["cu"] = torch.from_numpy(cu).to(dev)
    rows = int(cu[-1])
    if case["op"] in ("decode", "prefill"):
        s["q"] = torch.randn((rows, case["hq"], d), generator=g, device=dev).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = d ** -0.5
        # slopes 2^-1 .. 2^-8 over the heads
        s["slopes"] = torch.exp2(-8 * torch.arange(1, case["hq"] + 1, device=dev) / case["hq"]) if case["alibi"] else None
        s["prefix"] = torch.tensor([min(case["prefix"], n) for n in lens], dtype=torch.int32, device=dev) if case["prefix"] else None
        s["starts"] = None
        if case["doc"]:
            if case["op"] == "decode":
                v = [c // case["doc"] * case["doc"] for c in ctx]
            else:
                v = np.concatenate([np.arange(c, c + n) // case["doc"] * case["doc"] for c, n in zip(ctx, new)]).tolist()
            s["starts"] = torch.tensor(v, dtype=torch.int32, device=dev)
    elif case["op"] == "append":
        loud = torch.ones(d, device=dev)
        loud[torch.randperm(d, generator=g, device=dev)[:4]] = 10
        s["k"] = (torch.randn((rows, hkv, d), generator=g, device=dev) * loud).bfloat16()
        s["v"] = torch.randn((rows, hkv, d), generator=g, device=dev).bfloat16()
        s["q"] = torch.randn((rows, case["hq"], d), generator=g, device=dev).bfloat16()
        s["q_out"] = torch.empty_like(s["q"])
        s["positions"] = torch.from_numpy(_axis_positions(case)).to(dev)
        s["axis"] = _axis_of_pair(case)
        half = case["rotary"] // 2
        angle = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * torch.pow(
            torch.tensor(1e6, dtype=torch.float64, device=dev), -torch.arange(half, dtype=torch.float64, device=dev) / half)
        s["cs"] = torch.stack((angle.cos(), angle.sin()), -1).float()
        s["starts"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["read_cu"], s["rows"], s["most"] = s["cu"], rows, max(new)
    if case["op"] == "read":
        counts = [max(0, c - case["skip"]) for c in ctx]
        s["starts"] = torch.tensor([min(case["skip"], c) for c in ctx], dtype=torch.int32, device=dev)
        s["read_cu"] = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device=dev)
        s["rows"], s["most"], s["counts"], s["ctx"] = sum(counts), max(counts), counts, ctx
    if case["op"] in ("append", "read"):
        s["k_out"] = torch.empty((s["rows"], hkv, d), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        # the handles and the workspace that a program keeps from step to step: no data is touched
        import nvfp4_quantized_kv_b200 as nv

        s["nv"] = nv
        s["cache"] = nv.Cache(s["pool"], num_pages, hkv, d)
        s["seqs"] = nv.Seqs(table, s["kv_lens"], most * PAGE)
        if case["op"] in ("decode", "prefill"):
            s["mod"] = nv.ScoreMod(softcap=case["cap"], window=case["window"], alibi_slopes=s["slopes"],
                                   prefix_lens=s["prefix"], key_starts=s["starts"])
            size = (nv.nvkv_decode_workspace_bytes(len(lens), new[0], case["hq"], hkv, d, 0) if case["op"] == "decode"
                    else nv.nvkv_prefill_workspace_bytes(rows, case["hq"], d, 0))
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=dev)
    return s


# -------------------------------------------------------------- plain forms
def _pairs(raw):
    """Bytes of E2M1 code pairs -> their two values, along a new last axis."""
    m = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=raw.device)
    m = torch.cat((m, -m))
    both = torch.stack((m.repeat(16), m.repeat_interleave(16)), -1)  # [byte][low, high]
    return both[raw.int()]


def _cached(pool, pages, hkv, d):
    """The K and V rows of pages [...] as fp32 [..., hkv, 16, d]."""
    raw = pool.view(-1, hkv, 18 * d)[pages.long()]
    kc, ks, vc, vs = raw.split((8 * d, d, 8 * d, d), -1)
    scale = ks.unflatten(-1, (PAGE, d // 16)).contiguous().view(torch.float8_e4m3fn).float()
    k = _pairs(kc).flatten(-2).unflatten(-1, (PAGE, d // 16, 16)) * scale[..., None]
    scale = vs.unflatten(-1, (d // 16, 1, PAGE)).contiguous().view(torch.float8_e4m3fn).float()
    v = _pairs(vc).flatten(-2).unflatten(-1, (d // 16, 16, PAGE)) * scale
    return k.flatten(-2), v.flatten(-3, -2).transpose(-1, -2)


def _sequences(s):
    """Every sequence's cached rows, fp32 [batch][hkv][positions][d]."""
    k, v = _cached(s["pool"], s["table"].clamp(min=0), s["case"]["hkv"], s["case"]["d"])
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    c = s["case"]
    k, v = _sequences(s)
    batch, hkv, length, d = k.shape
    dev, most, group = k.device, max(s["new"]), c["hq"] // hkv
    # the rows of every sequence, padded to the longest chunk
    i = torch.arange(most, device=dev)
    cu, lens = s["cu"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    there = i < n[:, None]
    row = torch.where(there, cu[:-1, None] + i, 0)
    p = (lens - n)[:, None] + i
    q = s["q"].float()[row].unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    x = x.view(batch, hkv, group, most, length)
    j = torch.arange(length, device=dev)
    if s["slopes"] is not None:
        far = (p[..., None] - j).abs().float()
        x -= s["slopes"].view(hkv, group)[None, :, :, None, None] * far[:, None, None]
    low, high = torch.zeros_like(p), p + 1
    if s["starts"] is not None:
        st = s["starts"].long()
        low = torch.maximum(low, st[:, None] if c["op"] == "decode" else st[row])
    if c["window"]:
        low = torch.maximum(low, p - c["window"] + 1)
    if s["prefix"] is not None:
        ahead = s["prefix"].long()[:, None] - p
        high = torch.where(ahead > 0, p + (ahead.clamp(max=c["window"]) if c["window"] else ahead), high)
    high = torch.minimum(high, lens[:, None])
    seen = (j >= low[..., None]) & (j < high[..., None]) & (p >= 0)[..., None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp(min=-3e38)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = x.view(batch, hkv, -1, length) @ v / total.clamp(min=1e-30).view(batch, hkv, -1, 1)
    o = o.view(batch, hkv, group, most, d).permute(0, 3, 1, 2, 4)
    return o[there].reshape(-1, c["hq"], d).bfloat16()


def _plain_rotate(s, x):
    """x [rows][heads][d] with its first `rotary` elements turned: element i
    with element i + rotary/2, by the angle of its axis' position."""
    half = s["case"]["rotary"] // 2
    axis = torch.tensor(s["axis"], device=x.device)
    at = s["positions"].long()[axis]  # [pair][row]
    cs = s["cs"][at.t(), torch.arange(half, device=x.device)]  # [row][pair][2]
    # in 64 bits with the two fp32 roundings of the definition (the product
    # with the sine, and the sum): a value next to a border of the 4-bit
    # format must fall on its own side
    c, sn = cs[:, None, :, 0].double(), cs[:, None, :, 1].double()
    a, b, rest = x[..., :half].double(), x[..., half:2 * half].double(), x[..., 2 * half:].float()
    return torch.cat(((a * c - (b * sn).float().double()).float(), (b * c + (a * sn).float().double()).float(), rest), -1)


def _plain_quantise(x):
    """The values that the 4-bit cache holds for fp32 x."""
    sc = _scales(x).float()[..., None]
    g = x.unflatten(-1, (-1, PAGE))
    a = torch.where(sc > 0, g.abs(), torch.zeros_like(g))
    m = torch.zeros_like(a)
    for mid, step, even_below in ((0.25, 0.5, True), (0.75, 0.5, False), (1.25, 0.5, True), (1.75, 0.5, False),
                                  (2.5, 1.0, True), (3.5, 1.0, False), (5.0, 2.0, True)):
        m += step * (((a > mid * sc) if even_below else (a >= mid * sc)) & (sc > 0))
    return (torch.where(g < 0, -m, m) * sc).flatten(-2).bfloat16()


def _plain_read(s):
    k, v = _sequences(s)
    i = torch.arange(max(1, s["most"]), device=k.device)
    n = (s["read_cu"][1:] - s["read_cu"][:-1]).long()[:, None]
    b, r = (i < n).nonzero(as_tuple=True)
    at = s["starts"].long()[b] + r
    return k[b, :, at].bfloat16(), v[b, :, at].bfloat16()


def run(state):
    s = state
    c = s["case"]
    if own:
        nv = s["nv"]
        if c["op"] == "decode":
            nv.nvkv_decode_attn_mod(s["cache"], s["seqs"], s["q"], s["new"][0], c["hq"], s["scale"], s["mod"], 0,
                                    s["workspace"], s["out"])
            return s["out"]
        if c["op"] == "prefill":
            nv.nvkv_prefill_attn_mod(s["cache"], s["seqs"], s["q"], s["cu"], s["q"].shape[0], max(s["new"]), c["hq"],
                                     s["scale"], s["mod"], 0, s["workspace"], s["out"])
            return s["out"]
        if c["op"] == "append":
            nv.nvkv_append_rope_axes(s["cache"], s["seqs"], s["k"], s["v"], s["cu"], s["rows"], s["most"], s["cs"],
                                     c["rotary"], s["positions"], s["axis"], s["q"], s["q_out"])
        nv.nvkv_read_rows(s["cache"], s["seqs"], s["starts"], s["read_cu"], s["rows"], s["most"], s["k_out"], s["v_out"])
        if c["op"] == "append":
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        return {"k": s["k_out"], "v": s["v_out"]}
    if c["op"] in ("decode", "prefill"):
        return _plain_attention(s)
    if c["op"] == "append":
        return {"q": _plain_rotate(s, s["q"]).bfloat16(), "k": _plain_quantise(_plain_rotate(s, s["k"])),
                "v": _plain_quantise(s["v"].float())}
    k, v = _plain_read(s)
    return {"k": k, "v": v}


# --------------------------------------------------------------------- exact
def _e2m1(code):
    mag = code & 7
    v = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2.0, mag * 2.0 - 8.0)).double()
    return torch.where(code >= 8, -v, v)


def _e4m3(byte):
    e, m = (byte >> 3) & 15, byte & 7
    v = torch.where(e > 0, (8.0 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    return torch.where(byte >= 128, -v, v)


def _exact_rows(s, b, h):
    """The 64-bit K and V rows of kv-head h of sequence b."""
    c = s["case"]
    d, n = c["d"], s["lens"][b]
    raw = s["pool"].view(-1, c["hkv"], 18 * d)[s["table"][b, :-(-n // PAGE)].long(), h].to(torch.int32)
    ks, vs = _e4m3(raw[:, 8 * d:9 * d]), _e4m3(raw[:, 17 * d:])
    kc, vc = raw[:, :8 * d], raw[:, 9 * d:17 * d]
    k = torch.stack((_e2m1(kc & 15), _e2m1(kc >> 4)), -1).reshape(-1, PAGE, d // 16, 16)
    v = torch.stack((_e2m1(vc & 15), _e2m1(vc >> 4)), -1).reshape(-1, d, PAGE)
    k = (k * ks.reshape(-1, PAGE, d // 16, 1)).reshape(-1, d)
    v = (v * vs.reshape(-1, d // 16, PAGE).repeat_interleave(16, 1)).transpose(1, 2).reshape(-1, d)
    return k[:n], v[:n]


def _exact_attention(s):
    c = s["case"]
    lo, hi = _ranges(c)
    group, dev = c["hq"] // c["hkv"], s["pool"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    at = 0
    for b, n in enumerate(s["new"]):
        p = torch.arange(s["lens"][b] - n, s["lens"][b], device=dev)
        low, high = (torch.from_numpy(t[b]).to(dev) for t in (lo, hi))
        for h in range(c["hkv"]):
            k, v = _exact_rows(s, b, h)
            j = torch.arange(k.shape[0], device=dev)
            for r in range(0, n, 512):  # 512 rows at a time
                e = min(n, r + 512)
                seen = (j >= low[r:e, None]) & (j < high[r:e, None])
                for g in range(group):
                    x = s["q"][at + r:at + e, h * group + g].double() @ k.t() * s["scale"]
                    if c["cap"]:
                        x = c["cap"] * torch.tanh(x / c["cap"])
                    if c["alibi"]:
                        x = x - s["slopes"][h * group + g].double() * (p[r:e, None] - j).abs()
                    x = torch.where(seen, x, -math.inf)
                    top = x.amax(1, keepdim=True)
                    w = torch.where(seen, torch.exp(x - torch.where(top.isinf(), 0.0, top)), 0.0)
                    total = w.sum(1, keepdim=True)
                    out[at + r:at + e, h * group + g] = w @ v / torch.where(total > 0, total, 1.0)
        at += n
    return out


def _exact_turn(s, x):
    half = s["case"]["rotary"] // 2
    x = x.double()
    axis = torch.tensor(s["axis"], device=x.device)
    cs = s["cs"].double()[s["positions"].long()[axis], torch.arange(half, device=x.device)[:, None]]
    z = torch.complex(cs[..., 0], cs[..., 1]).t()[:, None] * torch.complex(x[..., :half], x[..., half:2 * half])
    return torch.cat((z.real, z.imag, x[..., 2 * half:]), -1)


def _exact_stored(x):
    """Nearest E4M3 scale of amax / 6, then nearest E2M1 multiples, ties to even."""
    g = x.double().unflatten(-1, (-1, 16))
    t = g.abs().amax(-1, keepdim=True) / 6
    unit = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    sc = (torch.round(t / unit) * unit).clamp(max=448.0)
    r = (g.abs() / torch.where(sc > 0, sc, 1.0)).clamp(max=6.0)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    return (torch.sign(g) * torch.round(r / step) * step * sc).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("decode", "prefill"):
        return _exact_attention(s)
    if case["op"] == "append":
        return {"q": _exact_turn(s, s["q"]), "k": _exact_stored(_exact_turn(s, s["k"])), "v": _exact_stored(s["v"])}
    out = {"k": [], "v": []}
    for b, n in enumerate(s["counts"]):
        a = s["ctx"][b] - n
        heads = [_exact_rows(s, b, h) for h in range(case["hkv"])]
        out["k"].append(torch.stack([k[a:] for k, _ in heads], 1))
        out["v"].append(torch.stack([v[a:] for _, v in heads], 1))
    return {n: torch.cat(t) for n, t in out.items()}
