"""GPU parity of nvkv_append_rope_axes: the pool bit-exact against the
oracle's one-axis rotating append fed a table that holds, for every cache
position, the several-axis angles of the row written there; the queries
against the 64-bit rotation."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv
import oracle

from mod_ref import bits

pytestmark = pytest.mark.gpu


def axis_lists(half, axes):
    """Sections in a row, interleaved axes, and one axis for all."""
    a = [min(axes - 1, i * axes // half) for i in range(half)]
    return {"sections": a, "interleaved": [i % axes for i in range(half)], "last": [axes - 1] * half}


class Setup:
    def __init__(self, Hq, Hkv, D, ctx, n, r, axes, kind="sections", seed=0, max_pos=700, fill=0xA5):
        rng = np.random.default_rng([seed, D, r, axes])
        self.Hq, self.Hkv, self.D, self.r = Hq, Hkv, D, r
        self.lens = np.array([c + k for c, k in zip(ctx, n)], np.int32)
        self.n, self.ctx = n, ctx
        per = [(int(l) + 15) // 16 for l in self.lens]
        self.num_pages = sum(per) + 3
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.pt = np.full((len(ctx), max(1, max(per))), -1, np.int32)
        at = 0
        for b, p in enumerate(per):
            self.pt[b, :p] = perm[at:at + p]
            at += p
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        rows = self.rows = int(self.cu[-1])
        self.k = bits(rng.standard_normal((rows, Hkv, D)) * np.where(rng.random(D) < 0.03, 10.0, 1.0))
        self.v = bits(rng.standard_normal((rows, Hkv, D)))
        self.q = bits(rng.standard_normal((rows, Hq, D)))
        self.axis = axis_lists(r // 2, axes)[kind]
        self.max_pos = max_pos
        self.positions = rng.integers(0, max_pos, (axes, rows)).astype(np.int32)
        self.table = np.ascontiguousarray(oracle.rope_table(max_pos, r, 1e6, 1.0), np.float32)
        self.fill = fill
        self.pool0 = rng.integers(0, 256, self.num_pages * oracle.page_bytes(Hkv, D)).astype(np.uint8) \
            if fill is None else np.full(self.num_pages * oracle.page_bytes(Hkv, D), fill, np.uint8)

    def row_table(self, row):
        """[r/2][2]: the (cos, sin) of each pair of one row."""
        i = np.arange(self.r // 2)
        p = np.clip(self.positions[np.array(self.axis), row], 0, self.max_pos - 1)
        return self.table[p, i]

    def want_pool(self, skip=()):
        """The oracle's append, one sequence row at a time through a table
        whose row at the cache position is that row's own; rows in `skip` are
        not written."""
        pool = self.pool0.copy()
        t = np.zeros((int(self.lens.max()) + 1, self.r // 2, 2), np.float32)
        for b in range(len(self.n)):
            for i in range(self.n[b]):
                row, pos = int(self.cu[b]) + i, self.ctx[b] + i
                if row in skip:
                    continue
                t[pos] = self.row_table(row)
                oracle.append_rope(pool, self.Hkv, self.D, self.pt[b:b + 1], np.array([pos + 1], np.int32),
                                   self.k[row:row + 1], self.v[row:row + 1], np.array([0, 1], np.int32), self.r, t)
        return pool

    def want_q(self):
        f = lambda x: (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        q = f(self.q)
        half = self.r // 2
        out = q.copy()
        for row in range(self.rows):
            cs = self.row_table(row).astype(np.float64)
            x, y = q[row, :, :half], q[row, :, half:self.r]
            out[row, :, :half] = x * cs[:, 0] - y * cs[:, 1]
            out[row, :, half:self.r] = y * cs[:, 0] + x * cs[:, 1]
        # two fp32 roundings of products no larger than |q| (2^-24 each, and
        # one of the sum), then one to bf16
        h = np.abs(q[..., :half]) + np.abs(q[..., half:self.r])
        size = np.concatenate([h, h, np.zeros_like(q[..., self.r:])], -1)
        return out, 2.0 ** -8 * np.abs(out) + 3 * 2.0 ** -24 * size * 1.01

    def run(self, with_q=True, stream=None, in_place=False, graph=False):
        dev = torch.device("cuda")
        bf = lambda x: torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        cache = nv.Cache(torch.from_numpy(self.pool0.copy()).to(dev), self.num_pages, self.Hkv, self.D)
        self.cache = cache
        self.seqs = nv.Seqs(torch.from_numpy(self.pt).to(dev), torch.from_numpy(self.lens).to(dev),
                            self.pt.shape[1] * 16, self.err)
        q = bf(self.q) if with_q else None
        qo = (q if in_place else torch.full_like(q, 7.0)) if with_q else None
        args = (cache, self.seqs, bf(self.k), bf(self.v), torch.from_numpy(self.cu).to(dev), self.rows,
                max(self.n), torch.from_numpy(self.table).to(dev), self.r,
                torch.from_numpy(self.positions).to(dev), self.axis, q, qo)
        nv.nvkv_append_rope_axes(*args, stream=stream)
        torch.cuda.synchronize()
        return cache.pool.cpu().numpy(), None if qo is None else qo.double().cpu().numpy()


CASES = [
    # Hq, Hkv, D, ctx, n, rotary, axes, kind
    (24, 4, 256, [30, 100, 0], [37, 5, 16], 256, 3, "sections"),
    (24, 4, 256, [301], [1], 256, 3, "interleaved"),
    (8, 2, 128, [15, 0, 31, 16], [1, 33, 2, 16], 128, 2, "interleaved"),
    (8, 2, 128, [7], [70], 32, 4, "sections"),
    (16, 2, 256, [5, 12], [50, 4], 64, 3, "sections"),
    (5, 5, 128, [3, 1], [18, 31], 96, 1, "last"),
    (9, 9, 256, [16], [16], 128, 2, "last"),
    (3, 1, 256, [0, 9, 0], [0, 7, 0], 256, 4, "interleaved"),
]


@pytest.mark.parametrize("fill", [0xA5, None], ids=["sentinel", "random"])
@pytest.mark.parametrize("c", CASES, ids=[f"{c[0]}_{c[1]}_{c[2]}_r{c[5]}_a{c[6]}" for c in CASES])
def test_pool_is_bit_exact_and_queries_turn(c, fill):
    s = Setup(*c, seed=1, fill=fill)
    pool, q = s.run()
    assert int(s.err.item()) == 0
    assert np.array_equal(pool, s.want_pool())
    want, tol = s.want_q()
    assert (np.abs(q - want) <= tol).all()


def test_without_queries_and_in_place():
    s = Setup(24, 4, 256, [30, 2], [9, 17], 128, 3, seed=2)
    pool, _ = s.run(with_q=False)
    assert np.array_equal(pool, s.want_pool())
    pool, q = s.run(in_place=True)
    assert np.array_equal(pool, s.want_pool())
    want, tol = s.want_q()
    assert (np.abs(q - want) <= tol).all()


def test_one_axis_equals_append_rope():
    """With every axis at the cache position the call is nvkv_append_rope."""
    s = Setup(24, 4, 256, [30, 2], [40, 17], 256, 3, seed=3)
    for b in range(2):
        s.positions[:, s.cu[b]:s.cu[b + 1]] = s.ctx[b] + np.arange(s.n[b])
    pool, _ = s.run()
    dev = torch.device("cuda")
    bf = lambda x: torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
    cache = nv.Cache(torch.from_numpy(s.pool0.copy()).to(dev), s.num_pages, s.Hkv, s.D)
    nv.nvkv_append_rope(cache, s.seqs, bf(s.k), bf(s.v), torch.from_numpy(s.cu).to(dev), s.rows, max(s.n),
                        torch.from_numpy(s.table).to(dev), s.r)
    torch.cuda.synchronize()
    assert np.array_equal(pool, cache.pool.cpu().numpy())


@pytest.mark.parametrize("D,Hq,Hkv", [(256, 24, 4), (128, 8, 2)])
def test_positions_outside_the_table_leave_their_rows_out(D, Hq, Hkv):
    s = Setup(Hq, Hkv, D, [10, 60], [20, 5], 64, 3, seed=4)
    s.positions[1, 3] = s.max_pos
    s.positions[2, 21] = -1
    s.positions[0, 24] = 2 ** 31 - 1
    pool, q = s.run()
    assert int(s.err.item()) == nv.DEVERR_LENGTH
    assert np.array_equal(pool, s.want_pool(skip=(3, 21, 24)))
    want, tol = s.want_q()
    ok = np.ones(s.rows, bool)
    ok[[3, 21, 24]] = False
    assert (np.abs(q - want) <= tol)[ok].all()
    assert (q[~ok] == 7.0).all()


def test_bad_page_and_bad_length():
    s = Setup(24, 4, 256, [10, 60], [20, 5], 64, 3, seed=5)
    good = s.pt[0, 1]
    s.pt[0, 1] = s.num_pages
    pool, q = s.run()
    assert int(s.err.item()) == nv.DEVERR_PAGE_ID
    s.pt[0, 1] = good
    skip = [i for i in range(20) if (10 + i) // 16 == 1]
    assert np.array_equal(pool, s.want_pool(skip=skip))
    want, tol = s.want_q()
    assert (np.abs(q - want) <= tol).all()
    s.lens[1] = 3  # fewer tokens than new rows
    pool, q = s.run()
    assert int(s.err.item()) == nv.DEVERR_LENGTH
    assert np.array_equal(pool, s.want_pool(skip=range(20, 25)))
    assert (q[20:] == 7.0).all()


def test_special_values_are_stored_as_the_plain_append_stores_them():
    """Zero rows, infinities and NaN: same bytes as nvkv_append at a zero angle."""
    s = Setup(4, 4, 256, [0], [16], 32, 1, "last", seed=6)
    s.positions[:] = 0  # cos 1, sin 0
    s.k[:, :, 32:] = s.k[:, :, 32:]
    s.v[0] = 0
    s.v[1, :, 5] = 0x7F80
    s.v[2, :, 9] = 0x7FC0
    s.k[3, :, 40] = 0xFF80
    s.k[4, :, 100] = 0x7FC0
    s.k[5] = 0
    s.v[6] = 0x8000
    pool, _ = s.run()
    dev = torch.device("cuda")
    bf = lambda x: torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
    cache = nv.Cache(torch.from_numpy(s.pool0.copy()).to(dev), s.num_pages, s.Hkv, s.D)
    nv.nvkv_append(cache, s.seqs, bf(s.k), bf(s.v), torch.from_numpy(s.cu).to(dev), 16, 16)
    torch.cuda.synchronize()
    assert np.array_equal(pool, cache.pool.cpu().numpy())


def test_python_refusals():
    s = Setup(8, 2, 128, [5], [3], 64, 2, seed=7)
    s.run()
    dev = "cuda"
    bf = lambda x: torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
    k, v, q = bf(s.k), bf(s.v), bf(s.q)
    cu, cs = torch.from_numpy(s.cu).to(dev), torch.from_numpy(s.table).to(dev)
    pos = torch.from_numpy(s.positions).to(dev)
    f = lambda **kw: nv.nvkv_append_rope_axes(*[{**dict(
        c=s.cache, s=s.seqs, k=k, v=v, cu=cu, t=3, m=3, cs=cs, r=64, pos=pos, a=s.axis, q=q, qo=q), **kw}[n]
        for n in ("c", "s", "k", "v", "cu", "t", "m", "cs", "r", "pos", "a", "q", "qo")])
    f()
    for kw in (dict(pos=pos[:, :2].contiguous()), dict(a=s.axis[:-1]), dict(qo=None), dict(k=k[:2]),
               dict(q=q[:2]), dict(r=32), dict(cu=cu[:1]), dict(k=k.cpu())):
        with pytest.raises(ValueError):
            f(**kw)
    with pytest.raises(nv.NvkvError):
        f(a=[2] * 32)


def test_every_value_under_every_scale_decides_as_the_plain_append():
    """V: every bf16 value up to 7 scales, under every positive scale (the
    group's first element is 6 scales): the bytes of nvkv_append."""
    e4m3 = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    values = torch.arange(0, 0x7F80, dtype=torch.int16).view(torch.bfloat16).double()
    groups = []
    for s in e4m3.tolist():
        v = values[(values <= 6.2 * s) & (values >= 0.1 * s)]
        v = v[: len(v) // 15 * 15] if len(v) >= 15 else torch.cat([v, v.new_zeros(15 - len(v))])
        v = v.reshape(-1, 15) * torch.where(torch.arange(15) % 2 == 0, 1.0, -1.0)
        groups.append(torch.cat([torch.full((len(v), 1), 6 * s, dtype=torch.float64), v], 1))
    g = torch.cat(groups)
    Hkv, D = 4, 256
    n = -(-len(g) // (Hkv * D // 16))
    flat = torch.zeros(n * Hkv * D // 16, 16, dtype=torch.float64)
    flat[: len(g)] = g
    v = flat.reshape(n, Hkv, D).bfloat16().cuda()
    assert torch.equal(v.double().cpu().reshape(-1, 16), flat)  # all exact bf16
    pages = -(-n // 16)
    seqs = nv.Seqs(torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                   torch.tensor([n], dtype=torch.int32, device="cuda"), pages * 16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cs = torch.zeros(1, 16, 2, device="cuda")
    cs[..., 0] = 1
    pos = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    a = nv.Cache.allocate(pages, Hkv, D, "cuda", fill=0)
    b = nv.Cache.allocate(pages, Hkv, D, "cuda", fill=0)
    nv.nvkv_append_rope_axes(a, seqs, v, v, cu, n, n, cs, 32, pos, [0] * 16)
    nv.nvkv_append(b, seqs, v, v, cu, n, n)
    torch.cuda.synchronize()
    assert torch.equal(a.pool, b.pool)


def test_fp32_neighbours_of_every_border_decide_as_the_plain_rotating_append():
    """K: fp32 values on every rounding border m * s and up to 6 floats beside
    it, for 40 scales, made by a table of (value, 0) under unit elements."""
    D, half = 256, 128
    rows = []
    for byte in range(8, 127, 3):
        s = torch.tensor([byte], dtype=torch.uint8).view(torch.float8_e4m3fn).float()
        vals = []
        for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            base = (s * m).view(torch.int32)
            vals += [(base + d).view(torch.float32) for d in range(-6, 7)]
        vals = torch.cat(vals)
        vals = torch.cat([vals, vals.new_zeros(-len(vals) % 15)]).reshape(-1, 15)
        rows.append(torch.cat([torch.full((len(vals), 1), 6.0) * s, vals], 1))
    g = torch.cat(rows)
    n = -(-len(g) // (half // 16))
    cs = torch.zeros(n, half, 2)
    flat = torch.zeros(n * half // 16, 16)
    flat[: len(g)] = g
    cs[..., 0] = flat.reshape(n, half)
    k = torch.zeros(n, 1, D, dtype=torch.bfloat16, device="cuda")
    k[..., :half] = torch.where(torch.arange(half) % 3 == 0, -1.0, 1.0)
    k[..., 0:half:16] = 1.0
    pages = -(-n // 16)
    seqs = nv.Seqs(torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                   torch.tensor([n], dtype=torch.int32, device="cuda"), pages * 16)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous()
    a = nv.Cache.allocate(pages, 1, D, "cuda", fill=0)
    b = nv.Cache.allocate(pages, 1, D, "cuda", fill=0)
    cs = cs.cuda()
    nv.nvkv_append_rope_axes(a, seqs, k, k, cu, n, n, cs, D, pos, [0] * half)
    nv.nvkv_append_rope(b, seqs, k, k, cu, n, n, cs, D)
    torch.cuda.synchronize()
    assert torch.equal(a.pool, b.pool)
