"""GPU parity of the masked attention (nvkv_decode_attn_mod,
nvkv_prefill_attn_mod) against a plain 64-bit form over caches that the
oracle wrote, for both cache formats and every kernel."""
import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv

from mod_ref import Case, Mod, assert_within, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def slopes(h):
    return [2.0 ** (-8 * (i + 1) / h) for i in range(h)]


# what a kernel rounds, by the kernel the step's shape runs on
def decode_slack(case, T):
    name = nv.nvkv_decode_mod_kernel_name(case.cache, T, case.Hq)
    return {"decode_simt": "fp32", "decode_qk4": "f16 weights", "prefill_mod": "f16 scores"}[name]


DECODE = [
    # name, Hq, Hkv, D, lens, T, mod (h: query heads, B: sequences)
    ("plain", 8, 2, 128, [1, 17, 300], 1, lambda h: Mod()),
    ("cap", 24, 4, 256, [1, 129, 700], 1, lambda h: Mod(cap=30.0)),
    ("small_cap", 24, 4, 256, [500, 2], 1, lambda h: Mod(cap=0.5)),
    ("window", 24, 4, 256, [1000, 64, 200, 129], 1, lambda h: Mod(window=65)),
    ("window_one", 24, 4, 256, [300, 1], 1, lambda h: Mod(window=1)),
    ("window_unit", 8, 4, 256, [641, 640, 128], 1, lambda h: Mod(window=128)),
    ("alibi", 24, 4, 256, [777, 5, 128], 1, lambda h: Mod(slopes=slopes(h))),
    ("starts", 24, 4, 256, [600, 400, 300], 1, lambda h: Mod(starts=[300, 400, -5])),
    ("all", 24, 4, 256, [900, 333], 1,
     lambda h: Mod(cap=20.0, window=500, slopes=slopes(h), prefix=[40, 400], starts=[700, 3])),
    ("all_128", 16, 4, 128, [900, 333, 31], 3,
     lambda h: Mod(cap=20.0, window=77, slopes=slopes(h), prefix=[899, 400, 30], starts=[300, 3, 0])),
    ("verify_window", 24, 4, 256, [400, 131, 4], 4, lambda h: Mod(window=100, cap=50.0)),
    ("verify_prefix", 24, 4, 256, [260, 20], 6, lambda h: Mod(prefix=[258, 17])),
    ("verify_alibi", 16, 2, 256, [513, 90], 2, lambda h: Mod(slopes=slopes(h), cap=15.0)),
    ("verify_start_inside", 24, 4, 256, [300, 128], 6, lambda h: Mod(starts=[297, 126])),
    ("wide_verify", 24, 4, 256, [350], 16, lambda h: Mod(window=30, slopes=slopes(h))),
    ("one_head", 4, 4, 256, [200, 70], 5, lambda h: Mod(window=64, cap=5.0)),
    ("chunked_128", 8, 2, 128, [700, 129, 16], 6, lambda h: Mod(cap=30.0, window=200)),
    ("alibi_128", 8, 2, 128, [777, 5, 128], 1, lambda h: Mod(slopes=slopes(h))),
    ("one_head_128", 4, 4, 128, [200, 70], 2, lambda h: Mod(prefix=[199, 3], cap=5.0)),
    ("many_sequences", 4, 4, 256, [1 + 37 * i % 300 for i in range(70)], 1, lambda h: Mod(window=40)),
    ("short_T", 24, 4, 256, [2, 3, 150], 6, lambda h: Mod(cap=30.0, prefix=[2, 1, 0])),
    ("empty_seq", 24, 4, 256, [0, 40, 0], 1, lambda h: Mod(window=16)),
    ("nothing_seen", 24, 4, 256, [40, 50], 1, lambda h: Mod(starts=[40, 1000])),
]


@pytest.mark.parametrize("kernel", ["default", "tc", "simt"])
@pytest.mark.parametrize("c", DECODE, ids=[c[0] for c in DECODE])
def test_decode(c, kernel, monkeypatch):
    name, Hq, Hkv, D, lens, T, mod = c
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    case = Case(Hq, Hkv, D, lens, [T] * len(lens), seed=len(name) + T).device()
    m, scale = mod(Hq), D ** -0.5
    ref, tol = case.reference(m, scale, True, decode_slack(case, T))
    for splits in (0, 1, 5):
        out = run_decode(case, m, T, scale, splits)
        assert int(case.err.item()) == 0
        assert_within(out, ref, tol, f"{name}/{kernel}/S{splits}")


@pytest.mark.parametrize("D,Hq,T", [(256, 8, 1), (256, 8, 4), (128, 8, 2)])
def test_decode_k8v4(D, Hq, T):
    case = Case(Hq, 2, D, [150, 33], [T, T], seed=3, k8=True).device()
    m = Mod(cap=10.0, window=70, slopes=slopes(Hq), starts=[100, 0])
    name = nv.nvkv_decode_mod_kernel_name(case.cache, T, Hq)
    ref, tol = case.reference(m, D ** -0.5, True, "fp32" if name == "decode_simt" else "f16 weights")
    assert_within(run_decode(case, m, T, D ** -0.5), ref, tol, name)
    assert int(case.err.item()) == 0


PREFILL = [
    ("plain", 8, 2, 128, [64, 17], [64, 3], lambda h, c: Mod()),
    ("plain_256", 24, 4, 256, [300, 5], [37, 5], lambda h, c: Mod()),
    ("cap", 24, 4, 256, [400, 64], [90, 1], lambda h, c: Mod(cap=30.0)),
    ("small_cap", 24, 4, 256, [130], [50], lambda h, c: Mod(cap=0.5)),
    ("window", 24, 4, 256, [500, 130, 1], [100, 130, 1], lambda h, c: Mod(window=65)),
    ("window_one", 24, 4, 256, [100], [70], lambda h, c: Mod(window=1)),
    ("window_tile", 12, 2, 128, [300, 64], [200, 64], lambda h, c: Mod(window=64, cap=20.0)),
    ("alibi", 24, 4, 256, [333], [60], lambda h, c: Mod(slopes=slopes(h))),
    ("prefix", 24, 4, 256, [200, 90], [200, 50], lambda h, c: Mod(prefix=[150, 1000])),
    ("prefix_window", 8, 2, 256, [200], [200], lambda h, c: Mod(prefix=[128], window=40)),
    ("documents", 24, 4, 256, [300, 70], [300, 20],
     lambda h, c: Mod(starts=[(c.lens[b] - c.n[b] + i) // 47 * 47
                              for b in range(len(c.lens)) for i in range(c.n[b])])),
    ("starts_ahead", 24, 4, 256, [200], [120],   # some rows see nothing
     lambda h, c: Mod(starts=[i * 3 for i in range(120)])),
    ("nothing_seen", 24, 4, 256, [90], [90], lambda h, c: Mod(starts=[90] * 90)),
    ("all", 16, 4, 128, [260, 100], [130, 100],
     lambda h, c: Mod(cap=20.0, window=77, slopes=slopes(h), prefix=[200, 64], starts=[i % 90 for i in range(230)])),
    ("all_256", 16, 2, 256, [260, 100], [130, 100],
     lambda h, c: Mod(cap=20.0, window=77, slopes=slopes(h), prefix=[200, 64], starts=[i % 90 for i in range(230)])),
    ("one_head", 4, 4, 256, [140], [140], lambda h, c: Mod(window=100, cap=5.0)),
    ("empty_seq", 24, 4, 256, [0, 40, 0], [0, 9, 0], lambda h, c: Mod(window=16)),
]


def prefill_slack(case, kernel):
    return "fp32" if kernel == "simt" or case.k8 else "f16 scores"


@pytest.mark.parametrize("kernel", ["default", "simt"])
@pytest.mark.parametrize("c", PREFILL, ids=[c[0] for c in PREFILL])
def test_prefill(c, kernel, monkeypatch):
    name, Hq, Hkv, D, lens, n, mod = c
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    case = Case(Hq, Hkv, D, lens, n, seed=len(name)).device()
    m, scale = mod(Hq, case), D ** -0.5
    ref, tol = case.reference(m, scale, False, prefill_slack(case, kernel))
    for splits in (0, 1, 3):
        out = run_prefill(case, m, scale, splits)
        assert int(case.err.item()) == 0
        assert_within(out, ref, tol, f"{name}/{kernel}/S{splits}")


@pytest.mark.parametrize("D", [128, 256])
def test_prefill_k8v4(D):
    case = Case(8, 2, D, [90, 20], [40, 20], seed=4, k8=True).device()
    m = Mod(cap=10.0, window=30, slopes=slopes(8), prefix=[60, 0])
    ref, tol = case.reference(m, D ** -0.5, False, "fp32")
    assert_within(run_prefill(case, m, D ** -0.5), ref, tol, "k8v4")
    assert int(case.err.item()) == 0


def test_long_context_window_reads_only_its_keys():
    """A window at the end of a long sequence: the pages before it may be gone
    from the table, in decode and in prefill, and nothing is reported."""
    L, W = 5000, 100
    for D, Hq, Hkv in ((256, 24, 4), (128, 8, 2)):
        for n, run in ((1, "decode"), (4, "decode"), (33, "prefill")):
            case = Case(Hq, Hkv, D, [L], [n], seed=11)
            lo = max(0, L - n - W + 1)
            case.pt[0, :lo // 16] = np.where(np.arange(lo // 16) % 2, -1, 10 ** 6)
            case.device()
            m = Mod(window=W, cap=30.0)
            if run == "decode":
                ref, tol = case.reference(m, D ** -0.5, True, decode_slack(case, n))
                out = run_decode(case, m, n, D ** -0.5)
            else:
                ref, tol = case.reference(m, D ** -0.5, False, "f16 scores")
                out = run_prefill(case, m, D ** -0.5)
            assert int(case.err.item()) == 0
            assert_within(out, ref, tol, f"{run}/{D}/{n}")


@pytest.mark.parametrize("kernel", ["default", "tc", "simt"])
@pytest.mark.parametrize("D,Hq,Hkv", [(256, 24, 4), (128, 8, 2)])
def test_nan_bytes_outside_the_interval_stay_out(D, Hq, Hkv, kernel, monkeypatch):
    """Cache bytes of keys that no query sees (before a window or a start,
    inside the same page too, and past the end) hold NaN scale patterns."""
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    L, lo = 150, 70
    for n in (1, 3, 20):
        case = Case(Hq, Hkv, D, [L], [n], seed=5, fill=0x7F)
        blk = 18 * D
        pages = case.pool.reshape(case.num_pages, Hkv, blk)
        for pos in list(range(lo)) + list(range(L, -(-L // 16) * 16)):
            p, s = case.pt[0, pos // 16], pos % 16
            pages[p, :, 8 * D + s * (D // 16):8 * D + (s + 1) * (D // 16)] = 0x7F  # K scales
            for g in range(D // 16):
                pages[p, :, 17 * D + g * 16 + s] = 0x7F                            # V scales
        case.device()
        if n <= 3:
            m = Mod(starts=[lo])
            ref, tol = case.reference(m, D ** -0.5, True, decode_slack(case, n))
            out = run_decode(case, m, n, D ** -0.5)
        else:
            m = Mod(starts=[lo] * n)
            ref, tol = case.reference(m, D ** -0.5, False, "f16 scores")
            out = run_prefill(case, m, D ** -0.5)
        assert_within(out, ref, tol, f"{n}")


@pytest.mark.parametrize("kernel", ["default", "tc", "simt"])
def test_bad_visible_pages_are_reported_and_left_out(kernel, monkeypatch):
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    Hq, Hkv, D, L = 24, 4, 256, 200
    for n in (1, 4, 30):
        case = Case(Hq, Hkv, D, [L], [n], seed=6)
        case.pt[0, 9] = case.num_pages  # positions 144..159
        case.device()
        # 64-bit form without those keys: their scores cannot win (an
        # enormous bias is not available, so the rows are dropped)
        keep = [j for j in range(L) if j // 16 != 9]
        m = Mod(window=120, cap=25.0)
        full = case.reference(m, D ** -0.5, n <= 16, "f16 scores")[1]
        out = (run_decode(case, m, n, D ** -0.5) if n <= 16 else run_prefill(case, m, D ** -0.5))
        assert int(case.err.item()) & nv.DEVERR_PAGE_ID
        q = case.q64()
        G = Hq // Hkv
        for hq in (0, 7, 23):
            k = torch.from_numpy(case.khat[0][:, hq // G])
            v = torch.from_numpy(case.vhat[0][:, hq // G])
            for i in range(n):
                p = L - n + i
                js = [j for j in keep if p - 120 < j <= p]
                x = 25.0 * torch.tanh(k[js] @ q[i, hq] * D ** -0.5 / 25.0)
                o = torch.softmax(x, 0) @ v[js]
                # one page of about eight fewer keys: the same kinds of error,
                # on weights at most 120/104 as large
                assert ((out[i, hq].double().cpu() - o).abs() <= 2 * full[i, hq] + 2 ** -8 * o.abs() + 4e-3).all()


def test_more_segments_than_the_list_holds():
    """One split over many one-unit pairs: the CTA's segments run past its
    list."""
    for D in (128, 256):
        case = Case(16, 16, D, [5, 130, 17, 9], [1] * 4, seed=21).device()
        m = Mod(cap=10.0, window=100)
        ref, tol = case.reference(m, D ** -0.5, True, decode_slack(case, 1))
        for splits in (1, 2):
            assert_within(run_decode(case, m, 1, D ** -0.5, splits), ref, tol, f"{D}/S{splits}")
        assert int(case.err.item()) == 0


def test_rows_behind_the_last_sequence_are_left_alone():
    Hq, Hkv, D = 24, 4, 256
    for d, hq, hkv in ((256, 24, 4), (128, 8, 2)):
        case = Case(hq, hkv, d, [100, 50], [20, 7], seed=8).device()
        total = 27
        out = torch.full((total + 5, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(nv.nvkv_prefill_workspace_bytes(total, hq, d, 0), dtype=torch.uint8, device="cuda")
        nv.nvkv_prefill_attn_mod(case.cache, case.seqs, case.q_dev, case.cu_dev, total, 20, hq, d ** -0.5,
                                 Mod(window=8).device("cuda"), 0, ws, out)
        torch.cuda.synchronize()
        assert (out[total:] == 7.0).all() and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("kernel", ["default", "tc", "simt"])
def test_bad_lengths_are_reported_and_give_zero_rows(kernel, monkeypatch):
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    case = Case(24, 4, 256, [100, 60], [1, 1], seed=9).device()
    case.seqs.kv_lens[0] = 16 * case.max_pages + 1
    ref, tol = case.reference(Mod(cap=9.0), 1 / 16, True, "f16 weights")
    out = run_decode(case, Mod(cap=9.0), 1, 1 / 16)
    assert int(case.err.item()) & nv.DEVERR_LENGTH
    assert (out[0] == 0).all()
    assert_within(out[1:], ref[1:], tol[1:], "the other sequence")


def test_large_scores_keep_their_order():
    """Queries 1e3 times as large under a cap: every score near +-cap."""
    for T, Hq in ((1, 24), (4, 24)):
        case = Case(Hq, 4, 256, [300, 140], [T, T], seed=10, q_gain=1e3).device()
        m = Mod(cap=30.0)
        out = run_decode(case, m, T, 1 / 16)
        ref, tol = case.reference(m, 1 / 16, True, "f16 weights")
        assert_within(out, ref, tol, f"T{T}")


def test_plain_mod_equals_the_plain_calls():
    """Without any modification the masked calls compute the plain attention."""
    case = Case(24, 4, 256, [300, 77], [1, 1], seed=12).device()
    out = run_decode(case, Mod(), 1, 1 / 16)
    ws = torch.empty(nv.nvkv_decode_workspace_bytes(2, 1, 24, 4, 256, 0), dtype=torch.uint8, device="cuda")
    plain = torch.empty_like(out)
    nv.nvkv_decode_attn(case.cache, case.seqs, case.q_dev, 1, 24, 1 / 16, 0, ws)
    nv.nvkv_combine(case.seqs, ws, 1, 24, 4, 256, 0, plain)
    _, tol = case.reference(Mod(), 1 / 16, True, "f16 weights")
    assert ((out.double() - plain.double()).abs().cpu() <= 2 * tol).all()


def test_graph_replay_follows_lengths_and_masks():
    """One captured decode step replays with new lengths, starts and queries."""
    case = Case(24, 4, 256, [400, 90], [1, 1], seed=13).device()
    starts = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    mod = nv.ScoreMod(softcap=20.0, window=64, key_starts=starts)
    ws = torch.empty(nv.nvkv_decode_workspace_bytes(2, 1, 24, 4, 256, 0), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 24, 256), dtype=torch.bfloat16, device="cuda")
    step = lambda: nv.nvkv_decode_attn_mod(case.cache, case.seqs, case.q_dev, 1, 24, 1 / 16, mod, 0, ws, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens, st in (([400, 90], [0, 0]), ([131, 17], [100, 3]), ([64, 1], [70, 0])):
        case.seqs.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        starts.copy_(torch.tensor(st, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        short = Case(24, 4, 256, [400, 90], [1, 1], seed=13)
        short.lens = lens
        short.khat = [k[:l] for k, l in zip(short.khat, lens)]
        short.vhat = [v[:l] for v, l in zip(short.vhat, lens)]
        ref, tol = short.reference(Mod(cap=20.0, window=64, starts=st), 1 / 16, True, "f16 weights")
        assert_within(got, ref, tol, str(lens))


def test_another_stream():
    case = Case(24, 4, 256, [300, 77], [1, 1], seed=14).device()
    want = run_decode(case, Mod(window=50), 1, 1 / 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(nv.nvkv_decode_workspace_bytes(2, 1, 24, 4, 256, 0), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    m = Mod(window=50).device("cuda")
    s.wait_stream(torch.cuda.current_stream())
    nv.nvkv_decode_attn_mod(case.cache, case.seqs, case.q_dev, 1, 24, 1 / 16, m, 0, ws, out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_long_context_offsets():
    """Bias and positions at 300,000 keys: distances are exact, offsets past
    the reach of small integers are not hit by the window's unit arithmetic."""
    L = 300001
    D, Hq, Hkv = 256, 4, 4
    g = torch.Generator().manual_seed(3)
    pages = -(-L // 16)
    # a pool of 64 real pages, repeated through the page table
    base = Case(Hq, Hkv, D, [64 * 16], [1], seed=15)
    base.pt = np.resize(base.pt[0], (1, pages)).astype(np.int32)
    base.lens, base.max_pages = [L], pages
    idx = torch.arange(L) % (64 * 16)
    base.khat = [base.khat[0][idx.numpy()]]
    base.vhat = [base.vhat[0][idx.numpy()]]
    base.device()
    for m in (Mod(slopes=[1e-5, 1e-4, 2 ** -8, 0.5]), Mod(window=70000, cap=40.0)):
        G = 1
        out = run_decode(base, m, 1, 1 / 16)
        assert int(base.err.item()) == 0
        q = base.q64()
        for h in range(4):
            k, v = torch.from_numpy(base.khat[0][:, h]), torch.from_numpy(base.vhat[0][:, h])
            x = k @ q[0, h] / 16
            x = m.cap * torch.tanh(x / m.cap) if m.cap else x
            j = torch.arange(L)
            if m.slopes:
                x = x - float(np.float32(m.slopes[h])) * (L - 1 - j)
            if m.window:
                x = torch.where(j > L - 1 - m.window, x, -math.inf)
            o = torch.softmax(x, 0) @ v
            # f16 weights (2^-11), scores off by about 1e-4 (distances to
            # 3e5 at 2^-24 each and the cap's 2^-19): relative to sum w |v - o|,
            # which softmax weights keep below 2 here, plus the bf16 rounding
            assert ((out[0, h].double().cpu() - o).abs() <= 2 ** -8 * o.abs() + 2 * (2 ** -11 + 3e-4)).all()


@pytest.mark.parametrize("D,Hq,Hkv", [(256, 24, 4), (128, 8, 2)])
def test_prefill_cap_from_linear_to_saturated(D, Hq, Hkv):
    """Scores from far below the cap to far above it, in one chunk: rows whose
    scores all lie in the polynomial's range and rows past it."""
    for gain, cap in ((0.1, 50.0), (1.0, 12.0), (30.0, 20.0)):
        case = Case(Hq, Hkv, D, [200], [200], seed=17, q_gain=gain).device()
        m = Mod(cap=cap)
        ref, tol = case.reference(m, D ** -0.5, False, "f16 scores")
        assert_within(run_prefill(case, m, D ** -0.5), ref, tol, f"{gain}/{cap}")


@pytest.mark.parametrize("kernel", ["default", "simt"])
@pytest.mark.parametrize("cap", [1e-30, 1e-5, 1e-3, 3e3, 2e4, 3e4, 1e7, 1e30])
@pytest.mark.parametrize("D,Hq,Hkv", [(256, 24, 4), (128, 8, 2)])
def test_caps_of_any_size(D, Hq, Hkv, cap, kernel, monkeypatch):
    """Caps far below and far above the scores; a cap above all of them
    leaves the scores as they are."""
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    for T in (1, 5):
        case = Case(Hq, Hkv, D, [300, 77], [T, T], seed=31, q_gain=3.0).device()
        case.q_dev[0, 0] = 0.0  # scores of exactly 0
        case.q[0, 0] = 0
        m = Mod(cap=cap)
        ref, tol = case.reference(m, D ** -0.5, True, decode_slack(case, T))
        assert_within(run_decode(case, m, T, D ** -0.5), ref, tol, f"decode of {T}")
    case = Case(Hq, Hkv, D, [200], [100], seed=32, q_gain=3.0).device()
    case.q_dev[0] = 0.0
    case.q[0] = 0
    ref, tol = case.reference(m, D ** -0.5, False, prefill_slack(case, kernel))
    assert_within(run_prefill(case, m, D ** -0.5), ref, tol, "prefill")


def test_a_loose_bound_of_the_chunk_lengths():
    """max_q is only an upper bound: the largest int32 gives the same rows."""
    case = Case(24, 4, 256, [200, 90], [40, 9], seed=33).device()
    m = Mod(cap=20.0, window=64).device("cuda")
    outs = []
    for max_q in (40, 2 ** 31 - 1):
        out = torch.full((49, 24, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
        nv.nvkv_prefill_attn_mod(case.cache, case.seqs, case.q_dev, case.cu_dev, 49, max_q, 24, 1 / 16, m, 1, None, out)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)


FEW = [  # rows of a kv-head: n * Hq / Hkv at most 32, and at most 64
    (24, 4, 256, [300, 77, 6], [5, 1, 3]),
    (24, 4, 256, [300, 77, 130], [10, 2, 9]),
    (16, 2, 128, [300, 77, 4], [4, 3, 4]),
    (16, 2, 128, [200, 65, 129], [8, 1, 7]),
    (10, 1, 256, [190], [1]),
    (4, 4, 128, [700, 64], [32, 31]),
    (4, 4, 256, [140, 900], [64, 33]),
]


@pytest.mark.parametrize("masks", ["none", "window", "all"])
@pytest.mark.parametrize("c", FEW, ids=[f"{c[0]}_{c[1]}_{c[2]}_{max(c[4])}" for c in FEW])
def test_prefill_of_few_rows(c, masks):
    """Chunks short enough for a tile to hold several copies of its rows."""
    Hq, Hkv, D, lens, n = c
    case = Case(Hq, Hkv, D, lens, n, seed=41).device()
    m = {"none": Mod(), "window": Mod(window=50, cap=12.0),
         "all": Mod(cap=20.0, window=77, slopes=slopes(Hq), prefix=[l - 2 for l in lens],
                    starts=[i * 5 % 90 for i in range(sum(n))])}[masks]
    ref, tol = case.reference(m, D ** -0.5, False, "f16 scores")
    for splits in (0, 1, 3):
        assert_within(run_prefill(case, m, D ** -0.5, splits), ref, tol, f"S{splits}")
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(256, 24, 4), (128, 16, 2)])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 150])
def test_the_same_call_gives_the_same_bits(D, Hq, Hkv, n):
    """Sums have a fixed order: 40 calls, one after another, agree."""
    case = Case(Hq, Hkv, D, [900, 333, 257], [min(n, 16)] * 3 if n <= 16 else [n, 90, 120], seed=43).device()
    m = Mod(cap=15.0, window=300, slopes=slopes(Hq))
    run = (lambda: run_decode(case, m, n, D ** -0.5)) if n <= 16 else (lambda: run_prefill(case, m, D ** -0.5))
    first = run()
    assert torch.isfinite(first).all()
    for _ in range(40):
        assert torch.equal(run(), first)
    if n <= 16:
        first = run_prefill(case, m, D ** -0.5)
        for _ in range(40):
            assert torch.equal(run_prefill(case, m, D ** -0.5), first)
