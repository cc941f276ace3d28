"""Captured masked attention behind nodes that are no kernels, and behind two
streams that join: its kernels are launched as dependents of the work before
them, whatever that is."""
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv

from mod_ref import Case, Mod, assert_within

pytestmark = pytest.mark.gpu


def captured(step):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    return g


@pytest.mark.parametrize("T,D,Hq,Hkv", [(1, 256, 24, 4), (1, 128, 8, 2), (4, 256, 24, 4), (0, 256, 24, 4), (0, 128, 8, 2)])
@pytest.mark.parametrize("before", ["copies", "join", "join_behind_a_copy"])
def test_replay_sees_what_was_written_just_before(T, D, Hq, Hkv, before):
    """Queries, lengths and starts come by copies (memcpy nodes) or from
    another stream's kernels right before the call, new ones for each replay."""
    n = T or 40
    case = Case(Hq, Hkv, D, [300, 190], [n, n], seed=95).device()
    q_src, len_src = torch.empty_like(case.q_dev), torch.empty_like(case.seqs.kv_lens)
    start = torch.zeros(2 if T else 2 * n, dtype=torch.int32, device="cuda")
    start_src = torch.empty_like(start)
    mod = nv.ScoreMod(softcap=20.0, window=150, key_starts=start)
    size = (nv.nvkv_decode_workspace_bytes(2, T, Hq, Hkv, D, 0) if T else nv.nvkv_prefill_workspace_bytes(2 * n, Hq, D, 0))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(case.q_dev)
    side = torch.cuda.Stream()

    def attend():
        if T:
            nv.nvkv_decode_attn_mod(case.cache, case.seqs, case.q_dev, T, Hq, D ** -0.5, mod, 0, ws, out)
        else:
            nv.nvkv_prefill_attn_mod(case.cache, case.seqs, case.q_dev, case.cu_dev, 2 * n, n, Hq, D ** -0.5, mod, 3, ws, out)

    def step():
        main = torch.cuda.current_stream()
        if before == "copies":
            out.zero_()
            start.copy_(start_src)
            case.seqs.kv_lens.copy_(len_src)
            case.q_dev.copy_(q_src)
        else:
            side.wait_stream(main)
            with torch.cuda.stream(side):  # kernels
                torch.add(len_src, 0, out=case.seqs.kv_lens)
                torch.add(start_src, 0, out=start)
            torch.mul(q_src, 1.0, out=case.q_dev)
            if before == "join_behind_a_copy":
                out.copy_(q_src)
            main.wait_stream(side)
        attend()
        attend()  # (the workspace again, right behind)

    def fill(lens, first, gain):
        len_src.copy_(torch.tensor(lens, dtype=torch.int32))
        start_src.copy_(torch.tensor([first, 0] if T else [first] * n + [0] * n, dtype=torch.int32))
        torch.mul(good, gain, out=q_src)

    good = case.q_dev.clone()
    fill([300, 190], 0, 1.0)
    g = captured(step)
    for lens, first, gain in (([300, 190], 0, 1.0), ([n, 190], 2, 2.0), ([131, 64], 100, 0.5)):
        fill(lens, first, gain)
        torch.cuda.synchronize()
        for _ in range(5):
            g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = Case(Hq, Hkv, D, [300, 190], [n, n], seed=95)
        want.lens = lens
        want.khat = [k[:l] for k, l in zip(want.khat, lens)]
        want.vhat = [v[:l] for v, l in zip(want.vhat, lens)]
        want.q64 = lambda: good.double().cpu() * gain  # (powers of two: exact)
        m = Mod(cap=20.0, window=150, starts=[first, 0] if T else [first] * n + [0] * n)
        ref, tol = want.reference(m, D ** -0.5, bool(T), "f16 weights")
        assert_within(got, ref, tol, f"{lens}")
    assert int(case.err.item()) == 0
