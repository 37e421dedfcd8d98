"""GPU tests of scans that are cut along time with a workspace: packed and batched calls of several
sequences, every form of states, bad bounds, graph capture; the workspace's size and refusals; and
the single-token calls replayed from a graph. Tolerances are those of tests/test_gpu_block.py."""
import random

import pytest
import torch

from tests import block_ref as R
from tests.test_gpu_block import _SDT, HALF, NAN, check_states, close, cu_of, gen, randn, ssm_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import gated_linear_attention_kda_gb300 as m
    return m


def guarded(nbytes, dtype=torch.uint8, margin=4096):
    """A buffer between two margins, and a check that the margins are as they were."""
    raw = torch.full((nbytes + 2 * margin,), 0x5a, dtype=torch.uint8, device="cuda")

    def untouched():
        return bool((raw[:margin] == 0x5a).all()) and bool((raw[margin + nbytes:] == 0x5a).all())
    return raw[margin:margin + nbytes].view(dtype), untouched


def check_cut(kda, B, T, H, P, G=1, lengths=None, state="fp32", init=True, final=True, in_place=False, strided=False, seed=0):
    g = gen(seed)
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, B, T, H, P, G, strided)
    cu = cu_of(lengths) if lengths is not None else None
    S = len(lengths) if lengths is not None else B
    st = randn(g, S, H, P, 128, dtype=_SDT[state], scale=0.3) if init else None
    ref, fin, mag, fmag = R.ssm(x, dt, b, c, A_log, D, dt_bias, st, cu)
    need = kda.ssm_workspace_bytes(S, B * T, H, P)
    assert need > 0  # the call is cut
    ws, untouched = guarded(need)
    ws.fill_(0xff)
    out = torch.full((B, T, H, P), NAN, dtype=torch.bfloat16, device="cuda")
    got = (st if in_place else torch.full((S, H, P, 128), NAN, dtype=_SDT[state], device="cuda")) if final else None
    kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, initial_state=st, final_state=got, cu_seqlens=cu, workspace=ws)
    kda.check_device_status()
    assert untouched()
    close(out, ref, HALF * ref.abs() + 2 * HALF * (1 + HALF) * mag + 1e-30, "out")
    rel = float((out.double() - ref).norm() / ref.norm())
    assert rel <= HALF, rel
    if final:
        check_states(got, fin, fmag, "state")


MIXED = [1500, 0, 1, 900, 2049]


@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("lengths,state,init,final,in_place", [
    (MIXED, "fp32", True, True, True), (MIXED, "bf16", True, True, True), (MIXED, "bf16", False, True, False), (MIXED, "fp32", True, False, False),
    (MIXED, "fp32", False, False, False), ([0, 2000, 1700, 0], "fp32", True, True, True), ([129, 128, 127, 3000], "fp32", True, True, False),
    ([1280, 2560], "bf16", True, True, True)])
def test_packed(kda, lengths, state, init, final, in_place, P):
    check_cut(kda, 1, sum(lengths), 2, P, lengths=lengths, state=state, init=init, final=final, in_place=in_place, seed=len(lengths) + P)


@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("B,T,in_place,final", [(3, 1500, True, True), (2, 1408, False, True), (3, 1700, False, False)])
def test_batched(kda, B, T, in_place, final, P):
    check_cut(kda, B, T, 2, P, in_place=in_place, final=final, seed=B + T)


def test_groups_of_heads_and_strided_tokens(kda):
    check_cut(kda, 1, 4450, 4, 64, G=2, lengths=MIXED, strided=True, seed=3)


def test_more_sequences_than_a_warp_looks_at_once(kda):
    """The search for a piece's sequence goes over 32 sequences at a time. Against the uncut call, which takes each sequence
    by itself: both round scores and states to bf16 (2^-8 of the outputs together, twice), the states not at all."""
    r = random.Random(1)
    lengths = [r.choice([0, 129, 5000, 7000]) for _ in range(40)]
    T, S = sum(lengths), len(lengths)
    need = kda.ssm_workspace_bytes(S, T, 1, 64)
    assert need > 0
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(gen(8), 1, T, 1, 64, 1)
    cu, got = cu_of(lengths), []
    for ws in (None, torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")):
        out, fin = torch.full((1, T, 1, 64), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((S, 1, 64, 128), NAN, device="cuda")
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, final_state=fin, cu_seqlens=cu, workspace=ws)
        got.append((out.double(), fin.double()))
    kda.check_device_status()
    (o0, f0), (o1, f1) = got
    for i in range(S):
        s0, s1 = int(cu[i]), int(cu[i + 1])
        if s1 > s0:
            assert float((o1[:, s0:s1] - o0[:, s0:s1]).norm() / o0[:, s0:s1].norm()) <= 2 * HALF
        assert float((f1[i] - f0[i]).norm()) <= 2.0 ** -15 * float(f0[i].norm())


@pytest.mark.parametrize("P", [64, 128])
def test_bad_bounds_of_a_cut_call_touch_nothing_else(kda, P):
    """Bounds that do not rise from 0 to T, sequences that overlap among them (more pieces than the workspace has room for)."""
    g = gen(7)
    T, H = 4450, 2
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 1, T, H, P, 1)
    for bad in ([0, 4500], [1, T], [0, 2000, 1500, T], [-3, T], [0, 4449], [0, T, 0, T, 0, T], [0, 1 << 40, T], [0, 3000, -1, T]):
        N = len(bad) - 1
        need = kda.ssm_workspace_bytes(N, T, H, P)
        assert need > 0
        ws, ws_ok = guarded(need)
        out, out_ok = guarded(2 * T * H * P, torch.bfloat16)
        fin, fin_ok = guarded(4 * N * H * P * 128, torch.float32)
        kda.ssm(x, dt, b, c, out.view(1, T, H, P), A_log, D, dt_bias, final_state=fin.view(N, H, P, 128), cu_seqlens=torch.tensor(bad, device="cuda"),
                workspace=ws)
        with pytest.raises(kda.KDAError, match="cu_seqlens"):
            kda.check_device_status()
        assert ws_ok() and out_ok() and fin_ok(), bad


def test_cut_calls_are_bitwise_repeatable(kda):
    g = gen(22)
    lengths = MIXED
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, 1, sum(lengths), 2, 128, 1)
    cu, need = cu_of(lengths), kda.ssm_workspace_bytes(5, sum(lengths), 2, 128)
    assert need > 0
    got = []
    for fill in (0, 0xff, 0x41):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        out, fin = torch.empty_like(x), torch.empty(5, 2, 128, 128, device="cuda")
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, final_state=fin, cu_seqlens=cu, workspace=ws)
        got.append((out, fin))
    kda.check_device_status()
    for o, f in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(f, got[0][1])


def test_workspace_is_never_larger_than_its_bound(kda):
    """One buffer of 24 x SMs x (P K + 1) bytes serves every call."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    r = random.Random(5)
    cut = 0
    for _ in range(4000):
        P = r.choice([64, 128])
        states, H = r.choice([1, 2, 3, r.randint(1, 400)]), r.choice([1, 2, 3, 8, 32, r.randint(1, 300)])
        tokens = int(2 ** r.uniform(0, 24))
        n = kda.ssm_workspace_bytes(states, tokens, H, P)
        cut += n > 0
        assert n <= 24 * sms * (P * 128 + 1), (states, tokens, H, P)
    assert cut > 400


def test_workspace_refusals(kda):
    g = gen(4)
    T, H, P = 2000, 2, 64
    x, dt, b, c, A_log, D, dt_bias = (v.contiguous() for v in ssm_inputs(g, 1, T, H, P, 1))
    out, fin = torch.full((1, T, H, P), NAN, dtype=torch.bfloat16, device="cuda"), torch.full((1, H, P, 128), NAN, device="cuda")
    need = kda.ssm_workspace_bytes(1, T, H, P)
    assert need > 0
    arena = torch.zeros(2 * need + 64, dtype=torch.uint8, device="cuda")
    inside = arena[need - 256:need - 256 + x.numel() * 2].view(torch.bfloat16).view(x.shape)
    state = arena[need - 256:need - 256 + fin.numel() * 4].view(torch.float32).view(fin.shape)
    for ws, match, over in ((arena[:need - 16], "workspace of", {}), (arena[:16], "workspace of", {}), (arena[8:need + 8], "16-byte aligned", {}),
                            (arena[:need], "workspace must not share memory with final_state", dict(final_state=state)),
                            (arena[:need], "workspace must not share memory with initial_state", dict(initial_state=state)),
                            (arena[:need], "workspace must not share memory with x", dict(x=inside)),
                            (arena.cpu(), "workspace must be a CUDA tensor", {}), (arena[:need].view(torch.bfloat16), "workspace must be torch.uint8", {})):
        with pytest.raises(ValueError, match=match):
            kda.ssm(**{**dict(x=x, dt=dt, b=b, c=c, out=out, A_log=A_log, D=D, dt_bias=dt_bias, final_state=fin, workspace=ws), **over})
    kda.check_device_status()
    assert torch.isnan(out).all() and torch.isnan(fin).all()


@pytest.mark.parametrize("lengths", [None, MIXED])
def test_a_cut_call_replays_from_a_graph(kda, lengths):
    g = gen(20)
    B, T = (1, sum(lengths)) if lengths else (3, 1500)
    S = len(lengths) if lengths else B
    x, dt, b, c, A_log, D, dt_bias = ssm_inputs(g, B, T, 2, 64, 1)
    cu = cu_of(lengths) if lengths else None
    need = kda.ssm_workspace_bytes(S, B * T, 2, 64)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    first = randn(g, S, 2, 64, 128, dtype=torch.float32)
    state, out = first.clone(), torch.empty(B, T, 2, 64, dtype=torch.bfloat16, device="cuda")

    def run():
        kda.ssm(x, dt, b, c, out, A_log, D, dt_bias, initial_state=state, final_state=state, cu_seqlens=cu, workspace=ws)

    run()
    ref = [(out.clone(), state.clone())]
    run()
    ref.append((out.clone(), state.clone()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    state.copy_(first)
    for o, s in ref:  # the state goes on from replay to replay
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(state, s)
    kda.check_device_status()


@pytest.mark.parametrize("state", ["fp32", "bf16"])
def test_single_token_calls_replay_from_a_graph(kda, state):
    """A layer's step: convolution, recurrence, gated norm, residual norm; three replays go on as three eager steps do."""
    g = gen(21)
    S, H, P = 5, 3, 64
    n = H * P + 256
    row, taps, bias = randn(g, S, n), randn(g, n, 4, dtype=torch.float32, scale=0.5), randn(g, n, dtype=torch.float32)
    dt, A_log, D, dt_bias = randn(g, S, H), torch.rand(H, generator=g, device="cuda"), randn(g, H, dtype=torch.float32), randn(g, H, dtype=torch.float32)
    z, res0 = randn(g, S, 1, H * P), randn(g, S, H * P, dtype=torch.float32)
    w = 1 + randn(g, H * P, dtype=torch.float32, scale=0.1)
    conv0, mix0 = randn(g, S, 3, n), randn(g, S, H, P, 128, dtype=_SDT[state])
    conv, mix, res = conv0.clone(), mix0.clone(), res0.clone()
    xbc, out, pre = torch.empty_like(row), torch.empty(S, H, P, dtype=torch.bfloat16, device="cuda"), torch.empty(S, H * P, dtype=torch.bfloat16, device="cuda")

    def run():
        kda.conv_step(row, taps, xbc, conv, bias)
        b, c = (xbc[:, H * P + 128 * i:H * P + 128 * (i + 1)].unflatten(-1, (1, 128)) for i in (0, 1))
        kda.ssm_step(xbc[:, :H * P].unflatten(-1, (H, P)), dt, b, c, out, mix, A_log, D, dt_bias)
        rows = out.flatten(-2).unsqueeze(-2)
        kda.gated_norm(rows, z, w, rows, act="silu", gate_first=True)
        kda.residual_norm(rows.squeeze(-2), res, res, w, pre)

    keep = (xbc, out, pre, conv, mix, res)
    ref = []
    for _ in range(3):
        run()
        ref.append([t.clone() for t in keep])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t, t0 in ((conv, conv0), (mix, mix0), (res, res0)):
        t.copy_(t0)
    for want in ref:
        graph.replay()
        torch.cuda.synchronize()
        for got, exp in zip(keep, want):
            assert torch.equal(got, exp)
    kda.check_device_status()
