"""kda.gdn's packed calls that hold sequences of up to 8 tokens among longer ones: they run in fp32, as alone. Tolerances: an
output is off by its bf16 rounding, 2^-8 of it, and sums by 8 times 2^-16 of the row's root mean square; a state by the latter."""
import pytest
import torch

from tests.test_gpu_gdn import BF16, F32, SCALE, check, kda, make, run, want  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths", [[1] * 9, [8, 1, 2, 3, 4, 5, 6, 7], [300, 1, 0, 8, 5, 70, 2], [1, 9, 0, 8]])
@pytest.mark.parametrize("init", [None, F32, BF16])
@pytest.mark.parametrize("l2", [True, False])
def test_gdn_short_sequences_of_a_packed_call(kda, lengths, init, l2):  # noqa: F811
    """A sequence of up to 8 tokens gives the same bits beside others as alone, in fp32."""
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    spans = list(zip(cu[:-1].tolist(), cu[1:].tolist()))
    d = make(1, sum(lengths), 4, 2, seed=len(lengths), nseq=len(lengths), init=init, l2=l2)
    out, fin = run(kda, d, cu, fin=init or F32, nseq=len(lengths))
    check(out, fin, *want(d, cu), spans, short=True)
    for i, (b, e) in enumerate(spans):
        if e - b > 8:
            continue
        one = {n: d[n][:, b:e] for n in ("q", "k", "v", "a", "beta")}
        one.update(A_log=d["A_log"], dt_bias=d["dt_bias"], init=None if init is None else d["init"][i:i + 1], l2=l2)
        alone, state = run(kda, one, fin=init or F32)
        assert torch.equal(alone, out[:, b:e]) and torch.equal(state[0], fin[i])


def test_gdn_short_sequences_in_place_and_in_a_graph(kda):  # noqa: F811
    """States handed on in the same buffer, a captured call among them; a NaN stays in its sequence."""
    lengths = [3, 100, 1, 8, 0, 9]
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    d = make(1, sum(lengths), 2, 2, seed=50, nseq=len(lengths), init=F32)
    d["v"][0, 1, 0, 3] = float("nan")
    out, fin = run(kda, d, cu, nseq=len(lengths))
    hit = ~torch.isfinite(out)
    assert hit[0, 1:3, 0, 3].all() and hit.sum() == 2
    state, o2 = d["init"].clone(), torch.empty_like(out)

    def call():
        kda.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, o2, d["A_log"], d["dt_bias"], state, state, cu, qk_l2norm=True)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    state.copy_(d["init"])
    g.replay()
    torch.cuda.synchronize()
    kda.check_device_status()
    assert torch.equal(o2.nan_to_num(5.0), out.nan_to_num(5.0)) and torch.equal(state.nan_to_num(5.0), fin.nan_to_num(5.0))


def test_gdn_two_calls_at_once(kda):  # noqa: F811
    """Calls of two streams that overlap in time, packed with short sequences and batched, give the bits of one after the other."""
    lengths = [2, 700, 1, 8, 90, 1]
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    one, two = make(1, sum(lengths), 8, 4, seed=60, nseq=len(lengths), init=F32), make(6, 500, 8, 8, seed=61)
    want_one, want_two = run(kda, one, cu, nseq=len(lengths)), run(kda, two)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st, d, c, n in ((streams[0], one, cu, len(lengths)), (streams[1], two, None, 6)):
            with torch.cuda.stream(st):
                out, fin = torch.empty_like(d["v"]), torch.empty(n, 8, 128, 128, device="cuda")
                kda.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, out, d["A_log"], d["dt_bias"], d["init"], fin, c, qk_l2norm=True)
                got.append((out, fin))
    torch.cuda.synchronize()
    kda.check_device_status()
    for i, (out, fin) in enumerate(got):
        o, f = (want_one, want_two)[i % 2]
        assert torch.equal(out, o) and torch.equal(fin, f)
