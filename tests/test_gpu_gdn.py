"""The gated delta rule (kda.gdn, kda.gdn_step) against the 64-bit recurrence.

Tolerances. Single tokens and prompts of up to 8 tokens run in fp32: an output is off by its bf16 rounding, 2^-8 of it at
most, and by fp32 sums of 128 terms over a few steps, held under 2^-16 of the row's norm; an fp32 state by the latter.
Longer prompts run in chunks whose operands are bf16: the carried state, its product with the keys, the inverse, the
corrected values (twice), the scores and the output itself, seven roundings of 2^-8 / sqrt(12) to 2^-9 / sqrt(3) of a term
at random signs. A rounding of random mantissas is 1.66e-3 of a term in the mean square, so seven of them are 4.4e-3 where
every term is as large as the result: 5e-3 of a head's norm for outputs, and for states, which see five of them and bf16's
own. An element's error is a sum of roundings of its own token's terms (of a state: its own value channel's), e.g.
sum_c S[v, c] q[c] d_c with |d_c| <= 2^-8, whose mean square goes with that row's and not with the head's: a row behind a
large initial state is larger than rows after it has decayed. So no element may be off by more than 8 times 5e-3 of the root
mean square of its row or of the head, whichever is larger (64 x 128 normal errors stay under 5 times).
Two of the seven, T[i, i] and P[i, i], are one number for all channels of a token, so that they average over tokens alone: a
sequence of fewer than 16 is given their largest values, 2^-8 each, on top."""
import pytest
import torch

from tests import mixer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
REL, FEW = 5e-3, 2.0 ** -16
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def kda():
    import gated_linear_attention_kda_gb300 as m
    return m


def make(B, T, H, HK, seed=0, nseq=None, init=None, l2=True, extra=0, gate=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    row = randn(B, T, (2 * HK + H) * 128 + extra)
    q, k, v = row[..., :HK * 128], row[..., HK * 128:2 * HK * 128], row[..., 2 * HK * 128:(2 * HK + H) * 128]
    if not l2:
        for t in (q, k):
            u = t.unflatten(-1, (HK, 128)).float()
            t.copy_((u / u.norm(dim=-1, keepdim=True)).flatten(-2))
    d = dict(q=q.unflatten(-1, (HK, 128)), k=k.unflatten(-1, (HK, 128)), v=v.unflatten(-1, (H, 128)),
             a=randn(B, T, H), beta=randn(B, T, H), A_log=torch.log(1 + 15 * torch.rand(H, generator=g, device="cuda")),
             dt_bias=randn(H, dtype=F32) - 4 + gate, init=None, l2=l2)
    if init is not None:
        d["init"] = randn(nseq or B, H, 128, 128, dtype=init, scale=0.1)
    return d


def run(kda, d, cu=None, fin=F32, nseq=None):
    B, T, H, _ = d["v"].shape
    out = torch.full((B, T, H, 128), 7.0, dtype=BF16, device="cuda")
    fin = None if fin is None else torch.full((nseq or B, H, 128, 128), 7.0, dtype=fin, device="cuda")
    kda.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, out, d["A_log"], d["dt_bias"], d["init"], fin, cu, qk_l2norm=d["l2"])
    kda.check_device_status()
    return out, fin


def want(d, cu=None):
    return ref.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, d["A_log"], d["dt_bias"], d["init"], cu, d["l2"])


def close(got, exp, rel, what, tokens=16):
    """got, exp [..., rows, 128] of one head, behind so many tokens."""
    if rel == REL and tokens < 16:
        rel += 2.0 ** -7
    err, rms = (got.double() - exp), exp.pow(2).mean(-1, keepdim=True).clamp(min=exp.pow(2).mean()).sqrt()
    assert torch.isfinite(got).all(), what
    assert err.norm() <= rel * exp.norm() + 1e-12, (what, float(err.norm() / exp.norm()))
    assert (err.abs() <= 8 * rel * rms + 2.0 ** -8 * exp.abs()).all(), (what, float((err.abs() / rms).max()))


def check(got, fin, exp, efin, spans, short=False):
    out, o = got.flatten(0, 1), exp.flatten(0, 1)
    for i, (b, e) in enumerate(spans):
        few = e - b <= 8 and short
        for h in range(o.shape[1]):
            if e > b and few:
                rms = o[b:e, h].pow(2).mean().sqrt()
                assert ((out[b:e, h].double() - o[b:e, h]).abs() <= 2.0 ** -8 * o[b:e, h].abs() + 8 * FEW * rms).all(), (i, h)
            elif e > b:
                close(out[b:e, h], o[b:e, h], REL, ("out", i, h), e - b)
            if fin is not None:
                state_rel = REL if not few else FEW + (2.0 ** -8 if fin.dtype == BF16 else 0.0)
                close(fin[i, h], efin[i, h], state_rel, ("state", i, h), e - b)


@pytest.mark.parametrize("T", [1, 2, 8, 9, 31, 53, 63, 64, 65, 127, 128, 129, 200, 517])
@pytest.mark.parametrize("H,HK,init,l2", [(2, 2, None, True), (4, 2, F32, True), (3, 1, BF16, False)])
def test_gdn_batched(kda, T, H, HK, init, l2):
    B = 2
    d = make(B, T, H, HK, seed=T, init=init, l2=l2)
    out, fin = run(kda, d, fin=init or F32)
    check(out, fin, *want(d), [(i * T, (i + 1) * T) for i in range(B)], short=True)


@pytest.mark.parametrize("lengths", [[1], [64, 64], [0, 5, 0, 130, 1, 63, 0], [200, 3, 64, 65, 1, 1, 90], [300, 0]])
@pytest.mark.parametrize("init", [None, F32, BF16])
def test_gdn_packed(kda, lengths, init):
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    d = make(1, sum(lengths), 4, 2, seed=len(lengths), nseq=len(lengths), init=init)
    out, fin = run(kda, d, cu, fin=init or F32, nseq=len(lengths))
    check(out, fin, *want(d, cu), list(zip(cu[:-1].tolist(), cu[1:].tolist())))


def test_gdn_no_dt_bias_no_states_strided_out(kda):
    d = make(2, 150, 4, 4, extra=64, seed=5)
    wide = torch.full((2, 150, 4 * 128 + 128), 3.0, dtype=BF16, device="cuda")
    out = wide[..., 64:64 + 512].unflatten(-1, (4, 128))
    kda.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, out, d["A_log"], qk_l2norm=True)
    kda.check_device_status()
    d["dt_bias"] = None
    exp, efin = want(d)
    check(out.contiguous(), None, exp, efin, [(0, 150), (150, 300)])
    assert (wide[..., :64] == 3).all() and (wide[..., 576:] == 3).all()


def test_gdn_state_in_place_and_split_calls(kda):
    """Two calls that hand the state on give what one call gives."""
    T, cut = 300, 133
    d = make(2, T, 4, 2, seed=9, init=F32)
    exp, efin = want(d)
    st, outs = d["init"].clone(), []
    for s in (slice(0, cut), slice(cut, T)):
        o = torch.empty(2, s.stop - s.start, 4, 128, dtype=BF16, device="cuda")
        part = {n: d[n][:, s].contiguous() for n in ("q", "k", "v", "a", "beta")}
        kda.gdn(*part.values(), SCALE, o, d["A_log"], d["dt_bias"], st, st, qk_l2norm=True)
        outs.append(o)
    kda.check_device_status()
    check(torch.cat(outs, 1), st, exp, efin, [(0, T), (T, 2 * T)])


def test_gdn_no_tokens(kda):
    d = make(2, 0, 2, 2, init=F32)
    _, fin = run(kda, d)
    assert torch.equal(fin, d["init"])
    d["init"] = None
    assert (run(kda, d)[1] == 0).all()


@pytest.mark.parametrize("gate", [-30.0, 4.0, 30.0])
def test_gdn_gates_at_their_ends(kda, gate):
    """Decays of nearly one and of nothing at all."""
    d = make(1, 190, 2, 1, seed=3, init=F32, gate=gate)
    out, fin = run(kda, d)
    check(out, fin, *want(d), [(0, 190)])


def test_gdn_closed_gate_between_open_ones(kda):
    """A token whose decay is nothing, however large its gate's input, forgets what came before and nothing else."""
    d = make(1, 190, 2, 1, seed=4, init=F32)
    d["a"][:, [10, 64, 100]] = 3e38
    out, fin = run(kda, d)
    check(out, fin, *want(d), [(0, 190)])


@pytest.mark.parametrize("T", [5, 100])
def test_gdn_long_keys(kda, T):
    """Keys and queries of any length with qk_l2norm, and zero keys."""
    d = make(1, T, 2, 2, seed=6)
    d["k"][:, ::3] *= 1000
    d["k"][:, 1::3] *= 0.001
    d["k"][:, 4] = 0
    d["q"][:, 2] = 0
    out, fin = run(kda, d)
    exp, efin = want(d)
    check(out, fin, exp, efin, [(0, T)], short=True)


def nan_where(x):
    return ~torch.isfinite(x)


@pytest.mark.parametrize("T", [7, 200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["v", "k", "q", "a", "beta"])
def test_gdn_no_number_reaches_no_earlier_token(kda, T, bad, name):
    """What is no number reaches what the formulas say: v its own channel, the others their head, from its token on
    (q its token alone), and no other sequence."""
    if name in ("a", "beta") and bad == float("inf"):
        bad = float("nan")  # an infinite gate or step is a number: no decay, or a step of one
    lengths, t0 = [T, T], T + T * 2 // 3
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    d = make(1, 2 * T, 2, 2, seed=8, nseq=2, init=F32)
    clean, cfin = want(d, cu)
    if name in ("a", "beta"):
        d[name][0, t0, 1] = bad
    else:
        d[name][0, t0, 1, 5] = bad
    out, fin = run(kda, d, cu, nseq=2)
    check(out[:, :t0], None, clean[:, :t0], None, [(0, T), (T, t0)])
    check(out[:, :, :1], None, clean[:, :, :1], None, [(0, T), (T, 2 * T)])
    close(fin[0, 0], cfin[0, 0], REL, "first sequence", T)
    close(fin[1, 0], cfin[1, 0], REL, "other head", T)
    hit = nan_where(out[0, t0:, 1])
    if name == "v":
        assert hit[:, 5].all() and not hit[:, :5].any() and not hit[:, 6:].any()
        other = [c for c in range(128) if c != 5]
        close(out[0, t0:, 1][:, other], clean[0, t0:, 1][:, other], REL, "other channels", T)
        assert nan_where(fin[1, 1, 5]).all() and torch.isfinite(fin[1, 1, other]).all()
    elif name == "q":
        assert hit[0].all() and not hit[1:].any() and torch.isfinite(fin).all()
    else:
        assert hit.all() and nan_where(fin[1, 1]).all()


@pytest.mark.parametrize("cu", [[0, 10, 300, 200], [0, -5, 200], [0, 100, 300], [1, 100, 200], [0, 1 << 40, 200]])
def test_gdn_bad_bounds_are_flagged(kda, cu):
    d = make(1, 200, 2, 2, seed=1, nseq=len(cu) - 1, init=F32)
    out = torch.zeros(1, 200, 2, 128, dtype=BF16, device="cuda")
    fin = torch.zeros(len(cu) - 1, 2, 128, 128, device="cuda")
    kda.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, out, d["A_log"], None, d["init"], fin, torch.tensor(cu).cuda())
    with pytest.raises(kda.KDAError):
        kda.check_device_status()
    kda.check_device_status()


@pytest.mark.parametrize("T", [4, 150])
def test_gdn_in_a_graph_and_on_another_stream(kda, T):
    d = make(2, T, 4, 2, seed=2, init=BF16)
    out, fin = run(kda, d, fin=BF16)
    o2, f2 = torch.empty_like(out), torch.empty_like(fin)

    def call():
        kda.gdn(d["q"], d["k"], d["v"], d["a"], d["beta"], SCALE, o2, d["A_log"], d["dt_bias"], d["init"], f2, qk_l2norm=True)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(f2, fin)
    for n in ("q", "k", "v"):
        d[n].mul_(0.5)
    exp, _ = run(kda, d, fin=BF16)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, exp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(o2, exp)


@pytest.mark.parametrize("S,H,HK,state,l2", [(1, 1, 1, F32, True), (3, 4, 2, BF16, True), (17, 6, 2, F32, False), (64, 8, 8, BF16, False)])
def test_gdn_step(kda, S, H, HK, state, l2):
    d = make(1, S, H, HK, seed=S, nseq=S, init=state, l2=l2, extra=32)
    tok = {n: d[n][0] for n in ("q", "k", "v", "a", "beta")}
    exp, efin = ref.gdn(*(t[:, None] for t in tok.values()), SCALE, d["A_log"], d["dt_bias"], d["init"], None, l2)
    out, st = torch.empty(S, H, 128, dtype=BF16, device="cuda"), d["init"].clone()
    kda.gdn_step(*tok.values(), SCALE, out, st, d["A_log"], d["dt_bias"], qk_l2norm=l2)
    kda.check_device_status()
    check(out[:, None], st, exp, efin, [(i, i + 1) for i in range(S)], short=True)


def test_gdn_steps_go_on_from_a_prompt(kda):
    T, n = 140, 6
    d = make(2, T, 4, 4, seed=12)
    exp, efin = want(d)
    st = torch.zeros(2, 4, 128, 128, device="cuda")
    part = {m: d[m][:, :T - n].contiguous() for m in ("q", "k", "v", "a", "beta")}
    first = torch.empty(2, T - n, 4, 128, dtype=BF16, device="cuda")
    kda.gdn(*part.values(), SCALE, first, d["A_log"], d["dt_bias"], st, st, qk_l2norm=True)
    outs = [first]
    for t in range(T - n, T):
        o = torch.empty(2, 4, 128, dtype=BF16, device="cuda")
        kda.gdn_step(*(d[m][:, t].contiguous() for m in ("q", "k", "v", "a", "beta")), SCALE, o, st, d["A_log"], d["dt_bias"], qk_l2norm=True)
        outs.append(o[:, None])
    kda.check_device_status()
    check(torch.cat(outs, 1), st, exp, efin, [(0, T), (T, 2 * T)])


@pytest.mark.parametrize("seed", range(16))
def test_gdn_random_shapes(kda, seed):
    import random
    r = random.Random(seed)
    HK = r.choice([1, 2, 3])
    lengths = [r.choice([0, 1, 63, 64, 65, r.randint(1, 600)]) for _ in range(r.randint(1, 6))] if r.random() < 0.5 else None
    if lengths is not None and sum(lengths) < 9:
        lengths[0] = 30
    B = 1 if lengths else r.randint(1, 3)
    T = sum(lengths) if lengths else r.randint(9, 700)
    init = r.choice([None, F32, BF16])
    d = make(B, T, HK * r.choice([1, 2, 4]), HK, seed=seed, nseq=len(lengths) if lengths else B, init=init, l2=r.random() < 0.6, extra=8 * r.randint(0, 5))
    cu = torch.tensor([0] + lengths).cumsum(0).cuda() if lengths else None
    out, fin = run(kda, d, cu, fin=init or F32, nseq=len(lengths) if lengths else B)
    spans = list(zip(cu[:-1].tolist(), cu[1:].tolist())) if lengths else [(i * T, (i + 1) * T) for i in range(B)]
    check(out, fin, *want(d, cu), spans)


def test_gdn_many_states_than_sms(kda):
    """More (sequence, head) pairs than the machine holds at once."""
    d = make(11, 70, 32, 16, seed=40, init=BF16)
    out, fin = run(kda, d, fin=BF16)
    exp, efin = want(d)
    for i in (0, 5, 10):
        for h in (0, 13, 31):
            close(out[i, :, h], exp[i, :, h], REL, ("out", i, h))
            close(fin[i, h], efin[i, h], REL, ("state", i, h))
    assert (out.double() - exp).norm() <= REL * exp.norm()


def test_gdn_repeated_keys(kda):
    """The worst that the roundings meet: one key for all tokens, steps b near one and no decay. A head's state is then k s^T
    with s the last value almost, and s_i = s_0 + sum_{j <= i} b n_j, n_j = sum_l T[j, l] (v_l - s_0) telescopes: what n_j
    adds n_{j+1} takes back. The inverse is known, T[j, j] = 1 and T[j, l] = -b (1 - b)^(j - l - 1), so its rounding to bf16 is
    too. Its rows no longer sum to about nothing: with b = sigmoid(6) what is off is .0014 of s_0 a token, .09 of it after a
    chunk. That has to be all beside the roundings of N and of P, 1.66e-3 of |n_j| = 2^0.5 |v| each in the mean square, which
    add up over i <= 64 tokens: 1.66e-3 (2 * 2 * 64)^0.5 = .0266, on top of REL."""
    d = make(1, 200, 2, 1, seed=41, gate=-20.0)
    d["k"][:] = d["k"][:, :1].clone()
    d["beta"][:] = 6.0
    out, fin = run(kda, d)
    exp, efin = want(d)
    assert (out.double() - exp).norm() <= .1 * exp.norm()
    b = torch.sigmoid(torch.tensor(6.0, dtype=torch.float64))
    m = torch.arange(64)[:, None] - torch.arange(64)
    T = torch.where(m == 0, 1.0, torch.where(m > 0, -b * (1 - b) ** (m - 1).clamp(min=0), 0.0)).to(BF16).double().cuda()
    k, q = d["k"].double()[0, :, 0], d["q"].double()[0, :, 0]
    kk = k / k.pow(2).sum(-1, keepdim=True).add(1e-6).sqrt()
    qq = q / q.pow(2).sum(-1, keepdim=True).add(1e-6).sqrt()
    p, v = (qq * kk).sum(-1) * SCALE, d["v"].double()[0]
    for h in range(2):
        s, rows = torch.zeros(128, dtype=torch.float64, device="cuda"), []
        for c in range(0, 200, 64):
            x = v[c:c + 64, h] - s
            at = s + b.cuda() * (T[:len(x), :len(x)] @ x).cumsum(0)
            rows.append(p[c:c + 64, None] * at)
            s = at[-1]
        rows = torch.cat(rows)
        assert (out[0, :, h].double() - rows).norm() <= (REL + .0266) * rows.norm()
        assert (fin[0, h].double() - torch.outer(s, kk[0])).norm() <= (REL + .0266) * s.norm()


@pytest.mark.parametrize("beta", [-200.0, -60.0, 60.0, float("inf"), float("-inf")])
@pytest.mark.parametrize("l2", [True, False])
def test_gdn_steps_at_their_ends(kda, beta, l2):
    """Steps of 0 and 1 among ordinary ones: a step of 0 leaves the state to its decay, and no logarithm of it shows."""
    d = make(1, 150, 2, 1, seed=43, init=F32, l2=l2)
    d["beta"][:, ::3] = beta
    out, fin = run(kda, d)
    exp, efin = want(d)
    check(out, fin, exp, efin, [(0, 150)])
    d["beta"][:] = beta
    out, fin = run(kda, d)
    exp, efin = want(d)
    if beta < 0:  # outputs are the decayed state's alone
        assert torch.isfinite(out).all() and (fin.double() - efin).norm() <= REL * efin.norm() + 1e-30
    else:
        check(out, fin, exp, efin, [(0, 150)])
