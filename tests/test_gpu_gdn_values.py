"""kda.gdn where its roundings count for more than with independent keys: sequences of few tokens, and keys and queries that
have much in common.

Tolerances. What the roundings of a chunk's operands make depends on the keys: where they are alike, an output is a sum of
products P[i, j] n[j] that take each other back, and a state one of n'[j] k[j]. So the chunks' algebra is done here in 64 bits with the operands rounded as the kernel's documentation says (the state, D1', T and N' to bf16, N and P cut off to
tf32), and without. The distance of the two is what those roundings make of this input. The kernel's own bits differ (its
inverse is tf32 between blocks of 8, an eighth to a quarter of the step of T's rounding, its sums fp32), so that it meets
other roundings of the same size: 1.5 times that distance is allowed over a head, which the inverse's share, 1.03 as squares
add, and the spread of a mean of some thousand squares stay far below; 1e-4 on top for fp32 sums and the hardware's
exponentials, and a bf16 output's or state's own rounding, 1.66e-3 in the mean square, as squares add."""
import pytest
import torch

from tests.test_gpu_gdn import BF16, F32, SCALE, kda, make, run  # noqa: F401

pytestmark = pytest.mark.gpu
F64 = torch.float64
C = 64


def bf16(x):
    return x.float().to(BF16).double()


def tf32(x):
    return (x.float().contiguous().view(torch.int32) & ~0x1fff).view(torch.float32).double()


def chunks(d, h, span, rounded):
    """One head of one sequence by the chunk algebra, on the CPU in 64 bits; rounded: operands as the kernel's."""
    low, short = (bf16, tf32) if rounded else (lambda x: x, lambda x: x)
    H, HK = d["v"].shape[2], d["q"].shape[2]
    q, k, v = (d[n].flatten(0, 1)[span[0]:span[1], i].double().cpu() for n, i in (("q", h // (H // HK)), ("k", h // (H // HK)), ("v", h)))
    if d["l2"]:
        q, k = (x / (x.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    a, beta = (d[n].flatten(0, 1)[span[0]:span[1], h].double().cpu() for n in ("a", "beta"))
    u = a + d["dt_bias"][h].double().cpu()
    keep = -torch.exp(d["A_log"][h].double().cpu()) * torch.logaddexp(u, torch.zeros_like(u))
    b, outs, S = torch.sigmoid(beta), [], torch.zeros(128, 128, dtype=F64)
    for c in range(0, len(v), C):
        K, Q, V, bc = k[c:c + C], q[c:c + C], v[c:c + C], b[c:c + C]
        G = keep[c:c + C].cumsum(0)
        decay = torch.exp(G[:, None] - G[None])
        A = torch.tril(decay * (K @ K.T), -1) * bc
        P = torch.tril(decay * (Q @ K.T)) * bc * SCALE
        T = torch.linalg.solve_triangular(torch.eye(len(V), dtype=F64) + A, torch.eye(len(V), dtype=F64), upper=False, unitriangular=True)
        S_op = low(S)
        N = low(T) @ V - low(T) @ low(torch.exp(G)[:, None] * (K @ S_op.T))
        outs.append(SCALE * torch.exp(G)[:, None] * (Q @ S_op.T) + short(P) @ short(N))
        S = torch.exp(G[-1]) * S + low((torch.exp(G[-1] - G) * bc)[:, None] * N).T @ K
    return torch.cat(outs), S


def holds(d, out, fin, spans, heads):
    """The kernel's distance from the definition against that of the rounded algebra; returns the largest ratio."""
    worst = 0.0
    for i, span in enumerate(spans):
        for h in heads:
            exact, rounded = (chunks(d, h, span, r) for r in (False, True))
            got = out.flatten(0, 1)[span[0]:span[1], h].double().cpu(), fin[i, h].double().cpu()
            for what, g, e, r, own in (("out", got[0], exact[0], rounded[0], 1.66e-3), ("state", got[1], exact[1], rounded[1], 1.66e-3 if fin.dtype == BF16 else 0.0)):
                expect = float((r - e).norm() / e.norm())
                err, limit = float((g - e).norm() / e.norm()), 1.5 * (expect ** 2 + own ** 2) ** 0.5 + 1e-4
                print(f"{what} {i} {h}: off by {err:.2e}, roundings {expect:.2e}")
                assert err <= limit, (what, i, h, err, expect)
                worst = max(worst, err / limit)
    return worst


def alike(T, cos, beta, gate, seed, nseq=1, other=0):
    """Keys and queries with the cosine ``cos`` to each other in the mean: a common direction (with ``other``, two that take
    turns) in each; steps about sigmoid(beta), or ordinary ones."""
    d = make(nseq, T, 2, 1, seed=seed, gate=gate)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    u = torch.randn(2, 128, generator=g, device="cuda")
    u = (u / u.norm(dim=-1, keepdim=True))[(torch.arange(T, device="cuda") % 2) * other]
    for n in ("q", "k"):
        x = d[n][:, :, 0].float()
        x = x / x.norm(dim=-1, keepdim=True)
        d[n][:, :, 0] = (8 * ((1 - cos) ** 0.5 * x + cos ** 0.5 * u)).to(BF16)
    if beta is not None:
        d["beta"][:] = beta
    return d


@pytest.mark.parametrize("cos", [0.0, 0.1, 0.3, 0.6, 0.9])
@pytest.mark.parametrize("beta", [None, 0.0, 3.0])
@pytest.mark.parametrize("gate", [0.0, -4.0])
def test_gdn_keys_with_a_common_part(kda, cos, beta, gate):  # noqa: F811
    T = 600
    d = alike(T, cos, beta, gate, int(100 * cos))
    out, fin = run(kda, d)
    holds(d, out, fin, [(0, T)], (0, 1))


@pytest.mark.parametrize("other", [0, 1])
@pytest.mark.parametrize("beta,gate", [(1.0, 0.0), (1.0, -4.0), (None, -1.0), (3.0, -4.0)])
def test_gdn_runs_of_one_key_and_of_two(kda, beta, gate, other):  # noqa: F811
    """What padding, indentation or a table's separators give: one key over and over, or two that take turns."""
    T = 300
    d = alike(T, 1.0, beta, gate, 7, other=other)
    out, fin = run(kda, d, fin=BF16)
    holds(d, out, fin, [(0, T)], (0, 1))


@pytest.mark.parametrize("T", [9, 10, 13, 15, 16, 20])
@pytest.mark.parametrize("fin", [F32, BF16])
def test_gdn_few_tokens_through_chunks(kda, T, fin):  # noqa: F811
    d = make(3, T, 2, 2, seed=T)
    out, st = run(kda, d, fin=fin)
    holds(d, out, st, [(i * T, (i + 1) * T) for i in range(3)], (0, 1))
