"""kda.attn_step where scores are infinite: what the softmax over the visible tokens gives, and nothing of the masked ones.
Tolerances as in test_gpu_paged.py: the weights' rounding to bf16, the output's, fp32 scores."""
import pytest
import torch

from tests import mixer_ref as ref
from tests.test_gpu_paged import BF16, caches, gen, kda, pages  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("D,HK,per", [(64, 1, 1), (128, 2, 3)])
@pytest.mark.parametrize("lens", [[1, 0, 40], [5000, 3, 129]])
@pytest.mark.parametrize("what", ["all", "all but one", "first half", "plus"])
def test_attn_step_infinite_scores(kda, workspace, D, HK, per, lens, what):  # noqa: F811
    """All visible scores -infinity: 0 / 0, no number, with a log sum of -infinity. Some: weights of 0 for those. One +infinity:
    no number. Sequences that see nothing beside them stay 0."""
    g, page = gen(30 + sum(lens)), 16
    table, total = pages(g, lens, page)
    kc, vc = caches(g, total, HK, page, D)
    for s, n in enumerate(lens):
        hit = {"all": range(n), "all but one": [t for t in range(n) if t != n // 2], "first half": range(n // 2), "plus": [n - 1] if n else []}[what]
        at = torch.tensor(list(hit), dtype=torch.long, device="cuda")
        kc[table[s].long()[at // page], :, at % page, 3] = INF if what == "plus" else -INF
    q = (torch.randn(len(lens), HK * per, D, generator=g, device="cuda")).to(BF16)
    q[..., 3] = 1.0
    pos = torch.tensor(lens, device="cuda") - 1
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.empty(kda.attn_step_workspace_bytes(len(lens), HK * per, HK, D), dtype=torch.uint8, device="cuda") if workspace else None
    kda.attn_step(q, kc, vc, table, pos, out, D ** -0.5, lse, ws)
    kda.check_device_status()
    for s, n in enumerate(lens):
        pg = table[s, :(n + page - 1) // page].long()
        for h in range(HK * per):
            if n == 0:
                assert (out[s, h] == 0).all() and lse[s, h] == -INF
                continue
            k, v = (c[pg, h // per].reshape(-1, D)[:n].double() for c in (kc, vc))
            x = D ** -0.5 * (k @ q[s, h].double())
            p, want = torch.softmax(x, 0), torch.logsumexp(x, 0)
            if torch.isnan(p).any():
                assert torch.isnan(out[s, h]).all(), (s, h)
                assert lse[s, h] == -INF if want == -INF else not torch.isfinite(lse[s, h])
                continue
            seen = torch.isfinite(x)
            size = float(D ** -0.5 * (k[seen].abs() @ q[s, h].double().abs()).max())
            tol = 2.0 ** -8 * (p @ v).abs() + (2.0 ** -8 + 2.0 ** -16 * size) * (p @ v.abs()) + 1e-30
            assert ((out[s, h].double() - p @ v).abs() <= tol).all(), (s, h)
            assert abs(float(lse[s, h]) - float(want)) <= 2.0 ** -17 * size + 2.0 ** -20 * (1 + abs(float(want)))
