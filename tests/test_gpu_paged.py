"""Query and key norm with rotation, the paged cache and attention of single tokens (kda.qk_rope, kda.kv_append,
kda.attn_step) against their 64-bit formulas.

Tolerances. A turned channel is off by its bf16 rounding, 2^-8 of it, and by a few fp32 roundings of its two terms (angle,
sine and cosine, norm: under 2^-20 of their sum). Attention rounds its weights to bf16 (2^-8 of sum p |v| at most) and its
output (2^-8); scores are fp32 sums of up to 128 products, off by 2^-17 of sum |q k| at most, and change a weight and the
log sum by as much."""
import pytest
import torch

from tests import mixer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    import gated_linear_attention_kda_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def freqs(R, base=10000.0):
    return None if R == 0 else (base ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)).float()


def near(got, exp, mag):
    assert torch.isfinite(got).all()
    bad = (got.double() - exp).abs() > 2.0 ** -8 * exp.abs() + 2.0 ** -20 * mag + 1e-30
    assert not bad.any(), (int(bad.sum()), float((got.double() - exp).abs().max()))


@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 32), (128, 48), (256, 64), (256, 256), (128, 0)])
@pytest.mark.parametrize("H,HK,M", [(1, 1, 1), (5, 2, 3), (16, 4, 77), (4, 0, 9)])
@pytest.mark.parametrize("norm,inter", [(True, False), (True, True), (False, False)])
def test_qk_rope(kda, D, R, H, HK, M, norm, inter):
    g = gen(D + R + M)
    row = randn(g, M, (H + HK) * D + 16, scale=2.0)
    q = row[:, :H * D].unflatten(-1, (H, D))
    k = row[:, H * D:(H + HK) * D].unflatten(-1, (HK, D)) if HK else None
    qw, kw = (1 + randn(g, D, dtype=F32, scale=0.1) for _ in range(2))
    pos = torch.randint(-100, 100000, (M,), generator=g, device="cuda")
    qo, ko = torch.full((M, H, D), 7.0, dtype=BF16, device="cuda"), torch.full((M, HK, D), 7.0, dtype=BF16, device="cuda") if HK else None
    kda.qk_rope(q, k, qo, ko, pos, freqs(R), qw, kw, norm=norm, interleaved=inter)
    kda.check_device_status()
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        if x is not None:
            near(got, *ref.rope(x, w, pos, freqs(R), norm, inter, 1e-6))


def test_qk_rope_many_tokens_in_place(kda):
    g = gen(1)
    row = randn(g, 3, 5001, 6 * 128)
    q, k = row[..., :512].unflatten(-1, (4, 128)), row[..., 512:].unflatten(-1, (2, 128))
    pos = torch.arange(5001, device="cuda").repeat(3, 1)
    exp = [ref.rope(x, None, pos, freqs(64), True, False, 1e-6) for x in (q, k)]
    kda.qk_rope(q, k, q, k, pos, freqs(64))
    kda.check_device_status()
    near(q, *exp[0])
    near(k, *exp[1])


@pytest.mark.parametrize("pos", [0, 1, 131071, (1 << 20) + 17, (1 << 31) - 1, 1 << 31, -5, -(1 << 30)])
def test_qk_rope_far_positions(kda, pos):
    """Angles of positions that no float holds: the reference's product is exact to 2^-53 of it."""
    g = gen(2)
    q = randn(g, 2, 3, 128)
    p = torch.tensor([pos, pos + 1], device="cuda")
    f = freqs(128, 500000.0)
    out = torch.empty_like(q)
    kda.qk_rope(q, None, out, None, p, f, norm=False)
    near(out, *ref.rope(q, None, p, f, False, False, 0.0))


@pytest.mark.parametrize("f", [0.0, 1e-30, 2.0 ** -126, 1e-40, 3.0, 1234.5, -0.25, 2.0 ** 30])
def test_qk_rope_any_frequency(kda, f):
    g = gen(3)
    q = randn(g, 4, 2, 64)
    p = torch.tensor([0, 1, 7, 1000], device="cuda")
    fr = torch.full((8,), f, device="cuda")
    out = torch.empty_like(q)
    kda.qk_rope(q, None, out, None, p, fr, norm=False)
    near(out, *ref.rope(q, None, p, fr, False, False, 0.0))


def test_qk_rope_no_numbers_stay_in_their_head(kda):
    g = gen(4)
    q = randn(g, 5, 4, 128)
    q[2, 1, 3] = float("nan")
    q[3, 2, 127] = float("inf")
    p = torch.arange(5, device="cuda")
    out = torch.empty_like(q)
    kda.qk_rope(q, None, out, None, p, freqs(128))
    bad = ~torch.isfinite(out).all(-1)
    assert bad[2, 1] and bad[3, 2] and bad.sum() == 2


def pages(g, held, page, spare=3):
    """A table of distinct pages in no order, and their count; entries behind the last are -1."""
    need = [(n + page - 1) // page for n in held]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda")[:sum(need)].to(torch.int32)
    table = torch.full((len(held), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


def caches(g, total, HK, page, D, joint=True):
    if joint:
        c = randn(g, total, 2, HK, page, D)
        return c[:, 0], c[:, 1]
    return randn(g, total, HK, page, D), randn(g, total, HK, page, D)


@pytest.mark.parametrize("D,R,page,HK", [(64, 64, 8, 1), (128, 32, 64, 3), (128, 0, 16, 2), (256, 128, 128, 1)])
@pytest.mark.parametrize("lengths,before", [([1], [0]), ([5, 1, 70], [3, 0, 64]), ([0, 130, 0, 9], [0, 7, 5, 100])])
@pytest.mark.parametrize("norm,inter,joint", [(True, False, True), (False, True, False)])
def test_kv_append_packed(kda, D, R, page, HK, lengths, before, norm, inter, joint):
    g = gen(D + R + sum(lengths))
    cu = torch.tensor([0] + lengths).cumsum(0).cuda()
    T = sum(lengths)
    table, total = pages(g, [a + b for a, b in zip(lengths, before)], page)
    kc, vc = caches(g, total, HK, page, D, joint)
    row = randn(g, 1, T, 2 * HK * D + 8)
    k, v = row[..., :HK * D].unflatten(-1, (HK, D)), row[..., HK * D:2 * HK * D].unflatten(-1, (HK, D))
    pos = torch.cat([torch.arange(b, b + n) for n, b in zip(lengths, before)]).cuda()[None]
    w = 1 + randn(g, D, dtype=F32, scale=0.1)
    old = kc.clone(), vc.clone()
    kda.kv_append(k, v, kc, vc, table, pos, freqs(R), w, norm=norm, interleaved=inter, cu_seqlens=cu)
    kda.check_device_status()
    y, mag = ref.rope(k[0], w, pos[0], freqs(R), norm, inter, 1e-6)
    t = 0
    for s, (n, b) in enumerate(zip(lengths, before)):
        for i in range(b, b + n):
            at = int(table[s, i // page]), i % page
            near(kc[at[0], :, at[1]], y[t], mag[t])
            assert torch.equal(vc[at[0], :, at[1]], v[0, t])
            old[0][at[0], :, at[1]], old[1][at[0], :, at[1]] = kc[at[0], :, at[1]], vc[at[0], :, at[1]]
            t += 1
    assert torch.equal(kc, old[0]) and torch.equal(vc, old[1])  # nothing else has changed


def test_kv_append_step_and_padding(kda):
    """One token per sequence; positions below zero are padding and leave the cache alone."""
    g, S, HK, D, page = gen(5), 40, 2, 128, 16
    pos = torch.randint(0, 200, (S,), generator=g, device="cuda")
    pos[[3, 17, 39]] = -1
    table, total = pages(g, (pos + 1).tolist(), page)
    kc, vc = caches(g, total, HK, page, D)
    old = kc.clone(), vc.clone()
    k, v = randn(g, S, HK, D), randn(g, S, HK, D)
    kda.kv_append(k, v, kc, vc, table, pos)
    kda.check_device_status()
    for s in range(S):
        if pos[s] >= 0:
            pg, sl = int(table[s, pos[s] // page]), int(pos[s] % page)
            old[0][pg, :, sl], old[1][pg, :, sl] = k[s], v[s]
    assert torch.equal(kc, old[0]) and torch.equal(vc, old[1])


def test_kv_append_batched_rows(kda):
    g, B, T, HK, D, page = gen(6), 3, 50, 2, 64, 32
    pos = torch.arange(T, device="cuda").repeat(B, 1)
    table, total = pages(g, [T] * B, page)
    kc, vc = caches(g, total, HK, page, D)
    k, v = randn(g, B, T, HK, D), randn(g, B, T, HK, D)
    kda.kv_append(k, v, kc, vc, table, pos)
    kda.check_device_status()
    for b in range(B):
        got = kc[table[b].long()].transpose(1, 2).reshape(-1, HK, D)[:T]
        assert torch.equal(got, k[b])


@pytest.mark.parametrize("what", ["position", "page", "negative page"])
def test_kv_append_bad_pages_are_flagged_and_not_written(kda, what):
    g, S, HK, D, page = gen(7), 4, 1, 64, 8
    table, total = pages(g, [20] * S, page)
    kc, vc = caches(g, total, HK, page, D)
    pos = torch.full((S,), 19, device="cuda")
    if what == "position":
        pos[1] = 24
    else:
        table[1, 2] = total if what == "page" else -7
    old = kc.clone()
    k, v = randn(g, S, HK, D), randn(g, S, HK, D)
    kda.kv_append(k, v, kc, vc, table, pos)
    with pytest.raises(kda.KDAError, match="page"):
        kda.check_device_status()
    for s in (0, 2, 3):
        old[int(table[s, 2]), :, 3] = k[s]
    assert torch.equal(kc, old)


def check_attn(kda, q, kc, vc, table, pos, scale, workspace=True, lse=True):
    S, H, D = q.shape
    HK = kc.shape[1]
    out, ls = torch.full_like(q, 7.0), torch.full((S, H), 7.0, device="cuda") if lse else None
    ws = torch.full((kda.attn_step_workspace_bytes(S, H, HK, D),), 255, dtype=torch.uint8, device="cuda") if workspace else None
    kda.attn_step(q, kc, vc, table, pos, out, scale, ls, ws)
    kda.check_device_status()
    exp, else_, mag, size = ref.attn_step(q, kc, vc, table, pos, scale)
    err = (out.double() - exp).abs()
    tol = 2.0 ** -8 * exp.abs() + (2.0 ** -8 + 2.0 ** -16 * size[..., None]) * mag + 1e-30
    assert (err <= tol).all(), float((err / tol).max())
    if lse:
        live = torch.isfinite(else_)
        assert torch.equal(torch.isfinite(ls), live) and (ls[~live] == -torch.inf).all()
        assert ((ls.double() - else_).abs()[live] <= 2.0 ** -17 * size[live] + 2.0 ** -20 * (1 + else_[live].abs())).all()
    return out, ls


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,HK", [(1, 1), (4, 4), (6, 2), (16, 2), (20, 1), (40, 1)])
@pytest.mark.parametrize("lens,page", [([1], 8), ([7, 0, 64, 65], 16), ([1000, 3, 257], 64), ([129, 128, 127], 128), ([513], 256)])
@pytest.mark.parametrize("workspace", [True, False])
def test_attn_step(kda, D, H, HK, lens, page, workspace):
    g = gen(D + H + sum(lens))
    table, total = pages(g, lens, page)
    kc, vc = caches(g, total, HK, page, D, joint=H % 2 == 0)
    row = randn(g, len(lens), H * D + 24)
    check_attn(kda, row[:, :H * D].unflatten(-1, (H, D)), kc, vc, table, torch.tensor(lens, device="cuda") - 1, D ** -0.5, workspace)


def test_attn_step_many_ragged_sequences(kda):
    g = gen(11)
    lens = torch.randint(0, 700, (70,), generator=g, device="cuda").tolist()
    table, total = pages(g, lens, 32)
    kc, vc = caches(g, total, 2, 32, 128)
    check_attn(kda, randn(g, 70, 8, 128), kc, vc, table, torch.tensor(lens, device="cuda") - 1, 128 ** -0.5)


@pytest.mark.parametrize("scale,size", [(0.09, 30.0), (-0.1, 1.0), (0.0, 1.0), (1.0, 20.0)])
def test_attn_step_large_scores(kda, scale, size):
    """Weights that leave one token, and scores in the hundreds."""
    g = gen(12)
    lens = [300, 5, 64]
    table, total = pages(g, lens, 16)
    kc, vc = caches(g, total, 2, 16, 128)
    check_attn(kda, randn(g, 3, 8, 128, scale=size), kc, vc, table, torch.tensor(lens, device="cuda") - 1, scale)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3.3e38])
def test_attn_step_rows_behind_the_position_are_not_used(kda, junk):
    """Whatever stands behind a position in its last page, and in pages that the table holds for later."""
    g, D, HK, page = gen(13), 128, 2, 64
    lens = [1, 63, 65, 200]
    table, total = pages(g, [256] * 4, page)
    kc, vc = caches(g, total, HK, page, D)
    for s, n in enumerate(lens):
        for t in range(n, 256):
            kc[int(table[s, t // page]), :, t % page] = junk
            vc[int(table[s, t // page]), :, t % page] = junk
    check_attn(kda, randn(g, 4, 8, D), kc, vc, table, torch.tensor(lens, device="cuda") - 1, D ** -0.5)


def test_attn_step_no_number_in_sight_reaches_its_heads_alone(kda):
    g, D, page = gen(14), 64, 16
    lens = [40, 40]
    table, total = pages(g, lens, page)
    kc, vc = caches(g, total, 2, page, D)
    q = randn(g, 2, 4, D)
    pos = torch.tensor(lens, device="cuda") - 1
    clean = check_attn(kda, q, kc, vc, table, pos, 0.125, workspace=False)[0].clone()
    vc[int(table[0, 1]), 1, 3, 7] = float("nan")
    out = torch.empty_like(q)
    kda.attn_step(q, kc, vc, table, pos, out, 0.125)
    hit = ~torch.isfinite(out)
    assert hit[0, 2:, 7].all() and hit.sum() == 2
    assert torch.equal(out[~hit], clean[~hit])
    vc[int(table[0, 1]), 1, 3, 7] = 0
    kc[int(table[1, 0]), 0, 2, 1] = float("nan")
    kda.attn_step(q, kc, vc, table, pos, out, 0.125)
    hit = ~torch.isfinite(out).all(-1)
    assert hit[1, :2].all() and hit.sum() == 2


@pytest.mark.parametrize("what", ["position", "page"])
def test_attn_step_bad_pages_are_flagged(kda, what):
    g, D, page = gen(15), 64, 8
    table, total = pages(g, [30, 30, 30], page)
    kc, vc = caches(g, total, 1, page, D)
    q, pos = randn(g, 3, 2, D), torch.full((3,), 29, device="cuda")
    good = torch.empty_like(q)
    kda.attn_step(q, kc, vc, table, pos, good, 0.125)
    kda.check_device_status()
    if what == "position":
        pos[1] = 32
    else:
        table[1, 1] = total + 5
    out = torch.empty_like(q)
    kda.attn_step(q, kc, vc, table, pos, out, 0.125)
    with pytest.raises(kda.KDAError, match="page"):
        kda.check_device_status()
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    if what == "position":
        assert (out[1] == 0).all()
    else:  # the bad page's tokens are left out
        live = [t for t in range(30) if t // page != 1]
        k, v = (torch.stack([c[int(table[1, t // page]), 0, t % page] for t in live]).double() for c in (kc, vc))
        exp = torch.softmax(0.125 * (q[1].double() @ k.T), -1) @ v
        assert (out[1].double() - exp).abs().max() <= 2.0 ** -6


def test_attn_step_far_offsets(kda):
    """A cache of more than 2^32 elements: pages near its end."""
    page, HK, D = 256, 8, 128
    total = (1 << 32) // (page * HK * D) + 40
    kc, vc = torch.zeros(total, HK, page, D, dtype=BF16, device="cuda"), torch.zeros(total, HK, page, D, dtype=BF16, device="cuda")
    g = gen(16)
    table = torch.tensor([[total - 1, 3, total - 2]], dtype=torch.int32, device="cuda")
    T = 3 * page - 5
    k, v = randn(g, 1, T, HK, D), randn(g, 1, T, HK, D)
    kda.kv_append(k, v, kc, vc, table, torch.arange(T, device="cuda")[None])
    q = randn(g, 1, 16, D)
    out = torch.empty_like(q)
    kda.attn_step(q, kc, vc, table, torch.tensor([T - 1], device="cuda"), out, D ** -0.5)
    kda.check_device_status()
    small = torch.stack([kc[i] for i in table[0].tolist()]), torch.stack([vc[i] for i in table[0].tolist()])
    exp, _, mag, size = ref.attn_step(q, *small, torch.tensor([[0, 1, 2]], device="cuda"), torch.tensor([T - 1]), D ** -0.5)
    assert ((out.double() - exp).abs() <= 2.0 ** -8 * exp.abs() + (2.0 ** -8 + 2.0 ** -16 * size[..., None]) * mag).all()


def test_one_layers_step_in_a_graph(kda):
    """rotation, append and attention as a decoding step runs them, captured, replayed as the sequences grow."""
    g, S, H, HK, D, page = gen(17), 5, 8, 2, 128, 16
    lens = [3, 100, 17, 64, 15]
    table, total = pages(g, [n + 4 for n in lens], page)
    kc, vc = caches(g, total, HK, page, D)
    ws = torch.empty(kda.attn_step_workspace_bytes(S, H, HK, D), dtype=torch.uint8, device="cuda")
    row, pos = randn(g, S, (H + 2 * HK) * D), torch.tensor(lens, device="cuda")
    q, k, v = (row[:, a * D:b * D].unflatten(-1, (b - a, D)) for a, b in ((0, H), (H, H + HK), (H + HK, H + 2 * HK)))
    qr, out, f = torch.empty(S, H, D, dtype=BF16, device="cuda"), torch.empty(S, H, D, dtype=BF16, device="cuda"), freqs(64)

    def step():
        kda.qk_rope(q, None, qr, None, pos, f)
        kda.kv_append(k, v, kc, vc, table, pos, f, norm=True)
        kda.attn_step(qr, kc, vc, table, pos, out, D ** -0.5, workspace=ws)

    step()
    kda.check_device_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        row.copy_(randn(g, *row.shape))
        pos.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        kda.check_device_status()
        y, _ = ref.rope(q, None, pos, f, True, False, 1e-6)
        assert (qr.double() - y).abs().max() <= 2.0 ** -7 * y.abs().max()
        exp, _, mag, size = ref.attn_step(qr, kc, vc, table, pos, D ** -0.5)
        assert ((out.double() - exp).abs() <= 2.0 ** -8 * exp.abs() + (2.0 ** -8 + 2.0 ** -16 * size[..., None]) * mag).all()


def test_two_graphs_may_share_a_workspace(kda):
    """Captured calls replayed one after the other on one stream, each over its own cache."""
    g, H, HK, D = gen(18), 8, 2, 64
    ws = torch.empty(kda.attn_step_workspace_bytes(4, H, HK, D), dtype=torch.uint8, device="cuda")
    graphs = []
    for lens, page in (([900, 3, 40, 0], 16), ([5000], 128)):
        table, total = pages(g, lens, page)
        kc, vc = caches(g, total, HK, page, D)
        q, pos = randn(g, len(lens), H, D), torch.tensor(lens, device="cuda") - 1
        out, ls = torch.empty_like(q), torch.empty(len(lens), H, device="cuda")
        kda.attn_step(q, kc, vc, table, pos, out, 0.125, ls, ws)
        torch.cuda.synchronize()
        want = out.clone(), ls.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.attn_step(q, kc, vc, table, pos, out, 0.125, ls, ws)
        graphs.append((graph, out, ls, want, (kc, vc, q)))
    for _ in range(3):
        for graph, out, ls, _, _ in graphs:
            out.zero_()
            ls.zero_()
            graph.replay()
    torch.cuda.synchronize()
    kda.check_device_status()
    for _, out, ls, want, _ in graphs:
        assert torch.equal(out, want[0]) and torch.equal(ls, want[1])


def test_attn_step_same_call_same_bits(kda):
    """Cuts follow the lengths alone and are joined in order: a call repeats its bits, also on another stream."""
    g = gen(19)
    lens = [3000, 17, 640]
    table, total = pages(g, lens, 32)
    kc, vc = caches(g, total, 4, 32, 128)
    q, pos = randn(g, 3, 16, 128), torch.tensor(lens, device="cuda") - 1
    ws = torch.empty(kda.attn_step_workspace_bytes(3, 16, 4, 128), dtype=torch.uint8, device="cuda")
    outs = []
    side = torch.cuda.Stream()
    for s in (torch.cuda.current_stream(), side, side, torch.cuda.current_stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            out = torch.empty_like(q)
            kda.attn_step(q, kc, vc, table, pos, out, 0.09, workspace=ws)
        torch.cuda.synchronize()
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_workspace_too_small_is_refused(kda):
    g = gen(20)
    table, total = pages(g, [5], 8)
    kc, vc = caches(g, total, 1, 8, 64)
    q, pos = randn(g, 1, 1, 64), torch.tensor([4], device="cuda")
    n = kda.attn_step_workspace_bytes(1, 1, 1, 64)
    assert n > 0 and kda.attn_step_workspace_bytes(500, 64, 8, 64) == n  # whatever the sizes
    with pytest.raises(ValueError, match="workspace of"):
        kda.attn_step(q, kc, vc, table, pos, q.clone(), 1.0, workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("seed", range(12))
def test_attn_step_random_shapes(kda, seed):
    import random
    r = random.Random(seed)
    S, HK, D, page = r.randint(1, 9), r.choice([1, 2, 3, 8]), r.choice([64, 128]), r.choice([8, 16, 64, 256])
    lens = [r.choice([0, 1, 15, 16, 17, r.randint(1, 3000)]) for _ in range(S)]
    g = gen(100 + seed)
    table, total = pages(g, lens, page)
    kc, vc = caches(g, total, HK, page, D, joint=r.random() < 0.5)
    check_attn(kda, randn(g, S, HK * r.choice([1, 3, 8, 17]), D), kc, vc, table, torch.tensor(lens, device="cuda") - 1, D ** -0.5, r.random() < 0.8, r.random() < 0.7)


def test_layers_hand_their_states_from_a_prompt_to_steps(kda):
    """examples/delta_attention_layers.py: prompts, then single tokens, against one longer prompt. Prompts go through the
    chunks of the delta rule (seven roundings), steps through fp32; convolution, norms, projections, weights and outputs
    round alike in number but not in place. Some sixteen roundings of at most 2^-8 that add as squares."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_attention_layers.py")
    spec = importlib.util.spec_from_file_location("delta_attention_layers", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main() <= 4 * 2.0 ** -8
