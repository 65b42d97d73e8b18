"""The router of a layer of experts and the move of tokens to their columns and back, against the formulas in 64 bits.

Integers are compared exactly.  Gates: expf is within 2 units in the last place (2^-22 relative), a sum of E such terms adds
(E + 2) 2^-24, a division 2^-23.  Sums of n products in fp32: (n + 1) 2^-24 of the sum of magnitudes.  Outputs in bf16 add
half a step, 2^-8.
"""
import math

import pytest
import torch

import sparse_gemm_nm_b200 as nm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


def padded(values, dtype, pad=0):
    """The matrix with 16-byte rows; what lies behind a row's end is NaN."""
    r, c = values.shape
    per = 8 if dtype == BF else 4
    ld = max((c + per - 1) // per * per + pad, per)
    out = torch.full((r, ld), math.nan, device=DEV, dtype=dtype)[:, :c]
    out.copy_(values)
    return out


def reference(logits, k, renorm):
    """(expert, gate, slot, source, offsets) chosen one after the other, in 64 bits."""
    l = logits.double().cpu()
    E, T = l.shape
    key = torch.where(l.isnan(), INF, l)  # NaN (and +inf behind it) first
    rank = l.isnan().double()
    expert = torch.full((k, T), -1, dtype=torch.int64)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-rank[e, t].item(), -key[e, t].item(), e))
        for j, e in enumerate(order[:k]):
            if l[e, t].item() != -INF:
                expert[j, t] = e
    z = torch.where(expert >= 0, l.gather(0, expert.clamp(min=0)), -INF)
    over = z if renorm else l
    top = over.max(0).values  # by differences: a log-sum-exp near the type's lowest value has no room for log 4
    total = (over - top).exp().sum(0)
    gate = torch.where(top == INF, torch.where(z == INF, math.nan, 0.0), (z - top).exp() / total)
    gate = torch.where(expert >= 0, torch.where(top.isnan(), math.nan, gate), 0.0)
    slot, source, offsets = torch.full((k, T), -1, dtype=torch.int64), [], [0]
    for e in range(E):
        for t, j in (expert == e).T.nonzero().tolist():
            slot[j, t] = len(source)
            source.append(j * T + t)
        offsets.append(len(source))
    source += [-1] * (k * T - len(source))
    return expert, gate, slot, torch.tensor(source, dtype=torch.int64), torch.tensor(offsets)


def check_route(logits, k, renorm):
    got = nm.experts_route(logits, k, renorm=renorm)
    want = reference(logits, k, renorm)
    for g, w, name in zip(got, want, ("expert", "gate", "slot", "source", "offsets")):
        assert g.shape == w.shape
        if name == "gate":
            err = (g.cpu().double() - w).abs()
            assert (err <= (logits.shape[0] + 16) * 2.0 ** -23 * w + 1e-38)[~w.isnan()].all(), name
            assert torch.equal(g.cpu().isnan(), w.isnan())
        else:
            assert torch.equal(g.cpu().long(), w), name
    return got, want


@pytest.mark.parametrize("E,T,k", [(1, 1, 1), (2, 5, 2), (7, 31, 3), (64, 16, 6), (64, 32, 8), (65, 33, 16), (8, 513, 2),
                                   (256, 100, 8), (1024, 40, 4), (33, 1500, 1), (16, 1024, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(E, T, k, dtype, renorm):
    g = torch.Generator(device=DEV).manual_seed(E + T + k)
    l = torch.randn((E, T), generator=g, device=DEV)
    if E > 4:  # ties, skewed experts, experts that a token may not use, tokens of padding
        l[1::3] = (l[1::3] * 2).round() / 2
        l[0] += 1.5
        l[torch.rand((E, T), generator=g, device=DEV) < 0.1] = -INF
        l[:, torch.rand(T, generator=g, device=DEV) < 0.1] = -INF
    check_route(padded(l, dtype, 8), k, renorm)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_special_values(dtype, renorm):
    low = torch.finfo(dtype).min
    l = torch.tensor([[0.0, -0.0, 1.0, INF, math.nan, low, -INF, low, 3.0],
                      [-0.0, 0.0, math.nan, 2.0, math.nan, low, -INF, low, low],
                      [0.0, 0.0, 0.5, 1.0, 0.0, low, -INF, -INF, low],
                      [-1e-30, -0.0, -INF, INF, INF, low, 4.0, -INF, low]], device=DEV)
    for k in (1, 2, 3, 4):
        got, want = check_route(padded(l, dtype), k, renorm)
    assert got[0][:, 0].tolist() == [0, 1, 2, 3]  # -0 ties with +0
    assert got[0][:, 6].tolist() == [3, -1, -1, -1] and got[1][1:, 6].tolist() == [0, 0, 0]


def test_route_nowhere():
    """No token may use any expert; and one expert takes all."""
    l = padded(torch.full((8, 70), -INF, device=DEV), BF)
    expert, gate, slot, source, offsets = nm.experts_route(l, 2)
    assert (expert == -1).all() and (gate == 0).all() and (slot == -1).all() and (source == -1).all() and (offsets == 0).all()
    l[5] = 1
    expert, gate, slot, source, offsets = nm.experts_route(l, 2)
    assert offsets.tolist() == [0] * 6 + [70] * 3 and source.tolist() == list(range(70)) + [-1] * 70
    assert (gate[0] == 1).all() and (gate[1] == 0).all()
    none = nm.experts_route(torch.empty((4, 0), dtype=BF, device=DEV), 2)
    assert none[0].shape == (2, 0) and none[4].tolist() == [0] * 5


def test_route_rows_of_any_stride():
    g = torch.Generator(device=DEV).manual_seed(2)
    wide = torch.randn((9, 51), generator=g, device=DEV)
    for dtype in (BF, F32):
        l = wide.to(dtype)[:, 1:46]
        got, want = check_route(l, 3, False)
        dgate = torch.randn((3, 45), generator=g, device=DEV)
        a = nm.experts_route_grad(l, got[0], got[1], dgate, renorm=False)
        assert torch.equal(a, nm.experts_route_grad(padded(l, dtype), got[0], got[1], dgate, renorm=False))


def test_route_many_tokens():
    """More groups of tokens than one pass over the counts takes at a time: a permutation, sorted, with the right counts."""
    g = torch.Generator(device=DEV).manual_seed(3)
    E, T, k = 48, 70001, 3
    l = padded(torch.randn((E, T), generator=g, device=DEV), BF)
    expert, gate, slot, source, offsets = nm.experts_route(l, k)
    assert torch.equal(torch.bincount(expert.flatten().long(), minlength=E).cumsum(0), offsets[1:].long())
    assert torch.equal(source.long().sort().values, torch.arange(k * T, device=DEV))
    assert torch.equal(slot.flatten().long()[source.long()], torch.arange(k * T, device=DEV))
    order = expert.flatten()[source.long()].long() * T + source.long() % T
    assert (order[1:] > order[:-1]).all()
    assert torch.equal(l.gather(0, expert.long()), l.topk(k, dim=0).values)


def gate_of(logits, expert, renorm):
    z = torch.where(expert >= 0, logits.gather(0, expert.clamp(min=0)), -INF)
    base = torch.logsumexp(z if renorm else logits, 0)
    return torch.where(expert >= 0, (z - torch.where(base == -INF, 0.0, base)).exp(), 0.0)


@pytest.mark.parametrize("E,T,k", [(1, 1, 1), (5, 33, 2), (64, 40, 8), (300, 70, 16)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient(E, T, k, dtype, renorm):
    g = torch.Generator(device=DEV).manual_seed(E * T)
    l = torch.randn((E, T), generator=g, device=DEV)
    if E > 4:
        l[torch.rand((E, T), generator=g, device=DEV) < 0.2] = -INF
        l[:, 3] = -INF
        l[1:, 4] = -INF
    l = padded(l, dtype)
    dgate = torch.randn((k, T), generator=g, device=DEV)
    expert, gate, *_ = nm.experts_route(l, k, renorm=renorm)
    got = nm.experts_route_grad(l, expert, gate, dgate, renorm=renorm)
    # the formula, in 64 bits
    e = expert.long()
    p = torch.zeros((E, T), dtype=torch.float64, device=DEV)
    up = torch.zeros_like(p)
    exact_gate = gate_of(l.double(), e, renorm)
    dg = torch.where(e >= 0, dgate.double(), 0.0)
    for j in range(k):
        p[e[j].clamp(min=0), torch.arange(T)] += exact_gate[j]
        up[e[j].clamp(min=0), torch.arange(T)] += dg[j]
    if not renorm:
        base = torch.logsumexp(l.double(), 0)
        p = (l.double() - torch.where(base == -INF, 0.0, base)).exp()
    ref = p * (up - (p * up).sum(0))
    mag = p * (up.abs() + (p * up.abs()).sum(0))
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    bound = (E + 3 * k + 24) * 2.0 ** -23 * mag + half * ref.abs() + 1e-38
    assert got.shape == l.shape and ((got.double() - ref).abs() <= bound).all()
    # differences of the gates themselves, for tokens whose choice does not move
    if dtype == F32 and E == 64:
        d, h = torch.randn((E, T), generator=g, device=DEV).double(), 1e-6
        l64 = l.double()
        f = [(gate_of(l64 + s * h * d, e, renorm) * dg).sum(0) for s in (1, -1)]
        slope = torch.where(l64 == -INF, 0.0, ref * d).sum(0)
        assert ((f[0] - f[1]) / (2 * h) - slope).abs().max() < 1e-6


MOVES = [  # rows, T, k, experts
    (1, 1, 1, 1), (3, 5, 2, 4), (17, 16, 6, 64), (64, 33, 2, 8), (129, 1000, 3, 8), (6, 9001, 2, 16), (5, 30000, 1, 8),
    (2, 60001, 1, 4), (3, 110001, 2, 8), (640, 7, 1, 3), (4096, 2, 2, 8),
    (1800, 1001, 3, 8), (905, 5003, 3, 16), (449, 16001, 1, 8), (1337, 8200, 2, 64), (891, 20000, 1, 4), (450, 33000, 1, 8),
    (470, 2100, 8, 32), (460, 16400, 2, 8), (300, 5000, 8, 64), (200, 16390, 8, 16), (5, 16001, 8, 16),
]


def moved(rows, T, k, E, g):
    l = torch.randn((E, T), generator=g, device=DEV)
    if T > 4:
        l[:, torch.rand(T, generator=g, device=DEV) < 0.1] = -INF
        if k > 1:
            l[1:, 2] = -INF
    return nm.experts_route(padded(l, BF), k)


@pytest.mark.parametrize("rows,T,k,E", MOVES)
def test_gather(rows, T, k, E):
    g = torch.Generator(device=DEV).manual_seed(rows + T)
    expert, gate, slot, source, offsets = moved(rows, T, k, E, g)
    X = padded(torch.randn((rows, T), generator=g, device=DEV), BF, 8)
    got = nm.experts_gather(X, source)
    src = source.long()
    want = torch.where(src >= 0, X[:, src.clamp(min=0) % T], 0.0)
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,T,k,E", MOVES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gated", [True, False])
def test_combine(rows, T, k, E, dtype, gated):
    g = torch.Generator(device=DEV).manual_seed(rows + T + 1)
    expert, gate, slot, source, offsets = moved(rows, T, k, E, g)
    Yg = padded(torch.randn((rows, k * T), generator=g, device=DEV), BF)
    Yg[:, int(offsets[-1]):] = math.nan  # columns of no expert
    got = nm.experts_combine(Yg, slot, gate if gated else None, out_dtype=dtype)
    w = torch.where(slot >= 0, gate if gated else torch.ones_like(gate), 0.0).double()
    y = torch.where(slot[:, None] >= 0, Yg[:, slot.clamp(min=0).long()].double().transpose(0, 1), 0.0)  # k x rows x T
    ref, mag = (w[:, None] * y).sum(0), (w[:, None] * y).abs().sum(0)
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    assert ((got.double() - ref).abs() <= (k + 1) * 2.0 ** -24 * mag + half * ref.abs() * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("rows,T,k,E", MOVES)
@pytest.mark.parametrize("gated", [True, False])
def test_combine_gradient(rows, T, k, E, gated):
    g = torch.Generator(device=DEV).manual_seed(rows + T + 2)
    expert, gate, slot, source, offsets = moved(rows, T, k, E, g)
    Yg = padded(torch.randn((rows, k * T), generator=g, device=DEV), BF, 16)
    Yg[:, int(offsets[-1]):] = math.nan
    dY = padded(torch.randn((rows, T), generator=g, device=DEV), BF)
    dyg, dgate = nm.experts_combine_grad(dY, Yg, slot, source, gate if gated else None)
    src = source.long().clamp(min=0)
    w = gate.flatten()[src].double() if gated else torch.ones(k * T, dtype=torch.float64, device=DEV)
    ref = torch.where(source >= 0, dY[:, src % T].double() * w, 0.0)
    assert ((dyg.double() - ref).abs() <= 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -7)).all()
    y = torch.where(slot[:, None] >= 0, Yg[:, slot.clamp(min=0).long()].double().transpose(0, 1), 0.0)
    prod = y * dY.double()
    assert ((dgate.double() - prod.sum(1)).abs() <= (rows + 1) * 2.0 ** -24 * prod.abs().sum(1)).all()
    assert (dgate[slot < 0] == 0).all()


def test_move_leaves_what_lies_behind_rows():
    """Rows end inside a 16-byte unit: the rest of it is the caller's."""
    g = torch.Generator(device=DEV).manual_seed(8)
    R, T, k = 13, 11, 3
    expert, gate, slot, source, offsets = moved(R, T, k, 4, g)
    S = k * T
    X = padded(torch.randn((R, T), generator=g, device=DEV), BF)
    xg, y = torch.full((R, 48), 5.0, device=DEV, dtype=BF), torch.full((R, 24), 5.0, device=DEV, dtype=BF)
    nm.nm_experts_gather(X, X.stride(0), R, T, source, S, xg, 48)
    nm.nm_experts_combine(xg, 48, S, R, T, k, slot, gate, y, 24)
    assert (xg[:, S:] == 5).all() and (y[:, T:] == 5).all()
    dyg, dgate = torch.full((R, 48), 5.0, device=DEV, dtype=BF), torch.empty((k, T), device=DEV)
    nm.nm_experts_combine_grad(X, X.stride(0), R, T, k, xg, 48, S, slot, source, gate, dyg, 48, dgate)
    assert (dyg[:, S:] == 5).all()
    # index arrays that start off 16 bytes
    odd = torch.empty(S + 1, dtype=torch.int32, device=DEV)[1:]
    odd.copy_(source)
    assert torch.equal(nm.experts_gather(X, odd), xg[:, :S])


def test_captured_with_other_tokens():
    g = torch.Generator(device=DEV).manual_seed(9)
    E, T, k, K = 16, 100, 4, 64
    logits = padded(torch.randn((E, T), generator=g, device=DEV), BF)
    X = padded(torch.randn((K, T), generator=g, device=DEV), BF)

    def step():
        expert, gate, slot, source, offsets = nm.experts_route(logits, k)
        xg = nm.experts_gather(X, source)
        y = nm.experts_combine(xg, slot, gate)
        dyg, dgate = nm.experts_combine_grad(X, xg, slot, source, gate)
        return expert, gate, slot, source, offsets, xg, y, dyg, dgate, nm.experts_route_grad(logits, expert, gate, dgate)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        logits.normal_()
        X.normal_()
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
