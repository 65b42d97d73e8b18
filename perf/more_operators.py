"""A layer of pruned experts and the clipping of its gradients, as cases to be measured.

Layout is the library's: activations are features x tokens with the tokens contiguous (rows padded to 16 bytes), every
expert's weight is 2:4 compressed (values E x R x K/2 bf16, positions in the tiled metadata, E x words).  Columns grouped by
expert: expert e has the columns offsets[e] .. offsets[e + 1] - 1.  ``own`` picks the side: False computes every operator
with elementary torch operations in 32 bits, True calls the library.

  route         nm.experts_route         the k experts of every token, their gates, and the columns grouped by expert
  route_both    ... and nm.experts_route_grad, the logits' gradient
  gather        nm.experts_gather        every column's token: Xg[:, s] = X[:, source[s] mod T]
  combine       nm.experts_combine       y_t = sum_j gate[j][t] Yg[:, slot[j][t]]
  combine_grad  nm.experts_combine_grad  its gradients: dYg and dgate
  spmm          nm.experts_spmm          Y[:, s] = W'_e X[:, s], e the expert of column s
  spmm_t        nm.experts_spmm_t        the input gradient of the same
  sddmm         nm.experts_sddmm         the gradients of every expert's stored survivors
  clip          nm.clip_grads            the norm over many gradients, which are scaled to max_norm where it is above
"""
import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One decoding step of 16 sequences: 6 of 64 experts each.
        {"name": "route_decode", "op": "route", "E": 64, "T": 16, "k": 6, "f32": True, "renorm": True},
        # Training on 16384 tokens, 8 of 64 experts each, with the gradient of the full softmax.
        {"name": "route_train", "op": "route_both", "E": 64, "T": 16384, "k": 8, "f32": False, "renorm": False},
        # Prompts of 8192 tokens laid out for two experts each.
        {"name": "gather_8k", "op": "gather", "K": 4096, "T": 8192, "k": 2},
        # ... and their outputs joined again.
        {"name": "combine_8k", "op": "combine", "K": 4096, "T": 8192, "k": 2},
        # The backward pass of the same join.
        {"name": "combine_grad_8k", "op": "combine_grad", "K": 4096, "T": 8192, "k": 2},
        # One token of one request at two experts of eight: a down projection of 4096 x 11008.
        {"name": "experts_token", "op": "spmm", "E": 8, "R": 4096, "K": 11008, "S": 2, "active": 2},
        # One decoding step of 16 sequences, every expert in use: an up projection of 11008 x 4096.
        {"name": "experts_decode", "op": "spmm", "E": 8, "R": 11008, "K": 4096, "S": 32, "active": 8},
        # Prompts of 8192 tokens at two experts each.
        {"name": "experts_prompt", "op": "spmm", "E": 8, "R": 11008, "K": 4096, "S": 16384, "active": 8},
        # Training on 4096 tokens: the input gradient, one expert without tokens.
        {"name": "experts_dx", "op": "spmm_t", "E": 8, "R": 11008, "K": 4096, "S": 8192, "active": 7},
        # ... and the gradients of the experts' survivors.
        {"name": "experts_dv", "op": "sddmm", "E": 8, "R": 11008, "K": 4096, "S": 8192, "active": 8},
        # Fine-tuning adapters: many small 32-bit gradients.
        {"name": "clip_adapters", "op": "clip", "tensors": 56, "total": 56 * 16 * 4096, "f32": 1.0},
        # A step of four layers: gradients of compressed values, and of the norms beside them in 32 bits.
        {"name": "clip_layers", "op": "clip", "tensors": 44, "total": 4 * (4 * 4096 + 3 * 11008) * 2048, "f32": 0.3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_both", "gather", "combine", "combine_grad", "spmm", "spmm", "spmm_t", "sddmm", "clip"])
    if op.startswith("route"):
        E = _log(rng, 2, 384)
        T = min(_log(rng, 1, 50432), 64 * 16384 // E)
        return {"op": op, "E": E, "T": T, "k": _log(rng, 1, min(E, 12)), "f32": rng.random() < 0.5,
                "renorm": rng.random() < 0.5}
    if op in ("gather", "combine", "combine_grad"):
        k = _log(rng, 1, 8)
        T = _log(rng, 1, 16384)
        K = min(_log(rng, 16, 13824), max(16, 4096 * 8192 * 2 // (T * k)))
        return {"op": op, "K": K, "T": T, "k": k}
    if op == "clip":
        return {"op": op, "tensors": _log(rng, 1, 60), "total": _log(rng, 400, 4 * (4 * 4096 + 3 * 11008) * 2048),
                "f32": rng.random()}
    E = _log(rng, 1, 96)
    K = 16 * _log(rng, 4, 688) if rng.random() < 0.5 else 128 * _log(rng, 1, 86)
    R = min(_log(rng, 8, 13824), max(8, 8 * 11008 * 4096 // (E * K)))
    S = min(_log(rng, 1, 16384), 11008 * 4096 * (16384 if op == "spmm" else 8192) // (R * K))
    return {"op": op, "E": E, "R": R, "K": K, "S": S, "active": rng.randint(1, min(E, S))}


# ------------------------------------------------------------------ inputs
def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _rows(g, rows, cols, std, dtype):
    """rows x cols with the rows padded to 16 bytes, as the library takes them."""
    per = 4 if dtype == torch.float32 else 8
    return _normal(g, (rows, (cols + per - 1) // per * per), std, dtype)[:, :cols]


def _pack_2of4(pairs, R, K):
    """Tiled metadata of one R x K weight from R x K/4 nibbles p0 | p1 << 2, padding groups 0x4."""
    rb, cb = (R + 15) // 16, (K + 127) // 128
    nib = torch.full((rb * 16, cb * 32), 4, dtype=torch.int32, device=pairs.device)
    nib[:R, :K // 4] = pairs
    nib = nib.view(rb, 2, 8, cb, 4, 2, 4)  # row block, row half, row, column block, quarter, column half, group
    words = torch.zeros((rb, 8, cb, 4, 2), dtype=torch.int32, device=pairs.device)
    for half in range(2):
        for group in range(4):
            words |= nib[:, half, :, :, :, :, group] << (16 * half + 4 * group)
    return words.permute(0, 2, 4, 1, 3).reshape(-1)  # row block, column block, column half, row, quarter


def _weights(g, E, R, K):
    """E 2:4 weights: values ~ N(0, 0.02), the two positions of every group uniform."""
    values = torch.empty((E, R, K // 2), dtype=torch.bfloat16, device=DEV)
    meta = torch.empty((E, (R + 15) // 16 * ((K + 127) // 128) * 64), dtype=torch.int32, device=DEV)
    table = torch.tensor([4, 8, 12, 9, 13, 14], dtype=torch.int32, device=DEV)  # p0 | p1 << 2 for p0 < p1
    for e in range(E):
        values[e].normal_(0, 0.02, generator=g)
        meta[e] = _pack_2of4(table[torch.randint(0, 6, (R, K // 4), generator=g, device=DEV)], R, K)
    return values, meta


def _ragged(seed, E, S, active):
    """offsets of S columns over `active` of E experts, of uneven sizes (one column at least each)."""
    r = random.Random(seed * 7919 + S)
    used = sorted(r.sample(range(E), active))
    weight = [r.uniform(0.2, 1.8) for _ in used]
    count = [1 + int((S - active) * w / sum(weight)) for w in weight]
    count[r.randrange(active)] += S - sum(count)
    sizes = [0] * E
    for e, n in zip(used, count):
        sizes[e] = n
    at = [0]
    for n in sizes:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _routed(g, T, k, E=8):
    """Of T tokens at k of max(E, k) experts: (slot k x T, source k T, gate k x T)."""
    E = max(E, k)
    score = torch.rand((E, T), generator=g, device=DEV) + torch.linspace(0, 0.3, E, device=DEV)[:, None]
    expert = score.topk(k, dim=0).indices
    order = (expert.reshape(-1) * T + torch.arange(T, device=DEV).repeat(k)).argsort()
    slot = torch.empty_like(order)
    slot[order] = torch.arange(k * T, device=DEV)
    gate = torch.softmax(torch.randn((k, T), generator=g, device=DEV), dim=0)
    return slot.view(k, T).to(torch.int32), order.to(torch.int32), gate


def _sizes(case):
    """Sizes of a clip case's gradients: uneven, the largest about 30 times the mean at most, some tiny."""
    r = random.Random(case["tensors"] * 31 + case["total"])
    n = case["tensors"]
    weight = [math.exp(r.gauss(0, 1.2)) for _ in range(n)]
    sizes = [max(1, int(case["total"] * w / sum(weight))) for w in weight]
    return sizes, [r.random() < case["f32"] for _ in range(n)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op.startswith("route"):
        E, T, k = case["E"], case["T"], case["k"]
        kind = torch.float32 if case["f32"] else torch.bfloat16
        # Experts differ in how often they are wanted; a few tokens are padding and go nowhere, and a few may not use some
        # experts.
        bias = _normal(g, (E, 1), 0.5, torch.float32)
        l = _rows(g, E, T, 1.0, torch.float32) + bias
        l = torch.where(torch.rand((E, T), generator=g, device=DEV) < 0.02, -math.inf, l)
        l = torch.where(torch.rand((1, T), generator=g, device=DEV) < 0.03, -math.inf, l)
        s["logits"] = _rows(g, E, T, 1.0, kind)
        s["logits"].copy_(l)
        if op == "route_both":
            s["dgate"] = torch.randn((k, T), generator=g, device=DEV)
        return s
    if op in ("gather", "combine", "combine_grad"):
        K, T, k = case["K"], case["T"], case["k"]
        s["slot"], s["source"], s["gate"] = _routed(g, T, k)
        if op != "combine":
            s["X"] = _rows(g, K, T, 1.0, torch.bfloat16)  # the tokens, or their gradients
        if op != "gather":
            s["Y"] = _rows(g, K, k * T, 1.0, torch.bfloat16)  # the experts' outputs
        return s
    if op == "clip":
        sizes, f32 = _sizes(case)
        s["grads"] = [_normal(g, (n,), 0.01, torch.float32 if f else torch.bfloat16) for n, f in zip(sizes, f32)]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        s["max_norm"] = 1.0 if sum(sizes) > 20000 else 0.5
        return s
    E, R, K, S = case["E"], case["R"], case["K"], case["S"]
    s["values"], s["meta"] = _weights(g, E, R, K)
    s["offsets"] = _ragged(int(seed), E, S, case["active"])
    if op != "spmm_t":
        s["X"] = _rows(g, K, S, 1.0, torch.bfloat16)
    if op != "spmm":
        s["dY"] = _rows(g, R, S, 1.0, torch.bfloat16)
    return s


# -------------------------------------------------------------- plain form
def _columns(meta, R, K):
    """R x K/2 column of every stored survivor of one weight."""
    rb, cb = (R + 15) // 16, (K + 127) // 128
    words = meta.view(rb, cb, 2, 8, 4, 1, 1)
    shift = 16 * torch.arange(2, device=meta.device).view(2, 1) + 4 * torch.arange(4, device=meta.device)
    nib = (words >> shift.to(torch.int32)) & 15  # row block, column block, column half, row, quarter, row half, group
    nib = nib.permute(0, 5, 3, 1, 4, 2, 6).reshape(rb * 16, cb * 32)[:R, :K // 4]
    first = 4 * torch.arange(K // 4, device=meta.device)
    return torch.stack([first + (nib & 3), first + (nib >> 2)], dim=2).reshape(R, K // 2)


def _dense(values, meta, R, K):
    w = torch.zeros((R, K), dtype=torch.float32, device=values.device)
    return w.scatter_(1, _columns(meta, R, K), values.float())


def _plain_route(s):
    E, T, k = s["E"], s["T"], s["k"]
    l = s["logits"].float()
    top, expert = l.sort(dim=0, descending=True, stable=True)
    top, expert = top[:k], expert[:k]
    has = top > -math.inf
    first = torch.where(has[:1], top[:1], 0.0)
    e = (top - first).exp()
    total = e.sum(0) if s["renorm"] else (l - first).exp().sum(0)
    gate = torch.where(has, e / torch.where(total > 0, total, 1.0), 0.0)
    expert = torch.where(has, expert, -1)
    flat = expert.reshape(-1)
    key = torch.where(flat < 0, E, flat) * T + torch.arange(T, device=l.device).repeat(k)
    order = key.argsort()
    count = torch.bincount(torch.where(flat < 0, E, flat), minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
    offsets[1:] = count.cumsum(0)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(k * T, device=l.device)
    slot = torch.where(has, slot.view(k, T), -1)
    source = torch.where(flat[order] < 0, -1, order)
    out = (expert.to(torch.int32), gate, slot.to(torch.int32), source.to(torch.int32), offsets.to(torch.int32))
    if s["op"] == "route":
        return out
    dot = (gate * s["dgate"]).sum(0)
    at = torch.where(has, expert, 0)
    dl = torch.zeros_like(l).scatter_add_(0, at, gate * (s["dgate"] - dot) if s["renorm"] else gate * s["dgate"])
    if not s["renorm"]:
        dl -= (l - first).exp() / torch.where(total > 0, total, 1.0) * dot
    return out + (dl.to(s["logits"].dtype),)


def _plain(s):
    op = s["op"]
    if op.startswith("route"):
        return _plain_route(s)
    if op == "gather":
        return s["X"][:, s["source"].long() % s["T"]]
    if op == "combine":
        y = torch.zeros((s["K"], s["T"]), dtype=torch.float32, device=s["Y"].device)
        for j in range(s["k"]):
            y += s["gate"][j] * s["Y"][:, s["slot"][j].long()].float()
        return y.to(torch.bfloat16)
    if op == "combine_grad":
        dy = s["X"].float()
        src = s["source"].long()
        dyg = (dy[:, src % s["T"]] * s["gate"].reshape(-1)[src]).to(torch.bfloat16)
        dgate = torch.stack([(dy * s["Y"][:, s["slot"][j].long()].float()).sum(0) for j in range(s["k"])])
        return dyg, dgate
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for t in s["grads"]:
            t = t.double()
            total += (t * t).sum()
        norm = total.sqrt()
        factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
        for t, o in zip(s["grads"], s["out"]):
            o.copy_(t.float() * factor)
        return [norm.float()] + s["out"]
    R, K, at = s["R"], s["K"], s["offsets"].tolist()
    if op == "sddmm":
        dv = torch.zeros(s["values"].shape, dtype=torch.bfloat16, device=s["dY"].device)
        for e in range(s["E"]):
            a, b = at[e], at[e + 1]
            if b > a:
                dv[e] = (s["dY"][:, a:b].float() @ s["X"][:, a:b].float().T).gather(1, _columns(s["meta"][e], R, K))
        return dv
    x = s["X"] if op == "spmm" else s["dY"]
    y = torch.empty((R if op == "spmm" else K, s["S"]), dtype=torch.bfloat16, device=x.device)
    for e in range(s["E"]):
        a, b = at[e], at[e + 1]
        if b > a:
            w = _dense(s["values"][e], s["meta"][e], R, K)
            y[:, a:b] = (w if op == "spmm" else w.T) @ x[:, a:b].float()
    return y


# ------------------------------------------------------------- the library
def _library(s):
    import sparse_gemm_nm_b200 as nm
    op = s["op"]
    if op.startswith("route"):
        out = nm.experts_route(s["logits"], s["k"], renorm=s["renorm"])
        if op == "route":
            return out
        return (*out, nm.experts_route_grad(s["logits"], out[0], out[1], s["dgate"], renorm=s["renorm"]))
    if op == "gather":
        return nm.experts_gather(s["X"], s["source"])
    if op == "combine":
        return nm.experts_combine(s["Y"], s["slot"], s["gate"])
    if op == "combine_grad":
        return nm.experts_combine_grad(s["X"], s["Y"], s["slot"], s["source"], s["gate"])
    if op == "clip":
        return [nm.clip_grads(s["grads"], s["max_norm"], out=s["out"])] + s["out"]
    if op == "spmm":
        return nm.experts_spmm(s["values"], s["meta"], 2, 4, s["K"], s["X"], s["offsets"])
    if op == "spmm_t":
        return nm.experts_spmm_t(s["values"], s["meta"], 2, 4, s["K"], s["dY"], s["offsets"])
    return nm.experts_sddmm(s["meta"], 2, 4, s["R"], s["K"], s["dY"], s["X"], s["offsets"])


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    """Each input read once and each output written once; products at the stored survivors only."""
    op = case["op"]
    if op.startswith("route"):
        E, T, k, l = case["E"], case["T"], case["k"], 4 if case["f32"] else 2
        if op == "route":
            return {"bytes": l * E * T + 16 * k * T + 4 * E, "flops": 4 * E * T}
        return {"bytes": 2 * l * E * T + 20 * k * T + 4 * E, "flops": 8 * E * T}
    if op in ("gather", "combine", "combine_grad"):
        K, T, S = case["K"], case["T"], case["k"] * case["T"]
        if op == "gather":
            return {"bytes": 2 * K * (T + S) + 4 * S, "flops": 0}
        if op == "combine":
            return {"bytes": 2 * K * (T + S) + 8 * S, "flops": 2 * K * S}
        return {"bytes": 2 * K * (T + 2 * S) + 16 * S, "flops": 3 * K * S}
    if op == "clip":
        sizes, f32 = _sizes(case)
        return {"bytes": 2 * sum(n * (4 if f else 2) for n, f in zip(sizes, f32)) + 4, "flops": 3 * sum(sizes)}
    E, R, K, S = case["E"], case["R"], case["K"], case["S"]
    flops = 2 * S * R * K // 2
    if op == "sddmm":
        return {"bytes": case["active"] * R * K // 8 + 2 * S * (R + K) + E * R * K + 4 * E, "flops": flops}
    return {"bytes": case["active"] * (R * K + R * K // 8) + 2 * S * (R + K) + 4 * E, "flops": flops}


# ---------------------------------------------------------------- 64 bits
def _dense64(values, meta, R, K):
    """One W' with every group's positions read word by word of the tiled layout: word 4l + q of block (i, j) holds
    rows 16i + l % 8 (low half) and 16i + 8 + l % 8, columns 128j + 32q + 16(l // 8) + 0..15, a nibble a group."""
    r = torch.arange(R, device=DEV)[:, None]
    c = torch.arange(K // 4, device=DEV)[None, :] * 4
    lane = r % 8 + 8 * (c % 32 // 16)
    word = ((r // 16) * -(-K // 128) + c // 128) * 64 + 4 * lane + c % 128 // 32
    nib = meta.long()[word] // (1 << (16 * (r % 16 // 8) + 4 * (c % 16 // 4))) % 16
    w = torch.zeros((R, K // 4, 4), dtype=torch.float64, device=DEV)
    w.scatter_(2, torch.stack([nib % 4, nib // 4], 2), values.double().view(R, K // 4, 2))
    return w.view(R, K)


def _exact_route(s):
    """Chosen one after the other: the first of the largest logits left."""
    E, T, k = s["E"], s["T"], s["k"]
    l = s["logits"].double()
    left, tokens = l.clone(), torch.arange(T, device=DEV)
    experts, chosen = [], []
    for _ in range(k):
        best = left.max(0).values
        e = (left == best).int().argmax(0)
        some = best > -math.inf
        experts.append(torch.where(some, e, -1))
        chosen.append(best)
        left[e, tokens] = -math.inf
    expert, z = torch.stack(experts), torch.stack(chosen)
    base = torch.logsumexp(z if s["renorm"] else l, 0)
    gate = torch.where(expert >= 0, (z - torch.where(base > -math.inf, base, 0.0)).exp(), 0.0)
    slot = torch.full((k, T), -1, dtype=torch.int64, device=DEV)
    source = torch.full((k * T,), -1, dtype=torch.int64, device=DEV)
    offsets, at = [0], 0
    for e in range(E):
        t, j = torch.nonzero((expert == e).T, as_tuple=True)
        n = t.numel()
        slot[j, t] = torch.arange(at, at + n, device=DEV)
        source[at:at + n] = j * T + t
        at += n
        offsets.append(at)
    out = [expert.int(), gate, slot.int(), source.int(), torch.tensor(offsets, dtype=torch.int32, device=DEV)]
    if s["op"] == "route_both":
        p = torch.zeros_like(l)
        if s["renorm"]:
            for j in range(k):
                p[expert[j].clamp(min=0), tokens] += gate[j]
        else:
            p = (l - torch.where(base > -math.inf, base, 0.0)).exp()
        up = torch.zeros_like(l)  # the gradient of each expert's probability
        for j in range(k):
            up[expert[j].clamp(min=0), tokens] += torch.where(expert[j] >= 0, s["dgate"][j].double(), 0.0)
        out.append(p * (up - (p * up).sum(0)))
    return tuple(out)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("route"):
        return _exact_route(s)
    if op in ("gather", "combine", "combine_grad"):
        K, T, k = s["K"], s["T"], s["k"]
        token = s["source"].long() % T
        if op == "gather":
            return s["X"].double().index_select(1, token)
        weight = s["gate"].double().view(-1).index_select(0, s["source"].long())  # of every column
        y = s["Y"].double()
        if op == "combine":
            return torch.zeros((K, T), dtype=torch.float64, device=DEV).index_add_(1, token, y * weight)
        dy = s["X"].double().index_select(1, token)
        dgate = torch.empty(k * T, dtype=torch.float64, device=DEV)
        dgate[s["source"].long()] = torch.einsum("rs,rs->s", dy, y)
        return dy * weight, dgate.view(k, T)
    if op == "clip":
        norm = torch.stack([torch.linalg.vector_norm(t.double()) for t in s["grads"]]).square().sum().sqrt()
        factor = min(1.0, s["max_norm"] / float(norm))
        return [norm] + [t.double() * factor for t in s["grads"]]
    E, R, K = s["E"], s["R"], s["K"]
    at = s["offsets"].tolist()
    if op == "sddmm":
        dv = torch.zeros(s["values"].shape, dtype=torch.float64, device=DEV)
        for e in range(E):
            if at[e + 1] > at[e]:
                full = s["dY"][:, at[e]:at[e + 1]].double() @ s["X"][:, at[e]:at[e + 1]].double().T
                kept = _dense64(torch.ones_like(s["values"][e]), s["meta"][e], R, K) != 0
                dv[e] = full[kept].view(R, K // 2)
        return dv
    x = s["X"] if op == "spmm" else s["dY"]
    out = []
    for e in range(E):
        if at[e + 1] > at[e]:
            w = _dense64(s["values"][e], s["meta"][e], R, K)
            out.append((w if op == "spmm" else w.T) @ x[:, at[e]:at[e + 1]].double())
    return torch.cat(out, 1)
