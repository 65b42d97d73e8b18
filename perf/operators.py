"""The operators around a pruned projection, as cases to be measured: layer norm, low-rank adapters, and the
cross entropy of a pruned output head.

Layout is the library's: activations are features x tokens with the tokens contiguous (rows padded to 16 bytes),
weights are 2:4 compressed (values R x K/2 bf16, positions in the tiled metadata).  ``own`` picks the side: False
computes every operator with elementary torch operations in 32 bits, True calls the library.

  norm         nm.layer_norm        y = (x - mean) * rstd * gamma + beta over the K features of each token
  norm_grad    nm.layer_norm_grad   its input, gamma and beta gradients
  lora         nm.spmm_lora         y_t = (W' Pi) x_t + s_a B_a A_a x_t, a the adapter of token t
  lora_dx      nm.spmm_lora_t       the input gradient of the same
  lora_grad    nm.lora_grad         the gradients of every adapter's A and B
  xent         nm.spmm_xent         loss_t = log sum_v exp(w'_v . x_t) - w'_target . x_t
  xent_grad    nm.spmm_xent_grad    its gradients: dX, and dV at the stored survivors of the head
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # One decoding step of 16 sequences through a norm in front of the 13824 x 5120 projection.
        {"name": "norm_decode", "op": "norm", "K": 5120, "T": 16, "x32": False, "affine": True},
        # The norm in front of a ViT-B layer on 256 images of 197 tokens.
        {"name": "norm_vit", "op": "norm", "K": 768, "T": 50432, "x32": False, "affine": True},
        # Training on 2048 tokens of width 4096, the residual stream kept in 32 bits.
        {"name": "norm_grad_2k", "op": "norm_grad", "K": 4096, "T": 2048, "x32": True, "affine": True},
        # The same backward pass for the ViT-B layer.
        {"name": "norm_grad_vit", "op": "norm_grad", "K": 768, "T": 50432, "x32": False, "affine": True},
        # One decoding step of 16 requests, each with its own fine-tuned adapter.
        {"name": "lora_decode", "op": "lora", "R": 13824, "K": 5120, "T": 16, "adapters": 16, "rank": 16,
         "permuted": False, "mixed": True},
        # Prompts of several requests side by side through a permuted 4096 x 4096 projection.
        {"name": "lora_prompts", "op": "lora", "R": 4096, "K": 4096, "T": 2048, "adapters": 8, "rank": 16,
         "permuted": True, "mixed": False},
        # Fine-tuning two adapters: the input gradient of the 4096 x 11008 projection.
        {"name": "lora_dx_4096x11008", "op": "lora_dx", "R": 4096, "K": 11008, "T": 2048, "adapters": 2, "rank": 32,
         "permuted": True, "mixed": False},
        # The adapters' own gradients beside the 11008 x 4096 projection.
        {"name": "lora_grad_11008x4096", "op": "lora_grad", "R": 11008, "K": 4096, "T": 2048, "adapters": 4,
         "rank": 64, "mixed": False},
        # Scoring a short answer of 37 tokens over a vocabulary of 32000.
        {"name": "xent_answer", "op": "xent", "R": 32000, "K": 4096, "T": 37, "permuted": False},
        # The loss of 2048 tokens.
        {"name": "xent_2k", "op": "xent", "R": 32000, "K": 4096, "T": 2048, "permuted": False},
        # A classifier of 1000 classes on 256 images of ViT-B features, gradients.
        {"name": "xent_grad_classes", "op": "xent_grad", "R": 1000, "K": 768, "T": 256, "permuted": False},
        # The gradients of the language model's loss on 2048 tokens.
        {"name": "xent_grad_2k", "op": "xent_grad", "R": 32000, "K": 4096, "T": 2048, "permuted": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "lora", "lora_dx", "lora_grad", "xent", "xent_grad"])
    T = _log(rng, 1, 50432)
    if op in ("norm", "norm_grad"):
        K = min(_log(rng, 8, 16384), max(8, 768 * 50432 // T))
        return {"op": op, "K": K, "T": T, "x32": rng.random() < 0.5, "affine": rng.random() < 0.8}
    T = min(T, 8192)
    if op.startswith("lora"):
        K = 8 * _log(rng, 2, 1376) if rng.random() < 0.7 else 128 * _log(rng, 1, 86)
        R = _log(rng, 6, 13824)
        T = max(1, min(T, 4096 * 11008 * 2048 // (R * K)))
        case = {"op": op, "R": R, "K": K, "T": T, "adapters": _log(rng, 1, 16), "rank": _log(rng, 1, 64),
                "mixed": rng.random() < 0.4}
        if op != "lora_grad":
            case["permuted"] = rng.random() < 0.5
        return case
    K = 8 * _log(rng, 8, 512) if rng.random() < 0.5 else 128 * _log(rng, 1, 32)
    R = _log(rng, 2, 50257)
    T = max(1, min(T, 32000 * 4096 * 2048 // (R * K)))
    return {"op": op, "R": R, "K": K, "T": T, "permuted": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs
def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _rows(g, rows, cols, std, dtype):
    """rows x cols with the rows padded to 16 bytes, as the library takes them."""
    per = 4 if dtype == torch.float32 else 8
    return _normal(g, (rows, (cols + per - 1) // per * per), std, dtype)[:, :cols]


def _pack_2of4(pairs, R, K):
    """Tiled metadata of R x K/4 nibbles p0 | p1 << 2 (int64), padding groups 0x4."""
    rb, cb = (R + 15) // 16, (K + 127) // 128
    nib = torch.full((rb * 16, cb * 32), 4, dtype=torch.int64, device=pairs.device)
    nib[:R, :K // 4] = pairs
    nib = nib.view(rb, 2, 8, cb, 4, 2, 4)  # row block, row half, row, column block, quarter, column half, group
    shift = 16 * torch.arange(2, device=nib.device).view(1, 2, 1, 1, 1, 1, 1) + 4 * torch.arange(4, device=nib.device)
    words = (nib << shift).sum(dim=(1, 6))  # row block, row, column block, quarter, column half
    words = words.permute(0, 2, 4, 1, 3).reshape(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _weights(g, R, K):
    """A 2:4 weight: values ~ N(0, 0.02), the two positions of every group uniform."""
    values = _normal(g, (R, K // 2), 0.02, torch.bfloat16)
    table = torch.tensor([4, 8, 12, 9, 13, 14], device=DEV)  # p0 | p1 << 2 for p0 < p1
    pairs = table[torch.randint(0, 6, (R, K // 4), generator=g, device=DEV)]
    return values, _pack_2of4(pairs, R, K)


def _adapter_map(g, T, adapters, mixed):
    """The adapter of each token (-1: none): runs of ragged length, or any order."""
    if mixed:
        a = torch.randint(0, adapters, (T,), generator=g, device=DEV)
        a = torch.where(torch.rand(T, generator=g, device=DEV) < 0.05, -1, a)
    else:
        cuts = torch.rand(adapters, generator=g, device=DEV).sort().values * T
        a = (torch.arange(T, device=DEV)[:, None] >= cuts[None, :]).sum(1) - 1
    return a.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    op, K, T = case["op"], case["K"], case["T"]
    if op in ("norm", "norm_grad"):
        x = torch.float32 if case["x32"] else torch.bfloat16
        s["X"] = _rows(g, K, T, 1.5, x)
        s["X"].add_(_normal(g, (K, 1), 0.5, torch.float32).to(x))  # features differ in their means
        s["gamma"] = 1 + _normal(g, (K,), 0.1, torch.float32) if case["affine"] else None
        s["beta"] = _normal(g, (K,), 0.1, torch.float32) if case["affine"] else None
        if op == "norm_grad":
            s["dY"] = _rows(g, K, T, 1.0, torch.bfloat16)
            x64 = s["X"].double()
            s["mean"] = x64.mean(0).float()
            s["rstd"] = (1 / (x64.var(0, unbiased=False) + 1e-5).sqrt()).float()
        return s
    R = case["R"]
    if op != "lora_grad":
        s["values"], s["meta"] = _weights(g, R, K)
        s["idx"] = torch.randperm(K, generator=g, device=DEV).to(torch.int32) if case["permuted"] else None
    if op.startswith("lora"):
        n, r = case["adapters"], case["rank"]
        s["A"] = _normal(g, (n, r, K), 1 / math.sqrt(K), torch.bfloat16)
        s["B"] = _normal(g, (n, R, r), 0.5 / math.sqrt(r), torch.bfloat16)
        s["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        s["adapter"] = _adapter_map(g, T, n, case["mixed"])
        if op != "lora_dx":
            s["X"] = _rows(g, K, T, 1.0, torch.bfloat16)
        if op != "lora":
            s["dY"] = _rows(g, R, T, 1.0, torch.bfloat16)
        return s
    s["X"] = _rows(g, K, T, 1.0, torch.bfloat16)
    s["target"] = torch.randint(0, R, (T,), generator=g, device=DEV).to(torch.int32)
    s["target"][torch.rand(T, generator=g, device=DEV) < 0.03] = -100  # tokens without a loss
    if op == "xent_grad":
        s["lse"] = torch.logsumexp(_dense(s["values"], s["meta"], R, K) @ _permuted(s["X"], s["idx"]), dim=0)
        s["dloss"] = torch.rand(T, generator=g, device=DEV) / T
    return s


# -------------------------------------------------------------- plain form
def _columns(meta, R, K):
    """R x K/2 column of every stored survivor."""
    rb, cb = (R + 15) // 16, (K + 127) // 128
    words = meta.to(torch.int64).view(rb, cb, 2, 8, 4, 1, 1)
    shift = 16 * torch.arange(2, device=meta.device).view(2, 1) + 4 * torch.arange(4, device=meta.device)
    nib = (words >> shift) & 15  # row block, column block, column half, row, quarter, row half, group
    nib = nib.permute(0, 5, 3, 1, 4, 2, 6).reshape(rb * 16, cb * 32)[:R, :K // 4]
    first = 4 * torch.arange(K // 4, device=meta.device)
    return torch.stack([first + (nib & 3), first + (nib >> 2)], dim=2).reshape(R, K // 2)


def _dense(values, meta, R, K):
    w = torch.zeros((R, K), dtype=torch.float32, device=values.device)
    return w.scatter_(1, _columns(meta, R, K), values.float())


def _permuted(X, idx):
    return X.float() if idx is None else X.float()[idx.long()]


def _low_rank(M, Z, s):
    """Per adapter M_a Z, only at the tokens that the adapter serves: adapters x rank x T."""
    n, r = s["adapters"], s["rank"]
    serves = s["adapter"][None, :] == torch.arange(n, device=Z.device)[:, None]
    return (M.reshape(n * r, -1) @ Z).view(n, r, -1) * serves[:, None, :]


def _plain(s):
    op, K = s["op"], s["K"]
    if op == "norm":
        x = s["X"].float()
        c = x - x.mean(0)
        var = (c * c).mean(0)
        rstd = 1 / (var + 1e-5).sqrt()
        y = c * rstd
        if s["gamma"] is not None:
            y = y * s["gamma"][:, None] + s["beta"][:, None]
        return y.to(torch.bfloat16), x.mean(0), rstd
    if op == "norm_grad":
        dy = s["dY"].float()
        h = (s["X"].float() - s["mean"]) * s["rstd"]
        gy = dy if s["gamma"] is None else dy * s["gamma"][:, None]
        dx = s["rstd"] * (gy - gy.mean(0) - h * (gy * h).mean(0))
        return dx.to(s["X"].dtype), (dy * h).sum(1), dy.sum(1)
    if op.startswith("lora"):
        n, r = s["adapters"], s["rank"]
        A, B, scale = s["A"].float(), s["B"].float(), s["scale"][:, None, None]
        if op == "lora":
            low = _low_rank(A, s["X"].float(), s) * scale
            y = _dense(s["values"], s["meta"], s["R"], K) @ _permuted(s["X"], s["idx"])
            return (y + B.permute(1, 0, 2).reshape(s["R"], n * r) @ low.view(n * r, -1)).to(torch.bfloat16)
        up = _low_rank(B.transpose(1, 2), s["dY"].float(), s) * scale
        if op == "lora_dx":
            dx = _dense(s["values"], s["meta"], s["R"], K).T @ s["dY"].float()
            if s["idx"] is not None:
                dx = torch.empty_like(dx).index_copy_(0, s["idx"].long(), dx)
            return (dx + A.reshape(n * r, K).T @ up.view(n * r, -1)).to(torch.bfloat16)
        x, dy = s["X"].float(), s["dY"].float()
        low = _low_rank(A, x, s) * scale
        return (up.view(n * r, -1) @ x.T).view(n, r, K), (low.view(n * r, -1) @ dy.T).view(n, r, -1).transpose(1, 2)
    w, x = _dense(s["values"], s["meta"], s["R"], K), _permuted(s["X"], s["idx"])
    logits = w @ x
    has = (s["target"] >= 0) & (s["target"] < s["R"])
    at = torch.where(has, s["target"], 0).long()
    if op == "xent":
        top = logits.max(0).values
        lse = top + (logits - top).exp().sum(0).log()
        return torch.where(has, lse - logits.gather(0, at[None, :])[0], 0.0), lse
    p = (logits - s["lse"]).exp()
    p.scatter_add_(0, at[None, :], torch.full_like(p[:1], -1.0))
    grad = p * torch.where(has, s["dloss"], 0.0)
    dx = w.T @ grad
    if s["idx"] is not None:
        dx = torch.empty_like(dx).index_copy_(0, s["idx"].long(), dx)
    dv = (grad @ x.T).gather(1, _columns(s["meta"], s["R"], K))
    return dx.to(torch.bfloat16), dv.to(torch.bfloat16)


# ------------------------------------------------------------- the library
def _library(s):
    import sparse_gemm_nm_b200 as nm
    op = s["op"]
    if op == "norm":
        return nm.layer_norm(s["X"], s["gamma"], s["beta"], eps=1e-5, out_dtype=torch.bfloat16)
    if op == "norm_grad":
        return nm.layer_norm_grad(s["dY"], s["X"], s["mean"], s["rstd"], s["gamma"])
    if op == "lora":
        return nm.spmm_lora(s["values"], s["meta"], 2, 4, s["K"], s["X"], s["A"], s["B"], s["adapter"], s["scale"],
                            idx=s["idx"])
    if op == "lora_dx":
        return nm.spmm_lora_t(s["values"], s["meta"], 2, 4, s["K"], s["dY"], s["A"], s["B"], s["adapter"],
                              s["scale"], idx=s["idx"])
    if op == "lora_grad":
        return nm.lora_grad(s["dY"], s["X"], s["A"], s["B"], s["adapter"], s["scale"], out_dtype=torch.float32)
    if op == "xent":
        return nm.spmm_xent(s["values"], s["meta"], 2, 4, s["K"], s["X"], s["target"], idx=s["idx"])
    return nm.spmm_xent_grad(s["values"], s["meta"], 2, 4, s["K"], s["X"], s["target"], s["lse"], s["dloss"],
                             idx=s["idx"])


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    """Each input read once and each output written once; products at the stored survivors only."""
    op, K, T = case["op"], case["K"], case["T"]
    if op == "norm":
        x = 4 if case["x32"] else 2
        return {"bytes": K * T * (x + 2) + 8 * K + 8 * T, "flops": 8 * K * T}
    if op == "norm_grad":
        x = 4 if case["x32"] else 2
        return {"bytes": K * T * (2 * x + 2) + 12 * K + 8 * T, "flops": 14 * K * T}
    R = case["R"]
    weights = R * K + R * K // 8  # values, and two bits for each
    if op.startswith("lora"):
        n, r = min(case["adapters"], T), case["rank"]
        low = 2 * n * r * (R + K)
        if op == "lora_grad":
            return {"bytes": 2 * T * (R + K) + 3 * low, "flops": 8 * T * r * (R + K)}
        return {"bytes": weights + 2 * T * (R + K) + low, "flops": 2 * T * (R * K // 2 + r * (R + K))}
    if op == "xent":
        return {"bytes": weights + 2 * K * T + 12 * T, "flops": 2 * T * R * K // 2}
    return {"bytes": weights + R * K + 4 * K * T + 12 * T, "flops": 3 * 2 * T * R * K // 2}


# ---------------------------------------------------------------- 64 bits
def _dense64(s):
    """W' with every group's positions read word by word of the tiled layout: word 4l + q of block (i, j) holds
    rows 16i + l % 8 (low half) and 16i + 8 + l % 8, columns 128j + 32q + 16(l // 8) + 0..15, a nibble a group."""
    R, K = s["R"], s["K"]
    r = torch.arange(R, device=DEV)[:, None]
    c = torch.arange(K // 4, device=DEV)[None, :] * 4
    lane = r % 8 + 8 * (c % 32 // 16)
    word = ((r // 16) * -(-K // 128) + c // 128) * 64 + 4 * lane + c % 128 // 32
    nib = s["meta"].long()[word] // (1 << (16 * (r % 16 // 8) + 4 * (c % 16 // 4))) % 16
    w = torch.zeros((R, K // 4, 4), dtype=torch.float64, device=DEV)
    v = s["values"].double().view(R, K // 4, 2)
    w.scatter_(2, torch.stack([nib % 4, nib // 4], 2), v)
    return w.view(R, K)


def exact(case, seed):
    s = prepare(case, seed)
    op, K, T = s["op"], s["K"], s["T"]
    if op == "norm":
        x = s["X"].double()
        mean = x.sum(0) / K
        rstd = ((x - mean).square().sum(0) / K + 1e-5).rsqrt()
        y = (x - mean) * rstd
        if s["gamma"] is not None:
            y = torch.addcmul(s["beta"].double()[:, None], y, s["gamma"].double()[:, None])
        return y, mean, rstd
    if op == "norm_grad":
        dy, x = s["dY"].double(), s["X"].double()
        rstd = s["rstd"].double()
        hat = (x - s["mean"].double()) * rstd
        up = dy if s["gamma"] is None else s["gamma"].double()[:, None] * dy
        dot = torch.einsum("kt,kt->t", up, hat)
        return rstd * (up - (up.sum(0) + hat * dot) / K), torch.einsum("kt,kt->k", dy, hat), dy.sum(1)
    if op.startswith("lora"):
        R, n, r = s["R"], s["adapters"], s["rank"]
        A, B, scale = s["A"].double(), s["B"].double(), s["scale"].double()
        which = [torch.nonzero(s["adapter"] == a)[:, 0] for a in range(n)]
        if op == "lora_grad":
            x, dy = s["X"].double(), s["dY"].double()
            dA, dB = torch.zeros_like(A), torch.zeros_like(B)
            for a, t in enumerate(which):
                dA[a] = scale[a] * (B[a].T @ dy[:, t]) @ x[:, t].T
                dB[a] = scale[a] * dy[:, t] @ (A[a] @ x[:, t]).T
            return dA, dB
        w = _dense64(s)
        if op == "lora":
            x = s["X"].double()
            y = w @ (x if s["idx"] is None else x[s["idx"].long()])
            for a, t in enumerate(which):
                y[:, t] += scale[a] * (B[a] @ (A[a] @ x[:, t]))
            return y
        dy = s["dY"].double()
        dx = w.T @ dy
        if s["idx"] is not None:
            dx = dx[torch.argsort(s["idx"].long())]
        for a, t in enumerate(which):
            dx[:, t] += scale[a] * (A[a].T @ (B[a].T @ dy[:, t]))
        return dx
    w, x = _dense64(s), s["X"].double()
    x = x if s["idx"] is None else x[s["idx"].long()]
    z = w @ x
    t = s["target"].long()
    at = torch.nonzero((t >= 0) & (t < s["R"]))[:, 0]
    if op == "xent":
        lse = torch.logsumexp(z, 0)
        loss = torch.zeros(T, dtype=torch.float64, device=DEV)
        loss[at] = lse[at] - z[t[at], at]
        return loss, lse
    grad = torch.zeros_like(z)
    grad[:, at] = torch.exp(z[:, at] - s["lse"].double()[at])
    grad[t[at], at] -= 1
    grad *= s["dloss"].double()
    dx = w.T @ grad
    if s["idx"] is not None:
        dx = dx[torch.argsort(s["idx"].long())]
    full = (grad @ x.T).view(s["R"], K // 4, 4)
    kept = torch.where(_kept64(s), full, torch.nan).view(-1)
    return dx, kept[~kept.isnan()].view(s["R"], K // 2)


def _kept64(s):
    """R x K/4 x 4 truth values: the positions that the metadata keeps."""
    ones = dict(s, values=torch.ones_like(s["values"]))
    return _dense64(ones).view(s["R"], s["K"] // 4, 4) != 0
