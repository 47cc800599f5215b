"""The measured operators of the MoE library: the router's balance loss with the gradient of its
logits, 8-bit rows with a scale for each token, the experts' product in 8-bit integers, and a whole
expert layer made of them.

Formulas (T tokens, E experts, k kept experts a token, S sequences of L = T / S tokens):

balance   p = softmax(logits); for sequence s: n_s unmasked tokens, c_se kept (token, slot) pairs of
          expert e, P_se the sum of p_te; loss = alpha / S * sum_s E / (k n_s^2) * sum_e c_se P_se.
gradient  dlogits_te = dloss * alpha / S * E / (k n_s^2) * p_te * (c_se - sum_i c_si p_ti) for an
          unmasked token t of sequence s, plus w_j (dw_j - sum_i w_i dw_i) at the expert of slot j.
quant     a = max |x| of the row, q = rint(127 x / a), scale = a / 127 (a = 0: q = 0, scale = 1).
product   y_rn = a_scale * w_scale_en * sum_i a_ri w_eni for the rows r of expert e; with "swiglu"
          the weights hold gate and up channels and out = gate / (1 + exp(-gate)) * up.
layer     quant, product with swiglu, quant, product, and the weighted sum of each token's rows.
"""
import math

import torch

own = False

ALPHA = 0.01
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _balance(name, T, S, E, k, masked, way, weights):
    return {"name": name, "kind": "balance", "T": T, "S": S, "E": E, "k": k, "masked": masked,
            "way": way, "weights": weights}


def _quant(name, T, H, dtype):
    return {"name": name, "kind": "quant", "T": T, "H": H, "dtype": dtype}


def _product(name, T, k, E, N, K, act, gather, dtype, skew):
    return {"name": name, "kind": "product", "T": T, "k": k, "E": E, "N": N, "K": K, "act": act,
            "gather": gather, "dtype": dtype, "skew": skew}


def _layer(name, T, k, E, H, inner, skew):
    return {"name": name, "kind": "layer", "T": T, "k": k, "E": E, "H": H, "I": inner, "skew": skew}


def listed():
    return [
        # a small micro-batch of the decode configuration: launches and latency
        _balance("balance 128 tokens", 128, 1, 256, 8, False, "both", False),
        # the forward pass of a prefill-sized training batch, the loss over the batch
        _balance("balance loss 4096", 4096, 1, 384, 8, False, "loss", False),
        # backward of a padded batch of odd length, the loss per sequence, one sequence empty
        _balance("balance grad padded", 8 * 1021, 8, 128, 4, True, "grad", True),
        # a long training batch, both passes, with the gradient of the routing weights
        _balance("balance 65536 tokens", 65536, 16, 256, 8, False, "both", True),
        # a decode batch's activations
        _quant("quant decode", 128, 7168, "bf16"),
        # fp32 activations of an odd batch and a hidden size that is no power of two
        _quant("quant f32 odd", 4099, 2064, "f32"),
        # one token through one matrix (a shared expert in decode): latency and bandwidth
        _product("product one token", 1, 1, 1, 4096, 7168, "none", False, "f32", 0.0),
        # gate and up of a decode batch: nearly all experts' weights for few rows each
        _product("product decode", 128, 8, 256, 2048, 7168, "swiglu", True, "bf16", 0.0),
        # down projection of the prefill batch: about 85 rows an expert
        _product("product prefill down", 4096, 8, 384, 7168, 2048, "none", False, "bf16", 0.0),
        # few experts with many rows each, uneven: bound by the matrix cores
        _product("product many rows", 8192, 4, 32, 2048, 4096, "swiglu", True, "bf16", 0.3),
        # sizes that fill no tile, uneven experts, fp32 results
        _product("product odd", 777, 3, 20, 1000, 2064, "none", True, "f32", 0.6),
        # a whole expert layer of a mid-sized batch
        _layer("expert layer 512", 512, 8, 64, 4096, 1408, 0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "quant", "product", "product", "layer"])
    if kind == "balance":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        k = rng.choice([1, 2, 4, 6, 8])
        S = rng.choice([1, 1, 2, 4, 8, 16])
        L = max(1, _log(rng, 1, 65536) // S)
        c = _balance("", S * L, S, E, k, rng.random() < 0.5, rng.choice(["loss", "grad", "both"]),
                     rng.random() < 0.5)
    elif kind == "quant":
        H = 16 * _log(rng, 4, 512)
        c = _quant("", min(_log(rng, 1, 32768), (1 << 27) // H), H, rng.choice(["bf16", "f32"]))
    elif kind == "product":
        E = rng.choice([1, 1, 4, 8, 16, 32, 60, 64, 128])
        k = min(rng.choice([1, 2, 4, 6, 8]), E)
        K = 16 * _log(rng, 4, 512)
        act = rng.choice(["none", "swiglu"])
        N = _log(rng, 32, max(33, min(8192, (1 << 30) // (E * K))))
        most = int(4e11 / (2.0 * N * K * k * (2 if act == "swiglu" else 1)))
        T = _log(rng, 1, max(2, min(16384 // k, most)))
        c = _product("", T, k, E, N, K, act, rng.random() < 0.7, rng.choice(["bf16", "f32"]),
                     rng.choice([0.0, 0.3, 0.6]))
    else:
        E = rng.choice([8, 16, 60, 64, 128])
        k = rng.choice([1, 2, 4, 6, 8])
        H = 16 * _log(rng, 8, 320)
        inner = 16 * _log(rng, 4, max(5, min(160, (1 << 29) // (16 * E * H))))
        c = _layer("", _log(rng, 1, 2048), k, E, H, inner, rng.choice([0.0, 0.3, 0.6]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------- inputs --
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _weights(g, E, N, K):
    """int8 weights [E, N, K] as rounding normal weights to 127 steps of their maximum gives them
    (about 3.7 standard deviations), and a scale for each channel."""
    w = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    flat = w.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, generator=g, device="cuda") * 34.0).round_().clamp_(-127, 127)
    scale = (0.5 + torch.rand((E, N), generator=g, device="cuda")) * (1.0 / (34.0 * math.sqrt(K)))
    return w, scale


def _route(g, T, k, E, skew):
    """Logits with expert popularity falling as (e + 1)^-skew, the kept ids and their weights."""
    logits = _normal(g, T, E)
    logits -= skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    top, idx = torch.topk(logits, k, dim=1)
    return logits, idx.to(torch.int32), torch.softmax(top, 1).contiguous()


def _layout(idx, E):
    """Rows in (expert, token, slot) order: offsets, the token of each row, the row of each slot."""
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device="cuda")
    return offsets, (order // k).to(torch.int32), row.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["kind"] == "balance":
        T, S, E, k = case["T"], case["S"], case["E"], case["k"]
        s["logits"], s["topk_idx"], s["topk_w"] = _route(g, T, k, E, 0.3)
        s["mask"] = None
        if case["masked"]:      # padding behind each sequence; the last of several is all padding
            lengths = torch.randint(1, T // S + 1, (S,), generator=g, device="cuda")
            if S > 1:
                lengths[S - 1] = 0
            s["mask"] = (torch.arange(T // S, device="cuda")[None, :] < lengths[:, None]).reshape(-1)
        s["dtopk_w"] = _normal(g, T, k) * (0.02 / T) if case["weights"] else None
        s["dloss"] = 0.5 + torch.rand(1, generator=g, device="cuda")
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        hit = s["topk_idx"].long() + (torch.arange(T, device="cuda") // (T // S) * E)[:, None]
        s["counts"] = torch.bincount(hit[keep].reshape(-1), minlength=S * E).to(torch.int32).view(S, E)
        s["seq_tokens"] = keep.view(S, -1).sum(1).to(torch.int32)
        s["out"] = {"loss": torch.empty(1, device="cuda"),
                    "expert_counts": torch.empty((S, E), dtype=torch.int32, device="cuda"),
                    "prob_sums": torch.empty((S, E), device="cuda"),
                    "seq_tokens": torch.empty(S, dtype=torch.int32, device="cuda"),
                    "dlogits": torch.empty((T, E), device="cuda")}
    elif case["kind"] == "quant":
        # activations with a few channels much larger than the rest
        T, H = case["T"], case["H"]
        channel = torch.exp(0.7 * _normal(g, H))
        s["x"] = (_normal(g, T, H) * channel).to(DTYPES[case["dtype"]])
        s["q"] = torch.empty((T, H), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(T, device="cuda")
    elif case["kind"] == "product":
        T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
        R = T * k
        _, idx, _ = _route(g, T, k, E, case["skew"])
        s["offsets"], row_token, _ = _layout(idx, E)
        s["row_token"] = row_token if case["gather"] else None
        rows = T if case["gather"] else R
        s["a"] = (_normal(g, rows, K) * 34.0).round_().clamp_(-127, 127).to(torch.int8)
        s["a_scale"] = (0.5 + torch.rand(rows, generator=g, device="cuda")) / 34.0
        s["w"], s["w_scale"] = _weights(g, E, 2 * N if case["act"] == "swiglu" else N, K)
        s["out"] = torch.empty((R, N), dtype=DTYPES[case["dtype"]], device="cuda")
    else:
        T, k, E, H, inner = case["T"], case["k"], case["E"], case["H"], case["I"]
        R = T * k
        _, idx, s["topk_w"] = _route(g, T, k, E, case["skew"])
        s["offsets"], s["row_token"], s["token_row"] = _layout(idx, E)
        s["x"] = _normal(g, T, H).to(torch.bfloat16)
        s["w1"], s["w1_scale"] = _weights(g, E, 2 * inner, H)
        s["w2"], s["w2_scale"] = _weights(g, E, H, inner)
        i8 = dict(dtype=torch.int8, device="cuda")
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        s["xq"], s["x_scale"] = torch.empty((T, H), **i8), torch.empty(T, device="cuda")
        s["h"] = torch.empty((R, inner), **bf16)
        s["hq"], s["h_scale"] = torch.empty((R, inner), **i8), torch.empty(R, device="cuda")
        s["y"], s["res"] = torch.empty((R, H), **bf16), torch.empty((T, H), **bf16)
    return s


# --------------------------------------------------------------------------------- plain form --
def _plain_probs(logits):
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_loss(s, p):
    T, S, E, k = s["T"], s["S"], s["E"], s["k"]
    hit = s["topk_idx"].long() + (torch.arange(T, device="cuda") // (T // S) * E)[:, None]
    one = torch.ones_like(s["topk_idx"])
    if s["mask"] is None:
        n = torch.full((S,), T // S, dtype=torch.int32, device="cuda")
    else:
        one = one * s["mask"][:, None]
        n = s["mask"].view(S, -1).sum(1, dtype=torch.int32)
        p = p * s["mask"][:, None]
    counts = torch.zeros(S * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, hit.reshape(-1), one.reshape(-1))
    counts = counts.view(S, E)
    sums = p.view(S, -1, E).sum(1, dtype=torch.float64)
    n64 = n.double().clamp(min=1)
    loss = ((counts * sums).sum(1) / (n64 * n64)).sum() * (ALPHA / S * E / k)
    return loss.float().view(1), counts, sums.float(), n


def _plain_grad(s, p, counts, n):
    T, S, E, k = s["T"], s["S"], s["E"], s["k"]
    # the probabilities add up to one, so any constant may be taken from the counts
    c = (counts - torch.round(n.float()[:, None] * (k / E))).repeat_interleave(T // S, 0)
    n32 = n.float().clamp(min=1)
    f = (s["dloss"] * (ALPHA / S * E / k) / (n32 * n32)).repeat_interleave(T // S)
    if s["mask"] is not None:
        f = f * s["mask"]
    d = f[:, None] * p * (c - (c * p).sum(1, keepdim=True))
    if s["dtopk_w"] is not None:
        w, dw = s["topk_w"], s["dtopk_w"]
        d.scatter_add_(1, s["topk_idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return d


def _plain_quant(x):
    x = x.double()                                  # quotients next to a rounding border
    a = x.abs().amax(1, keepdim=True)
    some = a > 0
    q = torch.where(some, torch.round(127 * x / torch.where(some, a, 1.0)), 0.0)
    scale = torch.where(some, a / torch.full_like(a, 127.0), 1.0)
    return q.to(torch.int8), scale.float().view(-1)


def _plain_product(a, a_scale, w, w_scale, offsets, row_token, act, dtype):
    E = w.shape[0]
    count = (offsets[1:] - offsets[:-1]).long()
    R = a.shape[0] if row_token is None else row_token.numel()
    r = torch.arange(R, device="cuda")
    src = r if row_token is None else row_token.long()
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), count)
    at = r - offsets.long()[e]
    rows = torch.zeros((E, int(count.max()), a.shape[1]), device="cuda")
    rows[e, at] = a[src].float()
    y = torch.bmm(rows, w.float().transpose(1, 2))[e, at]
    y = y * a_scale[src][:, None] * w_scale[e]
    if act == "swiglu":
        gate, up = y.chunk(2, 1)
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(dtype)


def _plain(s):
    if s["kind"] == "balance":
        p = _plain_probs(s["logits"])
        got, counts, n = {}, s["counts"], s["seq_tokens"]
        if s["way"] != "grad":
            got["loss"], counts, got["prob_sums"], n = _plain_loss(s, p)
            got["expert_counts"], got["seq_tokens"] = counts, n
        if s["way"] != "loss":
            got["dlogits"] = _plain_grad(s, p, counts, n)
        return got
    if s["kind"] == "quant":
        q, scale = _plain_quant(s["x"])
        return {"q": q, "scale": scale}
    if s["kind"] == "product":
        return _plain_product(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"],
                              s["row_token"], s["act"], DTYPES[s["dtype"]])
    q, scale = _plain_quant(s["x"])
    h = _plain_product(q, scale, s["w1"], s["w1_scale"], s["offsets"], s["row_token"], "swiglu",
                       torch.bfloat16)
    q, scale = _plain_quant(h)
    y = _plain_product(q, scale, s["w2"], s["w2_scale"], s["offsets"], None, "none", torch.bfloat16)
    rows = y[s["token_row"].long()].float().view(s["T"], s["k"], -1)
    return (rows * s["topk_w"][:, :, None]).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------------------------ kernels --
def _kernels(s):
    import combine_moe_route_03_amd as moe
    if s["kind"] == "balance":
        o, got, counts, n = s["out"], {}, s["counts"], s["seq_tokens"]
        if s["way"] != "grad":
            moe.moe_balance_loss(s["logits"], s["topk_idx"], ALPHA, n_seqs=s["S"],
                                 token_mask=s["mask"], loss=o["loss"],
                                 expert_counts=o["expert_counts"], prob_sums=o["prob_sums"],
                                 seq_tokens=o["seq_tokens"])
            counts, n = o["expert_counts"], o["seq_tokens"]
            got = {x: o[x] for x in ("loss", "expert_counts", "prob_sums", "seq_tokens")}
        if s["way"] != "loss":
            moe.moe_route_grad(s["logits"], s["topk_idx"], expert_counts=counts, seq_tokens=n,
                               alpha=ALPHA, n_seqs=s["S"], token_mask=s["mask"], dloss=s["dloss"],
                               topk_w=s["topk_w"] if s["weights"] else None, dtopk_w=s["dtopk_w"],
                               dlogits=o["dlogits"])
            got["dlogits"] = o["dlogits"]
        return got
    if s["kind"] == "quant":
        moe.moe_quant_rows(s["x"], q=s["q"], scale=s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if s["kind"] == "product":
        return moe.moe_expert_matmul_i8(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"],
                                        row_token=s["row_token"], act=s["act"], out=s["out"])
    moe.moe_quant_rows(s["x"], q=s["xq"], scale=s["x_scale"])
    moe.moe_expert_matmul_i8(s["xq"], s["x_scale"], s["w1"], s["w1_scale"], s["offsets"],
                             row_token=s["row_token"], act="swiglu", out=s["h"])
    moe.moe_quant_rows(s["h"], q=s["hq"], scale=s["h_scale"])
    moe.moe_expert_matmul_i8(s["hq"], s["h_scale"], s["w2"], s["w2_scale"], s["offsets"],
                             out=s["y"])
    return moe.moe_combine(s["y"], s["token_row"], s["topk_w"], s["res"])


def run(state):
    return _kernels(state) if own else _plain(state)


# --------------------------------------------------------------------------------------- work --
def _touched(T, k, E):
    """Experts that get a row, as many as even routing gives on average."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    if case["kind"] == "balance":
        T, S, E, k = case["T"], case["S"], case["E"], case["k"]
        loss, grad = case["way"] != "grad", case["way"] != "loss"
        b, f = 4.0 * T * E + (T if case["masked"] else 0), 5.0 * T * E
        if loss or case["weights"]:
            b += 4.0 * T * k
        if loss:
            b, f = b + 8.0 * S * E + 4 * S + 4, f + 1.0 * T * E
        if grad:
            b, f = b + 4.0 * T * E + (0 if loss else 4.0 * S * E), f + 4.0 * T * E
            if case["weights"]:
                b, f = b + 8.0 * T * k, f + 5.0 * T * k
        return {"bytes": b, "flops": f}
    if case["kind"] == "quant":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * ((2 if case["dtype"] == "bf16" else 4) + 1.0) + 4.0 * T, "flops": 4.0 * T * H}
    T, k, E = case["T"], case["k"], case["E"]
    R, used = T * k, _touched(T, k, E)
    if case["kind"] == "product":
        N, K = case["N"], case["K"]
        n = 2 * N if case["act"] == "swiglu" else N
        rows = T if case["gather"] else R
        return {"bytes": used * n * (K + 4.0) + rows * (K + 4.0) + (4.0 * R if case["gather"] else 0.0)
                + R * N * (2.0 if case["dtype"] == "bf16" else 4.0), "flops": 2.0 * R * n * K}
    H, inner = case["H"], case["I"]
    return {"bytes": used * (3.0 * H * inner + 8.0 * inner + 4.0 * H) + 4.0 * T * H + 12.0 * R,
            "flops": 6.0 * R * H * inner + 2.0 * R * H}


# -------------------------------------------------------------------------------------- exact --
def _exact_quant(x):
    x = x.double()
    top = x.abs().max(dim=1, keepdim=True).values
    q = torch.round((x * 127.0).div(torch.where(top == 0, torch.ones_like(top), top)))
    scale = torch.where(top == 0, torch.ones_like(top), top.div(torch.full_like(top, 127.0)))
    return q, scale


def _exact_product(a, a_scale, w, w_scale, offsets, row_token, act):
    bounds = offsets.tolist()
    parts = []
    for e in range(w.shape[0]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        src = torch.arange(lo, hi, device="cuda") if row_token is None else row_token[lo:hi].long()
        y = a[src].double() @ w[e].double().t()
        y = y * a_scale.double().view(-1)[src][:, None] * w_scale[e].double()
        if act == "swiglu":
            half = y.shape[1] // 2
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        parts.append(y)
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "balance":
        T, S, E, k = case["T"], case["S"], case["E"], case["k"]
        p = torch.softmax(s["logits"].double(), 1).view(S, T // S, E)
        keep = torch.ones(T, device="cuda") if s["mask"] is None else s["mask"]
        keep = keep.double().view(S, T // S)
        chosen = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        chosen.scatter_(1, s["topk_idx"].long(), 1.0)
        c = (chosen.view(S, T // S, E) * keep[:, :, None]).sum(1)
        n = keep.sum(1)
        sums = (p * keep[:, :, None]).sum(1)
        per = torch.where(n > 0, E / (k * n.clamp(min=1) ** 2), 0.0) * (ALPHA / S)
        got = {}
        if case["way"] != "grad":
            got["loss"] = (per * (c * sums).sum(1)).sum().view(1)
            got["expert_counts"], got["prob_sums"] = c.to(torch.int32), sums
            got["seq_tokens"] = n.to(torch.int32)
        if case["way"] != "loss":
            inner = (p * c[:, None, :]).sum(2, keepdim=True)
            d = (s["dloss"].double() * per)[:, None, None] * keep[:, :, None] * p * (c[:, None, :] - inner)
            d = d.reshape(T, E)
            if case["weights"]:
                # d/dlogit of each kept slot through w = softmax over the kept logits
                w, dw = s["topk_w"].double(), s["dtopk_w"].double()
                jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
                d.scatter_add_(1, s["topk_idx"].long(), (jac @ dw[:, :, None]).squeeze(2))
            got["dlogits"] = d
        return got
    if case["kind"] == "quant":
        q, scale = _exact_quant(s["x"])
        return {"q": q.to(torch.int8), "scale": scale.view(-1)}
    if case["kind"] == "product":
        return _exact_product(s["a"], s["a_scale"], s["w"], s["w_scale"], s["offsets"],
                              s["row_token"], case["act"])
    # the types that the layer's tensors are stored in belong to its definition
    q, scale = _exact_quant(s["x"])
    h = _exact_product(q, scale, s["w1"], s["w1_scale"], s["offsets"], s["row_token"], "swiglu")
    q, scale = _exact_quant(h.to(torch.bfloat16))
    y = _exact_product(q, scale, s["w2"], s["w2_scale"], s["offsets"], None, "none")
    rows = y.to(torch.bfloat16).double()[s["token_row"].long()].view(case["T"], case["k"], -1)
    return (rows * s["topk_w"].double()[:, :, None]).sum(1)
