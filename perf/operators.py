"""Cases for the 4-bit weight product, the expert router and the experts' products.

Three operators that a quantized decoder runs next to the library's 8-bit
projections:

``w4``       y = x W^T with 4-bit weights and a scale (and, if the checkpoint
             has them, a zero point) for each group of inputs,
``route``    a mixture-of-experts router: scores, balance bias, groups, top-k,
             renormalised weights,
``experts``  the routed tokens' products with their experts' 4-bit weights;
             ``combine`` sums a token's experts with the router's weights.

Weights: codes 0..15 packed two to a byte along K (the low nibble is the even
input), value (code - zero) * scale with zero 8 where no zero points are kept.
"""
import math

import torch

own = False

# ----------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------


def listed():
    return [
        # one token through a grouped-query key projection: a decode step's smallest product
        dict(name="w4 token k_proj", op="w4", M=1, N=1024, K=4096, group=128, zeros=False),
        # one token through the down projection: a decode step's long K, zero points kept
        dict(name="w4 token down", op="w4", M=1, N=4096, K=14336, group=128, zeros=True),
        # a decode batch through the gate projection
        dict(name="w4 batch gate", op="w4", M=16, N=14336, K=4096, group=64, zeros=False),
        # a ragged batch on a layer of odd width whose last group is short
        dict(name="w4 ragged", op="w4", M=77, N=1111, K=4128, group=64, zeros=True),
        # a prompt through the gate projection
        dict(name="w4 prompt gate", op="w4", M=2048, N=14336, K=4096, group=128, zeros=False),
        # one token's router in a decode step
        dict(name="route token", op="route", T=1, E=64, k=8, dtype="float32", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0),
        # a prompt chunk with a balance bias and limited groups
        dict(name="route chunk grouped", op="route", T=4099, E=256, k=8, dtype="float32", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5),
        # a long prompt's bf16 logits, plain softmax top-k
        dict(name="route prompt", op="route", T=16384, E=128, k=8, dtype="bfloat16", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0),
        # one token through its experts' gate and up rows
        dict(name="experts token up", op="experts", T=1, k=8, E=64, N=1536, K=2048, group=128, zeros=False,
             combine=False),
        # a small decode batch through the experts' down rows, summed with the router's weights
        dict(name="experts batch down", op="experts", T=7, k=8, E=64, N=2048, K=768, group=128, zeros=False,
             combine=True),
        # a prompt through the experts' gate and up rows
        dict(name="experts prompt up", op="experts", T=2048, k=8, E=64, N=1536, K=2048, group=128, zeros=False,
             combine=False),
        # a ragged prompt through the experts' down rows, with zero points
        dict(name="experts prompt down", op="experts", T=1019, k=8, E=64, N=2048, K=768, group=64, zeros=True,
             combine=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_MAX_MACS = 2048 * 14336 * 4096  # of the largest listed case


def draw(rng):
    op = rng.choice(["w4", "w4", "w4", "route", "route", "experts", "experts", "experts"])
    if op == "w4":
        while True:
            M, N = _log_int(rng, 1, 2048), _log_int(rng, 64, 14336)
            K = 32 * _log_int(rng, 8, 448)
            if M * N * K <= _MAX_MACS // 2:
                return dict(op=op, M=M, N=N, K=K, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
    if op == "route":
        while True:
            T, E = _log_int(rng, 1, 16384), rng.randint(8, 512)
            groups = rng.choice([1, 1, 2, 4, 8])
            if groups > 1:
                E = max(16, E // groups * groups)
                E -= E % groups
            k = rng.randint(1, 10)
            group_top = rng.choice([1, 2]) if groups > 1 else 1
            top_groups = rng.randint(1, groups)
            if T * E > 16384 * 256 or top_groups * (E // groups) < k or E // groups < group_top:
                continue
            return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["float32", "bfloat16"]),
                        score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                        top_groups=top_groups, group_top=group_top, renormalize=rng.random() < 0.7,
                        scale=rng.choice([1.0, 2.5]))
    while True:
        T, k, E = _log_int(rng, 1, 2048), rng.randint(1, 8), _log_int(rng, 8, 128)
        N, K = _log_int(rng, 128, 2048), 32 * _log_int(rng, 8, 64)
        if E * N * K <= 64 * 1536 * 2048 and T * k * N * K <= 2048 * 8 * 1536 * 2048:
            return dict(op=op, T=T, k=k, E=E, N=N, K=K, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.3,
                        combine=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _tokens(g, rows, K):
    """bf16 activations N(0, 1) with 1% outlier channels twenty times larger."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    outliers = torch.rand(K, generator=g, device="cuda") < 0.01
    return torch.where(outliers, x * 20.0, x).bfloat16()


def _hidden(g, rows, K):
    """bf16 gated activations silu(a) * b, as a down projection reads them."""
    a = torch.randn(rows, K, generator=g, device="cuda")
    b = torch.randn(rows, K, generator=g, device="cuda")
    return (a * torch.sigmoid(a) * b).bfloat16()


def _weights(g, rows, K, group, zeros):
    """Codes and scales of N(0, 0.02) weights quantized in groups along K."""
    groups = -(-K // group)
    w = torch.randn(rows, K, generator=g, device="cuda") * 0.02
    pad = groups * group - K
    wp = torch.nn.functional.pad(w, (0, pad)).view(rows, groups, group)
    if zeros:
        lo, hi = wp.amin(-1).clamp(max=0.0), wp.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / 15.0).bfloat16()
        z = torch.round(-lo / s.float()).clamp(0, 15)
        q = (torch.round(wp / s.float().unsqueeze(-1)) + z.unsqueeze(-1)).clamp(0, 15)
        z = z.to(torch.uint8)
    else:
        s = (wp.abs().amax(-1) / 7.0).bfloat16()
        q = torch.round(wp / s.float().unsqueeze(-1)).clamp(-7, 7) + 8.0
        z = None
    q = q.view(rows, groups * group)[:, :K].to(torch.uint8)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s.contiguous(), z


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "w4":
        x = _tokens(g, case["M"], case["K"])
        wq, sw, wz = _weights(g, case["N"], case["K"], case["group"], case["zeros"])
        return dict(x=x, wq=wq, sw=sw, wz=wz)
    if op == "route":
        T, E = case["T"], case["E"]
        # a router's logits: the experts' own popularity plus the token's preference
        logits = torch.randn(T, E, generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda") * 0.5
        bias = torch.randn(E, generator=g, device="cuda") * 0.05 if case["bias"] else None
        return dict(logits=logits.to(getattr(torch, case["dtype"])), bias=bias)
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    x = _hidden(g, T * k, K).view(T, k, K) if case["combine"] else _tokens(g, T, K)
    parts = [_weights(g, N, K, case["group"], case["zeros"]) for _ in range(E)]
    wq, sw = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    wz = torch.stack([p[2] for p in parts]) if case["zeros"] else None
    pref = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda") * 0.5
    top, ids = torch.topk(pref, k, dim=-1)
    weights = torch.exp(top - top[:, :1])
    weights = weights / weights.sum(-1, keepdim=True) if case["combine"] else None
    return dict(x=x, wq=wq, sw=sw, wz=wz, ids=ids.to(torch.int32).contiguous(), weights=weights)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        import fp8_linear_layers_b200 as ql
        st["ql"] = ql
        if case["op"] == "route":
            st["score"] = {"softmax": ql.ROUTE_SOFTMAX, "sigmoid": ql.ROUTE_SIGMOID}[case["score"]]
        else:
            # what a serving program keeps beside its weights: the checked handle and a workspace
            st["w4"] = ql.W4Weight(st["wq"], st["sw"], st["wz"], group=case["group"])
            if case["op"] == "w4":
                n = ql.forward_w4_workspace_bytes(case["M"], st["w4"])
            else:
                n = ql.experts_w4_workspace_bytes(case["T"], case["k"], st["w4"], combine=case["combine"])
            st["ws"] = ql.new_workspace(n)
    return st


# ----------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------


def _dequantize(wq, sw, wz, group):
    """Packed codes [..., K/2], scales [..., K/group] -> f32 weights [..., K]."""
    q = torch.stack((wq & 15, wq >> 4), dim=-1).flatten(-2).float()
    K = q.shape[-1]
    s = sw.float().repeat_interleave(group, dim=-1)[..., :K]
    z = 8.0 if wz is None else wz.float().repeat_interleave(group, dim=-1)[..., :K]
    return (q - z) * s


def _plain_route(st):
    c = st["case"]
    logits = st["logits"].double()
    T, E = logits.shape
    if c["score"] == "softmax":
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    # without a bias the scores' order is the logits' own
    choice = p + st["bias"].double() if c["bias"] else logits
    if c["groups"] > 1:
        value = choice if c["bias"] or c["group_top"] == 1 else p
        per = value.view(T, c["groups"], E // c["groups"])
        gs = torch.sort(per, dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
        keep = torch.sort(gs, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros_like(gs, dtype=torch.bool).scatter(1, keep, True)
        choice = choice.masked_fill(~mask.repeat_interleave(E // c["groups"], dim=1), -math.inf)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_experts(st):
    c = st["case"]
    x, ids = st["x"].float(), st["ids"].long()
    T, k = ids.shape
    E, N = st["wq"].shape[:2]
    y = torch.zeros(T, k, N, device=x.device)
    for e in torch.unique(ids).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        w = _dequantize(st["wq"][e], st["sw"][e], None if st["wz"] is None else st["wz"][e], c["group"])
        y[t, j] = (x[t, j] if c["combine"] else x[t]) @ w.t()
    if c["combine"]:
        y = (y * st["weights"].unsqueeze(-1)).sum(1)
    return y.bfloat16()


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        ql = st["ql"]
        if op == "w4":
            return ql.forward_w4(st["x"], st["w4"], workspace=st["ws"])
        if op == "route":
            return ql.route(st["logits"], c["k"], score=st["score"], bias=st["bias"], groups=c["groups"],
                            top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renormalize"],
                            scale=c["scale"])
        return ql.experts_w4(st["x"], st["ids"], st["w4"], weights=st["weights"], workspace=st["ws"])
    if op == "w4":
        return (st["x"].float() @ _dequantize(st["wq"], st["sw"], st["wz"], c["group"]).t()).bfloat16()
    return _plain_route(st) if op == "route" else _plain_experts(st)


# ----------------------------------------------------------------------------------------------
# Work and exact values
# ----------------------------------------------------------------------------------------------


def _weight_bytes(case):
    groups = -(-case["K"] // case["group"])
    return case["N"] * (case["K"] // 2 + groups * (3 if case["zeros"] else 2))


def work(case):
    op = case["op"]
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _weight_bytes(case) + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        # a score takes about ten operations, a selection one comparison an expert
        return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0), "flops": T * E * 11}
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token is expected to choose
    rows_in, rows_out = (T * k, T) if case["combine"] else (T, T * k)
    extra = 4 * T * k if case["combine"] else 0
    return {"bytes": int(used * _weight_bytes(case)) + 2 * rows_in * K + 2 * rows_out * N + 4 * T * k + extra,
            "flops": 2 * T * k * N * K}


def _exact_weights(wq, sw, wz, group, K):
    """[rows, K] in 64 bits, written per input index from the definition."""
    kk = torch.arange(K, device=wq.device)
    q = (wq[:, kk // 2].to(torch.int64) >> (4 * (kk % 2))) & 15
    z = 8 if wz is None else wz[:, kk // group].to(torch.int64)
    return (q - z).double() * sw[:, kk // group].double()


def _exact_route(case, inp):
    import numpy as np
    x = inp["logits"].double().cpu().numpy()
    T, E = x.shape
    k, G = case["k"], case["groups"]
    if case["score"] == "softmax":
        ex = np.exp(x - x.max(1, keepdims=True))
        p = ex / ex.sum(1, keepdims=True)
    else:
        ex = np.exp(-np.abs(x))
        p = np.where(x >= 0, 1.0, ex) / (1.0 + ex)
    c = p + inp["bias"].double().cpu().numpy() if case["bias"] else x
    allowed = np.ones((T, E), dtype=bool)
    if G > 1:
        size = E // G
        value = c if case["bias"] or case["group_top"] == 1 else p
        gs = -np.partition(-value.reshape(T, G, size), case["group_top"] - 1, axis=2)[:, :, :case["group_top"]].sum(2)
        rank = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1, kind="stable")
        allowed = np.repeat(rank < case["top_groups"], size, axis=1)
    order = np.argsort(np.where(allowed, -c, np.inf), axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, order, 1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(order.astype(np.int32)), torch.from_numpy(w * case["scale"])


def exact(case, seed):
    inp = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, inp)
    if case["op"] == "w4":
        w = _exact_weights(inp["wq"], inp["sw"], inp["wz"], case["group"], case["K"])
        return torch.einsum("mk,nk->mn", inp["x"].double(), w)
    T, k, N, K = (case[n] for n in ("T", "k", "N", "K"))
    x, flat = inp["x"].double(), inp["ids"].reshape(-1).long()
    rows = x.reshape(T * k, K) if case["combine"] else x
    y = torch.empty(T * k, N, dtype=torch.float64, device=x.device)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=case["E"]).tolist()
    at = 0
    for e, n in enumerate(counts):
        if n:
            r = order[at:at + n]
            w = _exact_weights(inp["wq"][e], inp["sw"][e], None if inp["wz"] is None else inp["wz"][e],
                               case["group"], K)
            y[r] = torch.einsum("rk,nk->rn", rows[r if case["combine"] else r // k], w)
            at += n
    y = y.view(T, k, N)
    if case["combine"]:
        return torch.einsum("tj,tjn->tn", inp["weights"].double(), y)
    return y
