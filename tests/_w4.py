"""Plain 64-bit restatements of the 4-bit product, the router and the experts'
products, with the tolerances the GPU tests use."""
import numpy as np
import torch


def make_weights(gen, lead, K, group, zeros, spread=1.0):
    """Random codes 0..15, bf16 scales around 2^-8 with random signs of the
    exponent, zero points 0..15 (or None)."""
    G = -(-K // group)
    q = torch.randint(0, 16, (*lead, K), generator=gen, dtype=torch.uint8)
    s = (2.0 ** (-8 + spread * torch.randn(*lead, G, generator=gen))).bfloat16()
    z = torch.randint(0, 16, (*lead, G), generator=gen, dtype=torch.uint8) if zeros else None
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), s, z


def dequantize(wq, sw, wz, group):
    """[..., K] float64 weights from the definition."""
    K = 2 * wq.shape[-1]
    k = torch.arange(K)
    q = (wq[..., k // 2].long() >> (4 * (k % 2))) & 15
    z = 8 if wz is None else wz[..., k // group].long()
    return (q - z).double() * sw[..., k // group].double()


def magnitudes(wq, sw, wz, group):
    """[..., K] float64: |q - z| |s|, the size of a weight."""
    return dequantize(wq, sw, wz, group).abs()


def product_limit(y, mag, K, zeros=False):
    """Largest allowed |kernel - exact|: the output's bf16 rounding (half a step:
    2^-8 of the value), and f32 sums of exact products: K / 16 tensor-core steps
    and at most 64 further additions, each off by at most 2^-22 of the sum of the
    magnitudes `mag` (a 17-term sum inside a step may truncate).

    With zero points a weight may be rounded once: q - z is an integer of up to 4
    bits (|q - z| <= 15), s has 8 significant bits, their product up to 12, and f16,
    in which the tensor cores take it, 11.  That rounding is off by at most half a
    step, 2^-11 of the weight, so by 2^-11 of |x w| in each term and 2^-11 `mag` in
    the sum.  (For z = 8, |q - z| <= 8 has at most 3 significant bits, the product
    11: exact.)"""
    return 2.0 ** -8 * y.abs() + ((K / 16 + 64) * 2.0 ** -22 + (2.0 ** -11 if zeros else 0.0)) * mag + 1e-38


def assert_product(got, x, wq, sw, wz, group, what=""):
    """got bf16 [M,N] against x [M,K] @ W[N,K]^T in float64."""
    w = dequantize(wq, sw, wz, group)
    y = x.double() @ w.t()
    mag = x.double().abs() @ magnitudes(wq, sw, wz, group).t()
    err = (got.double().cpu() - y).abs()
    lim = product_limit(y, mag, w.shape[1], wz is not None)
    bad = (~(err <= lim)).nonzero()
    assert bad.numel() == 0, (what, bad.shape[0], [(tuple(b.tolist()), got.double().cpu()[tuple(b)].item(),
                                                    y[tuple(b)].item(), lim[tuple(b)].item()) for b in bad[:4]])


def route64(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    """The router in float64 (numpy), token by token: ids, weights."""
    x = logits.double().numpy()
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    wts = np.zeros((T, k))
    b = None if bias is None else bias.double().numpy()
    fmax = float(np.finfo(np.float32).max)
    for t in range(T):
        l = np.minimum(x[t], fmax)
        logit_ok = l > -np.inf  # False for NaN too
        ok = logit_ok if b is None else logit_ok & (b > -np.inf)
        if not ok.any():
            continue
        m = l[logit_ok].max()
        with np.errstate(all="ignore"):
            if sigmoid:
                p = np.where(l >= 0, 1.0, np.exp(-np.abs(l))) / (1.0 + np.exp(-np.abs(l)))
            else:
                e = np.where(logit_ok, np.exp(l - m), 0.0)
                p = e / e.sum()
            c = l if b is None else p + b
        c = np.where(ok, c, -np.inf)
        if groups > 1:
            v = c if b is not None or group_top == 1 else np.where(ok, p, -np.inf)
            v = np.sort(v.reshape(groups, -1), axis=1)[:, ::-1]
            gs = v[:, 0] if group_top == 1 else v[:, 0] + v[:, 1]
            keep = np.argsort(-gs, kind="stable")[:top_groups]
            allowed = np.zeros(groups, bool)
            allowed[keep] = True
            c = np.where(np.repeat(allowed, E // groups), c, -np.inf)
        order = np.argsort(-c, kind="stable")[:k]
        order = order[c[order] > -np.inf]
        if not len(order):
            continue
        ids[t, :len(order)] = order
        lj = l[order]
        if renormalize:
            # exact ratios, also where the scores themselves would underflow
            if sigmoid:
                w = np.exp(np.minimum(lj, 0) - np.minimum(lj, 0).max()) / (1.0 + np.exp(-np.abs(lj)))
            else:
                w = np.exp(lj - lj.max())
            w = w / w.sum()
        else:
            w = p[order]
        wts[t, :len(order)] = w * scale
    return ids, wts


def experts64(x, ids, w, size, weights=None):
    """x [T,K] (gather) or [T,k,K] (combine), w [E,N,K] float64 and size its magnitudes ->
    (value, magnitude)."""
    T, k = ids.shape
    E, N, _ = w.shape
    shape = (T, N) if weights is not None else (T, k, N)
    y, mag = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            row = (x[t, j] if weights is not None else x[t]).double()
            v, m = w[e] @ row, size[e] @ row.abs()
            if weights is None:
                y[t, j], mag[t, j] = v, m
            else:
                g = float(weights[t, j])
                y[t] += g * v
                mag[t] += abs(g) * m
    return y, mag
