"""64-bit references of the serving-step operators (router, few-token expert layer, batched adapters), written from their
formulas, with element-wise error bounds.  Used by the tests only; nothing here calls the library."""
import numpy as np
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BF16_HALF_STEP = 2.0 ** -8       # largest relative error of one rounding to bf16
FP32_SUM = 2.0 ** -18            # relative to the sum of magnitudes: fp32 rounding of sums of up to some thousand terms


def values(q, sf):
    """Packed codes [rows, k/2] and 128x4-swizzled scales -> float64 e2m1 * ue4m3 [rows, k], on q's device."""
    rows, half = q.shape
    codes = torch.stack((q & 15, q >> 4), -1).reshape(rows, 2 * half).long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=q.device)
    r = torch.arange(rows, device=q.device)[:, None]
    c = torch.arange(half // 8, device=q.device)[None, :]
    groups = -(-(half // 8) // 4)
    code = sf.reshape(-1)[((r // 128) * groups + c // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + c % 4]
    scale = code.view(torch.float8_e4m3fn).double()
    return table[codes] * scale.repeat_interleave(16, 1)


def slice_error(x, chunk):
    """Largest error of four FP4 slices for every value of x [rows, k]: 1/1536 of its 16-value block's largest magnitude,
    or 1/786432 of its chunk's where that is more."""
    rows, k = x.shape
    pad = -(-k // chunk) * chunk
    a = torch.zeros((rows, pad), dtype=torch.float64, device=x.device)
    a[:, :k] = x.abs()
    block = a.view(rows, -1, 16).amax(-1).repeat_interleave(16, 1)
    whole = a.view(rows, -1, chunk).amax(-1).repeat_interleave(chunk, 1)
    return torch.maximum(block / 1536, whole / 786432)[:, :k]


def moe(x, ids, weights, w, E):
    """out and its error bound, float64 [t, k].  w: dict of gate, up, down -> (codes [E, ...], scales, amax [E])."""
    t, k = x.shape
    xd = x.double()
    ex = slice_error(xd, 256)
    out = torch.zeros((t, k), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    for e in range(E):
        at, slot = (ids == e).nonzero(as_tuple=True)
        if not at.numel():
            continue
        m = {name: values(q[e], sf[e]) * (amax[e].double() / 2688.0) for name, (q, sf, amax) in w.items()}
        xe, xerr = xd[at], ex[at]
        g, u = xe @ m["gate"].t(), xe @ m["up"].t()
        dg = (xerr + FP32_SUM * xe.abs()) @ m["gate"].abs().t()
        du = (xerr + FP32_SUM * xe.abs()) @ m["up"].abs().t()
        h = g * torch.sigmoid(g) * u
        # |d silu| <= 1.1 |dg|; a few fp32 roundings in silu and the product
        dh = 1.1 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du + 2.0 ** -20 * h.abs()
        dh = dh + slice_error(h.abs() + dh, 128)
        wt = weights[at, slot].double()[:, None]
        out.index_add_(0, at, (h @ m["down"].t()) * wt)
        err.index_add_(0, at, ((dh + FP32_SUM * h.abs()) @ m["down"].abs().t()) * wt.abs())
    return out, err + BF16_HALF_STEP * (out.abs() + err)


def lora_down(x, w, adapter):
    d = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(d)
    for a in range(w.shape[0]):
        at = (adapter == a).nonzero()[:, 0]
        d[at] = x[at].double() @ w[a].double().t()
        mag[at] = x[at].double().abs() @ w[a].double().abs().t()
    err = FP32_SUM * mag
    return d, err + BF16_HALF_STEP * (d.abs() + err)


def gemm_lora(a, b, a_sf, b_sf, alpha, d, l1, adapter, bias):
    av, bv, al = values(a, a_sf), values(b, b_sf), alpha.double()
    out = av @ bv.t() * al
    err = FP32_SUM * (av.abs() @ bv.abs().t()) * al.abs()
    for i in range(l1.shape[0]):
        at = (adapter == i).nonzero()[:, 0]
        out[at] += d[at].double() @ l1[i].double().t()
        # d / alpha is rounded to bf16 once
        err[at] += (BF16_HALF_STEP + FP32_SUM) * (d[at].double().abs() @ l1[i].double().abs().t())
    if bias is not None:
        out = out + bias.double()
    return out, err + BF16_HALF_STEP * (out.abs() + err)


def route(logits, topk, weighting):
    """ids and weights as numpy arrays, one token at a time: 0 softmax, 1 softmax over the selected, 2 sigmoid."""
    x = logits.double().cpu().numpy()
    big = float(np.finfo(np.float32).max)
    ids = np.full((x.shape[0], topk), -1, np.int32)
    w = np.zeros((x.shape[0], topk))
    for i, row in enumerate(x):
        ok = [(-min(v, big), e) for e, v in enumerate(row) if v > -np.inf]      # NaN compares false
        best = sorted(ok)[:topk]
        if not best:
            continue
        v = np.array([-b for b, _ in best])
        ids[i, :len(best)] = [e for _, e in best]
        if weighting == 2:
            w[i, :len(best)] = 1.0 / (1.0 + np.exp(-v))
        else:
            total = np.exp(v - v[0]).sum() if weighting == 1 else sum(np.exp(-b - v[0]) for b, _ in ok)
            w[i, :len(best)] = np.exp(v - v[0]) / total
    return ids, w


def assert_within(got, ref, err, what=""):
    d = (got.double() - ref).abs()
    bad = ~(d <= err)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; worst ratio {float((d / err).nan_to_num(float('inf')).max())}"
