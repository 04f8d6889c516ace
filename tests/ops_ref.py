"""64-bit references of the operators over channels-last frames, written from their formulas."""
import torch

F24 = 2.0 ** -24


def norm_forward(x, groups, weight, bias, act, alpha, beta, eps, lengths):
    """(y, mean, rstd, scale) in fp64; scale bounds the size of what is added up in u."""
    B, T, C = x.shape
    D = C // groups
    y = torch.zeros(B, T, C, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    mean = torch.zeros(B, groups, dtype=torch.float64, device=x.device)
    var = torch.zeros_like(mean)
    one = torch.ones(C, dtype=torch.float64, device=x.device)
    w = one if weight is None else weight.double()
    b = 0 * one if bias is None else bias.double()
    for i in range(B):
        n = T if lengths is None else min(max(int(lengths[i]), 0), T)
        if n == 0:
            continue
        xi = x[i, :n].double().view(n, groups, D)
        mean[i] = xi.mean(dim=(0, 2))
        var[i] = ((xi - mean[i][:, None]) ** 2).mean(dim=(0, 2))
        rs = 1 / torch.sqrt(var[i] + eps)
        xh = ((xi - mean[i][:, None]) * rs[:, None]).reshape(n, C)
        u = xh * w + b
        mag[i, :n] = (xh * w).abs() + b.abs() + (mean[i].abs() * rs).repeat_interleave(D) * w.abs()
        y[i, :n] = activation(u, act, alpha, beta)[0]
    return y, mean, 1 / torch.sqrt(var + eps), mag


def activation(u, act, alpha, beta):
    """(act(u), act'(u), d act / d alpha, d act / d beta)"""
    if act == "silu":
        s = torch.sigmoid(u)
        return u * s, s + u * s * (1 - s), None, None
    if act == "snake_beta":
        a, be = alpha.double(), beta.double() + 1e-9
        s, c = torch.sin(a * u), torch.cos(a * u)
        return u + s * s / be, 1 + 2 * a * s * c / be, 2 * u * s * c / be, -s * s / be ** 2
    return u, torch.ones_like(u), None, None


def activation_parts(u, act, alpha, beta):
    """The size of what is added or multiplied up in act'(u) and in the factors of dalpha and dbeta.  Each
    is computed with errors relative to these, not to its value: 1 + alpha sin(2 alpha u) / beta can
    cancel, and the errors of sin and cos are absolute, relative to 1."""
    if act == "silu":
        return torch.ones_like(u) + u.abs() * torch.sigmoid(u), None, None
    if act == "snake_beta":
        a, be = alpha.double(), beta.double()
        return 1 + (a / be).abs() + 0 * u, 2 * u.abs() / be.abs(), 1 / be ** 2 + 0 * u
    return torch.ones_like(u), None, None


def norm_backward(dy, x, groups, weight, bias, act, alpha, beta, mean, rstd, lengths):
    """dict of fp64 gradients and, for each, the sum of the sizes its errors are relative to; mean and
    rstd are taken as given."""
    B, T, C = x.shape
    D = C // groups
    z = torch.zeros(C, dtype=torch.float64, device=x.device)
    w = z + 1 if weight is None else weight.double()
    b = z if bias is None else bias.double()
    out = {"dx": torch.zeros(B, T, C, dtype=torch.float64, device=x.device)}
    mag = {"dx": torch.zeros_like(out["dx"])}
    for k in ("dweight", "dbias", "dalpha", "dbeta"):
        out[k], mag[k] = z.clone(), z.clone()
    for i in range(B):
        n = T if lengths is None else min(max(int(lengths[i]), 0), T)
        if n == 0:
            continue
        mu, rs = mean[i].double().repeat_interleave(D), rstd[i].double().repeat_interleave(D)
        g = dy[i, :n].double()
        xh = (x[i, :n].double() - mu) * rs
        u = xh * w + b
        _, slope, da, db = activation(u, act, alpha, beta)
        p_slope, p_da, p_db = activation_parts(u, act, alpha, beta)
        du, p_du = g * slope, g.abs() * p_slope
        for k, term, part in (("dweight", du * xh, p_du * xh.abs()), ("dbias", du, p_du),
                              ("dalpha", None if da is None else g * da, None if da is None else g.abs() * p_da),
                              ("dbeta", None if db is None else g * db, None if db is None else g.abs() * p_db)):
            if term is not None:
                out[k] += term.sum(0)
                mag[k] += part.sum(0)
        h = du * w
        m1 = h.view(n, groups, D).mean(dim=(0, 2)).repeat_interleave(D)
        m2 = (h * xh).view(n, groups, D).mean(dim=(0, 2)).repeat_interleave(D)
        p_h = p_du * w.abs()
        a1 = p_h.view(n, groups, D).mean(dim=(0, 2)).repeat_interleave(D)
        a2 = (p_h * xh.abs()).view(n, groups, D).mean(dim=(0, 2)).repeat_interleave(D)
        out["dx"][i, :n] = rs * (h - m1 - xh * m2)
        mag["dx"][i, :n] = rs * (p_h + a1 + xh.abs() * a2)
    return out, mag


def e4m3(v):
    """The e4m3 number nearest to each fp64 value (ties to even, at most 448 in magnitude; NaN stays)."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6).nan_to_num())[1].long() - 1
    step = ((e - 3 + 1023) << 52).view(torch.float64)  # exactly a power of two
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def quantize(x, block_rows):
    """(q, scale [K blocks, row blocks], the values they stand for), fp64.  The scale and the number that is
    rounded to e4m3 are fp32 by definition."""
    R, K = x.shape
    rb, kb = -(-R // block_rows), -(-K // 128)
    p = torch.zeros(rb * block_rows, kb * 128, dtype=torch.float64, device=x.device)
    p[:R, :K] = x.double()
    p = p.view(rb, block_rows, kb, 128)
    top = p.abs().amax(dim=(1, 3), keepdim=True).clamp(min=2.0 ** -100)
    scale = (top / 448).float().double()
    factor = (448 / top).float().double()
    q = e4m3((p * factor).float().double())
    v = (q * scale).view(rb * block_rows, kb * 128)[:R, :K]
    return q.view(rb * block_rows, kb * 128)[:R, :K], scale[:, 0, :, 0].t(), v


def dequantize(q, scale):
    """The fp64 values of a stored matrix (block rows from the scale's shape)."""
    R, K = q.shape
    rows = 1 if scale.shape[1] == R else 128
    at_r = torch.arange(R, device=q.device) // rows
    at_k = torch.arange(K, device=q.device) // 128
    return q.float().double() * scale.double()[at_k][:, at_r].t()
