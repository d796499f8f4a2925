"""Plain implementations in f64 of a layer's norm, routing and experts, and how far a
correct f32 computation may be from them.  Shared by the CPU and GPU tests; elementary
torch operations and loops, no code of the library."""
import math

import torch

# Half a step, relative to the value.
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def norm(x, weight, residual, eps, offset):
    """(y, s) in f64."""
    s = x.double() + (0 if residual is None else residual.double())
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return y * (1.0 if weight is None else offset + weight.double()), s


def norm_bounds(y, s, dtype, adds):
    """How far outputs may be off.  A sum s = x + r is one f32 rounding and one to the type.  For y:
    s (2^-24), the sum of squares (`adds` roundings of a partial sum that is at most the whole, and
    twice s's error; half of that counts in its root), the mean, + eps, root, reciprocal (each 2^-23 at
    most), two products and offset + weight (each 2^-24), then the rounding to the type."""
    u = 2.0 ** -24
    e = u + 0.5 * (adds + 2) * u + 4 * 2 * u + 3 * u
    return (e + HALF[dtype] * (1 + e)) * y.abs() + 1e-42, (u + HALF[dtype] * (1 + u)) * s.abs()


def route(logits, top_k, bias, sigmoid, groups, top_groups, group_top, renormalize, scale):
    """(ids, weights) in f64; of equal choices the lowest index, one token at a time."""
    x = logits.double().cpu()
    t, e = x.shape
    ids, weights = torch.zeros((t, top_k), dtype=torch.int32), torch.zeros((t, top_k), dtype=torch.float64)
    for i in range(t):
        row = x[i]
        if sigmoid:
            s = 1.0 / (1.0 + torch.exp(-row))
        else:
            m = row.max()
            s = torch.zeros(e, dtype=torch.float64) if m == -math.inf else torch.exp(row - m)
            s = s / s.sum() if s.sum() > 0 else s
        c = s if bias is None else s + bias.double().cpu()
        rank = (row if bias is None else c).tolist()
        c = c.tolist()
        size = e // groups
        if groups > 1:
            worth = [sum(sorted(c[g * size:(g + 1) * size], reverse=True)[:group_top]) for g in range(groups)]
            stays = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        else:
            stays = [0]
        pool = [j for g in stays for j in range(g * size, (g + 1) * size)]
        best = sorted(pool, key=lambda j: (-rank[j], j))[:top_k]
        w = torch.stack([s[j] for j in best])
        if renormalize:
            total = w.sum()
            w = w / total if total != 0 else torch.zeros_like(w)
        ids[i], weights[i] = torch.tensor(best, dtype=torch.int32), w * scale
    return ids, weights


def q4_values(w):
    """Q4_0 rows (uint8 [.., blocks * 18]) as f64."""
    b = w.reshape(*w.shape[:-1], -1, 18)
    d = b[..., :2].contiguous().view(torch.float16).double()
    q = b[..., 2:].to(torch.int32)
    return (torch.cat([q & 15, q >> 4], -1) - 8).double().mul(d).reshape(*w.shape[:-1], -1)


def q4_random(shape, k, gen, size=0.2):
    """Random Q4_0 rows whose products with rows near 1 are near 1."""
    x = torch.randint(0, 256, (*shape, k // 32, 18), dtype=torch.uint8, generator=gen)
    d = (0.5 + torch.rand((*shape, k // 32), generator=gen)) * (size / math.sqrt(k))
    d = torch.where(torch.rand(d.shape, generator=gen) < 0.5, d, -d).half()
    x[..., :2] = d.unsqueeze(-1).contiguous().view(torch.uint8)
    return x.reshape(*shape, k // 32 * 18)


def activate(a, kind):
    if kind == 1:
        return a * torch.sigmoid(a)
    if kind == 2:
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    return a


def experts(w_gate, w_up, w_down, x, ids, weights, kind):
    """(out, bound) in f64: the formula, and how far the library's may be off by what its header says of
    its precision.

    A product x_k w_k is off by p |x_k w_k| + 2^-38 max|x| |w_k|: f32 rows p = 2^-21; bf16 rows the
    weight's rounding to 11 bits, 2^-11, and for the inner activations theirs, 2^-11 more.  A sum of K
    products in f32 takes at most K additions, tensor cores 16 of them at a time and up to 3 times
    (pieces), each of which may cut off 2^-23 of a partial sum that is at most the sum of magnitudes:
    (3 K / 16 + 64) 2^-23 with the additions of parts.  Activations: the derivative is at most 1.13,
    their own evaluation 16 units of f32 of |a|.  The weighted sum: top_k roundings of partial sums."""
    u = 2.0 ** -24
    bf16 = x.dtype == torch.bfloat16
    t, k = ids.shape
    xd = x.double()
    out = torch.zeros((t, w_down.shape[1]), dtype=torch.float64, device=x.device)
    bound, size = torch.zeros_like(out), torch.zeros_like(out)

    def product(a, w, rounds):
        p = (2.0 ** -21 if not bf16 else 2.0 ** -11 * rounds) + (3 * a.shape[-1] / 16 + 64) * 2 * u
        mag = a.abs() @ w.abs().T
        return a @ w.T, p * mag + 2.0 ** -38 * a.abs().amax(-1, keepdim=True) * w.abs().sum(-1)

    for e in range(w_up.shape[0]):
        ti, ji = torch.nonzero(ids == e, as_tuple=True)
        if len(ti) == 0:
            continue
        up, eu = product(xd[ti], q4_values(w_up[e]), 1)
        if w_gate is not None:
            g, eg = product(xd[ti], q4_values(w_gate[e]), 1)
            a, ea = activate(g, kind), 1.13 * eg + 16 * u * g.abs()
            h, eh = a * up, ea * up.abs() + a.abs() * eu + ea * eu + 2 * u * (a * up).abs()
        else:
            h, eh = activate(up, kind), 1.13 * eu + 16 * u * up.abs()
        wd = q4_values(w_down[e])
        y, ey = product(h, wd, 2)
        ey = ey + eh @ wd.abs().T * 1.01
        w = weights[ti, ji].double().unsqueeze(-1)
        for n in range(len(ti)):  # (a token may have an expert twice)
            out[ti[n]] += (y * w)[n]
            bound[ti[n]] += (ey * w.abs())[n]
            size[ti[n]] += (y * w).abs()[n]
    bound = bound + (k + 2) * 2 * u * size
    return out, bound + HALF[x.dtype] * (out.abs() + bound) + 1e-40
