"""Plain 64-bit forms of the MXFP4 operators and of the layer, with bounds of what the kernels'
roundings can add (used by the MXFP4 and few-token tests).

Bounds, for one output element.  u = 2^-24 is fp32's half step; a sum of n terms on the tensor cores
is off by at most n * 2u of the sum of their magnitudes (each partial sum truncated or rounded).

* x of an MXFP4 layer is the sum of two e4m3 values under one scale for 32 neighbours: exact down to
  2^-13 of the block's largest magnitude m, off by at most 2^-21 m below.
* h is fp32 before it is stored.  MXFP4: hi is off by at most 2^-4 of h, lo (four bits again) by 2^-5
  of that: 2^-9 |h|, or 2^-21 m below lo's range.  bf16: 2^-8 |h|.
* silu(a) b in fp32 with the fast exponential and division: 2^-20 of it, and what a and b are off by:
  |silu'| <= 1.1.
* gates (softmax in fp32): 2^-20 of them.  Output: one rounding to bf16, 2^-8.
"""
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SUM = 2.0 ** -23


def quantize(w):
    """codes [.., cols / 2], scales [.., cols / 32] (uint8) of w by the definition, in 64 bits."""
    v = w.double().reshape(-1, 32)
    finite = torch.isfinite(v).all(dim=1, keepdim=True)
    a = torch.where(finite, v.abs(), torch.zeros_like(v))
    amax = a.amax(dim=1, keepdim=True)
    s = torch.floor(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)))) - 2
    s = torch.where(amax > 0, s, torch.full_like(s, -127)).clamp(min=-127)
    a = a / torch.exp2(s)
    grid = torch.tensor(GRID, dtype=torch.float64, device=w.device)
    dist = (a.unsqueeze(2) - grid).abs()
    best = dist.amin(dim=2, keepdim=True)
    # of the nearest codes (two at a tie) the even one
    order = torch.arange(8, device=w.device) + 8 * (torch.arange(8, device=w.device) % 2)
    code = torch.where(dist == best, order, 99).argmin(dim=2)
    code = code + 8 * torch.signbit(v).long()
    code = torch.where(finite, code, torch.zeros_like(code)).reshape(*w.shape[:-1], -1)
    scale = torch.where(finite, s + 127, torch.full_like(s, 255)).reshape(*w.shape[:-1], -1)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale.to(torch.uint8)


def values(codes, scales):
    """The matrix in 64 bits."""
    grid = torch.tensor(GRID + tuple(-m for m in GRID), dtype=torch.float64, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).long().flatten(-2)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return grid[c] * s.repeat_interleave(32, dim=-1)


def tile_scales(scales):
    """scales [.., rows, cols / 32] in blocks of 128 rows x 4 scales."""
    nb = scales.shape[-1]
    s = scales.reshape(-1, nb)
    out = torch.empty(s.numel(), dtype=torch.uint8)
    for r in range(s.shape[0]):
        for b in range(nb):
            out[(r // 128 * (nb // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4
                + b % 4] = s[r, b]
    return out.reshape(scales.shape)


def _block_max(v):
    return v.abs().reshape(v.shape[0], -1, 32).amax(dim=2).repeat_interleave(32, dim=1)


def layer(x, w_router, bias, w_gate, w_up, w_down, k, n_shared, routed_scale=1.0, mx=True):
    """(out, bound), 64 bits [T, d], of the layer whose weights are [G, rows, cols] in 64 bits (or
    callables g -> matrix)."""
    def mat(w, g):
        return w(g) if callable(w) else w[g]

    x = x.double()
    E = w_router.shape[0]
    logits = x @ w_router.double().T
    score = logits + (0 if bias is None else bias.double())
    top = torch.argsort(score, dim=1, descending=True, stable=True)[:, :k]
    gate = torch.softmax(logits.gather(1, top), dim=1) * routed_scale
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    for g in range(E + n_shared):
        if g < E:
            tok, slot = (top == g).nonzero(as_tuple=True)
            weight = gate[tok, slot].unsqueeze(1)
        else:
            tok, weight = torch.arange(x.shape[0], device=x.device), 1.0
        if tok.numel() == 0:
            continue
        xe, wg, wu, wd = x[tok], mat(w_gate, g), mat(w_up, g), mat(w_down, g)
        dx = 2.0 ** -21 * _block_max(xe) if mx else torch.zeros_like(xe)
        d, f = x.shape[1], wg.shape[0]
        a, b = xe @ wg.T, xe @ wu.T
        da = (dx + 2 * d * SUM * xe.abs()) @ wg.abs().T
        db = (dx + 2 * d * SUM * xe.abs()) @ wu.abs().T
        h = a * torch.sigmoid(a) * b
        dh = 1.1 * da * (b.abs() + db) + (a * torch.sigmoid(a)).abs() * db + 2.0 ** -20 * h.abs()
        dh = dh + (2.0 ** -9 * (h.abs() + dh) + 2.0 ** -21 * _block_max(h.abs() + dh) if mx
                   else 2.0 ** -8 * (h.abs() + dh))
        y = h @ wd.T
        dy = (dh + 2 * f * SUM * (h.abs() + dh)) @ wd.abs().T
        out.index_add_(0, tok, weight * y)
        err.index_add_(0, tok, weight * (dy + 2.0 ** -20 * y.abs()))
    err = err + (k + n_shared) * SUM * (out.abs() + err)
    return out, err + 2.0 ** -8 * (out.abs() + err) + 1e-37
