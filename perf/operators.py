"""Cases of the MXFP4 serving operators: what is called, on which inputs, and what it has to do.

Three operators, used one after the other by a program that serves a sparse-MoE layer from 4-bit
weights:

* ``quantise``: a matrix to MXFP4 and back.  Blocks of 32 neighbours of a row share a power-of-two
  scale 2^s, s = floor(log2 max|v|) - 2 (the largest e2m1 value is 6 = 1.5 * 2^2); every value
  becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times the scale, ties to the even code, larger
  ones 6.  The pass returns the values that the codes and scales stand for.
* ``layer``: the whole sparse-MoE layer with MXFP4 expert weights and bf16 activations, for any
  number of tokens (router, selection, experts, combine).
* ``few``: the whole layer for a few tokens in one launch, with bf16 or with MXFP4 expert weights.

Sizes: d_model 4096, 288 routed experts, top-8, d_ff 1280 and one shared expert are the layer's own
shape; 32 experts, d_ff 11264 (one expert, the dense FFN) and the small odd shapes are those of its
tests and benchmark.
"""
import math

import torch

own = False

_MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_FULL = dict(d=4096, E=288, k=8, f=1280, shared=1, bias="uniform")


def listed():
    return [
        # one decode batch's activations: a call that is all latency
        dict(name="quant_act_16x4096", op="quantise", rows=16, cols=4096, dtype="bf16"),
        # odd row count, a row length that is a multiple of the block only, fp32 master weights
        dict(name="quant_odd_f32_1013x1312", op="quantise", rows=1013, cols=1312, dtype="f32"),
        # one projection of all experts of a layer, as a checkpoint is converted
        dict(name="quant_experts_369920x4096", op="quantise", rows=289 * 1280, cols=4096,
             dtype="bf16"),
        # a small model with odd sizes
        dict(name="layer_odd_t77", op="layer", T=77, d=384, E=40, k=6, f=384, shared=1,
             bias="uniform"),
        # batched decode: a few tokens for each expert
        dict(name="layer_t256", op="layer", T=256, **_FULL),
        # a chunk whose routing is skewed: empty experts beside crowded ones
        dict(name="layer_skew_t4096", op="layer", T=4096, **dict(_FULL, bias="zipf")),
        # a prefill chunk, the largest batch
        dict(name="layer_t8192", op="layer", T=8192, **_FULL),
        # the dense FFN of the first layers
        dict(name="layer_dense_t1000", op="layer", T=1000, d=4096, E=1, k=1, f=11264, shared=0,
             bias="uniform"),
        # one token of one sequence: the latency of a single decode step
        dict(name="few_mx_t1", op="few", weights="mx", T=1, **_FULL),
        # four sequences with three drafted tokens each, verified together
        dict(name="few_mx_t16", op="few", weights="mx", T=16, **_FULL),
        # the same two from bf16 weights
        dict(name="few_bf16_t1", op="few", weights="bf16", T=1, **_FULL),
        dict(name="few_bf16_t16", op="few", weights="bf16", T=16, **_FULL),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "layer", "few"])
    if op == "quantise":
        cols = 32 * _log_int(rng, 1, 352)
        rows = _log_int(rng, 1, min(400000, 1_400_000_000 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]))
    E = rng.choice([1, 5, 16, 32, 40, 64, 128, 288])
    c = dict(op=op, d=128 * _log_int(rng, 1, 32), E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])),
             f=128 * _log_int(rng, 1, 10), shared=rng.choice([0, 1, 1]),
             bias=rng.choice(["uniform", "uniform", "zipf"]))
    if op == "few":
        c.update(T=_log_int(rng, 1, 64), weights=rng.choice(["mx", "bf16"]))
    else:
        c["T"] = _log_int(rng, 1, 8192)
    return c


# ------------------------------------------------------------------------------ inputs
def _nibble_table(device):
    """16-bit random word -> packed pair of e2m1 codes with the frequencies that a quantised
    N(0, 1) has when the largest of 32 neighbours (about 2.2 sigma) lies between 4 and 8 scale
    units: each byte of the word picks one code."""
    sigma = 2.5  # of the values in units of the scale
    edges = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    cdf = [math.erf(e / sigma / math.sqrt(2.0)) for e in edges] + [1.0]
    lut = []
    for b in range(128):  # magnitude from 7 bits, sign from the eighth
        u = (b + 0.5) / 128.0
        lut.append(next(i for i, c in enumerate(cdf) if u <= c))
    lut = torch.tensor(lut + [m + 8 for m in lut], dtype=torch.int32, device=device)
    w = torch.arange(65536, dtype=torch.int64, device=device)
    return (lut[w & 255] + 16 * lut[w >> 8]).to(torch.uint8)


def _mx_weights(gen, G, rows, cols, std, device):
    """codes [G, rows, cols / 2] and scales [G, rows, cols / 32] of N(0, std^2)-like weights."""
    table = _nibble_table(device)
    codes = torch.empty((G, rows, cols // 2), dtype=torch.uint8, device=device)
    for g0 in range(0, G, 16):
        part = codes[g0:g0 + 16]
        r = torch.randint(0, 65536, part.shape, generator=gen, device=device, dtype=torch.int32)
        torch.index_select(table, 0, r.view(-1), out=part.view(-1))
    # sigma = 2.5 scale units: the scale is the power of two next to std / 2.5
    s0 = 127 + round(math.log2(std / 2.5))
    u = torch.randint(0, 8, (G, rows, cols // 32), generator=gen, device=device,
                      dtype=torch.uint8)
    scales = (s0 + (u > 5).to(torch.int16) - (u < 1).to(torch.int16)).to(torch.uint8)
    return codes, scales


def _normal(gen, shape, std, device):
    return torch.randn(shape, generator=gen, device=device).mul_(std).to(torch.bfloat16)


def _bf16_weights(gen, G, rows, cols, std, device):
    out = torch.empty((G, rows, cols), dtype=torch.bfloat16, device=device)
    for g in range(0, G, 16):
        part = out[g:g + 16]
        part.copy_(_normal(gen, part.shape, std, device))
    return out


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "quantise":
        w = torch.randn((case["rows"], case["cols"]), generator=gen, device=dev,
                        dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        w.mul_(case["cols"] ** -0.5)
        w[::97, :32] = 0  # blocks of zeros, as pruned or padded rows have
        return dict(case=case, w=w)
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    G = E + case["shared"]
    s = dict(case=case)
    s["w_router"] = _normal(gen, (E, d), d ** -0.5, dev)
    if case["bias"] == "zipf":
        rank = torch.randperm(E, generator=gen, device=dev).float() + 1
        s["bias"] = -1.1 * torch.log(rank)
    else:
        s["bias"] = torch.rand(E, generator=gen, device=dev) * 0.2 - 0.1
    x = _normal(gen, (T, d), 1.0, dev)
    # a token whose k-th and (k+1)-th scores all but tie is drawn again: which of the two experts
    # it goes to is decided by the rounding of a sum, not by the operator
    for _ in range(100):
        score = x.double() @ s["w_router"].double().T + s["bias"].double()
        top = score.topk(min(E, k + 1), dim=1).values
        near = ((top[:, :-1] - top[:, 1:]).amin(dim=1) < 1e-4) if E > 1 else top[:, 0] > 1e300
        if not bool(near.any()):
            break
        n = int(near.sum())
        x[near] = _normal(gen, (n, d), 1.0, dev)
    s["x"] = x
    make = _mx_weights if case.get("weights", "mx") == "mx" else _bf16_weights
    for name, rows, cols in (("w_gate", f, d), ("w_up", f, d), ("w_down", d, f)):
        s[name] = make(gen, G, rows, cols, cols ** -0.5, dev)
    if own:
        import sparse_moe_layer_warp_b200 as moe

        cls = moe.MoELayerMXFP4 if make is _mx_weights else moe.MoELayer
        s["layer"] = cls(s["w_router"], s["bias"], s["w_gate"], s["w_up"], s["w_down"],
                         top_k=k, max_tokens=T, n_shared=case["shared"])
        s["layer"].workspace(T)
        s["out"] = torch.empty_like(x)
    return s


# ------------------------------------------------------------------------------ plain form
def _plain_quantise(w):
    v = w.float().view(w.shape[0], -1, 32)
    amax = v.abs().amax(dim=2, keepdim=True)
    exp = torch.frexp(amax).exponent - 3  # floor(log2 amax) - 2
    exp = torch.where(amax > 0, exp, torch.full_like(exp, -127)).clamp(-127, 125)
    a = torch.ldexp(v.abs(), -exp)
    # nearest of the eight magnitudes, ties to the even code, saturating at 6
    mag = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) \
        + (a >= 3.5).float() + 2.0 * (a > 5.0)
    return torch.ldexp(torch.copysign(mag, v), exp).view_as(w).to(w.dtype)


def _plain_matrix(w, g):
    """fp32 weights of expert g."""
    if not isinstance(w, tuple):
        return w[g].float()
    codes, scales = w[0][g], w[1][g]
    lut = torch.tensor(_MAG + tuple(-m for m in _MAG), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), dim=2).int()
    val = lut[pair].view(codes.shape[0], -1, 32)
    return torch.ldexp(val, scales.int().unsqueeze(2) - 127).view(codes.shape[0], -1)


def _plain_expert(s, g, xe):
    a = xe @ _plain_matrix(s["w_gate"], g).T
    b = xe @ _plain_matrix(s["w_up"], g).T
    h = a / (1.0 + torch.exp(-a)) * b
    return h @ _plain_matrix(s["w_down"], g).T


def _plain_layer(s):
    case, x = s["case"], s["x"].float()
    E, k = case["E"], case["k"]
    logits = x @ s["w_router"].float().T
    idx = torch.argsort(logits + s["bias"], dim=1, descending=True, stable=True)[:, :k]
    sel = logits.gather(1, idx)
    p = torch.exp(sel - sel.amax(dim=1, keepdim=True))
    gate = p / p.sum(dim=1, keepdim=True)
    out = torch.zeros_like(x)
    for e in torch.unique(idx).tolist():
        tok, slot = (idx == e).nonzero(as_tuple=True)
        out[tok] += gate[tok, slot].unsqueeze(1) * _plain_expert(s, e, x[tok])
    if case["shared"]:
        out += _plain_expert(s, E, x)
    return out.to(torch.bfloat16)


def run(state):
    op = state["case"]["op"]
    if not own:
        return _plain_quantise(state["w"]) if op == "quantise" else _plain_layer(state)
    import sparse_moe_layer_warp_b200 as moe

    if op == "quantise":
        codes, scales = moe.mxfp4_quantize(state["w"])
        return moe.mxfp4_dequantize(codes, scales, dtype=state["w"].dtype)
    if op == "few":
        return state["layer"].forward_few(state["x"], out=state["out"])
    return state["layer"].forward(state["x"], out=state["out"])


# ------------------------------------------------------------------------------ 64 bits
def _exact_block_values(w):
    """Definition of the quantisation by the distance to every magnitude, in fp64."""
    grid = torch.tensor(_MAG, dtype=torch.float64, device=w.device)
    mid = (grid[1:] + grid[:-1]) / 2
    v = w.double().reshape(-1, 32)
    amax = v.abs().max(dim=1, keepdim=True).values
    s = torch.exp2(torch.clamp(torch.floor(torch.log2(amax)) - 2, -127, 125))
    s = torch.where(amax == 0, torch.full_like(s, 2.0 ** -127), s)
    a = v.abs() / s
    code = torch.bucketize(a, mid)  # mid[i-1] < a <= mid[i]: a tie goes down
    tie_up = (a == mid[code.clamp(max=6)]) & (code < 7) & (code % 2 == 1)
    q = grid[code + tie_up.long()] * s
    return torch.where(v < 0, -q, q).reshape(w.shape)


def _exact_matrix(w, g):
    if not isinstance(w, tuple):
        return w[g].double()
    codes, scales = w[0][g].long(), w[1][g].double()
    grid = torch.tensor(_MAG, dtype=torch.float64, device=codes.device)
    nib = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=torch.long,
                      device=codes.device)
    nib[:, 0::2] = codes % 16
    nib[:, 1::2] = codes // 16
    val = torch.where(nib >= 8, -grid[nib % 8], grid[nib % 8])
    return val * torch.exp2(scales - 127.0).repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        out = torch.empty_like(s["w"], dtype=torch.float64)
        step = max(1, 50_000_000 // case["cols"])
        for r in range(0, case["rows"], step):
            out[r:r + step] = _exact_block_values(s["w"][r:r + step])
        return out
    x = s["x"].double()
    logits = x @ s["w_router"].double().T
    score = logits + s["bias"].double()
    chosen = score.topk(case["k"], dim=1).indices
    gates = torch.zeros_like(logits).scatter_(
        1, chosen, torch.softmax(logits.gather(1, chosen), dim=1))
    out = torch.zeros_like(x)
    for g in range(case["E"] + case["shared"]):
        if g < case["E"]:
            rows = torch.nonzero(gates[:, g] > 0).flatten()
            if rows.numel() == 0:
                continue
            weight = gates[rows, g].unsqueeze(1)
        else:
            rows = torch.arange(x.shape[0], device=x.device)
            weight = 1.0
        xe = x[rows]
        a = xe @ _exact_matrix(s["w_gate"], g).T
        h = a * torch.sigmoid(a) * (xe @ _exact_matrix(s["w_up"], g).T)
        out[rows] += weight * (h @ _exact_matrix(s["w_down"], g).T)
    return out


# ------------------------------------------------------------------------------ work
def _touched(E, k, T):
    """Expected number of routed experts that T tokens reach under even routing."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    if case["op"] == "quantise":
        n = case["rows"] * case["cols"]
        held = n / 2 + n / 32
        # read the matrix, write codes and scales, read them, write the values
        return dict(bytes=2 * n * (2 if case["dtype"] == "bf16" else 4) + 2 * held,
                    flops=4.0 * n)
    T, d, E, k, f = (case[n] for n in ("T", "d", "E", "k", "f"))
    per = 2.0 if case.get("weights") == "bf16" else 0.5 + 1.0 / 32
    experts = (_touched_skewed(E, k, T) if case["bias"] == "zipf" else _touched(E, k, T))
    nbytes = (experts + case["shared"]) * 3 * d * f * per + E * d * 2 + 2 * T * d * 2
    flops = 2.0 * T * (k + case["shared"]) * 3 * d * f + 2.0 * T * d * E
    return dict(bytes=nbytes, flops=flops)


def _touched_skewed(E, k, T):
    """The same with probabilities proportional to rank^-1.1 for each of the k picks."""
    p = [r ** -1.1 for r in range(1, E + 1)]
    z = sum(p)
    return sum(1.0 - (1.0 - min(1.0, k * q / z)) ** T for q in p)
