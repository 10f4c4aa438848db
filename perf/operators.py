"""The operators around the routed experts, as cases to measure: their plain forms in torch and the library's kernels.

Four operators, in the order a batch meets them:

  balance    the load-balance loss of a router with its per-expert counts and
             the loss's gradient with respect to the logits;
  quantize   E4M3 codes with one fp32 scale for each 1 x 128 piece of a row
             (activations) or each 128 x 128 block (weights);
  matmul     the product of two such matrices, dense or grouped by expert;
  swiglu     an expert's first half: gate and up products, SiLU(gate) * up, and
             the hidden rows quantised for the next product.

`own` chooses the library's kernels; without it `run` computes the plain form.
"""
import math

import torch

own = False

BLOCK = 128      # elements that share a scale along K, and rows of a weight block
E4M3_MAX = 448.0
ROWS = 4096      # rows of weights drawn at once by prepare()


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step of 32 sequences through an 8-expert router: all latency
        dict(name="balance T32 E8 k2", op="balance", T=32, E=8, k=2, dtype="f32", gate=0, seqs=1, masked=0.0, seed_skew=0.0),
        # a top-1 router with skewed load, bf16 logits, a batch of ragged sequences with padding tokens
        dict(name="balance T16384 E64 ragged", op="balance", T=16384, E=64, k=1, dtype="bf16", gate=0, seqs=37, masked=0.1, seed_skew=1.2),
        # many fine-grained experts with sigmoid affinities, one loss per sequence, a training batch
        dict(name="balance T32768 E256 k8", op="balance", T=32768, E=256, k=8, dtype="f32", gate=2, seqs=8, masked=0.0, seed_skew=0.5),
        # one token's activations before an expert product: all latency
        dict(name="quantize 1x7168", op="quantize", stack=1, rows=1, cols=7168, block_rows=1, dtype="bf16"),
        # a prefill batch's activations
        dict(name="quantize 8192x7168", op="quantize", stack=1, rows=8192, cols=7168, block_rows=1, dtype="bf16"),
        # a stack of expert weights, once when a model is loaded
        dict(name="quantize 8x14336x4096 w", op="quantize", stack=8, rows=14336, cols=4096, block_rows=128, dtype="bf16"),
        # one token through one wide projection: streaming the weights
        dict(name="matmul 1x14336x4096", op="matmul", M=1, N=14336, K=4096, E=0, skew=0.0, out="bf16", gates=False),
        # a dense (shared) expert's down projection over a prefill batch
        dict(name="matmul 8192x7168x2048", op="matmul", M=8192, N=7168, K=2048, E=0, skew=0.0, out="bf16", gates=False),
        # 32 decoding tokens, 8 experts each of 256: a row or two per expert, many without any
        dict(name="matmul 256 rows E256", op="matmul", M=256, N=2048, K=7168, E=256, skew=0.3, out="bf16", gates=False),
        # the down projections of 8 wide experts over a prefill batch, gate-weighted
        dict(name="matmul 8192 rows E8", op="matmul", M=8192, N=4096, K=14336, E=8, skew=0.2, out="bf16", gates=True),
        # the gate and up projections of 8 wide experts, 32 decoding tokens
        dict(name="swiglu 64 rows E8", op="swiglu", M=64, N=14336, K=4096, E=8, skew=0.2),
        # the same over a prefill batch: the layer's largest product
        dict(name="swiglu 8192 rows E8", op="swiglu", M=8192, N=14336, K=4096, E=8, skew=0.2),
    ]


def draw(rng):
    def spread(lo, hi):  # evenly over the logarithm
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["balance", "quantize", "matmul", "matmul", "swiglu"])
    if op == "balance":
        E = spread(2, 512)
        return dict(op=op, T=spread(1, min(65536, 8_000_000 // E)), E=E, k=rng.randint(1, min(8, E - 1)),
                    dtype=rng.choice(["f32", "bf16"]), gate=rng.randint(0, 2), seqs=spread(1, 64),
                    masked=rng.choice([0.0, 0.1, 0.5]), seed_skew=round(rng.uniform(0.0, 1.5), 2))
    if op == "quantize":
        weights = rng.random() < 0.5
        return dict(op=op, stack=rng.randint(1, 4) if weights else 1, rows=spread(1, 8192), cols=16 * spread(1, 512),
                    block_rows=128 if weights else 1, dtype=rng.choice(["f32", "bf16"]))
    M, N, K = spread(1, 8192), spread(8, 8192), 16 * spread(4, 512)
    E = rng.choice([0, 1, spread(2, 64)]) if op == "matmul" else rng.choice([1, spread(2, 64)])
    N, K = min(N, max(8, 2_000_000_000 // (max(1, E) * K))), K
    if op == "swiglu":
        return dict(op=op, M=min(M, 4096), N=16 * max(1, N // 16), K=K, E=E, skew=round(rng.uniform(0.0, 1.0), 2))
    return dict(op=op, M=M, N=N, K=K, E=E, skew=round(rng.uniform(0.0, 1.0), 2),
                out=rng.choice(["bf16", "bf16", "f32"]), gates=rng.random() < 0.5)


# ----------------------------------------------------------------- the inputs
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _gen(seed):
    return torch.Generator(device=_device()).manual_seed(seed)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _cut(total, parts, skew, g):
    """Lengths of `parts` consecutive runs that add up to `total`: even at skew 0, some empty at 1."""
    w = torch.exp(2.0 * skew * torch.randn(parts, generator=g, device=_device())).double()
    ends = torch.round(torch.cumsum(w, 0) / w.sum() * total).long().clamp_(0, total)
    ends[-1] = total
    return torch.cat([ends.new_zeros(1), ends]).to(torch.int32)


def _routed(total, parts, skew, g):
    """Row counts per expert as a router gives them: each row falls to an expert at random."""
    w = torch.exp(2.0 * skew * torch.randn(parts, generator=g, device=_device()))
    to = torch.multinomial(w, total, replacement=True, generator=g)
    counts = torch.zeros(parts, dtype=torch.int64, device=to.device).index_add_(0, to, torch.ones_like(to))
    return torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)


def _weights(stack, rows, cols, g):
    """A stack of quantised weights of standard deviation 1 / sqrt(cols): codes and block scales."""
    codes = torch.empty(stack, rows, cols, dtype=torch.uint8, device=_device())
    nb, kb = -(-rows // BLOCK), -(-cols // BLOCK)
    scales = torch.empty(stack, nb, kb, dtype=torch.float32, device=_device())
    for e in range(stack):
        for r in range(0, rows, ROWS):
            n = min(ROWS, rows - r)
            w = torch.randn(n, cols, generator=g, device=_device()) / math.sqrt(cols)
            c, s = _quantize_plain(w[None], BLOCK)
            codes[e, r:r + n] = c[0]
            scales[e, r // BLOCK:r // BLOCK + s.shape[1]] = s[0]
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    dev = _device()
    c = dict(case)
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        # a router's logits: unit spread, and a popularity of the experts that falls off with their rank
        pop = -c["seed_skew"] * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
        logits = (torch.randn(T, E, generator=g, device=dev) + pop).to(_dtype(c["dtype"]))
        idx = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
        mask = None
        if c["masked"] > 0:
            mask = torch.rand(T, generator=g, device=dev) >= c["masked"]
        cu = None if c["seqs"] == 1 else _cut(T, c["seqs"], 0.4, g)
        dloss = torch.rand(c["seqs"], generator=g, device=dev) * 0.01
        return dict(c=c, logits=logits, idx=idx, mask=mask, cu=cu, dloss=dloss)
    if c["op"] == "quantize":
        w = torch.empty(c["stack"], c["rows"], c["cols"], dtype=_dtype(c["dtype"]), device=dev)
        for e in range(c["stack"]):
            w[e] = torch.randn(c["rows"], c["cols"], generator=g, device=dev)
        # a few channels of large values, as activations and their weights have
        w[:, :, :: max(1, c["cols"] // 7)] *= 20
        return dict(c=c, w=w if c["block_rows"] > 1 else w[0])
    E, M, N, K = c["E"], c["M"], c["N"], c["K"]
    offsets = _routed(M, E, c["skew"], g) if E else None
    most = int((offsets[1:] - offsets[:-1]).max()) if E else M
    x = torch.randn(M, K, generator=g, device=dev)
    x[:, :: max(1, K // 5)] *= 20
    a, a_scales = _quantize_plain(x[None], 1)
    s = dict(c=c, a=a[0], a_scales=a_scales[0], offsets=offsets, most=most)
    names = ("W_g", "W_u") if c["op"] == "swiglu" else ("W",)
    for name in names:
        codes, scales = _weights(max(1, E), N, K, g)
        s[name], s[name + "_scales"] = (codes, scales) if E else (codes[0], scales[0])
    if c["op"] == "matmul":
        s["out"] = torch.zeros(M, N, dtype=_dtype(c["out"]), device=dev)
        s["gates"] = torch.rand(M, generator=g, device=dev) if c["gates"] else None
    return s


# ------------------------------------------------------------- the plain forms
def _balance_plain(logits, idx, gate, mask, cu, dloss):
    T, E = logits.shape
    k = idx.shape[1]
    r = logits.float()
    seqs = dloss.shape[0]
    t = torch.arange(T, device=r.device)
    seq = torch.zeros_like(t) if cu is None else torch.searchsorted(cu.long(), t, right=True) - 1
    live = torch.ones(T, dtype=torch.bool, device=r.device) if mask is None else mask
    member = torch.zeros(seqs, T, dtype=torch.float64, device=r.device)
    member[seq, t] = live.double()
    if gate == 2:
        z = torch.clamp(r, max=0.0) - torch.log1p(torch.exp(-r.abs()))  # log sigmoid
        slope = 1.0 / (1.0 + torch.exp(r))                             # 1 - sigmoid
    else:
        z, slope = r, torch.ones_like(r)
    p = torch.exp(z - z.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    n = member.sum(dim=1)
    counts = torch.zeros(seqs * E, dtype=torch.int64, device=r.device)
    counts.index_add_(0, (seq[:, None] * E + idx.long()).reshape(-1), live[:, None].expand(T, k).reshape(-1).long())
    counts = counts.view(seqs, E)
    psum = member @ p.double()
    some = n.clamp(min=1.0)
    loss = E * (counts * psum).sum(dim=1) / (some * some * k)
    # f - 1/E: as the p add up to 1 it gives the same difference as f, without f's cancellation
    f = ((counts * E - (some * k)[:, None]) / (some * k * E)[:, None]).float()[seq]
    scale = (dloss.double() * E / some).float()[seq] * live.float()
    d = scale[:, None] * p * slope * (f - (f * p).sum(dim=1, keepdim=True))
    return dict(loss=loss.float(), counts=counts.to(torch.int32), tokens=n.to(torch.int32), dlogits=d.to(logits.dtype))


def _quantize_plain(w, block_rows):
    """w [stack, rows, cols] -> codes (uint8) and fp32 scales, one for each block_rows x 128 block."""
    stack, rows, cols = w.shape
    nb, kb = -(-rows // block_rows), -(-cols // BLOCK)
    full = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - cols, 0, nb * block_rows - rows))
    full = full.view(stack, nb, block_rows, kb, BLOCK)
    top = full.abs().amax(dim=(2, 4))
    scales = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    codes = (full / scales[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes = codes.view(stack, nb * block_rows, kb * BLOCK)[:, :rows, :cols].contiguous()
    return codes, scales


def _values(codes, scales, block_rows):
    """fp32 values of codes [.., rows, cols] with their block scales."""
    rows, cols = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, dim=-1)[..., :cols]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return codes.view(torch.float8_e4m3fn).float() * s


def _product_plain(a, a_scales, w, w_scales, offsets, most):
    """fp32 rows of the dense or grouped product."""
    x = _values(a, a_scales, 1)
    y = _values(w, w_scales, BLOCK)
    if offsets is None:
        return x @ y.t()
    E, M = y.shape[0], x.shape[0]
    row = torch.arange(M, device=x.device)
    e = torch.searchsorted(offsets.long(), row, right=True) - 1
    at = row - offsets.long()[e]
    padded = x.new_zeros(E, most, x.shape[1])
    padded[e, at] = x
    return torch.bmm(padded, y.transpose(1, 2))[e, at]


# ------------------------------------------------------------------- one pass
def run(s):
    c = s["c"]
    if own:
        import sparse_mixture_experts_aux_b200 as moe
    if c["op"] == "balance":
        if own:
            loss, counts, tokens = moe.balance_loss(s["logits"], s["idx"], gate_mode=c["gate"], token_mask=s["mask"], cu_seqlens=s["cu"])
            d = moe.balance_loss_backward(s["dloss"], s["logits"], counts, tokens, c["k"], gate_mode=c["gate"], token_mask=s["mask"], cu_seqlens=s["cu"])
            return dict(loss=loss, counts=counts, tokens=tokens, dlogits=d)
        return _balance_plain(s["logits"], s["idx"], c["gate"], s["mask"], s["cu"], s["dloss"])
    if c["op"] == "quantize":
        if own:
            codes, scales = moe.quantize_fp8_block(s["w"], block_rows=c["block_rows"])
        else:
            w = s["w"] if c["block_rows"] > 1 else s["w"][None]
            codes, scales = _quantize_plain(w, c["block_rows"])
            codes, scales = codes.view(s["w"].shape), scales if c["block_rows"] > 1 else scales[0]
        return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales)
    if c["op"] == "matmul":
        if own:
            return moe.matmul_fp8_block(s["a"], s["a_scales"], s["W"], s["W_scales"], offsets=s["offsets"], row_scale=s["gates"], out=s["out"])
        y = _product_plain(s["a"], s["a_scales"], s["W"], s["W_scales"], s["offsets"], s["most"])
        s["out"].copy_(y if s["gates"] is None else y * s["gates"][:, None])
        return s["out"]
    if own:
        codes, scales = moe.swiglu_fp8_block(s["a"], s["a_scales"], s["W_g"], s["W_u"], s["W_g_scales"], s["W_u_scales"], offsets=s["offsets"])
    else:
        gate = _product_plain(s["a"], s["a_scales"], s["W_g"], s["W_g_scales"], s["offsets"], s["most"])
        up = _product_plain(s["a"], s["a_scales"], s["W_u"], s["W_u_scales"], s["offsets"], s["most"])
        h = gate / (1.0 + torch.exp(-gate)) * up
        codes, scales = _quantize_plain(h[None], 1)
        codes, scales = codes[0], scales[0]
    return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales)


def work(case):
    c = case
    if c["op"] == "balance":
        size = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["E"]
        # logits in for each direction, gradient out, choices in
        return dict(bytes=3 * n * size + 4 * c["T"] * c["k"] + 8 * c["seqs"] * c["E"], flops=16 * n)
    if c["op"] == "quantize":
        n = c["stack"] * c["rows"] * c["cols"]
        scales = c["stack"] * -(-c["rows"] // c["block_rows"]) * -(-c["cols"] // BLOCK)
        return dict(bytes=n * ((2 if c["dtype"] == "bf16" else 4) + 1) + 4 * scales, flops=3 * n)
    M, N, K = c["M"], c["N"], c["K"]
    E = max(1, c["E"])
    used = min(E, M)  # experts that any row can reach
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    mats = 2 if c["op"] == "swiglu" else 1
    read = M * K + 4 * M * kb + mats * used * (N * K + 4 * nb * kb)
    written = M * N + 4 * M * nb if c["op"] == "swiglu" else M * N * (2 if c["out"] == "bf16" else 4)
    return dict(bytes=read + written, flops=2.0 * mats * M * N * K)


# ------------------------------------------------- the definitions in 64 bits
def _round_e4m3(v):
    """Nearest E4M3 value (ties to even, saturating) of each fp64 value."""
    _, e = torch.frexp(v.abs())
    step = torch.exp2((e.clamp(min=-5) - 4).double())  # 4 significant bits, subnormals below 2^-6
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(x, block_rows=1):
    """E4M3 values and scales of fp64 rows, one scale for each block."""
    rows, cols = x.shape
    codes, scales = [], []
    for k in range(0, cols, BLOCK):
        part = x[:, k:k + BLOCK]
        top = part.abs().amax(dim=1)
        if block_rows > 1:
            pad = -(-rows // block_rows) * block_rows - rows
            top = torch.cat([top, top.new_zeros(pad)]).view(-1, block_rows).amax(dim=1)
        sc = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        scales.append(sc)
        per_row = sc if block_rows == 1 else sc.repeat_interleave(block_rows)[:rows]
        codes.append(_round_e4m3(part / per_row[:, None]))
    return torch.cat(codes, dim=1), torch.stack(scales, dim=1)


def _exact_matrix(codes, scales, block_rows):
    """fp64 matrix of one set of codes, block by block along K."""
    out = codes.view(torch.float8_e4m3fn).double()
    for k in range(scales.shape[1]):
        s = scales[:, k].double()
        if block_rows > 1:
            s = s.repeat_interleave(block_rows)[:out.shape[0]]
        out[:, k * BLOCK:(k + 1) * BLOCK] *= s[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "balance":
        r, idx, mask = s["logits"].double(), s["idx"].long(), s["mask"]
        T, E = r.shape
        cuts = [0, T] if s["cu"] is None else s["cu"].tolist()
        loss, counts, tokens = [], [], []
        d = torch.zeros_like(r)
        for i, (b, e) in enumerate(zip(cuts[:-1], cuts[1:])):
            live = torch.arange(b, e, device=r.device)
            if mask is not None:
                live = live[mask[b:e]]
            n = live.numel()
            count = torch.bincount(idx[live].reshape(-1), minlength=E)
            counts.append(count)
            tokens.append(n)
            if n == 0:
                loss.append(0.0)
                continue
            x = r[live].requires_grad_(True)
            with torch.enable_grad():
                if c["gate"] == 2:
                    p = torch.softmax(torch.nn.functional.logsigmoid(x), dim=1)
                else:
                    p = torch.softmax(x, dim=1)
                value = E * (count.double() / (n * c["k"]) * p.mean(dim=0)).sum()
                d[live] = torch.autograd.grad(value, x)[0] * s["dloss"][i].double()
            loss.append(float(value.detach()))
        return dict(loss=torch.tensor(loss, dtype=torch.float64), counts=torch.stack(counts).to(torch.int32),
                    tokens=torch.tensor(tokens, dtype=torch.int32), dlogits=d)
    if c["op"] == "quantize":
        if c["block_rows"] == 1:
            codes, scales = _exact_rows(s["w"].double())
        else:
            both = [_exact_rows(w.double(), c["block_rows"]) for w in s["w"]]
            codes, scales = torch.stack([b[0] for b in both]), torch.stack([b[1] for b in both])
        return dict(codes=codes, scales=scales)
    x = _exact_matrix(s["a"], s["a_scales"], 1)
    cuts = [0, c["M"]] if s["offsets"] is None else s["offsets"].tolist()

    def product(name):
        y = x.new_zeros(c["M"], c["N"])
        for e, (b, t) in enumerate(zip(cuts[:-1], cuts[1:])):
            if t > b:
                w, sc = (s[name][e], s[name + "_scales"][e]) if s["offsets"] is not None else (s[name], s[name + "_scales"])
                y[b:t] = x[b:t] @ _exact_matrix(w, sc, BLOCK).t()
        return y

    if c["op"] == "matmul":
        y = product("W")
        return y if s["gates"] is None else y * s["gates"].double()[:, None]
    g = product("W_g")
    codes, scales = _exact_rows(g * torch.sigmoid(g) * product("W_u"))
    return dict(codes=codes, scales=scales)
