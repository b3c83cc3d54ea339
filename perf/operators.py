"""The FP8 operators (E4M3 values, one fp32 scale per block of 128) as they are measured.

  fp8_quantize  bf16 / fp32 -> E4M3 with a scale per 1 x 128 row group or per 128 x 128 block
  fp8_gemm      D = A . B^T, A scaled per row and 128 columns, B per 128 x 128 block
  FP8MoeFFN     the routed feed-forward layer on such weights: top-k, gate/up, SwiGLU, down, combine

Sizes are the framework's own routed and dense workloads (hidden 2048 / 4096 / 5120, expert width
512 / 1024 / 17408, 16 decode rows, 512-token prefill chunks, 4096-token prefill) and ragged ones.
"""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0


# ------------------------------------------------------------------------------- the cases ----
def listed():
    return [
        # the decode step's 16 rows before a product: latency alone
        dict(name="quantize_decode", op="quantize", rows=16, K=2048, tile="rows", dtype="bf16"),
        # a 4096-token prefill's activations
        dict(name="quantize_prefill", op="quantize", rows=4096, K=5120, tile="rows", dtype="bf16"),
        # preparing a weight matrix from fp32, sizes that end inside a block
        dict(name="quantize_weights", op="quantize", rows=17400, K=5004, tile="blocks", dtype="f32"),
        # one decode row against a dense projection: every weight byte once
        dict(name="gemm_row", op="gemm", M=1, N=17408, K=5120, dtype="bf16"),
        # a batch of rows that ends inside every tile, fp32 out
        dict(name="gemm_ragged", op="gemm", M=77, N=2070, K=1003, dtype="f32"),
        # a decode batch against a square projection: few tiles, a long sum
        dict(name="gemm_batch", op="gemm", M=64, N=4096, K=4096, dtype="bf16"),
        # the dense layer's down projection at prefill: compute bound
        dict(name="gemm_prefill", op="gemm", M=4096, N=5120, K=17408, dtype="bf16"),
        # one token through 512 experts, ten of them touched
        dict(name="moe_token", op="moe", T=1, H=2048, I=512, E=512, k=10, zipf=0.0),
        # the decode batch
        dict(name="moe_decode", op="moe", T=16, H=2048, I=512, E=512, k=10, zipf=0.0),
        # a batch between decode and prefill on sizes that end inside a block
        dict(name="moe_ragged", op="moe", T=45, H=1040, I=336, E=20, k=3, zipf=0.0),
        # a prefill chunk with popular experts
        dict(name="moe_chunk", op="moe", T=512, H=2048, I=512, E=512, k=10, zipf=1.1),
        # a long prefill: compute bound
        dict(name="moe_prefill", op="moe", T=4096, H=4096, I=1024, E=256, k=8, zipf=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "moe", "moe"])
    if op == "quantize":
        rows = _log(rng, 1, 17408)
        return dict(op=op, rows=rows, K=_log(rng, 128, 17408), tile=rng.choice(["rows", "blocks"]),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "gemm":
        N, K = _log(rng, 256, 17408), _log(rng, 256, 17408)
        M = _log(rng, 1, max(1, min(8192, 4096 * 5120 * 17408 // (N * K))))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "f32"]))
    H, I = 16 * _log(rng, 16, 256), 16 * _log(rng, 8, 64)
    E = _log(rng, 1, 512)
    while E * H * I > 1 << 30:
        E = max(1, E // 2)
    k = rng.randint(1, min(E, 10))
    T = _log(rng, 1, max(1, min(4096, (4096 * 8 * 4096 * 1024) // (k * H * I))))
    return dict(op=op, T=T, H=H, I=I, E=E, k=k, zipf=rng.choice([0.0, 0.0, 1.1]) if T <= 512 else 0.0)


def _logits(T, E, zipf, gen, device):
    """Router logits N(0, 1), with a Zipf popularity bias over a random ranking of the experts."""
    lg = torch.randn(T, E, generator=gen, device=device)
    if zipf > 0:
        p = (torch.randperm(E, generator=gen, device=device).double() + 1.0).pow(-zipf)
        lg += torch.log(p / p.sum()).float()
    return lg


def work(case):
    """Bytes: every input once and every output once (for the layer, the weights of the experts that
    a batch of these sizes touches); flops: two per product term."""
    c = case
    nb = lambda n: -(-n // BLOCK)  # noqa: E731
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        scales = (c["rows"] if c["tile"] == "rows" else nb(c["rows"])) * nb(c["K"])
        return dict(bytes=n * (2 if c["dtype"] == "bf16" else 4) + n + 4 * scales, flops=2 * n)
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        scales = (M + nb(N)) * nb(K)
        return dict(bytes=M * K + N * K + 4 * scales + M * N * (2 if c["dtype"] == "bf16" else 4),
                    flops=2 * M * N * K)
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    lg = _logits(T, E, c["zipf"], torch.Generator().manual_seed(0), "cpu")
    active = torch.topk(lg, k, dim=1).indices.unique().numel()
    weights = active * (3 * H * I + 4 * (2 * nb(I) * nb(H) + nb(H) * nb(I)))
    return dict(bytes=weights + 2 * T * H * 2 + 4 * T * E, flops=6 * T * k * H * I)


# ----------------------------------------------------------------------- the plain forms ----
def _groups(x, rows):
    """x [..., R, K] padded with zeros to whole groups, as [..., R / rows, rows, K / 128, 128]."""
    R, K = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -R % rows))
    return x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, rows))


def _quantize(x, rows):
    """E4M3 values (held in fp32, shaped like x) and fp32 scales of the groups of rows x 128.
    Quotients are formed and rounded in 64 bits: the grid's borders are values of few bits."""
    R, K = x.shape[-2:]
    g = _groups(x.float(), rows)
    s = (g.abs().amax(dim=(-3, -1)).double() / FP8_MAX).float()
    q = g.double() / s.double()[..., :, None, :, None]
    q = torch.where(s[..., :, None, :, None] == 0, torch.zeros_like(q), q)
    power = (q.view(torch.int64) & 0x7FF0000000000000).view(torch.float64)  # the power of two at or below |q|
    step = power.clamp(min=2.0 ** -6) / 8                                   # 4 significant bits
    q = (torch.round(q / step) * step).clamp(-FP8_MAX, FP8_MAX).float()
    return q.flatten(-4, -3).flatten(-2, -1)[..., :R, :K], s


def _spread(s, rows, R, K):
    """Scales [..., R / rows, K / 128] repeated over their groups, [..., R, K]."""
    return s.repeat_interleave(rows, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :K]


def _values(codes, s, rows):
    return codes.float() * _spread(s, rows, *codes.shape[-2:])


def _plain_gemm(a, sa, b, sb, dtype):
    return (_values(a, sa, 1) @ _values(b, sb, BLOCK).T).to(dtype)


def _plain_moe(x, logits, w13, s13, w2, s2, k):
    """The layer over padded per-expert groups [active experts, most tokens of one, ...], in fp32."""
    T, E = logits.shape
    I = w13.shape[2]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)  # ties to the lower expert
    top, ids = top[:, :k], ids[:, :k]
    p = torch.exp(top - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    flat = ids.flatten()
    order = torch.sort(flat, stable=True).indices             # pairs in expert order
    counts = torch.bincount(flat, minlength=E)
    active = counts.nonzero().flatten()
    first = counts.cumsum(0) - counts
    expert = flat[order]
    slot = torch.arange(T * k, device=x.device) - first[expert]
    group = torch.zeros(E, dtype=torch.int64, device=x.device)
    group[active] = torch.arange(active.numel(), device=x.device)
    xq, xs = _quantize(x, 1)
    rows = torch.zeros(active.numel(), int(counts.max()), x.shape[1], device=x.device)
    rows[group[expert], slot] = (xq * _spread(xs, 1, *xq.shape))[order // k]
    gu = rows @ _values(w13[active], s13[active], BLOCK).flatten(1, 2).transpose(1, 2)
    gate, up = gu[..., :I], gu[..., I:]
    hq, hs = _quantize(gate / (1 + torch.exp(-gate)) * up, 1)
    y = (hq * _spread(hs, 1, *hq.shape[-2:])) @ _values(w2[active], s2[active], BLOCK).transpose(1, 2)
    pairs = torch.empty(T * k, y.shape[2], device=x.device)
    pairs[order] = y[group[expert], slot]
    return (pairs.view(T, k, -1) * p[..., None]).sum(1).to(torch.bfloat16)


# ----------------------------------------------------------------------- inputs and passes ----
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(rows, K, gen):
    """N(0, 1) with one channel in a hundred twenty times as large."""
    x = torch.randn(rows, K, generator=gen, device="cuda")
    x[:, torch.randperm(K, generator=gen, device="cuda")[: K // 100]] *= 20.0
    return x


def _matrix(x, rows):
    """x as an E4M3 matrix whose rows start every multiple of 16 bytes, and its scales."""
    q, s = _quantize(x, rows)
    pitch = -(-x.shape[-1] // 16) * 16
    codes = torch.zeros(*x.shape[:-1], pitch, dtype=torch.float8_e4m3fn, device="cuda")
    codes[..., : x.shape[-1]] = q.to(torch.float8_e4m3fn)
    return codes[..., : x.shape[-1]], s


def _expert_weights(E, N, K, gen):
    """E matrices [N, K] of N(0, 1 / K), a few experts at a time."""
    codes = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), device="cuda")
    some = max(1, (1 << 27) // (N * K))
    for e in range(0, E, some):
        w = torch.randn(min(some, E - e), N, K, generator=gen, device="cuda") / math.sqrt(K)
        q, scales[e:e + some] = _quantize(w, BLOCK)
        codes[e:e + some] = q.to(torch.float8_e4m3fn)
    return codes, scales


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    if c["op"] == "quantize":
        x = _activations(c["rows"], c["K"], gen) if c["tile"] == "rows" else \
            torch.randn(c["rows"], c["K"], generator=gen, device="cuda") / math.sqrt(c["K"])
        return dict(c, x=x.to(_DTYPE[c["dtype"]]))
    if c["op"] == "gemm":
        a, sa = _matrix(_activations(c["M"], c["K"], gen).to(torch.bfloat16), 1)
        b, sb = _matrix(torch.randn(c["N"], c["K"], generator=gen, device="cuda") / math.sqrt(c["K"]), BLOCK)
        return dict(c, a=a, sa=sa, b=b, sb=sb)
    x = _activations(c["T"], c["H"], gen).to(torch.bfloat16)
    logits = _logits(c["T"], c["E"], c["zipf"], gen, "cuda")
    w13, s13 = _expert_weights(c["E"] * 2, c["I"], c["H"], gen)   # gate then up of each expert
    w2, s2 = _expert_weights(c["E"], c["H"], c["I"], gen)
    state = dict(c, x=x, logits=logits, w13=w13.unflatten(0, (-1, 2)), s13=s13.unflatten(0, (-1, 2)), w2=w2, s2=s2)
    if own:  # the handle a program keeps: the weights as they are, and a workspace
        from nvfp4_mixture_experts_w4a4_b200 import ops
        state["layer"] = ops.FP8MoeFFN(ops.FP8Experts(state["w13"], state["s13"], w2, s2), c["k"])
    return state


def run(state):
    s = state
    if own:
        from nvfp4_mixture_experts_w4a4_b200 import ops
        if s["op"] == "quantize":
            return ops.fp8_quantize(s["x"], tile=ops.FP8_ROWS if s["tile"] == "rows" else ops.FP8_BLOCKS)
        if s["op"] == "gemm":
            return ops.fp8_gemm(s["a"], s["sa"], s["b"], s["sb"], out_dtype=_DTYPE[s["dtype"]])
        return s["layer"](s["x"], s["logits"])
    if s["op"] == "quantize":
        q, scale = _quantize(s["x"], 1 if s["tile"] == "rows" else BLOCK)
        return q.to(torch.float8_e4m3fn), scale
    if s["op"] == "gemm":
        return _plain_gemm(s["a"], s["sa"], s["b"], s["sb"], _DTYPE[s["dtype"]])
    return _plain_moe(s["x"], s["logits"], s["w13"], s["s13"], s["w2"], s["s2"], s["k"])


# -------------------------------------------------------------------------------- in 64 bits ----
def _grid():
    """Every non-negative E4M3 value, ascending."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_codes(x, s):
    """The grid value nearest to x / s (elementwise; ties to the even code)."""
    grid = _grid()
    q = torch.where(s == 0, torch.zeros_like(x), x / torch.where(s == 0, torch.ones_like(s), s))
    a = q.abs()
    border = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(border, a.contiguous())             # borders strictly below a
    tie = (i < border.numel()) & (border[i.clamp(max=border.numel() - 1)] == a)
    i = torch.where(tie & (i % 2 == 1), i + 1, i)
    return torch.copysign(grid[i], q)


def _exact_rows(x):
    """x [R, K] in 64 bits -> its row-quantised values' codes and the scales spread over the columns."""
    codes, scale = torch.empty_like(x), torch.empty_like(x)
    for j in range(0, x.shape[1], BLOCK):
        part = x[:, j:j + BLOCK]
        s = (part.abs().amax(1, keepdim=True) / FP8_MAX).float().double()
        codes[:, j:j + BLOCK] = _exact_codes(part, s.expand_as(part))
        scale[:, j:j + BLOCK] = s
    return codes, scale


def _wide(codes, s):
    """A block-scaled matrix [N, K] in 64 bits."""
    w = codes.double()
    for i in range(s.shape[0]):
        w[i * BLOCK:(i + 1) * BLOCK] *= s[i].double().repeat_interleave(BLOCK)[: w.shape[1]]
    return w


def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e14:
        return None
    s = prepare(c, seed)
    if c["op"] == "quantize":
        x = s["x"]
        R, K = x.shape
        rows = 1 if c["tile"] == "rows" else BLOCK
        codes = torch.empty(R, K, dtype=torch.float64, device="cuda")
        scale = torch.empty(-(-R // rows), -(-K // BLOCK), dtype=torch.float64, device="cuda")
        for j in range(scale.shape[1]):
            part = x[:, j * BLOCK:(j + 1) * BLOCK].double()
            most = part.abs().amax(1)
            if rows > 1:
                most = torch.stack([m.amax() for m in most.split(rows)])
            scale[:, j] = most / FP8_MAX
            used = scale[:, j].float().double().repeat_interleave(rows)[:R, None].expand_as(part)
            codes[:, j * BLOCK:(j + 1) * BLOCK] = _exact_codes(part, used)
        return codes, scale
    if c["op"] == "gemm":
        a = s["a"].double()
        for j in range(s["sa"].shape[1]):
            a[:, j * BLOCK:(j + 1) * BLOCK] *= s["sa"][:, j:j + 1].double()
        return a @ _wide(s["b"], s["sb"]).T
    T, k = c["T"], c["k"]
    lg = s["logits"].double()
    chosen = []
    for _ in range(k):                                           # the largest left, lowest index first
        best = lg.amax(1, keepdim=True)
        at = torch.where(lg == best, torch.arange(c["E"], device="cuda"), c["E"]).amin(1, keepdim=True)
        chosen.append((at, best))
        lg = lg.scatter(1, at, -math.inf)
    ids = torch.cat([a for a, _ in chosen], 1)
    p = torch.softmax(torch.cat([b for _, b in chosen], 1), 1)
    xc, xs = _exact_rows(s["x"].double())
    x = xc * xs
    out = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        g = x[t] @ _wide(s["w13"][e, 0], s["s13"][e, 0]).T
        u = x[t] @ _wide(s["w13"][e, 1], s["s13"][e, 1]).T
        hc, hs = _exact_rows(g * torch.sigmoid(g) * u)
        out.index_add_(0, t, p[t, j][:, None] * ((hc * hs) @ _wide(s["w2"][e], s["s2"][e]).T))
    return out
