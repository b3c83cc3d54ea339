"""The FP8 operators (E4M3 with a scale per block of 128) on the GPU against their definitions in 64
bits.

Tolerances.  Quantised codes and scales are exact: scale = rn(amax / 448), code = the E4M3 value nearest
to the real quotient.  Products: with S = sum |a b| (scaled values), a tensor-core sum of 128 exact
products is taken to lose at most 2^-22 of S per addition (twice an fp32 half-step), the two scales
cost 2^-24 each and the additions over the blocks nkb 2^-24, so |error| <= (4 * 128 + nkb + 2) 2^-24 S, plus
half a step of the output type, finfo(t).eps / 2 of the value.  The layer: see layer_reference."""
import math
import weakref

import pytest
import torch

from nvfp4_mixture_experts_w4a4_b200 import _lib as C
from nvfp4_mixture_experts_w4a4_b200 import ops

pytestmark = pytest.mark.gpu

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2
F32_HALF = torch.finfo(torch.float32).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def blocks(n):
    return -(-n // 128)


# ---------------------------------------------------------------------- definitions, 64 bits ----
def grid():
    return torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()


def nearest(q):
    """The E4M3 value nearest to q (fp64), ties to the even code, saturating."""
    g = grid()
    a = q.abs()
    mid = (g[1:] + g[:-1]) / 2
    lo = torch.searchsorted(mid, a.contiguous(), right=False)
    hi = torch.searchsorted(mid, a.contiguous(), right=True)   # differs from lo at a tie alone
    i = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
    return torch.copysign(torch.where(a.isnan(), a, g[i]), q)


def spread(s, rows, shape):
    """Scales repeated over their groups."""
    return s.repeat_interleave(rows, 0)[: shape[0]].repeat_interleave(128, 1)[:, : shape[1]]


def quantised(x, rows):
    """(codes as fp64 values, scales as fp64 holding fp32 values) of a matrix."""
    R, K = x.shape
    x = x.double()
    s = torch.empty(-(-R // rows), blocks(K), dtype=torch.float64, device=x.device)
    for i in range(s.shape[1]):
        part = x[:, i * 128:(i + 1) * 128].abs()
        m = part.amax(1)
        pad = torch.zeros(s.shape[0] * rows - R, dtype=torch.float64, device=x.device)
        s[:, i] = torch.cat([m, pad]).view(-1, rows).amax(1)
    s = (s / 448).float().double()
    d = spread(s, rows, x.shape)
    return torch.where(d == 0, torch.zeros_like(x), nearest(x / d)), s


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=777.0, posinf=888.0), torch.nan_to_num(b.double(), nan=777.0, posinf=888.0))


# ------------------------------------------------------------------------------- quantiser ----
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", [ops.FP8_ROWS, ops.FP8_BLOCKS])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 128), (3, 127), (129, 129), (130, 1000), (257, 336), (64, 2048),
                                    (5, 4099)])
def test_quantize(dtype, tile, rows, K):
    x = torch.randn(rows, K, generator=gen(rows + K), device="cuda")
    x[:, ::17] *= 30.0
    x = x.to(dtype)
    codes, scale = ops.fp8_quantize(x, tile=tile)
    q, s = quantised(x, 1 if tile == ops.FP8_ROWS else 128)
    assert codes.shape == x.shape and codes.dtype == torch.float8_e4m3fn and codes.stride(0) % 16 == 0
    assert torch.equal(scale.double(), s)
    assert torch.equal(codes.double(), q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile", [ops.FP8_ROWS, ops.FP8_BLOCKS])
@pytest.mark.parametrize("values", ["borders", "exact scales", "tiny", "subnormal", "huge", "zeros", "not finite"])
def test_quantize_at_the_edges(dtype, tile, values):
    g = gen(11)
    x = torch.randn(200, 700, generator=g, device="cuda")
    power = torch.exp2(torch.randint(-20, 4, x.shape, generator=g, device="cuda").float())
    if values == "borders":            # scale 1: every eighth and sixteenth between codes, small ones too
        x = torch.randint(-255, 256, x.shape, generator=g, device="cuda").float() / 16 * power.clamp(min=2.0 ** -8)
        x[:, ::128], x[::128] = 448.0, 448.0
    elif values == "exact scales":     # amax of 7, 14, ... times a power of two divides exactly
        x = x.bfloat16().float() * power
        x[:, ::128] = 7.0 * torch.exp2(torch.randint(0, 5, x[:, ::128].shape, generator=g, device="cuda").float())
    elif values == "tiny":
        x *= 2.0 ** -110
    elif values == "subnormal":
        x *= 2.0 ** -135
    elif values == "huge":
        x *= 2.0 ** 120
    elif values == "zeros":
        x[:130] = 0.0
        x[130:, :256] = -0.0
    else:
        x[3, 5], x[7, 300], x[140, 699] = math.nan, math.inf, -math.inf
    x = x.to(dtype)
    codes, scale = ops.fp8_quantize(x, tile=tile)
    q, s = quantised(x, 1 if tile == ops.FP8_ROWS else 128)
    assert same(scale, s)
    assert same(codes.float(), q)


def test_quantize_layouts():
    """Batches, pitches, slices and outputs of the caller's own; bytes outside them stay."""
    g = gen(5)
    wide = torch.randn(3, 40, 300, generator=g, device="cuda")
    for x in (wide[:, ::2, 3:260], wide[:, :, :256].bfloat16()[:, 5:], wide[1:2, :1, :200]):
        for tile, rows in ((ops.FP8_ROWS, 1), (ops.FP8_BLOCKS, 128)):
            B, R, K = x.shape
            store = torch.full((B, R + 1, K + 7), 99, dtype=torch.uint8, device="cuda")
            sstore = torch.full((B, -(-R // rows) + 1, blocks(K) + 1), -1.0, device="cuda")
            codes, scale = store[:, :R, :K], sstore[:, :-1, :-1]
            c, s = ops.fp8_quantize(x, tile=tile, codes=codes, scale=scale)
            assert c is codes and s is scale
            for b in range(B):
                q, t = quantised(x[b], rows)
                assert torch.equal(codes[b].clone().view(torch.float8_e4m3fn).double(), q)
                assert torch.equal(scale[b].double(), t)
            assert (store[:, R:] == 99).all() and (store[:, :, K:] == 99).all()
            assert (sstore[:, -1] == -1).all() and (sstore[:, :, -1] == -1).all()
    c, s = ops.fp8_quantize(torch.empty(0, 64, device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0, 1)


def test_quantize_past_32_bits():
    """More than 2^32 elements: the last rows are the last rows."""
    rows, K = 66000, 65552
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, generator=gen(2), device="cuda").bfloat16()
    codes, scale = ops.fp8_quantize(x)
    q, s = quantised(x[-3:], 1)
    assert torch.equal(codes[-3:].double(), q) and torch.equal(scale[-3:].double(), s)
    assert not codes[-4].view(torch.uint8).any()


# --------------------------------------------------------------------------------- product ----
def matrices(M, N, K, seed, pitch=0):
    g = gen(seed)
    a = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    a[:, ::13] *= 20.0
    b = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
    out = []
    for x, tile in ((a, ops.FP8_ROWS), (b, ops.FP8_BLOCKS)):
        store = torch.full((x.shape[0], -(-K // 16) * 16 + pitch), 0x7F, dtype=torch.uint8, device="cuda")
        codes = store.view(torch.float8_e4m3fn)[:, :K]
        out += ops.fp8_quantize(x, tile=tile, codes=codes)
    return out


def check_gemm(d, a, sa, b, sb):
    K = a.shape[1]
    A, B = a.double() * spread(sa.double(), 1, a.shape), b.double() * spread(sb.double(), 128, b.shape)
    ref, size = A @ B.T, A.abs() @ B.abs().T
    half = BF16_HALF if d.dtype == torch.bfloat16 else F32_HALF
    bound = (4 * 128 + blocks(K) + 2) * 2.0 ** -24 * size * (1 + half) + half * ref.abs()
    assert ((d.double() - ref).abs() <= bound).all(), ((d.double() - ref).abs() / bound).max()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 129, 16), (2, 7, 130), (16, 256, 2048), (33, 300, 1003), (77, 2070, 520), (128, 128, 128),
    (129, 257, 272), (200, 1000, 4096), (256, 512, 640), (300, 700, 2000), (513, 1025, 300), (1000, 2048, 512),
    (2500, 640, 144), (5, 4000, 8192),
])
def test_gemm(M, N, K, out_dtype):
    """Every way the product is split: single tiles, 128 and 256 columns, K over clusters, pairs of
    CTAs, sizes that end inside each."""
    a, sa, b, sb = matrices(M, N, K, M + N)
    d = ops.fp8_gemm(a, sa, b, sb, out_dtype=out_dtype)
    check_gemm(d, a, sa, b, sb)
    assert torch.equal(d, ops.fp8_gemm(a, sa, b, sb, out_dtype=out_dtype))
    assert ops.device_status() == 0


def test_gemm_pitches_and_outputs():
    """Rows further apart than their length (NaN bytes between them), views of wider scales, an output
    inside a larger matrix whose surroundings stay, odd pitches and offsets."""
    for M, N, K in ((150, 333, 392), (40, 96, 1000), (700, 520, 256)):
        a, sa, b, sb = matrices(M, N, K, 3, pitch=32)
        wa = torch.full((M, blocks(K) + 3), math.nan, device="cuda")
        wa[:, 1:1 + blocks(K)] = sa
        wb = torch.full((blocks(N), blocks(K) + 2), math.nan, device="cuda")
        wb[:, :blocks(K)] = sb
        for dtype in (torch.bfloat16, torch.float32):
            for left in (0, 1, 16):
                store = torch.full((M + 2, N + 19), -7.0, dtype=dtype, device="cuda")
                out = store[1:-1, left:left + N]
                d = ops.fp8_gemm(a, wa[:, 1:1 + blocks(K)], b, wb[:, :blocks(K)], out=out)
                assert d is out
                check_gemm(d, a, sa, b, sb)
                keep = torch.ones_like(store, dtype=torch.bool)
                keep[1:-1, left:left + N] = False
                assert (store[keep] == -7).all()
    a, sa, b, sb = matrices(4, 8, 64, 1)
    assert ops.fp8_gemm(a[:0], sa[:0], b, sb).shape == (0, 8)
    assert torch.equal(ops.fp8_gemm(a.view(torch.uint8), sa, b.view(torch.uint8), sb), ops.fp8_gemm(a, sa, b, sb))


def test_gemm_keeps_rows_and_blocks_apart():
    """A NaN or infinite scale, or a NaN code, of one row stays in that row; of one block of B in its
    columns; a zero scale gives zeros."""
    a, sa, b, sb = matrices(300, 520, 384, 9)
    clean = ops.fp8_gemm(a, sa, b, sb, out_dtype=torch.float32)
    sa, sb, a = sa.clone(), sb.clone(), a.clone()
    sa[7, 1], sa[150] = math.nan, 0.0
    a.view(torch.uint8)[290, 5] = 0x7F
    sb[2, 0] = math.inf                     # columns 256..383
    d = ops.fp8_gemm(a, sa, b, sb, out_dtype=torch.float32)
    rows = torch.tensor([r for r in range(300) if r not in (7, 150, 290)], device="cuda")
    cols = torch.tensor([c for c in range(520) if not 256 <= c < 384], device="cuda")
    assert torch.equal(d[rows][:, cols], clean[rows][:, cols])
    assert d[7].isnan().all() and d[290].isnan().all()
    assert (d[150][cols] == 0).all()
    assert not d[rows][:, 256:384].isfinite().any()


def test_gemm_output_past_32_bits():
    M, N, K = 70000, 33000, 32
    a, sa, b, sb = matrices(M, N, K, 4)
    d = ops.fp8_gemm(a, sa, b, sb)
    for r in (0, 35000, M - 130):
        check_gemm(d[r:r + 130], a[r:r + 130], sa[r:r + 130], b, sb)


def test_gemm_needs_aligned_rows():
    a, sa, b, sb = matrices(4, 8, 64, 1)
    odd = torch.zeros(4, 72, dtype=torch.float8_e4m3fn, device="cuda")[:, :64]
    with pytest.raises(C.Nvfp4MoeError, match="16 bytes"):
        ops.fp8_gemm(odd, sa, b, sb)
    with pytest.raises(ValueError, match="unit stride"):
        ops.fp8_gemm(torch.zeros(64, 4, dtype=torch.float8_e4m3fn, device="cuda").T, sa, b, sb)


# ----------------------------------------------------------------------------------- layer ----
def experts(E, I, H, seed):
    g = gen(seed)
    w = [torch.randn(E, I, H, generator=g, device="cuda") / math.sqrt(H) for _ in range(2)]
    return ops.FP8Experts.from_float(*w, torch.randn(E, H, I, generator=g, device="cuda") / math.sqrt(I))


def in_tiles(T, E, k, launch=C.LAUNCH_AUTO):
    """Whether a batch runs in row tiles, whose rows of the output wait for the combine in fp16."""
    P = T * k
    return (T > 16 or launch == C.LAUNCH_MULTI) and (T > 256 or P > 20 * min(P, E))


def layer_reference(w, x, logits, k, tiles):
    """(out, bound) in 64 bits.  The kernels' gate and up sums differ from the real ones by at most
    eg = (4 * 128 + nkb + 2) 2^-24 of the sums of magnitudes; silu (slope at most 1.1) and its fast
    exponential and division add 2^-18 of h, so h is off by at most
      eh = 1.1 eg(g) |u| + |silu(g)| eg(u) + 2^-18 |h|
    (products of errors are below that).  Its group's scale moves by at most max(eh) / 448 + 2^-24 of it.
    A code of h can then differ where the real quotient is nearer to a border than the quotient's own
    error; it differs by the grid's step there (at most |code| / 8, or 2^-9), or a scale that rounds
    elsewhere moves the dequantised value by its relative change.  The output is off by those, weighted
    by the down weights and the routing, by the product's own bound, by the softmax's 2^-21 and by half
    a step of bf16; and where rows wait in fp16, by half a step of it, 2^-11 of the value or, for those below
    2^-28 of the largest in 128 columns (which is scaled to 2^14 or more), 2^-25 / 2^14 of that."""
    T, E = logits.shape
    H, I = w.H, w.I
    lg = logits.double()
    order = torch.sort(lg + 0.0, dim=1, descending=True, stable=True)
    ids, p = order.indices[:, :k], torch.softmax(order.values[:, :k], 1)
    xq, xs = quantised(x, 1)
    xd = xq * spread(xs, 1, x.shape)
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    es = lambda n: (4 * 128 + blocks(n) + 2) * 2.0 ** -24  # noqa: E731
    codes = lambda t: t.view(torch.float8_e4m3fn).double()  # noqa: E731
    mid = (grid()[1:] + grid()[:-1]) / 2
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        wg, wu = (codes(w.w13_codes[e, i].view(torch.uint8)) * spread(w.w13_scale[e, i].double(), 128, (I, H)) for i in (0, 1))
        wd = codes(w.w2_codes[e].view(torch.uint8)) * spread(w.w2_scale[e].double(), 128, (H, I))
        xe = xd[t]
        g, u = xe @ wg.T, xe @ wu.T
        s = g * torch.sigmoid(g)
        h = s * u
        eh = 1.1 * es(H) * (xe.abs() @ wg.abs().T) * u.abs() + s.abs() * es(H) * (xe.abs() @ wu.abs().T) + 2.0 ** -18 * h.abs()
        hq, hs = quantised(h, 1)
        S = spread(hs, 1, h.shape)
        pad = torch.nn.functional.pad(eh, (0, blocks(I) * 128 - I)).view(len(t), -1, 128).amax(2)
        rel = torch.where(hs > 0, pad / (448 * hs).clamp(min=1e-300), torch.zeros_like(pad)) + 2.0 ** -23
        rel = spread(rel, 1, h.shape)                                   # relative change of the scale
        q = torch.where(S > 0, h.abs() / S.clamp(min=1e-300), torch.zeros_like(h))
        eq = torch.where(S > 0, eh / S.clamp(min=1e-300), torch.zeros_like(h)) + q * rel
        near = torch.searchsorted(mid, (q - eq).contiguous()) != torch.searchsorted(mid, (q + eq).contiguous(), right=True)
        step = (q / 8).clamp(min=2.0 ** -9) * 1.2
        dh = S * (near * step + hq.abs() * rel)
        y = (hq * S) @ wd.T
        size = (hq * S).abs() @ wd.abs().T
        c = p[t, j][:, None]
        out.index_add_(0, t, c * y)
        slot = 2.0 ** -11 * (y.abs() + es(I) * size) + 2.0 ** -39 * y.abs().amax(1, keepdim=True) if tiles else 0.0
        bound.index_add_(0, t, c * (dh @ wd.abs().T + (es(I) + 2.0 ** -21 + k * 2.0 ** -24) * size + slot))
    return out, bound * (1 + BF16_HALF) + BF16_HALF * out.abs()


def check_layer(w, x, logits, k, y, launch=C.LAUNCH_AUTO):
    ref, bound = layer_reference(w, x, logits, k, in_tiles(*logits.shape, k, launch))
    err = (y.double() - ref).abs()
    assert (err <= bound).all(), (err / bound.clamp(min=1e-300)).max()


CASES = [
    # T, H, I, E, k
    (1, 256, 128, 8, 2), (1, 2048, 512, 64, 10), (1, 1024, 4096, 1, 1), (2, 16, 16, 3, 3), (3, 144, 80, 5, 1),
    (8, 256, 128, 8, 2), (15, 1040, 336, 20, 3), (16, 512, 256, 512, 10), (16, 400, 144, 1024, 32), (17, 768, 384, 12, 4),
    (32, 2048, 128, 40, 8), (32, 256, 128, 1, 1), (33, 256, 128, 8, 2), (64, 400, 144, 64, 2), (65, 400, 144, 64, 2), (40, 6144, 144, 4, 4), (45, 1040, 336, 20, 3), (130, 640, 208, 7, 2),
    (300, 384, 512, 3, 1), (600, 272, 128, 300, 5), (16, 7168, 128, 6, 2), (5, 6144, 256, 4, 2), (256, 640, 208, 64, 5),
    (257, 640, 208, 64, 5), (90, 1040, 656, 3, 1), (700, 1552, 96, 5, 2), (1500, 256, 128, 1, 1),
]


@pytest.mark.parametrize("T,H,I,E,k", CASES)
def test_layer(T, H, I, E, k):
    w = experts(E, I, H, T + E)
    g = gen(T)
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, ::29] *= 15.0
    x, logits = x.bfloat16(), torch.randn(T, E, generator=g, device="cuda")
    layer = ops.FP8MoeFFN(w, k)
    y = layer(x, logits)
    check_layer(w, x, logits, k, y)
    assert torch.equal(y, layer(x, logits))
    assert ops.device_status() == 0


@pytest.mark.parametrize("T", [1, 7, 16])
@pytest.mark.parametrize("launch", [C.LAUNCH_SINGLE, C.LAUNCH_MULTI])
def test_layer_launches(T, launch):
    """Both ways of running a small batch, workspaces reused across changing routings."""
    w = experts(24, 272, 528, 1)
    layer = ops.FP8MoeFFN(w, 4, launch=launch)
    for seed in range(4):
        g = gen(seed)
        x = torch.randn(T, 528, generator=g, device="cuda").bfloat16()
        logits = torch.randn(T, 24, generator=g, device="cuda")
        if seed == 1:      # one expert gets every token
            logits[:, 5] += 100.0
        if seed == 2:      # equal logits: the lowest experts
            logits[:] = 0.25
        if seed == 3:      # one token alone among the others' experts
            logits[0] = -logits[0]
        check_layer(w, x, logits, 4, layer(x, logits), launch)
    assert ops.device_status() == 0


@pytest.mark.parametrize("T", [12, 100])
def test_layer_rows_stay_apart(T):
    """A token of NaN, one of infinities and one of zeros leave the other tokens' bits alone."""
    w = experts(6, 128, 256, 2)
    g = gen(3)
    x, logits = torch.randn(T, 256, generator=g, device="cuda").bfloat16(), torch.randn(T, 6, generator=g, device="cuda")
    layer = ops.FP8MoeFFN(w, 2)
    clean = layer(x, logits)
    x[2], x[5, 100], x[7] = math.nan, math.inf, 0.0
    y = layer(x, logits)
    others = torch.tensor([t for t in range(T) if t not in (2, 5, 7)], device="cuda")
    assert torch.equal(y[others], clean[others])
    assert y[2].isnan().all() and not y[5].isfinite().any() and (y[7] == 0).all()


def test_layer_rows_of_any_size():
    """Rows that wait in fp16 keep their precision whatever their size: down weights from 2^-100 to 2^100."""
    T, H, I = 300, 256, 128
    g = gen(4)
    x, logits = torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.zeros(T, 1, device="cuda")
    w = experts(1, I, H, 7)
    for e in (-100, -20, 0, 20, 100):
        v = ops.FP8Experts(w.w13_codes, w.w13_scale, w.w2_codes, w.w2_scale * 2.0 ** e)
        check_layer(v, x, logits, 1, ops.FP8MoeFFN(v, 1)(x, logits))


def test_layer_inputs_and_outputs():
    """Strided x and logits, other logit types, an output of the caller's own, an empty batch."""
    w = experts(8, 128, 256, 4)
    layer = ops.FP8MoeFFN(w, 2)
    g = gen(6)
    x, logits = torch.randn(40, 512, generator=g, device="cuda").bfloat16(), torch.randn(40, 16, generator=g, device="cuda")
    y = layer(x[::2, :256], logits[::2, ::2])
    assert torch.equal(y, layer(x[::2, :256].contiguous(), logits[::2, ::2].contiguous()))
    half = logits[::2, ::2].bfloat16()
    assert torch.equal(layer(x[::2, :256], half), layer(x[::2, :256], half.float()))
    out = torch.empty(20, 256, dtype=torch.bfloat16, device="cuda")
    assert layer(x[::2, :256], logits[::2, ::2], out=out) is out and torch.equal(out, y)
    assert layer(x[:0, :256], logits[:0, :8]).shape == (0, 256)
    for bad in (dict(x=x[:4].float()[:, :256], logits=logits[:4, :8]), dict(x=x[:4], logits=logits[:4, :8]),
                dict(x=x[:4, :256], logits=logits[:5, :8]), dict(x=x[:4, :256], logits=logits[:4, :8], out=out)):
        with pytest.raises(ValueError):
            layer(**bad)
    with pytest.raises(C.Nvfp4MoeError, match="single launch"):
        ops.FP8MoeFFN(w, 2, launch=C.LAUNCH_SINGLE)(x[:17, :256], logits[:17, :8])
    with pytest.raises(C.Nvfp4MoeError, match="multiple of 16"):
        ops.FP8MoeFFN(experts(2, 24, 256, 1), 1)(x[:4, :256], logits[:4, :2])


def test_experts_from_codes():
    """from_fp8 keeps codes and scales as they are; from_float is fp8_quantize's blocks."""
    g = gen(8)
    ws = [torch.randn(3, n, k, generator=g, device="cuda") for n, k in ((144, 272), (144, 272), (272, 144))]
    q = [ops.fp8_quantize(v, tile=ops.FP8_BLOCKS) for v in ws]
    a, b = ops.FP8Experts.from_fp8(*q), ops.FP8Experts.from_float(*ws)
    for n in ("w13_codes", "w2_codes"):
        assert torch.equal(getattr(a, n).view(torch.uint8), getattr(b, n).view(torch.uint8))
    assert torch.equal(a.w13_scale, b.w13_scale) and torch.equal(a.w2_scale, b.w2_scale)
    for i, (c, s) in enumerate(q):
        for e in range(3):
            r, t = quantised(ws[i][e], 128)
            assert torch.equal(c[e].double(), r) and torch.equal(s[e].double(), t)


# ---------------------------------------------------------------------- streams, graphs, together ----
@pytest.mark.parametrize("T", [4, 60])
def test_graphs_share_a_workspace(T):
    """Two captured calls on one layer's workspace, replayed in turn with an eager call between, and on
    a stream of their own."""
    w = experts(16, 256, 512, 5)
    layer = ops.FP8MoeFFN(w, 3)
    g = gen(T)
    xs = [torch.randn(T, 512, generator=g, device="cuda").bfloat16() for _ in range(4)]
    ls = [torch.randn(T, 16, generator=g, device="cuda") for _ in range(4)]
    want = [layer(x, l) for x, l in zip(xs, ls)]
    a, b = ops.GraphedMoeFFN(layer, T), ops.GraphedMoeFFN(layer, T)
    for i in range(4):
        assert torch.equal(a(xs[i], ls[i]), want[i])
        assert torch.equal(layer(xs[i ^ 1], ls[i ^ 1]), want[i ^ 1])
        assert torch.equal(b(xs[3 - i], ls[3 - i]), want[3 - i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [layer(x, l) for x, l in zip(xs, ls)]
    side.synchronize()
    assert all(torch.equal(y, z) for y, z in zip(got, want))
    io = ops.GraphedMoeFFN(layer, T, host_io=True)
    y = io(xs[0].cpu(), ls[0].cpu())
    torch.cuda.synchronize()
    assert torch.equal(y.cuda(), want[0])


def test_quantize_and_gemm_on_streams_and_in_graphs():
    g = gen(1)
    x, wt = torch.randn(70, 640, generator=g, device="cuda").bfloat16(), torch.randn(900, 640, generator=g, device="cuda")
    b, sb = ops.fp8_quantize(wt, tile=ops.FP8_BLOCKS)
    want = ops.fp8_gemm(*ops.fp8_quantize(x), b, sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.fp8_gemm(*ops.fp8_quantize(x), b, sb)
    side.synchronize()
    assert torch.equal(got, want)
    graph, static = torch.cuda.CUDAGraph(), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        out = ops.fp8_gemm(*ops.fp8_quantize(static), b, sb)
    static.copy_(x)
    graph.replay()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1, 24, 200])
def test_a_block_of_a_model(T):
    """The operators as a model's block uses them: a projection, the router on its output, the routed
    layer, a projection back; each against its definition on the inputs that it got."""
    g = gen(T)
    H, E, k = 512, 12, 3
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    proj, sp = ops.fp8_quantize(torch.randn(H, H, generator=g, device="cuda") / math.sqrt(H), tile=ops.FP8_BLOCKS)
    router, sr = ops.fp8_quantize(torch.randn(E, H, generator=g, device="cuda") / math.sqrt(H), tile=ops.FP8_BLOCKS)
    w = experts(E, 256, H, 3)
    a, sa = ops.fp8_quantize(x)
    y = ops.fp8_gemm(a, sa, proj, sp)
    check_gemm(y, a, sa, proj, sp)
    b, sb = ops.fp8_quantize(y)
    logits = ops.fp8_gemm(b, sb, router, sr, out_dtype=torch.float32)
    check_gemm(logits, b, sb, router, sr)
    z = ops.FP8MoeFFN(w, k)(y, logits)
    check_layer(w, y, logits, k, z)
    c, sc = ops.fp8_quantize(z)
    check_gemm(ops.fp8_gemm(c, sc, proj, sp), c, sc, proj, sp)
    assert ops.device_status() == 0


def test_two_layers_on_two_streams():
    """Two layers with workspaces of their own, their launches interleaved on two streams."""
    g = gen(9)
    layers = [ops.FP8MoeFFN(experts(12, 256, 512, s), 3) for s in (1, 2)]
    calls = [[(torch.randn(T, 512, generator=g, device="cuda").bfloat16(), torch.randn(T, 12, generator=g, device="cuda"))
              for T in (3, 16, 40, 300)] for _ in layers]
    want = [[layer(*c) for c in cs] for layer, cs in zip(layers, calls)]
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i in range(4):
            for n, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[n].append(layers[n](*calls[n][i]))
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(y, want[n][i % 4]) for i, y in enumerate(got[n]))
    assert ops.device_status() == 0


def test_weights_can_be_replaced():
    """A layer reads the experts' tensors as they are at the call."""
    a, b = experts(4, 128, 256, 1), experts(4, 128, 256, 2)
    g = gen(3)
    x, logits = torch.randn(9, 256, generator=g, device="cuda").bfloat16(), torch.randn(9, 4, generator=g, device="cuda")
    want = ops.FP8MoeFFN(b, 2)(x, logits)
    layer = ops.FP8MoeFFN(a, 2)
    assert not torch.equal(layer(x, logits), want)
    a.w13_codes, a.w13_scale, a.w2_codes, a.w2_scale = b.w13_codes, b.w13_scale, b.w2_codes, b.w2_scale
    assert torch.equal(layer(x, logits), want)


@pytest.mark.parametrize("T", [1, 16, 24, 200])
def test_calls_that_follow_at_once(T):
    """Launches set themselves up while the one before still runs: a chain of calls, each on what the
    last one wrote into buffers that are used again, gives what it gives with a wait after every call."""
    g = gen(T)
    H, E, k = 512, 12, 3
    w = [torch.randn(E, 256, H, generator=g, device="cuda") / math.sqrt(H) for _ in range(2)]
    w.append(torch.randn(E, H, 256, generator=g, device="cuda") / math.sqrt(256))
    fp8 = ops.FP8MoeFFN(ops.FP8Experts.from_float(*w), k)
    fp4 = ops.MoeFFN(ops.NVFP4Experts.from_float(*w), k, None, combine=C.COMBINE_ORDERED)
    proj, sp = ops.fp8_quantize(torch.randn(H, H, generator=g, device="cuda") / math.sqrt(H), tile=ops.FP8_BLOCKS)
    router, sr = ops.fp8_quantize(torch.randn(E, H, generator=g, device="cuda") / math.sqrt(H), tile=ops.FP8_BLOCKS)
    x0 = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    codes, scale = ops.fp8_quantize(x0)
    x, y, logits = x0.clone(), torch.empty_like(x0), torch.empty(T, E, device="cuda")

    def chain(wait):
        seen = []
        x.copy_(x0)
        wait()
        for i in range(12):
            ops.fp8_quantize(x, codes=codes, scale=scale), wait()
            ops.fp8_gemm(codes, scale, router, sr, out=logits), wait()
            ops.fp8_gemm(codes, scale, proj, sp, out=y), wait()
            fp8(y, logits, out=x), wait()
            fp8(x, logits, out=y), wait()
            ops.fp8_gemm(codes, scale, proj, sp, out=x), wait()
            if i % 3 == 2:
                (fp4(y, logits, out=x), wait(), ops.fp8_gemm(codes, scale, router, sr, out=logits), wait(),
                 fp8(x, logits, out=y), wait())
            seen += [x.clone(), y.clone(), logits.clone()]
        return seen

    want = chain(torch.cuda.synchronize)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))
    assert ops.device_status() == 0


def fork_and_join(x, proj, sp, fp8, logits, z, seen):
    """What calls may follow: a copy, a fill, a wait for another stream, a kernel and such a wait at once."""
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    codes, scale = ops.fp8_quantize(x)
    y = ops.fp8_gemm(codes, scale, proj, sp)          # after a kernel
    side.wait_stream(main)
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000)
        a = ops.fp8_gemm(codes, scale, proj, sp)      # after a kernel of another stream, and a delay
        other = fp8[0](a, logits)
        z.copy_(other)
    b = fp8[1](y, logits)                             # while the other stream works
    main.wait_stream(side)
    c = fp8[1](z, logits)                             # after a kernel and the other stream's copy
    z.zero_()
    z[:1].copy_(c[:1])
    d = fp8[1](z, logits)                             # after a copy
    e, se = ops.fp8_quantize(d)
    side.wait_stream(main)
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000)
        e.zero_()
    main.wait_stream(side)
    seen += [y, a, other, b, c, d, ops.fp8_gemm(e, se, proj, sp)]  # after the fill
    return seen


@pytest.mark.parametrize("T", [3, 40, 200])
def test_what_calls_follow(T):
    """Eager and captured, calls wait for all that their stream waits for."""
    g = gen(T)
    H, E, k = 512, 12, 3
    w = experts(E, 256, H, 3)
    proj, sp = ops.fp8_quantize(torch.randn(H, H, generator=g, device="cuda") / math.sqrt(H), tile=ops.FP8_BLOCKS)
    x, logits = torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda")
    fp8, z = [ops.FP8MoeFFN(w, k) for _ in range(2)], torch.empty_like(x)
    # one call at a time, each after a wait
    want = []
    y = ops.fp8_gemm(*ops.fp8_quantize(x), proj, sp)
    torch.cuda.synchronize()
    b = fp8[0](y, logits)
    torch.cuda.synchronize()
    c = fp8[0](b, logits)
    torch.cuda.synchronize()
    first = torch.zeros_like(x)
    first[:1] = c[:1]
    torch.cuda.synchronize()
    want = [y, y, b, b, c, fp8[0](first, logits), torch.zeros_like(y)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = fork_and_join(x, proj, sp, fp8, logits, z, [])
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph, static, out = torch.cuda.CUDAGraph(), torch.zeros_like(x), []
    with torch.cuda.graph(graph):
        static.copy_(x)
        fork_and_join(static, proj, sp, fp8, logits, z, out)
    for _ in range(3):
        for t in out:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert ops.device_status() == 0


def test_experts_refuse_other_tensors():
    w = experts(4, 128, 256, 1)
    for name, t, match in (("w2_codes", w.w13_codes[:, 0], "w2_codes must be"), ("w2_scale", w.w2_scale.double(), "fp32"),
                           ("w13_codes", w.w13_codes.float(), "float8"), ("w13_scale", w.w13_scale.cpu(), "CUDA")):
        with pytest.raises(ValueError, match=match):
            setattr(w, name, t)
    wide = torch.zeros(4, 256, 256, dtype=torch.uint8, device="cuda")
    w.w2_codes = wide[..., :128]
    assert w.w2_codes.is_contiguous()


def test_quantize_matrices_that_share_rows():
    """One matrix seen as a batch, and codes whose rows lie between those of another matrix."""
    g = gen(5)
    x = torch.randn(130, 256, generator=g, device="cuda")
    for tile in (ops.FP8_ROWS, ops.FP8_BLOCKS):
        want, scale = ops.fp8_quantize(x, tile=tile)
        codes, s = ops.fp8_quantize(x.expand(3, 130, 256), tile=tile)
        assert all(same(c.float(), want.float()) and torch.equal(t, scale) for c, t in zip(codes, s))
        between = torch.zeros(130, 2, 256, dtype=torch.float8_e4m3fn, device="cuda").transpose(0, 1)
        ops.fp8_quantize(torch.stack([x, -x]), tile=tile, codes=between)
        assert same(between[0].float(), want.float()) and same(between[1].float(), (-want.float()))
        with pytest.raises(RuntimeError, match="overlap"):
            ops.fp8_quantize(torch.stack([x, x]), tile=tile, codes=want.expand(2, 130, 256))


LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("T", [5, 40, 100, 300])
@pytest.mark.parametrize("mask", [-math.inf, LOWEST])
def test_layer_masked_experts(T, mask):
    """Experts masked with -inf or the type's lowest value: all but one, all but k, and (the lowest value)
    all, which leaves a uniform choice of the first k; a token whose experts are all -inf has no softmax
    and gives NaN, and the other tokens keep their bits."""
    E, k = 10, 3
    w = experts(E, 128, 256, 4)
    g = gen(T)
    x, logits = torch.randn(T, 256, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda")
    layer = ops.FP8MoeFFN(w, k)
    logits[0, 1:] = mask
    logits[1, :7] = mask
    logits[2, 1::2] = mask
    if mask == LOWEST:
        logits[3] = mask
    y = layer(x, logits)
    check_layer(w, x, logits, k, y)
    if mask == -math.inf:
        logits[3] = mask
        z = layer(x, logits)
        assert z[3].isnan().all()
        others = torch.arange(T, device="cuda") != 3
        if T > 16:  # (moving a token moves rows to other tiles; a row's sums do not depend on that)
            assert torch.equal(z[others], y[others])
        else:       # (a single launch splits its sums by the number of experts that are touched)
            check_layer(w, x[others], logits[others], k, z[others])
    assert ops.device_status() == 0


def test_layer_rows_past_32_bits():
    """560,000 rows of 4096: rows, codes and scales past 2^31 elements.  A row's sums do not depend on the
    batch, so the last tokens get what a small batch of them gets."""
    T, H, E, k = 70_000, 4096, 16, 8
    g = gen(1)
    w = experts(E, 128, H, 1)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    layer = ops.FP8MoeFFN(w, k)
    y = layer(x, logits)
    for part in (slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)):
        assert torch.equal(y[part], ops.FP8MoeFFN(w, k)(x[part], logits[part]))
    assert ops.device_status() == 0


def twins(E, I, H, seed):
    """Experts 2e and 2e + 1 that differ by the factor -(1 + 2^-9) of their down weights alone."""
    w = experts(E, I, H, seed)
    twice = lambda t: t.repeat_interleave(2, 0)  # noqa: E731
    s2 = twice(w.w2_scale)
    s2[1::2] *= -(1 + 2.0 ** -9)
    return w, ops.FP8Experts(twice(w.w13_codes.view(torch.uint8)), twice(w.w13_scale),
                             twice(w.w2_codes.view(torch.uint8)), s2)


@pytest.mark.parametrize("T", [5, 100, 300])
def test_layer_rows_that_cancel(T):
    """A token whose two experts' rows nearly cancel: out = -2^-9 y / 2, where y is the layer of one of the
    twins alone (read in bf16: half a step, 2^-9 of y; the output's own: the same).  The rows' fp32 sums, one
    block of I, lose at most 2^-24 each in the two scales' product, the scaling, the weighting and the sum: four of
    2^-24 for each of two rows, over 2^-9: 2^-12 of the output."""
    H, I = 256, 128
    one, two = twins(1, I, H, 5)
    x = torch.randn(T, H, generator=gen(T), device="cuda").bfloat16()
    y = ops.FP8MoeFFN(one, 1)(x, torch.zeros(T, 1, device="cuda")).double()
    got = ops.FP8MoeFFN(two, 2)(x, torch.zeros(T, 2, device="cuda")).double()
    want = -y * 2.0 ** -10
    assert ((got - want).abs() <= want.abs() * (2 * BF16_HALF + 2.0 ** -12) * (1 + BF16_HALF)).all()


@pytest.mark.parametrize("T", [5, 100, 300])
@pytest.mark.parametrize("e", [-40, 0, 40])
def test_layer_columns_stay_apart(T, e):
    """A NaN code in one row of the down weights makes one column of the output NaN, and no other bit
    changes, whatever the size of its neighbours."""
    H, I = 256, 128
    w = experts(1, I, H, 6)
    x, logits = torch.randn(T, H, generator=gen(T), device="cuda").bfloat16(), torch.zeros(T, 1, device="cuda")
    w.w2_scale = w.w2_scale * 2.0 ** e
    clean = ops.FP8MoeFFN(w, 1)(x, logits)
    codes = w.w2_codes.view(torch.uint8).clone()
    codes[0, 5, 3], codes[0, 200, 7] = 0x7F, 0xFF
    got = ops.FP8MoeFFN(ops.FP8Experts(w.w13_codes, w.w13_scale, codes, w.w2_scale), 1)(x, logits)
    hit = torch.zeros(H, dtype=torch.bool, device="cuda")
    hit[[5, 200]] = True
    assert got[:, hit].isnan().all()
    assert torch.equal(got[:, ~hit], clean[:, ~hit])


@pytest.mark.parametrize("T", [4, 40, 300])
def test_layers_take_other_experts(T):
    """Other experts, of other sizes, and another top_k on a layer that has run: the bits of a layer made with
    them, before and after."""
    first, second = experts(64, 256, 256, 1), experts(8, 128, 528, 2)
    g = gen(T)
    xs = [torch.randn(T, w.H, generator=g, device="cuda").bfloat16() for w in (first, second)]
    ls = [torch.randn(T, w.E, generator=g, device="cuda") for w in (first, second)]
    layer = ops.FP8MoeFFN(first, 8)
    for w, k, x, l in ((first, 8, xs[0], ls[0]), (second, 2, xs[1], ls[1]), (second, 3, xs[1], ls[1]),
                       (first, 1, xs[0], ls[0]), (first, 8, xs[0], ls[0])):
        layer.w, layer.top_k = w, k
        assert torch.equal(layer(x, l), ops.FP8MoeFFN(w, k)(x, l))
    assert ops.device_status() == 0


@pytest.mark.parametrize("T", [4, 40])
def test_graphs_refuse_replaced_weights(T):
    """A captured call holds the tensors that it reads, follows values written into them, and refuses to run
    once the layer has others; a new capture takes those.  The NVFP4 layer's graphs go on with what they hold."""
    a, b = experts(8, 128, 256, 1), experts(8, 128, 256, 2)
    g = gen(T)
    x, logits = torch.randn(T, 256, generator=g, device="cuda").bfloat16(), torch.randn(T, 8, generator=g, device="cuda")
    want = [ops.FP8MoeFFN(w, 2)(x, logits) for w in (a, b)]
    layer = ops.FP8MoeFFN(a, 2)
    graph = ops.GraphedMoeFFN(layer, T)
    assert torch.equal(graph(x, logits), want[0])
    old = [(n, getattr(a, n)) for n in ("w13_codes", "w13_scale", "w2_codes", "w2_scale")]
    refs = [weakref.ref(t) for _, t in old]
    for n, t in old:
        setattr(a, n, getattr(b, n))
        with pytest.raises(RuntimeError, match=n):
            graph(x, logits)
        setattr(a, n, t)
    assert torch.equal(graph(x, logits), want[0])
    for n, _ in old:
        setattr(a, n, getattr(b, n))
    del old, t
    assert all(r() is not None for r in refs)
    assert torch.equal(ops.GraphedMoeFFN(layer, T)(x, logits), want[1])
    for n, r in zip(("w13_codes", "w13_scale", "w2_codes", "w2_scale"), refs):
        setattr(a, n, r())
    assert torch.equal(graph(x, logits), want[0])
    for name, value in (("w", b), ("top_k", 3), ("launch", C.LAUNCH_MULTI)):
        was = getattr(layer, name)
        setattr(layer, name, value)
        with pytest.raises(RuntimeError, match=name):
            graph(x, logits)
        setattr(layer, name, was)
    for n in ("w13_codes", "w2_codes"):
        getattr(a, n).view(torch.uint8).copy_(getattr(b, n).view(torch.uint8))
    a.w13_scale.copy_(b.w13_scale), a.w2_scale.copy_(b.w2_scale)
    assert torch.equal(graph(x, logits), want[1])

    ws = [torch.randn(4, n, k, generator=g, device="cuda") for n, k in ((128, 256), (128, 256), (256, 128))]
    fp4 = ops.MoeFFN(ops.NVFP4Experts.from_float(*ws), 2, None)
    graph, want = ops.GraphedMoeFFN(fp4, T), fp4(x, logits[:, :4])
    assert torch.equal(graph(x, logits[:, :4]), want)
    refs = [weakref.ref(fp4.w.w13_codes), weakref.ref(fp4.w.w2_sf), weakref.ref(fp4.w)]
    fp4.w = ops.NVFP4Experts.from_float(*[-w for w in ws])
    assert all(r() is not None for r in refs)
    assert torch.equal(graph(x, logits[:, :4]), want)


@pytest.mark.parametrize("M,N,K", [(5, 40, 64), (77, 300, 1003), (40, 96, 4000), (1300, 4200, 300)])
@pytest.mark.parametrize("ea,eb", [(-100, -38), (-20, -115), (-110, -40), (70, 60), (30, 97), (100, -100), (-90, 100)])
def test_gemm_scales_of_any_size(M, N, K, ea, eb):
    """Scales whose product is below the smallest ordinary fp32 number or above the largest, where D is
    neither: the codes are made large or small to match.  (2^-149 an addition where a block's share is no
    ordinary number.)"""
    a, sa, b, sb = matrices(M, N, K, M + K)
    if ea + eb > 64:   # codes of at most 2^-5: a block's sum is below 2^-2
        a, b = ((t.float() * 2.0 ** -14).to(torch.float8_e4m3fn) for t in (a, b))
        a, b = (torch.nn.functional.pad(t.view(torch.uint8), (0, -K % 16))[:, :K].view(torch.float8_e4m3fn) for t in (a, b))
    sa, sb = sa / sa.amax() * 1.37 * 2.0 ** ea, sb / sb.amax() * 1.23 * 2.0 ** eb
    sa[:, ::3] *= 2.0 ** -5      # a row's blocks, and an accumulator's rows, on both sides of the border
    sa[::2] *= 2.0 ** 4
    d = ops.fp8_gemm(a, sa, b, sb, out_dtype=torch.float32)
    A, B = a.double() * spread(sa.double(), 1, a.shape), b.double() * spread(sb.double(), 128, b.shape)
    ref, size = A @ B.T, A.abs() @ B.abs().T
    bound = (4 * 128 + blocks(K) + 3) * 2.0 ** -24 * size + F32_HALF * ref.abs() + (blocks(K) + 1) * 2.0 ** -149
    most = torch.finfo(torch.float32).max
    fits = ref.abs() + bound < most
    assert fits.any() and ((d.double() - ref).abs() <= bound)[fits].all()


@pytest.mark.parametrize("T", [5, 40, 300])
@pytest.mark.parametrize("ex,eg,eu,ed", [(-100, -30, 120, 60), (-60, -70, 110, 60), (0, 0, -91, -36), (100, 50, -110, -60)])
def test_layer_scales_of_any_size(T, ex, eg, eu, ed):
    """x and weights whose scales' products are no ordinary numbers: 2^(ex + eg) for the gate, 2^(ex + eu) for
    the up and, of h's size, by 2^ed for the down.  Where the gate's is above the largest, weights meet the small
    elements of x alone, so that the sums are not."""
    H, I = 336, 208
    g = gen(T)
    x, logits = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, 3, generator=g, device="cuda")
    w = [torch.randn(3, I, H, generator=g, device="cuda") / math.sqrt(H) for _ in range(2)]
    w = ops.FP8Experts.from_float(*w, torch.randn(3, H, I, generator=g, device="cuda") / math.sqrt(I))
    codes, s = w.w13_codes.view(torch.uint8).clone(), w.w13_scale.clone()
    if ex + eg > 128:
        x *= 2.0 ** -16
        x[:, ::16] = 1.0
        codes[..., ::16] = 0
        codes = (codes.view(torch.float8_e4m3fn).float() * 2.0 ** -14).to(torch.float8_e4m3fn)
    s[:, 0] *= 2.0 ** eg
    s[:, 1] *= 2.0 ** eu
    w = ops.FP8Experts(codes, s, w.w2_codes, w.w2_scale * 2.0 ** ed)
    x = (x * 2.0 ** ex).bfloat16()
    y = ops.FP8MoeFFN(w, 2)(x, logits)
    assert y.isfinite().all() and (y != 0).any()
    ref, bound = layer_reference(w, x, logits, 2, False)
    assert ((y.double() - ref).abs() <= bound + 2.0 ** -134).all()   # half of bf16's last step


@pytest.mark.parametrize("T", [5, 40, 300])
@pytest.mark.parametrize("gate", [-20.0, -80.0, -87.8, -88.5, -95.0, 30.0, 95.0])
def test_layer_gates_far_from_zero(T, gate):
    """silu(g) u where e^-g leaves fp32's range: x has one element, so g is the one product within 2^-22 of it
    (88 * 2^-22 of the exponential, below 2^-14), u (2^120 at most) brings h back towards one, and all of a row's h are equal
    (code 448, exact).  2^-12 of the exponential where it is below the ordinary numbers (-95: 2^-137, in steps
    of 2^-149), half a step of bf16 for the output."""
    H, I = 256, 128
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    x[:, 3] = 1.0
    silu = gate / (1 + math.exp(-gate))
    wg, wu = torch.zeros(1, I, H, device="cuda"), torch.zeros(1, I, H, device="cuda")
    wg[..., 3], wu[..., 3] = gate, math.copysign(min(1 / abs(silu), 2.0 ** 120), silu)
    w = ops.FP8Experts.from_float(wg, wu, torch.eye(I, device="cuda").repeat(2, 1)[None])
    y = ops.FP8MoeFFN(w, 1)(x, torch.zeros(T, 1, device="cuda"))
    g = w.w13_scale[0, 0, 0, 0].double() * 448 * math.copysign(1, gate)
    u = w.w13_scale[0, 1, 0, 0].double() * 448 * math.copysign(1, silu)
    want = g / (1 + torch.exp(-g)) * u
    slack = 2.0 ** -14 + (2.0 ** -12 if gate < -87.3 else 0.0) + BF16_HALF * (1 + 2.0 ** -7)
    assert ((y.double() - want).abs() <= slack * want.abs()).all()


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1300, 4200, 300), (2000, 5000, 1003), (1536, 4000, 1200), (300, 7001, 2304),  # pairs of CTAs
    (16, 24576, 1536), (100, 20000, 700), (90, 24001, 400),                        # 256 columns, whole sums
    (2311, 432, 2969), (2953, 140, 7046), (30, 18500, 9000),                       # 256 columns, split sums
])
def test_gemm_in_wide_tiles(M, N, K, out_dtype):
    """Sums of several blocks, scales of more than one batch of eight, and sizes that end inside a block or
    tile, for the forms that 148 SMs give these sizes."""
    a, sa, b, sb = matrices(M, N, K, M + K)
    d = ops.fp8_gemm(a, sa, b, sb, out_dtype=out_dtype)
    check_gemm(d, a, sa, b, sb)
    assert torch.equal(d, ops.fp8_gemm(a, sa, b, sb, out_dtype=out_dtype))
    assert ops.device_status() == 0


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_weights_written_right_before_a_call(T):
    """The layer reads weights, scales and logits that the launches right before it wrote in place."""
    g = gen(T)
    E, I, H = 6, 256, 512
    ws = [[torch.randn(E, *s, generator=g, device="cuda") / math.sqrt(s[1]) for s in ((I, H), (I, H), (H, I))] for _ in range(2)]
    fixed = [ops.FP8Experts.from_float(*w) for w in ws]
    w = ops.FP8Experts.from_float(*ws[0])
    layer = ops.FP8MoeFFN(w, 2)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    router, sr = ops.fp8_quantize(torch.randn(E, H, generator=g, device="cuda"), tile=ops.FP8_BLOCKS)
    codes, scale = ops.fp8_quantize(x)
    logits = ops.fp8_gemm(codes, scale, router, sr, out_dtype=torch.float32)
    want = [[ops.FP8MoeFFN(f, 2)(x, l) for l in (logits, -logits)] for f in fixed]
    torch.cuda.synchronize()
    now, minus = torch.empty_like(logits), torch.full_like(logits, -1.0)
    for i in range(24):
        a, b = i & 1, i >> 1 & 1
        for n, (c, s) in enumerate(((w.w13_codes[:, 0], w.w13_scale[:, 0]), (w.w13_codes[:, 1], w.w13_scale[:, 1]),
                                    (w.w2_codes, w.w2_scale))):
            ops.fp8_quantize(ws[a][n], tile=ops.FP8_BLOCKS, codes=c, scale=s)
        ops.fp8_gemm(codes, scale, router, sr, out=now)
        if b:
            now.mul_(minus)
            ops.fp8_quantize(ws[a][2], tile=ops.FP8_BLOCKS, codes=w.w2_codes, scale=w.w2_scale)
        assert torch.equal(layer(x, now), want[a][b]), i
    assert ops.device_status() == 0


@pytest.mark.parametrize("T,H,I,E,k", [c for c in CASES if in_tiles(c[0], c[3], c[4])])
def test_layer_in_tiles_keeps_fp32_rows(T, H, I, E, k):
    """The bound of the other forms, without layer_reference's allowance for rows that wait in fewer bits."""
    w = experts(E, I, H, T + E + 1)
    g = gen(T + 1)
    x, logits = torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.randn(T, E, generator=g, device="cuda")
    ref, bound = layer_reference(w, x, logits, k, False)
    assert ((ops.FP8MoeFFN(w, k)(x, logits).double() - ref).abs() <= bound).all()
    assert ops.device_status() == 0


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_on_a_device_that_is_not_current():
    """Eager and captured calls on the tensors' device, another being current."""
    with torch.cuda.device(1):
        w = experts(8, 128, 256, 1)
        x, logits = torch.randn(4, 256, device="cuda").bfloat16(), torch.randn(4, 8, device="cuda")
        want = ops.FP8MoeFFN(w, 2)(x, logits)
    torch.cuda.synchronize(1)
    layer = ops.FP8MoeFFN(w, 2)
    assert torch.equal(layer(x, logits), want)
    assert torch.equal(ops.GraphedMoeFFN(layer, 4)(x, logits), want)
