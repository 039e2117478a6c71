"""The operators of the layer's 8-bit path, as cases to measure: the RMSNorm in front of the
layer (residual added, bf16 rows for the router and 8-bit rows for the experts) and its
backward pass, the quantisation of rows and of expert weights, the grouped product of 8-bit
rows with 8-bit expert weights, and the gate/up product with SwiGLU and an 8-bit output.

The 8-bit form of a matrix: e4m3 values and, for each block of 128 along the reduction
dimension (rows: 1 x 128, weights: 128 x 128), a power of two (e8m0, one byte), the smallest
2^k with max|block| <= 448 2^k, k >= -126. A row of C values has 4 ceil(C / 512) scale
bytes; those past ceil(C / 128) hold 1.0. A matrix entry is its e4m3 value times its scale.

With `own` false, run() computes each operator from elementary torch operations in fp32;
with `own` true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def listed():
    return [
        # one decode step of the V4-shaped layer: 16 token rows, latency counts
        dict(name="norm_decode_t16", op="norm", T=16, d=7168),
        # the V3-shaped prefill batch
        dict(name="norm_prefill", op="norm", T=8192, d=7168),
        # training steps of the GShard-shaped and 2B-shaped layers
        dict(name="norm_bwd_gshard", op="norm_bwd", T=4096, d=1024),
        dict(name="norm_bwd_2b", op="norm_bwd", T=16384, d=1280),
        # rows of the tiny layer, where a call is all latency
        dict(name="quant_rows_tiny", op="quant_rows", R=512, C=256),
        # one projection of 32 V3-shaped experts, quantised at load time
        dict(name="quant_weights_slice", op="quant_weights", E=32, N=2048, K=7168),
        # down projection in decode: 16 tokens x top-9 over 48 V4-shaped experts, weights streamed
        dict(name="product_decode", op="product", E=48, R=144, N=7168, K=2048, skew=0.0),
        # down projection of the fine-grained GShard shape: K = 704 ends inside a block
        dict(name="product_gshard", op="product", E=64, R=32768, N=1024, K=704, skew=0.5),
        # down projection of 32 V3-shaped experts over 8192 rows
        dict(name="product_prefill", op="product", E=32, R=8192, N=7168, K=2048, skew=0.2),
        # gate/up of the tiny layer: 512 tokens x top-7, F = one scale block
        dict(name="gated_tiny", op="gated", E=64, R=3584, N=128, K=256, skew=0.5),
        # gate/up in decode: 16 tokens x top-9 over 48 V4-shaped experts
        dict(name="gated_decode", op="gated", E=48, R=144, N=2048, K=7168, skew=0.0),
        # gate/up of 32 V3-shaped experts over 8192 rows: the largest
        dict(name="gated_prefill", op="gated", E=32, R=8192, N=2048, K=7168, skew=0.2),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even in its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "quant_rows", "quant_weights", "product", "gated"])
    if op in ("norm", "norm_bwd"):
        return dict(op=op, T=_log(rng, 1, 8192), d=_log(rng, 64, 7168, 64))
    if op == "quant_rows":
        return dict(op=op, R=_log(rng, 1, 16384), C=_log(rng, 16, 7168, 16))
    if op == "quant_weights":
        return dict(op=op, E=_log(rng, 1, 32), N=_log(rng, 64, 2048, 8), K=_log(rng, 64, 7168, 16))
    E, R = _log(rng, 1, 64), _log(rng, 1, 16384)
    K = _log(rng, 64, 7168, 16)
    N = _log(rng, 64, 2048, 16) if op == "gated" else _log(rng, 64, 7168, 8)
    # expert weights of at most 48 matrices of 7168 x 2048, and no more products than the
    # largest listed case
    while E * N * K > 48 * 7168 * 2048:
        E = max(1, E // 2)
    while R * N * K > 8192 * 7168 * 2048:
        R = max(1, R // 2)
    return dict(op=op, E=E, R=R, N=N, K=K, skew=rng.choice([0.0, 0.2, 0.5, 1.1]))


# ------------------------------------------------------------------------------- inputs
def scale_cols(C):
    """Scale bytes of a row of C values."""
    return 4 * (-(-C // 512))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, R, C):
    """Activations: normal, with a spread of row sizes and a few outlier columns."""
    x = torch.randn((R, C), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((R, 1), generator=g, device="cuda"))
    x *= 1 + 20 * (torch.rand((1, C), generator=g, device="cuda") < 0.002)
    return x.bfloat16()


def _weights(g, E, N, K):
    return (torch.randn((E, N, K), generator=g, device="cuda") / math.sqrt(K)).bfloat16()


def _offsets(case, seed):
    """Rows of each expert, as routing gives them: a multinomial over Zipf weights in a random order."""
    E, R = case["E"], case["R"]
    rng = np.random.RandomState(seed % (1 << 31))
    p = rng.permutation(1.0 / np.arange(1, E + 1) ** case["skew"])
    return np.concatenate([[0], np.cumsum(rng.multinomial(R, p / p.sum()))]).astype(np.int32)


_handles = {}


def _handle(d, tokens):
    """The layer handle that the program keeps (one for each width and batch size)."""
    import mixture_experts_layer_score_b200 as M
    if (d, tokens) not in _handles:
        _handles[(d, tokens)] = M.dsmoe_create(M.make_cfg(d_model=d, n_routed=1, top_k=1, d_ff=64, max_tokens=tokens))
    return _handles[(d, tokens)]


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _q8_buffers(R, C):
    return _empty((R, C), F8), _empty((R, scale_cols(C)), E8)


def prepare(case, seed):
    s, g, op = dict(case), _gen(seed), case["op"]
    if op in ("norm", "norm_bwd"):
        T, d = case["T"], case["d"]
        s["w"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")).bfloat16()
        if op == "norm":
            s["x"], s["residual"] = 0.3 * _rows(g, T, d), _rows(g, T, d)
            s["out"] = (_empty((T, d), torch.bfloat16), _empty((T, d), torch.bfloat16), *_q8_buffers(T, d))
        else:
            s["r"] = _rows(g, T, d)
            s["dy"] = torch.randn((T, d), generator=g, device="cuda")
            s["dres"] = torch.randn((T, d), generator=g, device="cuda").bfloat16()
            s["out"] = (_empty((T, d), torch.bfloat16), _empty((d,), torch.float32))
        if own:
            s["handle"] = _handle(d, T)
        return s
    if op == "quant_rows":
        s["x"] = _rows(g, case["R"], case["C"])
        s["out"] = _q8_buffers(case["R"], case["C"])
    elif op == "quant_weights":
        E, N, K = case["E"], case["N"], case["K"]
        s["W"] = _weights(g, E, N, K)
        s["out"] = (_empty((E, N, K), F8), _empty((E, -(-N // 128), scale_cols(K)), E8))
    else:
        E, R, N, K = case["E"], case["R"], case["N"], case["K"]
        off = _offsets(case, seed)
        s["offsets"], s["most"] = torch.from_numpy(off).cuda(), int(np.diff(off).max())
        s["a"], s["a_scale"] = plain_quantize_rows(_rows(g, R, K))
        s["W"], s["W_scale"] = plain_quantize_weights(_weights(g, E, N, K))
        if op == "gated":
            s["Wu"], s["Wu_scale"] = plain_quantize_weights(_weights(g, E, N, K))
            s["out"] = _q8_buffers(R, N)
        else:
            s["out"] = _empty((R, N), torch.bfloat16)
    if own:
        s["handle"] = _handle(64, 1)
    return s


# -------------------------------------------------------------------------- plain forms
def _blocks(x, dim, size=128):
    """x, padded with zeros along `dim` to whole blocks, with that dimension split in two."""
    n = x.shape[dim]
    pad = -n % size
    if pad:
        shape = list(x.shape)
        shape[dim] = pad
        x = torch.cat([x, x.new_zeros(shape)], dim)
    return x.unflatten(dim, (-1, size))


def _scale_byte(amax):
    """The e8m0 byte of the smallest 2^k >= amax / 448, k >= -126; 255 where amax is not finite."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1, and 448 = 0.875 2^9
    byte = torch.where(amax > 0, e - 9 + (m > 0.875) + 127, 1).clamp(1, 254)
    return torch.where(torch.isfinite(amax), byte, 255)


def _power(exponent):
    """2^exponent in fp32 for integers in [-126, 127]."""
    return ((exponent + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(xb, byte):
    """e4m3 values of the blocked fp32 values xb under the scale bytes (broadcast)."""
    q = xb * _power(127 - byte.clamp(max=254))
    return torch.where(byte == 255, math.nan, q).to(F8)


def _pad_scales(byte, C):
    out = torch.full((*byte.shape[:-1], scale_cols(C)), 127, dtype=torch.uint8, device=byte.device)
    out[..., :byte.shape[-1]] = byte.to(torch.uint8)
    return out.view(E8)


def plain_quantize_rows(x):
    C = x.shape[-1]
    xb = _blocks(x.float(), -1)
    byte = _scale_byte(xb.abs().amax(-1))
    q = _encode(xb, byte[..., None]).flatten(-2)[..., :C].contiguous()
    return q, _pad_scales(byte, C)


def plain_quantize_weights(W):
    E, N, K = W.shape
    wb = _blocks(_blocks(W.float(), 2), 1)  # [E, N/128, 128, K/128, 128]
    byte = _scale_byte(wb.abs().amax((2, 4)))
    q = _encode(wb, byte[:, :, None, :, None]).flatten(3).flatten(1, 2)[:, :N, :K].contiguous()
    return q, _pad_scales(byte, K)


def plain_dequantize_rows(q, scale):
    C = q.shape[-1]
    v = scale.float()[..., :-(-C // 128)].repeat_interleave(128, -1)[..., :C]
    return q.float() * v


def plain_dequantize_weights(q, scale):
    return plain_dequantize_rows(q, scale.float().repeat_interleave(128, 1)[:, :q.shape[1]])


def plain_norm(x, residual, w):
    r = (x.float() + residual.float()).bfloat16()
    rf = r.float()
    u = (rf * torch.rsqrt((rf * rf).mean(-1, keepdim=True) + EPS) * w.float()).bfloat16()
    return (r, u, *plain_quantize_rows(u))


def plain_norm_backward(dy, dres, r, w):
    rf, g = r.float(), dy * w.float()
    rstd = torch.rsqrt((rf * rf).mean(-1, keepdim=True) + EPS)
    c = (g * rf).mean(-1, keepdim=True)
    dx = dres.float() + rstd * g - rf * (rstd * rstd * rstd * c)
    return dx.bfloat16(), (dy * rf * rstd).sum(0)


def plain_grouped(a, offsets, most, weights):
    """rows of expert e times weights[e]^T for each of the weights, in fp32: the experts' rows side by side,
    padded to the longest, and one batched product."""
    R, E = a.shape[0], offsets.shape[0] - 1
    off = offsets.long()
    rows = off[:-1, None] + torch.arange(most, device=a.device)
    padded = torch.where((rows < off[1:, None])[..., None], a[rows.clamp(max=R - 1)], 0.0)
    at = torch.arange(R, device=a.device)
    e = torch.searchsorted(off[1:].contiguous(), at, right=True)
    return [torch.bmm(padded, W.transpose(1, 2))[e, at - off[e]] for W in weights]


def run(s):
    op = s["op"]
    if own:
        import mixture_experts_layer_score_b200 as M
        h, out = s["handle"], s["out"]
        if op == "norm":
            M.dsmoe_norm_q8(h, s["T"], s["x"], s["residual"], s["w"], EPS, *out)
        elif op == "norm_bwd":
            M.dsmoe_norm_backward(h, s["T"], s["dy"], s["dres"], s["r"], s["w"], EPS, *out)
        elif op == "quant_rows":
            M.dsmoe_q8_quantize(h, s["R"], s["C"], s["x"], *out)
        elif op == "quant_weights":
            M.dsmoe_q8_quantize_weights(h, s["E"], s["N"], s["K"], s["W"], *out)
        elif op == "product":
            M.dsmoe_q8_matmul(h, s["E"], s["R"], s["N"], s["K"], s["offsets"], s["a"], s["a_scale"], s["W"],
                              s["W_scale"], out)
        else:
            M.dsmoe_q8_gated_matmul(h, s["E"], s["R"], s["N"], s["K"], s["offsets"], s["a"], s["a_scale"], s["W"],
                                    s["W_scale"], s["Wu"], s["Wu_scale"], *out)
        return out
    if op == "norm":
        return plain_norm(s["x"], s["residual"], s["w"])
    if op == "norm_bwd":
        return plain_norm_backward(s["dy"], s["dres"], s["r"], s["w"])
    if op == "quant_rows":
        return plain_quantize_rows(s["x"])
    if op == "quant_weights":
        return plain_quantize_weights(s["W"])
    a = plain_dequantize_rows(s["a"], s["a_scale"])
    W = plain_dequantize_weights(s["W"], s["W_scale"])
    if op == "product":
        return plain_grouped(a, s["offsets"], s["most"], [W])[0].bfloat16()
    g, u = plain_grouped(a, s["offsets"], s["most"], [W, plain_dequantize_weights(s["Wu"], s["Wu_scale"])])
    return plain_quantize_rows(g / (1 + torch.exp(-g)) * u)


def work(case):
    """Inputs read once and outputs written once (of the expert weights, those that some row uses)."""
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, d = case["T"], case["d"]
        if op == "norm":
            return dict(bytes=T * (d * (2 + 2 + 2 + 2 + 1) + scale_cols(d)) + 2 * d, flops=8 * T * d)
        return dict(bytes=T * d * (4 + 2 + 2 + 2) + 6 * d, flops=12 * T * d)
    if op == "quant_rows":
        return dict(bytes=case["R"] * (3 * case["C"] + scale_cols(case["C"])), flops=3 * case["R"] * case["C"])
    E, N, K = case["E"], case["N"], case["K"]
    weight = N * K + -(-N // 128) * scale_cols(K)
    if op == "quant_weights":
        return dict(bytes=E * (2 * N * K + weight), flops=3 * E * N * K)
    R = case["R"]
    used = E * (1 - (1 - 1 / E) ** R) if E > 1 else 1
    rows, two = R * (K + scale_cols(K)), 2 if op == "gated" else 1
    out = R * (N + scale_cols(N)) if op == "gated" else 2 * R * N
    return dict(bytes=rows + used * two * weight + out + 4 * (E + 1), flops=2.0 * two * R * N * K)


# ------------------------------------------------------------------- definition in 64 bits
def _two(k):
    """2^k in 64 bits for integers k."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(v):
    """v rounded to the nearest e4m3 value (ties to even): 4 significant bits, steps of at least 2^-9."""
    _, e = torch.frexp(v)
    step = _two((e - 1).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_scale(amax):
    k = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448)).clamp(min=-126)
    k = torch.where(448 * _two(k - 1) >= amax, k - 1, k).clamp(min=-126)  # where log2 rounded across
    return torch.where(448 * _two(k) < amax, _two(k + 1), _two(k))


def _exact_rows(y):
    """Values and scales of the 64-bit rows y, with the scales' pad columns."""
    C, n = y.shape[-1], -(-y.shape[-1] // 128)
    q, scales = torch.empty_like(y), torch.ones((*y.shape[:-1], scale_cols(C)), dtype=y.dtype, device=y.device)
    for b in range(n):
        part = y[..., 128 * b:128 * b + 128]
        s = _exact_scale(part.abs().amax(-1))
        scales[..., b] = s
        q[..., 128 * b:128 * b + 128] = _exact_e4m3(part / s[..., None])
    return q, scales


def _exact_weights(q, scale):
    """64-bit weights [N, K] of one expert from its values and scales."""
    N, K = q.shape
    W = q.double()
    for i in range(-(-N // 128)):
        for j in range(-(-K // 128)):
            W[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= scale[i, j].double()
    return W


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        r = (s["x"].double() + s["residual"].double()).bfloat16()
        rd = r.double()
        u = rd / torch.sqrt((rd * rd).mean(-1, keepdim=True) + EPS) * s["w"].double()
        return (rd, u, *_exact_rows(u.bfloat16().double()))
    if op == "norm_bwd":
        rd, dy, w = s["r"].double(), s["dy"].double(), s["w"].double()
        d = rd.shape[1]
        inv = 1 / torch.sqrt((rd * rd).sum(-1, keepdim=True) / d + EPS)
        n = rd * inv
        dn = dy * w
        dx = inv * (dn - n * (dn * n).sum(-1, keepdim=True) / d) + s["dres"].double()
        return dx, (dy * n).sum(0)
    if op == "quant_rows":
        return _exact_rows(s["x"].double())
    if op == "quant_weights":
        W = s["W"]
        E, N, K = W.shape
        q = torch.empty((E, N, K), dtype=torch.float64, device=W.device)
        scales = torch.ones((E, -(-N // 128), scale_cols(K)), dtype=torch.float64, device=W.device)
        for i in range(-(-N // 128)):
            for j in range(-(-K // 128)):
                part = W[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128].double()
                v = _exact_scale(part.abs().amax((1, 2)))
                scales[:, i, j] = v
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _exact_e4m3(part / v[:, None, None])
        return q, scales
    K, off = case["K"], s["offsets"].tolist()
    a = s["a"].double()
    for j in range(-(-K // 128)):
        a[:, 128 * j:128 * j + 128] *= s["a_scale"][:, j:j + 1].double()
    y = torch.zeros((case["R"], case["N"]), dtype=torch.float64, device=a.device)
    for e in range(case["E"]):
        rows = a[off[e]:off[e + 1]]
        if rows.shape[0] == 0:
            continue
        v = rows @ _exact_weights(s["W"][e], s["W_scale"][e]).T
        if op == "gated":
            v = v / (1 + torch.exp(-v)) * (rows @ _exact_weights(s["Wu"][e], s["Wu_scale"][e]).T)
        y[off[e]:off[e + 1]] = v
    return y if op == "product" else _exact_rows(y)
