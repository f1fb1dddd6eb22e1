"""Timing cases for the microscaled (MX) operators: 4-bit quantisation and product, and
activation checkpoints in 8 bits with their use in the backward pass.

An MX block is 32 elements along a row with one power-of-two scale (an E8M0 byte b stands
for 2^(b - 127)).  Elements are E2M1 (4 bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives, two to a byte, the even column in the low half) or E4M3 (8 bits).  A row holds
whole blocks.  The scales sit in tiles of 128 rows x 4 blocks, 512 bytes: byte
(row, block) at ((row / 128) * ceil(blocks / 4) + block / 4) * 512
+ (row % 32) * 16 + ((row % 128) / 32) * 4 + block % 4.

``own`` chooses who computes: the plain form in elementary torch operations, or the
package's operators.  ``exact`` is the definition in 64 bits, written separately.
"""

import math

import torch

own = False

BLOCK = 32
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MOST_ELEMENTS = 1 << 27  # of one elementwise case
MOST_PRODUCT = 8192 ** 3


def listed():
    return [
        # One token's activations on their way into a 4-bit linear layer.
        {"name": "quantize_token", "op": "quantize", "format": "e2m1", "rows": 1, "cols": 4096, "transpose": False,
         "type": "f16"},
        # A square weight, quantised along its other axis for the backward product.
        {"name": "quantize_weight_t", "op": "quantize", "format": "e2m1", "rows": 8192, "cols": 8192, "transpose": True,
         "type": "bf16"},
        # A layer's input saved in 8 bits, with sizes that end inside blocks and tiles.
        {"name": "quantize_ragged", "op": "quantize", "format": "e4m3", "rows": 4000, "cols": 3001, "transpose": False,
         "type": "f32"},
        # Decoding one sequence: one token against a square weight.
        {"name": "product_token", "op": "product", "m": 1, "n": 4096, "k": 4096, "out": "f16", "bias": False,
         "activation": "none", "residual": False},
        # Decoding a small batch through the widening layer of a feed-forward block.
        {"name": "product_batch", "op": "product", "m": 16, "n": 16384, "k": 4096, "out": "bf16", "bias": True,
         "activation": "silu", "residual": False},
        # The repository's ragged GEMM, in 4 bits.
        {"name": "product_ragged", "op": "product", "m": 4000, "n": 3000, "k": 1000, "out": "f32", "bias": False,
         "activation": "none", "residual": False},
        # The repository's fused GEMM (bias, GELU, residual) over a prompt, in 4 bits.
        {"name": "product_fused", "op": "product", "m": 4096, "n": 4096, "k": 4096, "out": "f16", "bias": True,
         "activation": "gelu", "residual": True},
        # The repository's largest GEMM, in 4 bits.
        {"name": "product_large", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "f16", "bias": False,
         "activation": "none", "residual": False},
        # A few rows of an odd width through an activation that saves its input.
        {"name": "forward_small", "op": "forward", "rows": 7, "cols": 4095, "activation": "gelu", "type": "f16"},
        # A prompt's widened activations.
        {"name": "forward_prompt", "op": "forward", "rows": 4096, "cols": 16384, "activation": "gelu_tanh",
         "type": "bf16"},
        # The backward pass of a small layer of odd width, in fp32.
        {"name": "backward_ragged", "op": "backward", "rows": 1000, "cols": 3001, "activation": "gelu", "type": "f32"},
        # The backward pass over a training batch's widened activations.
        {"name": "backward_batch", "op": "backward", "rows": 8192, "cols": 16384, "activation": "silu",
         "type": "bf16"},
    ]


def _size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "forward", "backward"))
    if op == "product":
        m = _size(rng, 1, 64) if rng.random() < 0.5 else _size(rng, 64, 8192)
        n, k = _size(rng, 32, 16384), _size(rng, 32, 16384)
        while m * n * k > MOST_PRODUCT:
            n, k = max(32, n // 2 + 1), max(32, k // 2 + 1)
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(("f32", "f16", "bf16")),
                "bias": rng.random() < 0.5, "activation": rng.choice(("none", "relu", "gelu", "silu", "gelu_tanh")),
                "residual": rng.random() < 0.5}
    rows, cols = _size(rng, 1, 16384), _size(rng, 1, 16384)
    while rows * cols > MOST_ELEMENTS // 2:
        rows = rows // 2 + 1
    case = {"op": op, "rows": rows, "cols": cols, "type": rng.choice(("f32", "f16", "bf16"))}
    if op == "quantize":
        case["format"] = rng.choice(("e2m1", "e4m3"))
        case["transpose"] = rng.random() < 0.5
    else:
        case["activation"] = rng.choice(("relu", "gelu", "silu", "gelu_tanh"))
    return case


# ------------------------------------------------------------------ the plain form


def _pow2(e):
    """2^e as fp32 for integer e in [-127, 127], built from its bits."""
    normal = ((e + 127) << 23).to(torch.int32)
    return torch.where(e > -127, normal, torch.full_like(normal, 1 << 22)).view(torch.float32)


def _quantize(x, fmt):
    """The MX values of fp32 rows x (rows x cols) as (elements, exponents): blocks of 32 along
    the row, the last one padded with zeros."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    mant, ex = torch.frexp(v.abs().amax(dim=2))
    ex = ex.to(torch.int64)
    if fmt == "e2m1":
        e = ex - 3  # floor(log2(amax)) - 2: the largest element lands in [4, 8), over 6 saturates
    else:
        e = torch.where(mant <= 0.875, ex - 9, ex - 8)  # the smallest power of two with amax <= 448 * 2^e
    e = torch.where(mant == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    t = v * _pow2(-e.clamp(max=126)).unsqueeze(2)
    a = t.abs()
    if fmt == "e2m1":
        q = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
        q = q.clamp(max=6)
    else:
        step = _pow2((torch.frexp(a)[1].to(torch.int64) - 1).clamp(min=-6) - 3)
        q = (torch.round(a / step) * step).clamp(max=448)
    return torch.copysign(q, t), e


def _values(q, e, cols):
    return (q * _pow2(e).unsqueeze(2)).reshape(q.shape[0], -1)[:, :cols]


def _tiled(e):
    """Scale bytes (rows x blocks, as exponents) in the tiled layout, zeros in the padding."""
    rows, nb = e.shape
    rt, ct = -(-rows // 128), -(-nb // 4)
    b = torch.zeros((rt * 128, ct * 4), dtype=torch.uint8, device=e.device)
    b[:rows, :nb] = (e + 127).to(torch.uint8)
    return b.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _untiled(s, rows, nb):
    rt, ct = -(-rows // 128), -(-nb // 4)
    return s.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:rows, :nb].to(torch.int64) - 127


def _packed(q, fmt):
    """Element bytes of rows x blocks x 32 element values."""
    rows = q.shape[0]
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, -1).contiguous()
    table = torch.tensor(LEVELS, device=q.device)
    code = torch.bucketize(q.abs(), table) + torch.where(torch.signbit(q), 8, 0)
    code = code.to(torch.uint8).view(rows, -1, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous()


def _unpacked(Q, S, fmt, cols):
    """fp32 values of stored elements and scales."""
    rows = Q.shape[0]
    nb = Q.shape[1] // (16 if fmt == "e2m1" else 32)
    if fmt == "e4m3":
        q = Q.view(torch.float8_e4m3fn).to(torch.float32)
    else:
        table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=Q.device)
        q = torch.stack((table[(Q & 15).to(torch.int64)], table[(Q >> 4).to(torch.int64)]), dim=2)
    return _values(q.reshape(rows, nb, BLOCK), _untiled(S, rows, nb), cols)


def _activate(act, x):
    if act == "relu":
        return torch.clamp(x, min=0)
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(x * -math.sqrt(0.5))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _slope(act, x):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu":
        return 0.5 * torch.special.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


# ------------------------------------------------------------------ inputs


def _activations(gen, rows, cols, dtype):
    """Rows of activations: normal values, channels of different size, and a few all-zero rows
    (the padding of a batch)."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((1, cols), generator=gen, device="cuda"))
    if rows >= 16:
        x[rows - rows // 16:] = 0
    return x.to(dtype)


def _stored(x, fmt):
    q, e = _quantize(x.float(), fmt)
    return _packed(q, fmt), _tiled(e)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case)
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        state["A"], state["SA"] = _stored(_activations(gen, m, k, torch.float32), "e2m1")
        w = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
        state["B"], state["SB"] = _stored(w, "e2m1")
        dt = TYPES[case["out"]]
        state["bias_v"] = None
        if case["bias"]:
            bias = torch.rand((n,), generator=gen, device="cuda") - 0.5
            state["bias_v"] = bias.to(torch.bfloat16 if case["out"] == "bf16" else torch.float16)
        state["residual_v"] = None
        if case["residual"]:
            state["residual_v"] = (torch.rand((m, n), generator=gen, device="cuda") * 2 - 1).to(dt)
        return state
    rows, cols, dt = case["rows"], case["cols"], TYPES[case["type"]]
    if case["op"] == "quantize":
        x = _activations(gen, rows, cols, dt)
        state["X"] = x.t().contiguous() if case["transpose"] else x
    elif case["op"] == "forward":
        state["Z"] = _activations(gen, rows, cols, dt)
    else:
        state["Q"], state["S"] = _stored(_activations(gen, rows, cols, dt), "e4m3")
        state["dY"] = torch.randn((rows, cols), generator=gen, device="cuda").to(dt)
    return state


# ------------------------------------------------------------------ one pass


def _run_plain(s):
    if s["op"] == "quantize":
        x = s["X"].t() if s["transpose"] else s["X"]
        q, e = _quantize(x.float(), s["format"])
        return _values(q, e, s["cols"]).to(TYPES[s["type"]])
    if s["op"] == "product":
        c = _unpacked(s["A"], s["SA"], "e2m1", s["k"]) @ _unpacked(s["B"], s["SB"], "e2m1", s["k"]).t()
        if s["bias_v"] is not None:
            c = c + s["bias_v"].float()
        c = _activate(s["activation"], c)
        if s["residual_v"] is not None:
            c = c + s["residual_v"].float()
        return c.to(TYPES[s["out"]])
    if s["op"] == "forward":
        z = s["Z"].float()
        q, e = _quantize(z, "e4m3")
        dt = TYPES[s["type"]]
        return _activate(s["activation"], z).to(dt), _values(q, e, s["cols"]).to(dt)
    z = _unpacked(s["Q"], s["S"], "e4m3", s["cols"])
    dz = s["dY"].float() * _slope(s["activation"], z)
    return dz.to(TYPES[s["type"]]), dz.sum(dim=0, dtype=torch.float64).float()


def _run_own(s):
    import tiled_dense_gemm_tlg_b200 as tlg

    if s["op"] == "quantize":
        Q, S = tlg.tlg_mx_quantize(s["X"], format=s["format"], op="T" if s["transpose"] else "N")
        return tlg.tlg_mx_dequantize(Q, S, s["cols"], format=s["format"], out=s["type"])
    if s["op"] == "product":
        return tlg.tlg_gemm_mxfp4(s["A"], s["SA"], s["B"], s["SB"], bias=s["bias_v"], activation=s["activation"],
                                  residual=s["residual_v"], out=s["out"])
    if s["op"] == "forward":
        Y, Q, S = tlg.tlg_act_forward_mx(s["Z"], s["activation"])
        return Y, tlg.tlg_mx_dequantize(Q, S, s["cols"], format="e4m3", out=s["type"])
    return tlg.tlg_act_backward_mx(s["dY"], s["Q"], s["S"], s["activation"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work


def work(case):
    """Each input read once, each output written once; what is stored in between (elements and
    scales, in the quantize and forward cases) written once."""
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        nb = -(-k // BLOCK)
        b = (m + n) * nb * 17 + m * n * BYTES[case["out"]] * (2 if case["residual"] else 1)
        return {"bytes": b + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    rows, cols, t = case["rows"], case["cols"], BYTES[case["type"]]
    nb = -(-cols // BLOCK)
    per_block = 17 if case.get("format") == "e2m1" else 33
    b = rows * cols * t * 2 + rows * nb * per_block
    if case["op"] == "forward":
        b += rows * cols * t  # the activation, beside the saved values
    if case["op"] == "backward":
        b += 4 * cols
    return {"bytes": b, "flops": rows * cols * {"quantize": 4, "forward": 16, "backward": 16}[case["op"]]}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_quantized(x, fmt):
    """For each block the scale by search over powers of two, for each element the nearest
    representable value by search in the sorted list of them (ties: the even code)."""
    x = x.double()
    rows, cols = x.shape
    dev = x.device
    if fmt == "e2m1":
        grid = torch.tensor(LEVELS, dtype=torch.float64, device=dev)
    else:  # code 0..126 of E4M3: subnormals m/8 * 2^-6, then (1 + m/8) * 2^(x - 7)
        c = torch.arange(127, device=dev, dtype=torch.float64)
        ex, m = torch.floor(c / 8), torch.remainder(c, 8)
        grid = torch.where(ex == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(ex - 7))
    powers = torch.exp2(torch.arange(-127, 128, device=dev, dtype=torch.float64))
    nb = -(-cols // BLOCK)
    pad = torch.zeros((rows, nb * BLOCK), dtype=torch.float64, device=dev)
    pad[:, :cols] = x
    amax = pad.abs().view(rows, nb, BLOCK).max(dim=2).values
    if fmt == "e2m1":  # the largest power of two with 4 * power <= amax
        at = torch.searchsorted(4 * powers, amax.contiguous(), right=True) - 1
    else:  # the smallest one with amax <= 448 * power
        at = torch.searchsorted(448 * powers, amax.contiguous(), right=False)
    scale = powers[at.clamp(0, 254)].repeat_interleave(BLOCK, dim=1)[:, :cols]
    a = (x.abs() / scale).contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(a >= grid[-1], torch.full_like(code, grid.numel() - 1), code)
    return torch.sign(x) * grid[code] * scale


def _exact_stored(Q, S, fmt, cols):
    rows = Q.shape[0]
    dev = Q.device
    nb = Q.shape[1] // (16 if fmt == "e2m1" else 32)
    r = torch.arange(rows, device=dev).unsqueeze(1)
    j = torch.arange(cols, device=dev).unsqueeze(0)
    b = j // BLOCK
    at = ((r // 128) * (-(-nb // 4)) + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4
    scale = torch.exp2(S[at].double() - 127)
    if fmt == "e2m1":
        code = (Q[:, torch.arange(cols, device=dev) // 2].to(torch.int32) >> (4 * (j % 2)).to(torch.int32)) & 15
        mag, sign = code & 7, code >> 3
        ex, m = mag >> 1, (mag & 1).double()
        val = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(ex.double() - 1))
    else:
        code = Q[:, :cols].to(torch.int32)
        mag, sign = code & 127, code >> 7
        ex, m = mag >> 3, (mag & 7).double()
        val = torch.where(ex == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(ex.double() - 7))
    return torch.where(sign == 1, -val, val) * scale


def _exact_act(act, x, slope=False):
    """The activation, or its derivative, of float64 values."""
    if act == "none":
        return torch.ones_like(x) if slope else x
    if act == "relu":
        return torch.where(x > 0, torch.ones_like(x) if slope else x, torch.zeros_like(x))
    if act == "gelu":
        cdf = torch.special.ndtr(x)
        return cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi) if slope else x * cdf
    # x * sigmoid(u(x)), u = x or, for the tanh form, 2 sqrt(2/pi) (x + 0.044715 x^3)
    c = 0.0 if act == "silu" else 0.044715
    w = 1.0 if act == "silu" else 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(w * (x + c * x ** 3))
    if not slope:
        return x * s
    return s + x * s * torch.sigmoid(-w * (x + c * x ** 3)) * w * (1 + 3 * c * x * x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["X"].t() if case["transpose"] else s["X"]
        return _exact_quantized(x, case["format"])
    if case["op"] == "product":
        c = torch.matmul(_exact_stored(s["A"], s["SA"], "e2m1", case["k"]),
                         _exact_stored(s["B"], s["SB"], "e2m1", case["k"]).t())
        if s["bias_v"] is not None:
            c = c + s["bias_v"].double()
        c = _exact_act(case["activation"], c)
        return c if s["residual_v"] is None else c + s["residual_v"].double()
    if case["op"] == "forward":
        z = s["Z"].double()
        return _exact_act(case["activation"], z), _exact_quantized(z, "e4m3")
    z = _exact_stored(s["Q"], s["S"], "e4m3", case["cols"])
    dz = s["dY"].double() * _exact_act(case["activation"], z, slope=True)
    return dz, dz.sum(dim=0)
