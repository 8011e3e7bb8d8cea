"""Timing cases of the operators on microscaled 4-bit floating point (blocks of 32 e2m1 values with one
e8m0 scale): quantization of activations, the product of activations with 4-bit weights, and the
gated feed-forward projection act(x Wg^T) * (x Wu^T) over such weights.  The products take activations
in 16 bits as they are, or quantized to the same 4-bit format.

`run` computes one pass, either in plain torch operations (`own` false) or through the package's entry
points (`own` true); both take the same state.  Codes are uint8 [rows, K / 2], the even element in the
low four bits (bit 3 the sign, bits 2..0 one of 0 0.5 1 1.5 2 3 4 6); scales are uint8 [rows, K / 32],
2 ** (byte - 127).  Sizes follow from the case alone, values from the seed.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_LARGEST = 4096 * 8192 * 28672          # multiply-adds of the largest listed case


# ---- cases ---------------------------------------------------------------------------------------

def _quantize(name, rows, inner, dtype):
    return {"name": name, "op": "quantize", "rows": rows, "inner": inner, "dtype": dtype}


def _product(name, rows, inner, outer, x, dtype):
    return {"name": name, "op": "product", "rows": rows, "inner": inner, "outer": outer, "x": x, "dtype": dtype}


def _gated(name, rows, inner, outer, x, act, dtype):
    return {"name": name, "op": "gated", "rows": rows, "inner": inner, "outer": outer, "x": x, "act": act,
            "dtype": dtype}


def listed():
    return [
        # one token's hidden state before a 4-bit product: latency
        _quantize("quantize_one_row", 1, 4096, "bf16"),
        # a prompt chunk of odd length, the inputs of a down projection
        _quantize("quantize_prompt", 2777, 14336, "f16"),
        # one user chatting: one row through an up projection, weights in 4 bits, the row as it is
        _product("product_one_row", 1, 4096, 14336, "16", "bf16"),
        # a decode batch, activations as they are
        _product("product_decode_batch", 16, 8192, 28672, "16", "f16"),
        # a decode batch in 4 bits on both sides
        _product("product_decode_batch_mx", 61, 8192, 8192, "mx", "bf16"),
        # a short prompt: more rows than a decode batch, too few to fill the card with large tiles
        _product("product_short_prompt_mx", 257, 4096, 4096, "mx", "bf16"),
        # a ragged chunk against an odd number of outputs, inputs that end inside a tile
        _product("product_ragged_mx", 1301, 4160, 4001, "mx", "f16"),
        # a prompt with activations as they are
        _product("product_prompt", 2048, 4096, 14336, "16", "bf16"),
        # the compute-bound end
        _product("product_prompt_mx", 4096, 8192, 28672, "mx", "bf16"),
        # one token through both projections of a feed-forward block
        _gated("gated_one_row", 1, 4096, 14336, "16", "silu", "bf16"),
        # a decode batch through the block
        _gated("gated_decode_batch", 48, 4096, 14336, "16", "gelu_tanh", "f16"),
        # a prompt through the block, 4 bits on both sides
        _gated("gated_prompt_mx", 2003, 8192, 14336, "mx", "silu", "bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    op = rng.choice(["quantize", "product", "product", "product", "gated", "gated"])
    inner = 32 * _log_int(rng, 4, 448)
    if op == "quantize":
        return _quantize("drawn", _log_int(rng, 1, 8192), inner, dtype)
    outer = _log_int(rng, 40, 28672 if op == "product" else 14336)
    if rng.random() < 0.5:
        outer = -(-outer // 32) * 32
    room = _LARGEST // (inner * outer * (1 if op == "product" else 2))
    rows = rng.choice([_log_int(rng, 1, 64), _log_int(rng, 1, 64), _log_int(rng, 65, 512), _log_int(rng, 65, 4096)])
    rows = max(1, min(rows, room))
    x = rng.choice(["16", "mx"])
    if op == "product":
        return _product("drawn", rows, inner, outer, x, dtype)
    return _gated("drawn", rows, inner, outer, x, rng.choice(["silu", "gelu_tanh"]), dtype)


def work(case):
    rows, inner = case["rows"], case["inner"]
    packed = inner / 2 + inner / 32                     # bytes of a quantized row
    if case["op"] == "quantize":
        # x in, codes and scales out, and the values read back from them
        return {"bytes": int(rows * (2 * inner + 2 * packed + 2 * inner)), "flops": 4 * rows * inner}
    outer, sides = case["outer"], 2 if case["op"] == "gated" else 1
    x = packed if case["x"] == "mx" else 2 * inner
    return {"bytes": int(sides * outer * packed + rows * x + 2 * rows * outer),
            "flops": 2 * sides * rows * inner * outer}


# ---- the plain forms -----------------------------------------------------------------------------

def _plain_quantize(x):
    """(codes, scales): the block's scale is 2 ** (floor(log2 max|x|) - 2) within 2 ** +-127, a value the
    nearest of the format's after division by it, ties to the even code, past 6 to 6."""
    rows, inner = x.shape
    blocks = x.float().reshape(rows, inner // 32, 32)
    most = blocks.abs().amax(-1)
    exponent = torch.frexp(most).exponent - 3
    exponent = torch.where(most > 0, exponent.clamp(-127, 127), torch.full_like(exponent, -127))
    size = (blocks.double() * torch.exp2(-exponent.double())[..., None]).abs()
    code = ((size > 0.25).to(torch.uint8) + (size >= 0.75) + (size > 1.25) + (size >= 1.75) + (size > 2.5)
            + (size >= 3.5) + (size > 5.0)).to(torch.uint8)
    code = (code + 8 * torch.signbit(blocks).to(torch.uint8)).reshape(rows, inner)
    return code[:, 0::2] + 16 * code[:, 1::2], (exponent + 127).to(torch.uint8)


def _plain_values(codes, scales):
    """float32 [rows, K] of codes and scales."""
    rows = codes.shape[0]
    sixteen = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
    pair = torch.stack((sixteen.repeat(16), sixteen.repeat_interleave(16)), -1)      # by byte: low, high
    value = pair[codes.int()].reshape(rows, -1, 32)
    return (value * torch.exp2(scales.float() - 127.0)[..., None]).reshape(rows, -1)


def _plain_act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain(s):
    c = s["case"]
    dt = _DTYPES[c["dtype"]]
    if c["op"] == "quantize":
        codes, scales = _plain_quantize(s["x"])
        return {"values": _plain_values(codes, scales).to(dt), "scales": scales}
    x = s["x"].float() if c["x"] == "16" else _plain_values(s["x_codes"], s["x_scales"])
    if c["op"] == "product":
        return torch.matmul(x, _plain_values(s["w_codes"], s["w_scales"]).t()).to(dt)
    gate = torch.matmul(x, _plain_values(s["g_codes"], s["g_scales"]).t())
    return (_plain_act(gate, c["act"]) * torch.matmul(x, _plain_values(s["u_codes"], s["u_scales"]).t())).to(dt)


# ---- state ---------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 2 + 1)
    rows, inner = case["rows"], case["inner"]
    state = {"case": case}

    # activations: normal values, some inputs several times larger than the others in every row
    size = torch.empty(inner, device=dev).normal_(0.0, 0.5, generator=gen).exp_()
    x = torch.empty((rows, inner), device=dev).normal_(generator=gen).mul_(size).to(_DTYPES[case["dtype"]])
    if case["op"] == "quantize":
        return state | {"x": x}
    if case["x"] == "mx":
        state["x_codes"], state["x_scales"] = _plain_quantize(x)
    else:
        state["x"] = x

    def weights(std):
        # rows of different size, quantized as a checkpoint holds them
        w = torch.empty((case["outer"], inner), device=dev).normal_(0.0, std, generator=gen)
        w *= torch.empty((case["outer"], 1), device=dev).normal_(0.0, 0.3, generator=gen).exp_()
        step = max(1, (1 << 26) // inner)
        parts = [_plain_quantize(w[i:i + step]) for i in range(0, case["outer"], step)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])

    for side in ("w",) if case["op"] == "product" else ("g", "u"):
        state[side + "_codes"], state[side + "_scales"] = weights(inner ** -0.5)
    return state


# ---- the package's entry points ------------------------------------------------------------------

def _own_run(s):
    import weight_only_quantized_amd as wq
    c = s["case"]
    dt = _DTYPES[c["dtype"]]
    if c["op"] == "quantize":
        t = wq.MXTensor.quantize(s["x"])
        return {"values": t.dequantize(dt), "scales": t.scales}
    if "layer" not in s:                      # a program lays its weights out once, when it loads them
        if c["op"] == "product":
            s["layer"] = wq.MXLinear(wq.MXTensor(s["w_codes"], s["w_scales"]))
        else:
            s["layer"] = wq.MXGatedLinear(wq.MXTensor(s["g_codes"], s["g_scales"]),
                                          wq.MXTensor(s["u_codes"], s["u_scales"]), activation=c["act"])
        if c["x"] == "mx":
            s["x"] = wq.MXTensor(s["x_codes"], s["x_scales"])
    return s["layer"].gemm(s["x"], dtype=dt)


def run(state):
    return _own_run(state) if own else _plain(state)


# ---- 64 bits, from the definitions ---------------------------------------------------------------

def _exact_quantized(x):
    """(values, scales) of x quantized: values on the grid of steps 2 ** (floor(log2 size) - 1), at least 0.5."""
    blocks = x.double().reshape(x.shape[0], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    # log2 rounds: a size just below a power of two belongs to the binade under it
    power = torch.where(torch.exp2(power) > top, power - 1, power)
    power = torch.where(top > 0, (power - 2).clamp(-127, 127), torch.full_like(top, -127))
    scaled = blocks / torch.exp2(power)
    step = torch.where(scaled.abs() < 2, 0.5, torch.where(scaled.abs() < 4, 1.0, 2.0))
    value = (torch.round(scaled / step) * step).clamp(-6, 6) * torch.exp2(power)
    return value.reshape(x.shape), (power.squeeze(-1) + 127).to(torch.uint8)


def _exact_values(codes, scales):
    nibble = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    sign = 1.0 - 2.0 * (nibble >> 3).double()
    exponent, odd = (nibble >> 1) & 3, (nibble & 1).double()
    size = torch.where(exponent == 0, 0.5 * odd, (1 + 0.5 * odd) * torch.exp2(exponent.double() - 1))
    return sign * size * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_product(x, codes, scales):
    out = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.float64, device=x.device)
    for i in range(0, codes.shape[0], 4096):
        part = slice(i, i + 4096)
        out[:, part] = x @ _exact_values(codes[part], scales[part]).t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        values, scales = _exact_quantized(s["x"])
        return {"values": values, "scales": scales}
    x = s["x"].double() if case["x"] == "16" else _exact_values(s["x_codes"], s["x_scales"])
    if case["op"] == "product":
        return _exact_product(x, s["w_codes"], s["w_scales"])
    gate = _exact_product(x, s["g_codes"], s["g_scales"])
    up = _exact_product(x, s["u_codes"], s["u_scales"])
    if case["act"] == "silu":
        return gate * torch.sigmoid(gate) * up
    return torch.nn.functional.gelu(gate, approximate="tanh") * up
