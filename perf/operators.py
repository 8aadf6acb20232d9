"""Cases and plain forms of the int8 linear and of the gradients around it.

Operators (all over packed weight rows as written by ``quantize_pack``,
canonical layout):

* ``forward``: x bf16 [M, K] is quantized per token to 8 bits (one scale per
  token) and multiplied in integers with the b-bit codes of the rows (one
  scale per row): y bf16 [M, N].
* ``backward``: from dy bf16 [M, N] the gradient of x through the packed rows
  (bf16 [M, K]) and the gradient of W from the 8-bit codes of x that the
  forward pass kept ([N, K], bf16 or fp32).
* ``step``: quantize, forward and backward of one linear, as one training or
  calibration step calls them.

``run`` computes the plain form unless ``own`` is set.
"""
import math

import torch

own = False

XQ = 127  # largest 8-bit code


def _case(name, op, M, N, K, bits, dw="none"):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "bits": bits, "dw": dw}


def listed():
    return [
        # one token through the smallest matrix of a decoder layer (k or v): latency
        _case("decode_1_kv", "forward", 1, 1024, 5120, 5),
        # one token through the largest matrix (gate or up): the weight stream
        _case("decode_1_gate", "forward", 1, 17408, 5120, 6),
        # eight sequences decoded together, output projection
        _case("decode_8_o", "forward", 8, 5120, 6144, 6),
        # a batch of decoded and drafted tokens
        _case("batch_48", "forward", 48, 4096, 4096, 4),
        # a short prompt of odd length through the down projection
        _case("prompt_333_down", "forward", 333, 5120, 17408, 7),
        # prefill of 2048 tokens, largest matrix at the recipe's usual width
        _case("prefill_2048_up", "forward", 2048, 17408, 5120, 6),
        # prefill through 8-bit rows
        _case("prefill_2048_w8", "forward", 2048, 5120, 5120, 8),
        # gradients of a small matrix for a short calibration sequence
        _case("backward_64_kv", "backward", 64, 1024, 5120, 5, "bf16"),
        # gradients of the largest matrix for a full micro-batch
        _case("backward_2048_up", "backward", 2048, 17408, 5120, 6, "bf16"),
        # fp32 weight gradients, as calibration statistics accumulate them
        _case("backward_1000_o_fp32", "backward", 1000, 5120, 6144, 7, "fp32"),
        # sizes that no tile or 16-byte row divides
        _case("backward_odd", "backward", 515, 1031, 777, 8, "bf16"),
        # one whole step of a square matrix
        _case("step_256", "step", 256, 4096, 4096, 4, "bf16"),
    ]


def draw(rng):
    def log_between(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["forward", "forward", "forward", "backward", "backward", "step"])
    bits = rng.randint(4, 8)
    M = log_between(1 if op == "forward" else 16, 2048)
    if rng.random() < 0.3 and M > 8:
        M -= M % 8
    N = log_between(256, 17408)
    K = log_between(256, 17408)
    while N * K > 17408 * 5120:
        N, K = (N // 2, K) if N > K else (N, K // 2)
    if rng.random() < 0.6:  # most matrices have sizes of whole 64s
        N, K = max(64, N - N % 64), max(64, K - K % 64)
    return {"op": op, "M": M, "N": N, "K": K, "bits": bits,
            "dw": "none" if op == "forward" else rng.choice(["bf16", "bf16", "fp32"])}


def _row_bytes(K, bits):
    return 16 * ((K * bits + 127) // 128)


def _pack(q, bits):
    """Codes int [N, K] -> canonical rows uint8 [N, row bytes], LSB first along K."""
    N, K = q.shape
    u = (q & ((1 << bits) - 1)).to(torch.uint8)
    b = (u.unsqueeze(-1) >> torch.arange(bits, device=q.device, dtype=torch.uint8)) & 1
    rb = _row_bytes(K, bits)
    b = torch.nn.functional.pad(b.reshape(N, K * bits), (0, 8 * rb - K * bits)).reshape(N, rb, 8)
    b <<= torch.arange(8, device=q.device, dtype=torch.uint8)
    return b.sum(-1, dtype=torch.uint8)


def prepare(case, seed):
    M, N, K, bits = case["M"], case["N"], case["K"], case["bits"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q = (1 << (bits - 1)) - 1
    W = torch.randn((N, K), generator=g, device="cuda") * 0.02
    scales = W.abs().amax(1) / Q
    packed = _pack(torch.round(W / scales[:, None]).to(torch.int32), bits)
    del W
    # activations of a normalised hidden state with a few large channels
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")] *= 8.0
    x = x.to(torch.bfloat16)
    st = {"case": dict(case), "packed": packed, "scales": scales}
    if case["op"] != "backward":
        st["x"] = x
    if case["op"] != "forward":
        st["dy"] = (torch.randn((M, N), generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
    if case["op"] == "backward":  # what the forward pass kept of x
        xf = x.float()
        st["sx"] = xf.abs().amax(1) / XQ
        xq = torch.round(xf / st["sx"][:, None]).to(torch.int8)
        st["xq"] = torch.nn.functional.pad(xq, (0, -K % 16)).view(torch.uint8)
    return st


# ---- plain forms ----------------------------------------------------------


def _plain_codes(packed, K, bits):
    k = torch.arange(K, device=packed.device) * bits
    p = torch.nn.functional.pad(packed, (0, 1)).to(torch.int32)
    u = ((p[:, k >> 3] | (p[:, (k >> 3) + 1] << 8)) >> (k & 7).to(torch.int32)) & ((1 << bits) - 1)
    return (u - ((u >> (bits - 1)) << bits)).float()


def _plain_quantize_x(x):
    xf = x.float()
    m = xf.abs().amax(1)
    sx = torch.where(m == 0, torch.ones_like(m), m) / XQ
    return torch.round(xf / sx[:, None]).clamp(-XQ, XQ), sx


def _plain_forward(codes, sx, q, scales):
    return ((codes @ q.T) * scales * sx[:, None]).to(torch.bfloat16)


def _plain_grad_x(dy, q, scales):
    return (dy.float() @ (q * scales[:, None])).to(torch.bfloat16)


def _plain_grad_w(dy, codes, sx, dtype):
    return (dy.float().T @ (codes * sx[:, None])).to(dtype)


# ---- one pass -------------------------------------------------------------


def _dw_dtype(case):
    return torch.float32 if case["dw"] == "fp32" else torch.bfloat16


def run(state):
    c = state["case"]
    K, bits, packed, scales = c["K"], c["bits"], state["packed"], state["scales"]
    if own:
        import mixed_precision_weight_row_b200 as mpw

        out = {}
        if c["op"] == "backward":
            xq, sx = state["xq"], state["sx"]
        else:
            xq, sx = mpw.quantize_x_int8(state["x"])
            out["y"] = mpw.qlinear_int8(None, packed, scales, bits, xq=xq, sx=sx, K=K)
        if c["op"] != "forward":
            out["dx"] = mpw.qlinear_grad_x(state["dy"], packed, scales, bits, K)
            out["dW"] = mpw.qlinear_grad_w_int8(state["dy"], xq, sx, K, dtype=_dw_dtype(c))
        return out
    out = {}
    q = _plain_codes(packed, K, bits)
    if c["op"] == "backward":
        codes, sx = state["xq"].view(torch.int8)[:, :K].float(), state["sx"]
    else:
        codes, sx = _plain_quantize_x(state["x"])
        out["y"] = _plain_forward(codes, sx, q, scales)
    if c["op"] != "forward":
        out["dx"] = _plain_grad_x(state["dy"], q, scales)
        out["dW"] = _plain_grad_w(state["dy"], codes, sx, _dw_dtype(c))
    return out


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    weights = N * _row_bytes(K, case["bits"]) + 4 * N
    nbytes, products = weights, 0
    if case["op"] != "backward":
        nbytes += 2 * M * K + 2 * M * N
        products += 1
    else:
        nbytes += M * K + 4 * M
    if case["op"] != "forward":
        nbytes += 2 * M * N + 2 * M * K + (4 if case["dw"] == "fp32" else 2) * N * K
        products += 2
    return {"bytes": nbytes, "flops": 2 * M * N * K * products}


# ---- the definition in 64 bits ---------------------------------------------


def _exact_codes(packed, K, bits):
    """Each code from its own bits: sum of bit j times 2^j, the top one negative."""
    place = torch.tensor([2.0 ** j for j in range(bits - 1)] + [-(2.0 ** (bits - 1))], dtype=torch.float64,
                         device=packed.device)
    rows = []
    for part in packed.split(512):
        b = torch.stack([(part >> i) & 1 for i in range(8)], dim=-1).reshape(part.shape[0], -1)
        rows.append(b[:, :K * bits].reshape(part.shape[0], K, bits).double() @ place)
    return torch.cat(rows)


def exact(case, seed):
    st = prepare(case, seed)
    K, bits = case["K"], case["bits"]
    w = _exact_codes(st["packed"], K, bits) * st["scales"].double()[:, None]
    if case["op"] == "backward":
        x8 = st["xq"].to(torch.int16)
        x8 = (x8 - 256 * (x8 > 127))[:, :K].double() * st["sx"].double()[:, None]
    else:
        # the scale and the quotient are 32-bit values by definition
        x = st["x"].double()
        top = x.abs().max(dim=1, keepdim=True).values
        s = (torch.where(top > 0, top, torch.ones_like(top)) / 127.0).float().double()
        x8 = torch.clamp((x / s).float().double().round(), -127, 127) * s
    out = {}
    if case["op"] != "backward":
        out["y"] = torch.einsum("mk,nk->mn", x8, w)
    if case["op"] != "forward":
        dy = st["dy"].double()
        out["dx"] = torch.einsum("mn,nk->mk", dy, w)
        out["dW"] = torch.einsum("mn,mk->nk", dy, x8)
    return out
