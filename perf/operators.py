"""The 8-bit operators, with the cases they are measured on.

Three operators, each in its plain form (elementary torch operations) and as the
calls of the package:

  int8_linear  y = x W^T + bias from 8-bit integers: each token x_t is scaled by
               its largest magnitude a_t and rounded to q = nearest(127 x / a_t)
               (ties to even), the weights are already 8-bit integers with one
               scale for each output channel, and
               y[t, o] = (sum_k q[t, k] w[o, k]) (a_t / 127) scale[o] + bias[o].
  checkpoint   an activation matrix stored in 8 bits and restored: blocks of 32
               entries of a row share the smallest power of two s with
               max |x| <= 127 s, and |x| / s is rounded to one of its two
               neighbouring integers without bias, by 16 random bits for each
               entry (Philox4x32-10 keyed by the seed).
  wgrad        the weight gradient of a linear layer from such a checkpoint:
               dW[o, i] = sum_t dY[t, o] s[t, i / 32] q[t, i].

An 8-bit matrix lies in rows of a whole number of 32 bytes (checkpoint: blocks
of 32 entries; its scale bytes in rows of a whole number of 16 bytes, the byte b
standing for 2^(b - 127)), which is how the package's own calls lay it out.
"""
import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_STREAM = 2  # third counter word of the checkpoint's Philox blocks


def listed():
    return [
        # one new token through a square projection: latency
        {"name": "token", "op": "int8_linear", "m": 1, "n": 4096, "k": 4096, "type": "bf16", "bias": False},
        # a few sequences, one token each, odd layer sizes, float32 activations
        {"name": "tokens, odd sizes", "op": "int8_linear", "m": 7, "n": 3001, "k": 4099, "type": "fp32", "bias": True},
        # a serving batch, one token for each sequence, through a wide layer
        {"name": "batch", "op": "int8_linear", "m": 64, "n": 16384, "k": 4096, "type": "bf16", "bias": True},
        # a prompt of a thousand tokens, odd layer sizes, half precision
        {"name": "prompt, odd sizes", "op": "int8_linear", "m": 1000, "n": 4099, "k": 3001, "type": "fp16", "bias": True},
        # many prompts at once through a layer's narrowing projection: throughput
        {"name": "prompts", "op": "int8_linear", "m": 16384, "n": 4096, "k": 16384, "type": "bf16", "bias": False},
        # the activations of a few tokens (a short sequence, an expert's share)
        {"name": "store few", "op": "checkpoint", "t": 64, "k": 4096, "type": "bf16"},
        # an odd number of tokens and of features, float32
        {"name": "store, odd sizes", "op": "checkpoint", "t": 3001, "k": 777, "type": "fp32"},
        # a training batch's activations of one layer
        {"name": "store", "op": "checkpoint", "t": 16384, "k": 4096, "type": "bf16"},
        # weight gradient of a square projection over a training batch
        {"name": "gradient", "op": "wgrad", "t": 16384, "o": 4096, "k": 4096, "type": "bf16"},
        # ragged batch and layer sizes, half precision
        {"name": "gradient, odd sizes", "op": "wgrad", "t": 777, "o": 1000, "k": 3001, "type": "fp16"},
        # a small layer (an adapter, a head) over many tokens: the sum is the long axis
        {"name": "gradient, long sum", "op": "wgrad", "t": 65536, "o": 512, "k": 512, "type": "bf16"},
        # float32 gradients over a medium batch
        {"name": "gradient, float32", "op": "wgrad", "t": 4096, "o": 4096, "k": 1024, "type": "fp32"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm; half of them multiples of 64 where that is in range."""
    v = int(round(2.0 ** rng.uniform(np.log2(lo), np.log2(hi))))
    if v >= 64 and rng.random() < 0.5:
        v -= v % 64
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["int8_linear", "checkpoint", "wgrad"])
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "int8_linear":
        c = {"op": op, "m": _log(rng, 1, 16384), "n": _log(rng, 64, 16384), "k": _log(rng, 64, 16384), "type": kind,
             "bias": rng.random() < 0.5}
        while c["m"] * c["n"] * c["k"] > 1 << 40:
            c["m"] = c["m"] // 2 + 1
        return c
    if op == "checkpoint":
        c = {"op": op, "t": _log(rng, 1, 16384), "k": _log(rng, 64, 16384), "type": kind}
        while c["t"] * c["k"] > 1 << 26 or (kind == "fp32" and c["t"] * c["k"] > 1 << 25):
            c["t"] = c["t"] // 2 + 1
        return c
    c = {"op": op, "t": _log(rng, 1, 65536), "o": _log(rng, 64, 4096), "k": _log(rng, 64, 4096), "type": kind}
    while c["t"] * c["o"] * c["k"] > (1 << 38 if kind == "bf16" else 1 << 36):
        c["t"] = c["t"] // 2 + 1
    return c


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _padded(rows, cols, to):
    """Zeroed bytes, int8, in rows of a whole number of `to` bytes: the [rows, cols] part of them."""
    return torch.zeros((rows, (cols + to - 1) // to * to), dtype=torch.int8, device="cuda")[:, :cols]


def _activations(g, t, k, kind):
    """Normal entries, token norms log-normal, one feature in a hundred 20 times larger."""
    x = torch.randn((t, k), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((t, 1), generator=g, device="cuda"))
    x *= torch.where(torch.rand((1, k), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(_TYPES[kind])


def _weights8(g, n, k):
    """Student-t weights (four degrees of freedom) in 8-bit integers, one scale for each row."""
    w = 0.02 * torch.randn((n, k), generator=g, device="cuda")
    c = sum(torch.randn((n, k), generator=g, device="cuda") ** 2 for _ in range(4))
    w = w / torch.sqrt(c / 4)
    a = w.abs().amax(1, keepdim=True)
    q = _padded(n, k, 32)
    q.copy_(torch.round(w * (127 / a)))
    return q, (a / 127).reshape(n)


def _store8(x):
    """A checkpoint of float32 x, rounded to nearest: its integers and its scale bytes."""
    t, k = x.shape
    blocks = (k + 31) // 32
    full = torch.zeros((t, blocks * 32), device="cuda")
    full[:, :k] = x
    e = torch.ceil(torch.log2(full.reshape(t, blocks, 32).abs().amax(2).clamp_min(1e-30) / 127))
    q, b = _padded(t, k, 32), _padded(t, blocks, 16).view(torch.uint8)
    v = torch.round(full.reshape(t, blocks, 32) / torch.exp2(e)[:, :, None]).clamp(-127, 127)
    q.copy_(v.reshape(t, -1)[:, :k])
    b.copy_(e + 127)
    return q, b


def prepare(case, seed):
    g = _rng(seed)
    if case["op"] == "int8_linear":
        w, scale = _weights8(g, case["n"], case["k"])
        bias = torch.randn(case["n"], generator=g, device="cuda") if case["bias"] else None
        return {"op": "int8_linear", "x": _activations(g, case["m"], case["k"], case["type"]), "w": w, "scale": scale,
                "bias": bias}
    if case["op"] == "checkpoint":
        return {"op": "checkpoint", "x": _activations(g, case["t"], case["k"], case["type"]), "seed": 1000 + seed}
    q, b = _store8(_activations(g, case["t"], case["k"], "fp32"))
    dy = 1e-3 * torch.randn((case["t"], case["o"]), generator=g, device="cuda")
    dy *= torch.exp(torch.randn((case["t"], 1), generator=g, device="cuda"))
    dy *= torch.where(torch.rand(dy.shape, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    return {"op": "wgrad", "dy": dy.to(_TYPES[case["type"]]), "q": q, "b": b}


def _random16(seed, t, k):
    """16 random bits for each entry: entry j of row r takes half j & 1 of word (j >> 1) & 3 of the Philox4x32-10 block
    with counter (j >> 3, r, 2, 0) and key (low, high word of the seed)."""
    low = 0xFFFFFFFF
    n = (k + 7) // 8
    c0 = torch.arange(n, device="cuda").expand(t, n)
    c1 = torch.arange(t, device="cuda")[:, None].expand(t, n)
    c2 = torch.full((), _STREAM, device="cuda", dtype=torch.int64).expand(t, n)
    c3 = torch.zeros((), device="cuda", dtype=torch.int64).expand(t, n)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits are exact, and with them both halves
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack((c0, c1, c2, c3), 2)
    return torch.stack((words & 0xFFFF, words >> 16), 3).reshape(t, n * 8)[:, :k]


def _linear_plain(x, w, scale, bias):
    x = x.float()
    a = x.abs().amax(1, keepdim=True)
    # in 64 bits: whether 127 x / a lies above or below a half decides the integer
    q = torch.round(x.double() * 127 / a.double().clamp_min(1e-300)).float()
    y = (q @ w.float().T) * (a / 127) * scale
    return y if bias is None else y + bias


def _checkpoint_plain(x, seed):
    t, k = x.shape
    blocks = (k + 31) // 32
    full = torch.zeros((t, blocks * 32), device="cuda")
    full[:, :k] = x
    m = full.reshape(t, blocks, 32).abs()
    big = m.amax(2, keepdim=True)
    mantissa, exponent = torch.frexp(big)  # mantissa in [0.5, 1), 127 = (127 / 128) 2^7
    exponent = torch.clamp(exponent - 7 + (mantissa > 127 / 128), min=-126)
    s = torch.ldexp(torch.ones_like(big), exponent)
    v = m / s
    low = torch.floor(v)
    up = _random16(seed, t, blocks * 32).reshape(t, blocks, 32) < torch.round((v - low) * 65536)
    v = torch.where(full.reshape(t, blocks, 32) < 0, -1.0, 1.0) * (low + up) * s
    return v.reshape(t, -1)[:, :k]


def _wgrad_plain(dy, q, b):
    s = torch.exp2(b.float() - 127).repeat_interleave(32, dim=1)[:, : q.shape[1]]
    return dy.float().T @ (q.float() * s)


def run(state):
    if state["op"] == "int8_linear":
        if own:
            from entropy_constrained_unbiased_b200 import linear as L

            return L.int8_linear(state["x"], state["w"], state["scale"], state["bias"])
        return _linear_plain(state["x"], state["w"], state["scale"], state["bias"]).to(state["x"].dtype)
    if state["op"] == "checkpoint":
        if own:
            from entropy_constrained_unbiased_b200 import ecasq as E

            q, b = E.checkpoint8(state["x"], state["seed"])
            return E.checkpoint8_restore(q, b, state["x"].dtype)
        return _checkpoint_plain(state["x"], state["seed"]).to(state["x"].dtype)
    if own:
        from entropy_constrained_unbiased_b200 import ecasq as E

        return E.checkpoint8_wgrad(state["dy"], state["q"], state["b"])
    return _wgrad_plain(state["dy"], state["q"], state["b"]).to(state["dy"].dtype)


def work(case):
    if case["op"] == "int8_linear":
        m, n, k, w = case["m"], case["n"], case["k"], _SIZE[case["type"]]
        return {"bytes": m * k * w + n * k + 4 * n + (4 * n if case["bias"] else 0) + m * n * w, "flops": 2 * m * n * k}
    if case["op"] == "checkpoint":
        t, k, w = case["t"], case["k"], _SIZE[case["type"]]
        # read, stored (integers and scale bytes) and restored
        return {"bytes": t * k * 2 * w + t * k + t * ((k + 31) // 32), "flops": 4 * t * k}
    t, o, k, w = case["t"], case["o"], case["k"], _SIZE[case["type"]]
    return {"bytes": t * o * w + t * k + t * ((k + 31) // 32) + o * k * w, "flops": 2 * t * o * k}


def _philox_np(seed, rows, n):
    """The words of the blocks (0 .. n-1) of the given rows, in numpy's unsigned 64-bit arithmetic: [rows, n, 4]."""
    u = np.uint64
    low, shift = u(0xFFFFFFFF), u(32)
    x = [np.broadcast_to(np.arange(n, dtype=u), (len(rows), n)), np.broadcast_to(rows.astype(u)[:, None], (len(rows), n)),
         np.full((len(rows), n), _STREAM, u), np.zeros((len(rows), n), u)]
    keys = [u(seed & 0xFFFFFFFF), u(seed >> 32)]
    for r in range(10):
        p, s = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(s >> shift) ^ x[1] ^ keys[0], s & low, (p >> shift) ^ x[3] ^ keys[1], p & low]
        keys = [u((int(keys[0]) + 0x9E3779B9) & 0xFFFFFFFF), u((int(keys[1]) + 0xBB67AE85) & 0xFFFFFFFF)]
    return np.stack(x, -1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "int8_linear":
        x = state["x"].double()
        out = torch.empty((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        w = state["w"].double()
        for r in range(0, case["m"], 2048):
            part = x[r : r + 2048]
            a = part.abs().max(dim=1, keepdim=True).values
            z = part * 127 / a
            z[a.expand_as(z) == 0] = 0
            f = torch.floor(z)
            d = z - f
            f += (d > 0.5) | ((d == 0.5) & (torch.remainder(f, 2) == 1))
            out[r : r + 2048] = torch.einsum("tk,ok->to", f, w) * a / 127 * state["scale"].double()
        return out if state["bias"] is None else out + state["bias"].double()
    if case["op"] == "checkpoint":
        x = state["x"].double().cpu().numpy()
        t, k = x.shape
        out = np.empty((t, k))
        blocks = (k + 31) // 32
        for r in range(0, t, 1024):
            rows = np.arange(r, min(t, r + 1024))
            part = np.zeros((len(rows), blocks * 32))
            part[:, :k] = x[rows]
            size = np.abs(part).reshape(len(rows), blocks, 32)
            top = size.max(2)
            s = np.exp2(np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 127)), -126))
            s = np.where(top > 127 * s, 2 * s, s)  # the logarithm's last bit
            s = np.where((top <= 127 * s / 2) & (s > 2.0**-126), s / 2, s)
            z = size / s[:, :, None]
            words = _philox_np(state["seed"], rows, blocks * 4)
            bits = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1).reshape(z.shape).astype(np.float64)
            near = np.floor(z) + (bits < np.rint((z - np.floor(z)) * 65536))
            out[rows] = np.copysign(near * s[:, :, None], part.reshape(z.shape)).reshape(len(rows), -1)[:, :k]
        return torch.from_numpy(out)
    t, k = state["q"].shape
    total = torch.zeros((case["o"], k), dtype=torch.float64, device="cuda")
    for r in range(0, t, 8192):
        s = torch.pow(2.0, state["b"][r : r + 8192].double() - 127)
        block = torch.arange(k, device="cuda") // 32
        total += torch.einsum("to,ti->oi", state["dy"][r : r + 8192].double(), state["q"][r : r + 8192].double() * s[:, block])
    return total
