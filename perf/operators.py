"""What the microscaled 4-bit (MXFP4) operators compute, in plain torch, and the sizes they are
measured at.

A block is 32 consecutive values of a row: sixteen bytes of e2m1 codes (the even position in the
low nibble) and one power of two, 2^(s - 127), held in a byte.  Four operators stand on it:

  quantize   rows of f32 / f16 / bf16 to blocks, and blocks back to the values they stand for
  product    rows in blocks times weight rows in blocks, for each expert's group of rows
  experts    SwiGLU experts with weights and activations in blocks, over dispatched rows
  tokens     a whole layer (router, top-k, SwiGLU experts, combine) for a few tokens, weights in
             blocks and activations in 16 bits

run() computes the plain form, or calls the package's operators where `own` is true.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# magnitudes of the eight e2m1 codes, and the borders between neighbours; a value on a border goes
# to the even code, which is the upper one where the flag is set
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
UPPER = (False, True, False, True, False, True, False)


def listed():
    return [
        # one token's hidden state on its way into a 4-bit product: pure latency
        dict(name="quantize one token", op="quantize", rows=1, K=2048, pad=0, dtype="bf16"),
        # a batch whose width is no multiple of a block, cut out of a wider buffer
        dict(name="quantize odd slice", op="quantize", rows=4099, K=1357, pad=7, dtype="f32"),
        # all tokens of a long prompt batch at the widest hidden size
        dict(name="quantize prompt", op="quantize", rows=16384, K=7168, pad=0, dtype="bf16"),
        # a few rows for each expert, some experts idle: the weights' bytes count
        dict(name="product few rows", op="product", rows=64, E=16, N=768, K=2048, zipf=1.1, dtype="bf16"),
        # ragged groups and sizes that end inside every tile, 32-bit results
        dict(name="product ragged", op="product", rows=3001, E=7, N=1000, K=1376, zipf=0.6, dtype="f32"),
        # one large dense projection
        dict(name="product dense", op="product", rows=8192, E=1, N=8192, K=8192, zipf=0.0, dtype="bf16"),
        # a decoding batch over many small experts
        dict(name="experts decode", op="experts", T=256, k=8, E=128, H=2048, I=768, zipf=1.1, dtype="bf16"),
        # a prompt batch over many experts with a skewed load
        dict(name="experts skewed", op="experts", T=2048, k=8, E=32, H=7168, I=2048, zipf=1.2, dtype="f16"),
        # a long prompt over few wide experts
        dict(name="experts prefill", op="experts", T=8192, k=2, E=8, H=4096, I=14336, zipf=0.0, dtype="bf16"),
        # the next token of one request, small experts: latency
        dict(name="tokens single", op="tokens", T=1, k=8, E=128, H=2048, I=768, dtype="bf16"),
        # one token for each of a few requests, few wide experts
        dict(name="tokens wide", op="tokens", T=7, k=2, E=8, H=4096, I=14336, dtype="f16"),
        # a small decoding batch over many large experts: the active weights are read once
        dict(name="tokens many experts", op="tokens", T=32, k=8, E=256, H=7168, I=2048, dtype="bf16"),
    ]


def _size(rng, lo, hi, unit=1):
    """A number of units between lo and hi, spread over the logarithm: odd, or a power of two."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return unit * (n | 1 if rng.random() < 0.6 else 1 << (n.bit_length() - 1))


def draw(rng):
    op = rng.choice(("quantize", "product", "experts", "tokens"))
    if op == "quantize":
        K = _size(rng, 32, 8192)
        rows = _size(rng, 1, min(65536, 16384 * 7168 // K - 1))
        return dict(op=op, rows=rows, K=K, pad=rng.choice((0, 0, 8, 5)), dtype=rng.choice(tuple(TYPES)))
    if op == "product":
        E, N, K = _size(rng, 1, 32), _size(rng, 32, 8192), _size(rng, 2, 255, BLOCK)
        while E * N * K > 1 << 28:
            E, N = max(1, E // 2), N // 2 | 1
        return dict(op=op, rows=_size(rng, 1, 8191), E=E, N=N, K=K, zipf=rng.choice((0.0, 0.6, 1.2)), dtype=rng.choice(tuple(TYPES)))
    E = _size(rng, 4, 256 if op == "tokens" else 64)
    unit = 128 if op == "tokens" else rng.choice((32, 32, 8))
    H, I = _size(rng, max(1, 256 // unit), 7167 // unit, unit), _size(rng, max(1, 128 // unit), 14335 // unit, unit)
    while E * H * I > (1 << 31 if op == "tokens" else 1 << 28):
        E, I = max(4, E // 2), unit * (I // unit // 2 | 1)
    k = rng.randint(1, min(E, 8))
    dtype = rng.choice(("f16", "bf16"))
    if op == "tokens":
        return dict(op=op, T=_size(rng, 1, 63), k=k, E=E, H=H, I=I, dtype=dtype)
    return dict(op=op, T=_size(rng, 1, 4095), k=k, E=E, H=H, I=I, zipf=rng.choice((0.0, 0.6, 1.2)), dtype=dtype)


# ----------------------------------------------------------------------------- blocks, plainly
def _quantize(x):
    """(codes, scales) of the rows of x: the exponent is that of the block's largest magnitude
    less two, each value goes to the nearest code (ties to even, past the last one to it), and a
    block with an infinity or a NaN gets the scale byte 255."""
    K = x.shape[-1]
    blocks = -(-K // BLOCK)
    f = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - K)).unflatten(-1, (blocks, BLOCK))
    top = f.abs().amax(-1)
    odd = ~torch.isfinite(f).all(-1)
    top = torch.where(odd, 0.0, top)
    e = torch.where(top > 0, torch.frexp(top).exponent.int() - 3, -127).clamp(-127, 127)
    v = torch.where(odd[..., None], 0.0, f)
    # the power of two in two steps, each of which a normal 32-bit number can hold
    half = (-e).div(2, rounding_mode="floor")
    v = torch.ldexp(torch.ldexp(v, half[..., None]), (-e - half)[..., None])
    m = v.abs()
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for border, up in zip(BORDERS, UPPER):
        code += (m >= border) if up else (m > border)
    code += 8 * torch.signbit(v).to(torch.uint8)
    code = torch.where(odd[..., None], 0, code).flatten(-2)
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = torch.where(odd, 255, e + 127).to(torch.uint8)
    return codes, torch.nn.functional.pad(scales, (0, -blocks % 4))


def _values(codes, scales):
    """The 32-bit values that the blocks stand for; rows end where the last block ends."""
    v = torch.tensor(MAGNITUDES, device=codes.device)
    v = torch.cat((v, -v))
    at = torch.arange(256, device=codes.device)
    pairs = torch.stack((v[at & 15], v[at >> 4]), -1)
    s = torch.arange(256, device=codes.device, dtype=torch.float32)
    power = torch.where(s == 255, torch.nan, torch.ldexp(torch.ldexp(torch.ones_like(s), (s - 127).int() // 2), (s - 127).int() - (s - 127).int() // 2))
    f = pairs[codes.long()].flatten(-2)
    blocks = f.shape[-1] // BLOCK
    return (f.unflatten(-1, (blocks, BLOCK)) * power[scales[..., :blocks].long()][..., None]).flatten(-2)


def _by_group(a, b, offsets, most):
    """rows of a [rows, K] times the transposed b [E, N, K] of their group, in 32 bits."""
    E = b.shape[0]
    row = torch.arange(a.shape[0], device=a.device)
    e = torch.searchsorted(offsets[1:].long(), row, right=True)
    at = row - offsets.long()[e]
    full = a.new_zeros(E, most, a.shape[1])
    full[e, at] = a
    return torch.bmm(full, b.transpose(1, 2))[e, at]


def _fit(v, K):
    return v[..., :K]


# --------------------------------------------------------------------------------- the inputs
def _weights(g, E, N, K, dev):
    """[E, N, K] weights of standard deviation K^-1/2 in blocks: rows drawn from a pool."""
    pool = min(E * N, 2048)
    codes, scales = _quantize(torch.randn(pool, K, generator=g, device=dev) * K**-0.5)
    at = torch.randint(0, pool, (E * N,), generator=g, device=dev)
    return codes[at].view(E, N, -1), scales[at].view(E, N, -1)


def _groups(g, rows, E, zipf, k, dev):
    """The sizes of the experts' groups of rows: top-k of normal scores with a Zipf bias."""
    bias = -zipf * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    bias = bias[torch.randperm(E, generator=g, device=dev)]
    score = torch.randn(rows, E, generator=g, device=dev) + bias
    count = torch.bincount(score.topk(k).indices.flatten(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = count.cumsum(0)
    return offsets, int(count.max())


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = dict(case)
    if op == "quantize":
        wide = case["K"] + case["pad"]
        # activations: a normal body, a scale for each row and some outlying columns
        x = torch.randn(case["rows"], wide, generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(case["rows"], 1, generator=g, device=dev))
        x *= 1 + 15 * (torch.rand(1, wide, generator=g, device=dev) < 0.004)
        s["x"] = x.to(dt)[:, : case["K"]]
    elif op == "product":
        s["offsets"], s["most"] = _groups(g, case["rows"], case["E"], case["zipf"], 1, dev)
        s["a"] = _quantize(torch.randn(case["rows"], case["K"], generator=g, device=dev))
        s["b"] = _weights(g, case["E"], case["N"], case["K"], dev)
    else:
        E, H, I, T = case["E"], case["H"], case["I"], case["T"]
        s["gate"], s["up"] = (_weights(g, E, I, H, dev) for _ in range(2))
        s["down"] = _weights(g, E, H, I, dev)
        rows = T * case["k"] if op == "experts" else T
        s["x"] = torch.randn(rows, H, generator=g, device=dev).to(dt)
        if op == "experts":
            s["offsets"], s["most"] = _groups(g, T, E, case["zipf"], case["k"], dev)
        else:
            # router rows of different lengths, so that some experts are chosen more often
            r = torch.randn(E, H, generator=g, device=dev) * H**-0.5
            s["router"] = (r * (0.7 + 0.6 * torch.rand(E, 1, generator=g, device=dev))).to(dt)
    return s


# ---------------------------------------------------------------------------------- the passes
def run(s):
    return _own(s) if own else _plain(s)


def _plain(s):
    op, dt = s["op"], TYPES[s["dtype"]]
    if op == "quantize":
        return {"values": _fit(_values(*_quantize(s["x"])), s["K"]).to(dt)}
    if op == "product":
        return {"out": _by_group(_values(*s["a"]), _values(*s["b"]), s["offsets"], s["most"]).to(dt)}
    gate, up, down = s["gate"], s["up"], s["down"]
    H, I = s["H"], s["I"]
    if op == "experts":
        # activations in blocks in front of both products; the SwiGLU result is not rounded first
        x = _values(*_quantize(s["x"]))
        g = _by_group(x, _values(*gate), s["offsets"], s["most"])
        u = _by_group(x, _values(*up), s["offsets"], s["most"])
        a = _values(*_quantize(torch.nn.functional.sigmoid(g) * g * u))
        return {"y": _by_group(a, _values(*down), s["offsets"], s["most"]).to(dt)}
    # tokens: which experts are taken is decided in 64 bits; activations stay in 16 bits
    T, k = s["T"], s["k"]
    logits = s["x"].double() @ s["router"].double().T
    top, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    w = torch.softmax(top[:, :k], -1).float()
    at = idx[:, :k].flatten()

    def times(v, m, n):  # each slot's vector times its expert's matrix
        return torch.bmm(_fit(_values(m[0][at], m[1][at]), n), v[:, :, None])[:, :, 0]

    x = s["x"].float().repeat_interleave(k, 0)
    g, u = times(x, gate, H), times(x, up, H)
    a = (torch.nn.functional.sigmoid(g) * g * u).to(dt).float()
    return {"out": (times(a, down, I).view(T, k, H) * w[:, :, None]).sum(1).to(dt)}


def _own(s):
    import mixture_experts_routing_moe_gb300 as moe

    op, dt = s["op"], TYPES[s["dtype"]]
    if op == "quantize":
        codes, scales = moe.moe_mx4_quantize(s["x"])
        return {"values": moe.moe_mx4_dequantize(codes, scales, s["K"], dt)}
    if op == "product":
        return {"out": moe.moe_mx4_product(*s["a"], *s["b"], offsets=s["offsets"], dtype=dt)}
    if op == "experts":
        return {"y": moe.moe_mx4_experts_forward_dispatched(s["x"], s["offsets"], s["gate"], s["up"], s["down"])}
    return {"out": moe.moe_mx4_forward_tokens(s["x"], s["router"], s["gate"], s["up"], s["down"], s["k"])}


# ------------------------------------------------------------------------------ what it has to do
def _block_bytes(rows, K):
    return rows * (-(-K // BLOCK)) * (BLOCK // 2 + 1)


def _used(n, E):
    """How many of E experts n independent choices reach, on the average."""
    return E * (1 - (1 - 1 / E) ** n)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op == "quantize":  # to blocks and back: the values, the blocks twice, the values
        rows, K = case["rows"], case["K"]
        return {"bytes": 2 * rows * K * size + 2 * _block_bytes(rows, K), "flops": 4 * rows * K}
    E = case["E"]
    if op == "product":
        rows, N, K = case["rows"], case["N"], case["K"]
        return {"bytes": _block_bytes(rows, K) + _used(rows, E) * _block_bytes(N, K) + rows * N * size, "flops": 2 * rows * N * K}
    H, I, T, k = case["H"], case["I"], case["T"], case["k"]
    one = 2 * _block_bytes(I, H) + _block_bytes(H, I)
    if op == "experts":
        rows = T * k
        return {"bytes": _used(rows, E) * one + 2 * rows * H * size, "flops": 6 * rows * H * I}
    return {"bytes": E * H * size + _used(T * k, E) * one + 2 * T * H * size, "flops": 6 * T * k * H * I + 2 * T * E * H}


# --------------------------------------------------------------- the definitions, in 64 bits
def _nearest64(x):
    """The values of x's rows after a trip through blocks, in 64 bits."""
    K = x.shape[-1]
    f = torch.nn.functional.pad(x.double(), (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = f.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp_min(1e-300)))
    e = (torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e)) - 2).clamp(-127, 127)
    v = f * torch.exp2(-e)
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return (torch.sign(v) * (torch.round(m / step) * step).clamp_max(6.0) * torch.exp2(e)).flatten(-2)[..., :K]


def _decode64(codes, scales):
    """(-1)^s 2^(x - 1) (1 + m / 2), or (-1)^s m / 2 where x = 0, times 2^(scale - 127)."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    sign = 1 - 2 * torch.floor(n / 8)
    n = n % 8
    x, m = torch.floor(n / 2), n % 2
    v = sign * torch.where(x > 0, torch.exp2(x - 1) * (1 + m / 2), m / 2)
    p = torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)
    return v * p[..., : v.shape[-1]]


def exact(case, seed):
    w = work(case)
    if w["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"values": _nearest64(s["x"])}
    if op in ("product", "experts"):
        edges = s["offsets"].tolist()
        a = _decode64(*s["a"]) if op == "product" else _nearest64(s["x"])
        parts = []
        for e in range(case["E"]):
            rows = a[edges[e] : edges[e + 1]]
            if op == "product":
                parts.append(rows @ _decode64(s["b"][0][e], s["b"][1][e]).T)
                continue
            wide = torch.nn.functional.pad(rows, (0, -case["H"] % BLOCK))
            g = wide @ _decode64(s["gate"][0][e], s["gate"][1][e]).T
            u = wide @ _decode64(s["up"][0][e], s["up"][1][e]).T
            h = _nearest64(g / (1 + torch.exp(-g)) * u)
            h = torch.nn.functional.pad(h, (0, -case["I"] % BLOCK))
            parts.append(h @ _decode64(s["down"][0][e], s["down"][1][e]).T)
        return {"out" if op == "product" else "y": torch.cat(parts)}
    H, I, k, dt = case["H"], case["I"], case["k"], TYPES[case["dtype"]]
    x = s["x"].double()
    logits = x @ s["router"].double().T
    idx = torch.argsort(-logits, dim=-1, stable=True)[:, :k]
    p = torch.exp(logits - logits.amax(-1, keepdim=True)).gather(1, idx)
    p = p / p.sum(-1, keepdim=True)
    out = torch.zeros_like(x)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        g = x[t] @ _decode64(s["gate"][0][e], s["gate"][1][e])[:, :H].T
        u = x[t] @ _decode64(s["up"][0][e], s["up"][1][e])[:, :H].T
        h = (g / (1 + torch.exp(-g)) * u).to(dt).double()
        out.index_add_(0, t, (h @ _decode64(s["down"][0][e], s["down"][1][e])[:, :I].T) * p[t, j, None])
    return {"out": out}
