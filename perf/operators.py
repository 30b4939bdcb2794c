"""Workloads of the operators around a DiT block's quantized linears.

Three operators, each with a plain torch form and the call a user of the
package makes:

* ``adapter``: one quantized projection shared by the rows of many requests,
  each row with the low-rank adapter of its own request (or none),
  Y[i] = X[i] w_hat^T + s_a (X[i] D_a^T) U_a^T with a = rows[i];
* ``qk_norm_rope``: root-mean-square norms of queries and keys and the rotary
  position rotation in one pass;
* ``rope``: the rotation alone, interleaved or half layout, part of the head,
  several position axes, frequencies scaled for long contexts, and inverse.
"""
import math

import numpy as np
import torch

own = False

GROUP = 128
_AXES3 = 3                      # frame, row and column positions of a video token


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token through an attention output projection, the smallest call
        dict(name="adapter_1x5120x5120_b4_r16", op="adapter", m=1, n=5120, k=5120, bits=4, adapters=8, rank=16,
             mix="tokens", out="bf16"),
        # 16 tokens of 16 requests, each with its own adapter, fused qkv of the block
        dict(name="adapter_16x15360x5120_b5_r16_each", op="adapter", m=16, n=15360, k=5120, bits=5, adapters=16,
             rank=16, mix="tokens", out="bf16"),
        # an odd number of tokens through the block's down projection, float32 output
        dict(name="adapter_37x5120x13824_b6_r64_f32", op="adapter", m=37, n=5120, k=13824, bits=6, adapters=5,
             rank=64, mix="tokens", out="f32"),
        # requests of ragged lengths in one batch, some without an adapter
        dict(name="adapter_1001x5120x5120_b4_r32", op="adapter", m=1001, n=5120, k=5120, bits=4, adapters=6, rank=32,
             mix="requests", out="bf16"),
        # an ordinary prompt batch through the block's up projection
        dict(name="adapter_4096x13824x5120_b5_r16", op="adapter", m=4096, n=13824, k=5120, bits=5, adapters=8,
             rank=16, mix="requests", out="bf16"),
        # a whole video's tokens through the fused qkv, the largest call
        dict(name="adapter_32760x15360x5120_b4_r32", op="adapter", m=32760, n=15360, k=5120, bits=4, adapters=4,
             rank=32, mix="requests", out="bf16"),
        # one token: latency
        dict(name="qknorm_1x40x128_head", op="qk_norm_rope", batch=1, tokens=1, hq=40, hk=40, dim=128, rot=128,
             norm="head", layout="interleaved", axes=1, fused=True, dtype="bf16", scaling="none", far=1000),
        # the video's tokens, q and k as slices of the fused qkv output
        dict(name="qknorm_32760x40x128_head", op="qk_norm_rope", batch=1, tokens=32760, hq=40, hk=40, dim=128,
             rot=128, norm="head", layout="interleaved", axes=_AXES3, fused=True, dtype="bf16", scaling="none", far=0),
        # two guidance branches, the norm over all heads of the token
        dict(name="qknorm_2x4099x40x128_token", op="qk_norm_rope", batch=2, tokens=4099, hq=40, hk=40, dim=128,
             rot=128, norm="token", layout="half", axes=_AXES3, fused=True, dtype="bf16", scaling="none", far=0),
        # shared key heads, an odd length, part of the head rotated, float32
        dict(name="qknorm_3x1009x24x96_head_f32", op="qk_norm_rope", batch=3, tokens=1009, hq=24, hk=8, dim=96,
             rot=64, norm="head", layout="half", axes=1, fused=False, dtype="f32", scaling="ntk", far=30000),
        # long context: scaled frequencies, far positions, part of the head
        dict(name="rope_2x16384x24x128_half_yarn", op="rope", batch=2, tokens=16384, hq=24, hk=0, dim=128, rot=64,
             norm="none", layout="half", axes=1, fused=False, dtype="bf16", scaling="yarn", far=900000, inverse=False),
        # the inverse rotation of a few float32 rows (the gradient of the rotation)
        dict(name="rope_1x257x16x72_inverse_f32", op="rope", batch=1, tokens=257, hq=16, hk=0, dim=72, rot=72,
             norm="none", layout="interleaved", axes=1, fused=True, dtype="f32", scaling="linear", far=5000,
             inverse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            m = _log(rng, 1, 32760)
            n = 16 * _log(rng, 8, 960)
            k = 128 * _log(rng, 4, 108)
            if m * n * k <= 32760 * 15360 * 5120:
                break
        rank = rng.choice([8, 16, 24, 32, 64, 128])
        most = 2048 if m <= 1024 else 256
        adapters = rng.randint(1, max(1, min(24, most // rank)))
        return dict(op="adapter", m=m, n=n, k=k, bits=rng.choice([3, 4, 5, 6, 7]), adapters=adapters, rank=rank,
                    mix=rng.choice(["tokens", "requests"]), out=rng.choice(["bf16", "bf16", "f32"]))
    op = rng.choice(["qk_norm_rope", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        dim = rng.choice([64, 72, 80, 96, 128, 128, 160, 256])
        hq = _log(rng, 1, 40)
        hk = rng.choice([h for h in range(1, hq + 1) if hq % h == 0]) if op == "qk_norm_rope" else 0
        batch = rng.randint(1, 4)
        tokens = _log(rng, 1, 32760)
        size = 2 if dtype == "bf16" else 4
        if batch * tokens * (hq + hk) * dim * size <= 32760 * 80 * 128 * 2:
            break
    axes = rng.choice([1, _AXES3])
    case = dict(op=op, batch=batch, tokens=tokens, hq=hq, hk=hk, dim=dim,
                rot=rng.choice([dim, dim // 2 // 2 * 2]),
                norm=rng.choice(["head", "head", "token"]) if op == "qk_norm_rope" else "none",
                layout=rng.choice(["interleaved", "half"]), axes=axes, fused=rng.random() < 0.5, dtype=dtype,
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]) if axes == 1 else "none",
                far=_log(rng, 1, 1000000) if axes == 1 else 0)
    if op == "rope":
        case["inverse"] = rng.random() < 0.3
    return case


def work(case):
    if case["op"] == "adapter":
        m, n, k, b, r = (case[x] for x in ("m", "n", "k", "bits", "rank"))
        used = min(case["adapters"], m)
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * m * k + n * k * b // 8 + n * k // 32 + used * (2 * r * (n + k) + 4) + 4 * m + out * m * n,
                "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    size = 2 if case["dtype"] == "bf16" else 4
    rows = case["batch"] * case["tokens"]
    elements = rows * (case["hq"] + case["hk"]) * case["dim"]
    weights = 0
    if case["norm"] != "none":
        weights = 2 * case["dim"] if case["norm"] == "head" else (case["hq"] + case["hk"]) * case["dim"]
    return {"bytes": 2 * elements * size + weights * size + 4 * rows * case["axes"] + 4 * case["rot"],
            "flops": elements * (3 if case["norm"] == "none" else 7)}


# -------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantized(gen, n, k, bits):
    """The stored record of an N(0, 0.02^2) weight: codes of `bits` bits in one
    most-significant-bit-first stream, and float32 scales per 128 inputs."""
    half = (1 << (bits - 1)) - 1
    packed, scales = [], []
    place = torch.arange(7, -1, -1, device="cuda", dtype=torch.int64) * bits
    byte = torch.arange(bits - 1, -1, -1, device="cuda", dtype=torch.int64) * 8
    for r0 in range(0, n, 2048):
        rows = min(2048, n - r0)
        w = torch.randn(rows, k // GROUP, GROUP, device="cuda", generator=gen) * 0.02
        step = 2.0 * (w.abs().amax(-1) * 1.01) / float((1 << bits) - 1)
        q = torch.round(w / step[..., None]).clamp_(-half, half).to(torch.int64) + half
        word = (q.view(-1, 8) << place).sum(-1)
        packed.append(((word[:, None] >> byte) & 255).to(torch.uint8).view(-1))
        scales.append(step)
    return torch.cat(packed), torch.cat(scales).contiguous()


def _request_rows(case, seed):
    """The adapter of every row: drawn row by row, or runs of ragged lengths
    (requests one after another); about one in eight is without an adapter."""
    rng = np.random.default_rng([seed, 11])
    m, a = case["m"], case["adapters"]
    if case["mix"] == "tokens":
        rows = rng.integers(0, a, m)
        if m >= a:                                   # every adapter in use
            rows[rng.permutation(m)[:a]] = np.arange(a)
        if m >= 8:
            rows[rng.random(m) < 0.06] = -1
        return rows.astype(np.int32)
    cuts = np.sort(rng.integers(0, m + 1, a))
    rows = np.searchsorted(cuts, np.arange(m), side="right") - 1
    return rows.astype(np.int32)                     # rows before the first cut: -1, no adapter


def _scaled_frequencies(pairs, scaling):
    """(frequencies, amplitude) of `pairs` pairs, base 10000, for contexts
    longer than the model's by a factor of 4 (8192 positions originally)."""
    rot, base, factor, original = 2 * pairs, 10000.0, 4.0, 8192.0
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2.0))
    freqs = [base ** (-2.0 * i / rot) for i in range(pairs)]
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    if scaling == "yarn":
        def pair_of(turns):
            return rot * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        low = max(math.floor(pair_of(32.0)), 0)
        high = min(math.ceil(pair_of(1.0)), rot - 1)
        for i in range(pairs):
            ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
            freqs[i] = freqs[i] * (1.0 - ramp) + freqs[i] / factor * ramp
        return freqs, 0.1 * math.log(factor) + 1.0
    return freqs, 1.0


def _positions(case):
    s = case["tokens"]
    if case["axes"] == 1:
        return np.arange(s, dtype=np.int64)[:, None] + case["far"]
    w = max(1, int(math.sqrt(s / 8.0)))
    t = np.arange(s, dtype=np.int64)
    return np.stack([t // (w * w), t // w % w, t % w], -1)


def _sections(case):
    """Pairs of each position axis: the first axis takes what three equal parts leave."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return (pairs,)
    part = pairs // 3
    return (pairs - 2 * part, part, part)


def prepare(case, seed):
    gen = _generator(seed)
    if case["op"] == "adapter":
        m, n, k, b, a, r = (case[x] for x in ("m", "n", "k", "bits", "adapters", "rank"))
        packed, scales = _quantized(gen, n, k, b)
        state = dict(case=case,
                     x=torch.randn(m, k, device="cuda", generator=gen).bfloat16(), packed=packed, scales=scales,
                     down=(torch.randn(a, r, k, device="cuda", generator=gen) / math.sqrt(k)).bfloat16(),
                     up=(torch.randn(a, n, r, device="cuda", generator=gen) * 0.1).bfloat16(),
                     weight=torch.rand(a, device="cuda", generator=gen) * 1.5 + 0.25,
                     rows=torch.from_numpy(_request_rows(case, seed)).cuda())
        if own:
            from dit_dequant_gemm_amd import api
            state["record"] = api.QWeight(packed, scales, b, n, k, k)
            state["pool"] = api.AdapterPool(state["down"], state["up"], state["weight"])
        return state
    b, s, hq, hk, d = (case[x] for x in ("batch", "tokens", "hq", "hk", "dim"))
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["fused"]:
        # slices of the fused projection's output; the value part is there too
        buf = torch.randn(b, s, (hq + 2 * hk) * d, device="cuda", generator=gen, dtype=dtype)
        q = buf[..., :hq * d].view(b, s, hq, d)
        kk = buf[..., hq * d:(hq + hk) * d].view(b, s, hk, d)
    else:
        q = torch.randn(b, hq, s, d, device="cuda", generator=gen, dtype=dtype).transpose(1, 2)
        kk = torch.randn(b, hk, s, d, device="cuda", generator=gen, dtype=dtype).transpose(1, 2)
    state = dict(case=case, q=q, k=kk, positions=torch.from_numpy(_positions(case).astype(np.int32)).cuda())
    freqs, amplitude = [], 1.0
    for pairs in _sections(case):
        f, amplitude = _scaled_frequencies(pairs, case["scaling"])
        freqs += f
    state["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    state["amplitude"] = amplitude
    if case["norm"] != "none":
        for name, heads in (("q_weight", hq), ("k_weight", hk)):
            size = d if case["norm"] == "head" else heads * d
            state[name] = (1.0 + 0.2 * torch.randn(size, device="cuda", generator=gen)).to(dtype)
    return state


# ---------------------------------------------------------------- plain forms
def _plain_adapter(state):
    case = state["case"]
    n, k, b, a, r = (case[x] for x in ("n", "k", "bits", "adapters", "rank"))
    # codes of the packed stream, eight at a time from `bits` bytes
    byte = torch.arange(b - 1, -1, -1, device="cuda", dtype=torch.int64) * 8
    place = torch.arange(7, -1, -1, device="cuda", dtype=torch.int64) * b
    word = (state["packed"].view(-1, b).to(torch.int64) << byte).sum(-1)
    q = ((word[:, None] >> place) & ((1 << b) - 1)) - ((1 << (b - 1)) - 1)
    w = (q.float().view(n, k // GROUP, GROUP) * state["scales"][..., None]).view(n, k)
    w = w.bfloat16().float()                         # the stored format's weight is bf16
    x = state["x"].float()
    t = (x @ state["down"].view(a * r, k).float().t()).view(-1, a, r)
    mine = state["rows"][:, None] == torch.arange(a, device="cuda", dtype=torch.int32)
    t = torch.where(mine[..., None], t * state["weight"][:, None], torch.zeros((), device="cuda"))
    up = state["up"].permute(0, 2, 1).reshape(a * r, n).float()
    y = x @ w.t() + t.view(-1, a * r) @ up
    return y.bfloat16() if case["out"] == "bf16" else y


def _angles(state):
    """cos and sin (batch of tokens x pairs), the angles in 64 bits."""
    case = state["case"]
    axis = torch.repeat_interleave(torch.arange(case["axes"], device="cuda"),
                                   torch.tensor(_sections(case), device="cuda"), output_size=case["rot"] // 2)
    angle = state["positions"].double()[:, axis] * state["freqs"]
    if case.get("inverse"):
        angle = -angle
    return (torch.cos(angle).float() * state["amplitude"])[:, None], (torch.sin(angle).float() * state["amplitude"])[:, None]


def _plain_rotate(x, cos, sin, case):
    rot = case["rot"]
    y = x.clone()
    if case["layout"] == "interleaved":
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = u * cos - v * sin
        y[..., 1:rot:2] = v * cos + u * sin
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = u * cos - v * sin
        y[..., rot // 2:rot] = v * cos + u * sin
    return y


def _plain_norm(x, weight, case):
    x = x.float()
    if case["norm"] == "head":
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rstd = torch.rsqrt((x * x).mean((-1, -2), keepdim=True) + 1e-6)
    return x * rstd * weight.float().view(x.shape[-2], x.shape[-1])


def run(state):
    case = state["case"]
    if own:
        from dit_dequant_gemm_amd import api
        if case["op"] == "adapter":
            return api.adapter_gemm(state["x"], state["record"], state["pool"], state["rows"],
                                    out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        rotary = dict(layout=case["layout"], sections=_sections(case), amplitude=state["amplitude"])
        if case["op"] == "rope":
            return api.rope(state["q"], state["positions"], state["freqs"], inverse=case["inverse"], **rotary)
        return api.qk_norm_rope(state["q"], state["k"], state["positions"], state["freqs"],
                                q_weight=state["q_weight"], k_weight=state["k_weight"], eps=1e-6,
                                norm=case["norm"], **rotary)
    if case["op"] == "adapter":
        return _plain_adapter(state)
    cos, sin = _angles(state)
    if case["op"] == "rope":
        return _plain_rotate(state["q"].float(), cos, sin, case).to(state["q"].dtype)
    return tuple(_plain_rotate(_plain_norm(state[t], state[t + "_weight"], case), cos, sin, case).to(state[t].dtype)
                 for t in ("q", "k"))


# ------------------------------------------------------------------ 64 bits
def _exact_weight(state, n, k, bits):
    """The record's bf16 weight as float64: every code's bits read one by one
    from the stream."""
    out = torch.empty(n, k, dtype=torch.float64, device="cuda")
    shift = torch.arange(7, -1, -1, device="cuda", dtype=torch.uint8)
    row_bytes = k * bits // 8
    for r0 in range(0, n, 512):
        rows = min(512, n - r0)
        part = state["packed"][r0 * row_bytes:(r0 + rows) * row_bytes]
        stream = ((part[:, None] >> shift) & 1).view(rows * k, bits)
        code = torch.zeros(rows * k, dtype=torch.int32, device="cuda")
        for j in range(bits):
            code = 2 * code + stream[:, j]
        level = (code - (2 ** (bits - 1) - 1)).view(rows, k // GROUP, GROUP).float()
        w = level * state["scales"][r0:r0 + rows].unsqueeze(2)
        out[r0:r0 + rows] = w.view(rows, k).to(torch.bfloat16).double()
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "adapter":
        x = state["x"].double()
        y = x @ _exact_weight(state, case["n"], case["k"], case["bits"]).T
        rows = state["rows"].cpu().numpy()
        for a in range(case["adapters"]):
            ids = torch.from_numpy(np.flatnonzero(rows == a)).cuda()
            if ids.numel():
                t = x[ids] @ state["down"][a].double().T
                y[ids] += float(state["weight"][a]) * (t @ state["up"][a].double().T)
        return y
    pairs, rot = case["rot"] // 2, case["rot"]
    axis = np.concatenate([np.full(c, i) for i, c in enumerate(_sections(case))])
    angle = _positions(case).astype(np.float64)[:, axis] * state["freqs"].cpu().numpy()
    if case.get("inverse"):
        angle = -angle
    # each pair as a complex number, turned by its angle
    turn = torch.from_numpy(np.exp(1j * angle) * state["amplitude"]).cuda()[None, :, None]

    def rotated(x):
        head, rest = x[..., :rot], x[..., rot:]
        if case["layout"] == "interleaved":
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], pairs, 2).contiguous()) * turn
            head = torch.view_as_real(z).reshape(head.shape)
        else:
            z = torch.complex(head[..., :pairs].contiguous(), head[..., pairs:].contiguous()) * turn
            head = torch.cat([z.real, z.imag], -1)
        return torch.cat([head, rest], -1)

    def one(x, weight):
        out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 26) // max(1, x.shape[2] * x.shape[3]))      # tokens at a time: bounded memory
        nonlocal turn
        whole = turn
        for b in range(x.shape[0]):
            for s0 in range(0, x.shape[1], step):
                v = x[b:b + 1, s0:s0 + step].double()
                if weight is not None:
                    dims = (3,) if case["norm"] == "head" else (2, 3)
                    v = v / torch.sqrt(v.square().mean(dims, keepdim=True) + 1e-6)
                    v = v * weight.double().view((1, -1) if case["norm"] == "head" else (x.shape[2], x.shape[3]))
                turn = whole[:, s0:s0 + step]
                out[b:b + 1, s0:s0 + step] = rotated(v)
        turn = whole
        return out

    if case["op"] == "rope":
        return one(state["q"], None)
    return one(state["q"], state["q_weight"]), one(state["k"], state["k_weight"])
