"""Cases that measure the bf16 expert products, the bf16 SwiGLU and the AdamW step.

Each case is one pass through one operator, in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, through the package's binding, as a program that trains
or serves a mixture-of-experts layer calls it.
"""
import math

import numpy as np
import torch

own = False   # set from outside: False computes the plain forms, True calls the package

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest MoE layer of the tests and the benchmark: launch latency counts
        dict(name="fwd_tiny", op="fwd", T=512, k=1, E=4, K=256, N=512, skew=0.0),
        # one token through the gate/up projection of the FFN layer: serving, bound by the weights
        dict(name="fwd_one_token", op="fwd", T=1, k=8, E=32, K=7168, N=4096, skew=0.0),
        # the FFN layer's gate/up projection over a training batch
        dict(name="fwd_ffn", op="fwd", T=16384, k=8, E=32, K=7168, N=4096, skew=0.0),
        # a small ragged layer, sizes that no tile divides, some experts without rows
        dict(name="dgrad_odd", op="dgrad", T=1013, k=3, E=23, K=1112, N=712, skew=1.2),
        # input gradient of the down projection with 128 experts of very uneven popularity
        dict(name="dgrad_skewed", op="dgrad", T=4096, k=8, E=128, K=4096, N=1536, skew=1.2),
        # weight gradient of a small ragged layer: few rows per expert, the output dominates
        dict(name="wgrad_odd", op="wgrad", T=517, k=4, E=24, K=1544, N=1064, skew=1.2),
        # weight gradient of the FFN layer's down projection
        dict(name="wgrad_ffn", op="wgrad", T=16384, k=8, E=32, K=2048, N=7168, skew=0.0),
        # activation of a few routed rows while serving
        dict(name="swiglu_fwd_serving", op="swiglu_fwd", R=8, I=2048),
        # backward of the activation over the FFN layer's routed rows
        dict(name="swiglu_bwd_ffn", op="swiglu_bwd", R=131072, I=2048),
        # optimizer over many small tensors (norms, biases, routers, a small layer's weights)
        dict(name="adamw32_many_small", op="adamw", bits=32, tensors=96, elems=700_001, param="bf16", grad="bf16",
             stochastic=False, clip=1.0),
        # 8-bit states over weights of odd sizes, bf16 parameters without a master copy
        dict(name="adamw8_odd", op="adamw", bits=8, tensors=37, elems=117_440_519, param="bf16", grad="fp32",
             stochastic=True, clip=1.0),
        # fp32 parameters with a bf16 copy for the products, fp32 states: a whole layer's weights
        dict(name="adamw32_layer", op="adamw", bits=32, tensors=8, elems=402_653_184, param="fp32", grad="fp32",
             stochastic=False, clip=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: an odd multiple of 256 (whole tiles), or of 8 (the finest that rows may have)."""
    unit = 256 if rng.random() < 0.4 else 8
    v = max(1, _log(rng, lo, hi) // unit)
    return unit * (v if v % 2 else v + 1)


def draw(rng):
    op = rng.choice(["fwd", "fwd", "dgrad", "dgrad", "wgrad", "wgrad", "swiglu_fwd", "swiglu_bwd", "adamw", "adamw"])
    if op.startswith("swiglu"):
        I = _width(rng, 64, 4096)
        R = min(_log(rng, 1, 131072), 131072 * 2048 // I)
        return dict(op=op, R=R, I=I)
    if op == "adamw":
        param = rng.choice(["bf16", "fp32"])
        elems = _log(rng, 20_000, 200_000_000) | 1
        return dict(op=op, bits=rng.choice([8, 32]), tensors=min(_log(rng, 1, 200), elems // 50), elems=elems, param=param,
                    grad=rng.choice(["bf16", "fp32"]), stochastic=param == "bf16" and rng.random() < 0.5,
                    clip=rng.choice([0.0, 1.0]))
    E = rng.choice([1, 3, 8, 16, 32, 60, 128])
    k = rng.randint(1, min(8, E))
    T, K, N = _log(rng, 1, 16384), _width(rng, 64, 7168), _width(rng, 64, 7168)
    skew = rng.choice([0.0, 1.2])
    while E * N * K > 950_000_000:
        E = max(1, E // 2)
        k = min(k, E)
    # the plain form pads every expert to the fullest one
    while T > 1 and E * min(T, (4 * T * k // E + 64) if skew == 0.0 else T) * max(N * K / 2.9e7, (N + K) / 11264) > 131072:
        T = max(1, T * 2 // 3)
    return dict(op=op, T=T, k=k, E=E, K=K, N=N, skew=skew)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _bf16(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).bfloat16()


def _routing(case, seed):
    """Rows per expert of top-k routing; with skew, expert popularity falls with its rank and every ninth expert gets no rows."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 1)
    T, E, k = case["T"], case["E"], case["k"]
    score = torch.randn(T, E, generator=g)
    if case["skew"]:
        u = torch.rand(T, E, generator=g).clamp_(1e-20, 1.0)
        rank = torch.randperm(E, generator=g) + 1.0
        logp = -case["skew"] * torch.log(rank)
        dead = torch.arange(E) % 9 == 4
        score = logp - torch.log(-torch.log(u))
        if E - int(dead.sum()) >= k:
            score[:, dead] = -math.inf
    ids = torch.topk(score, k, dim=1).indices
    return torch.bincount(ids.reshape(-1), minlength=E)


def _sizes(case):
    """Element counts of an optimizer's tensors: weights, biases and scalars of very different sizes, most of them odd."""
    n, total = case["tensors"], case["elems"]
    w = [4.0 ** ((7 * i) % 5) for i in range(n)]
    s = [max(1, int(total * x / sum(w)) // 3 * 2 - i) for i, x in enumerate(w)]
    s[n // 2] += max(0, total - sum(s))
    return s


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=dict(case))
    op = case["op"]
    if op.startswith("swiglu"):
        R, I = case["R"], case["I"]
        st["a"] = _bf16((R, 2 * I), g, 2.0)
        if op == "swiglu_fwd":
            st["h"] = torch.empty(R, I, dtype=torch.bfloat16, device=DEV)
        else:
            st["dh"] = _bf16((R, I), g, 1e-2)
            st["da"] = torch.empty(R, 2 * I, dtype=torch.bfloat16, device=DEV)
        return st
    if op == "adamw":
        sizes = _sizes(case)
        first = [0]
        first += [int(x) for x in np.cumsum([-(-n // 32) * 32 for n in sizes])]   # every tensor starts on a 32-element boundary
        P = first[-1]
        real = torch.zeros(P, dtype=torch.bool, device=DEV)
        decay = torch.zeros(P // 32, device=DEV)                                  # weight decay by block of 32: none for the small tensors
        st["wd"] = [0.1 if n >= 4096 else 0.0 for n in sizes]
        starts = torch.tensor(first[:-1], device=DEV)
        lens = torch.tensor(sizes, device=DEV)
        which = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), torch.tensor([(b - a) // 32 for a, b in zip(first, first[1:])], device=DEV))
        decay.copy_(torch.tensor(st["wd"], device=DEV)[which])
        real.view(-1, 32).copy_(torch.arange(P, device=DEV).view(-1, 32) - starts[which, None] < lens[which, None])
        mag = torch.exp(torch.randn(P // 32, 1, generator=g, device=DEV))         # gradients differ in size from row to row

        def flat(std):
            x = torch.randn(P, generator=g, device=DEV)
            x.view(-1, 32).mul_(mag)
            return x.mul_(std).mul_(real)
        dt = dict(bf16=torch.bfloat16, fp32=torch.float32)
        st["p"] = (torch.randn(P, generator=g, device=DEV) * 0.02).mul_(real).to(dt[case["param"]])
        st["g"] = flat(1e-3).to(dt[case["grad"]])
        m, r = flat(3e-4), flat(1e-3).abs_()
        if case["bits"] == 8:
            st["m"], st["ms"] = _encode_m(m, None)
            st["r"], st["rs"] = _encode_r(r, None)
            st["values"] = torch.zeros(2, P, dtype=torch.bfloat16, device=DEV)
        else:
            st["m"], st["v"] = m, r.square_()
        if case["param"] == "fp32":
            st["copy"] = torch.zeros(P, dtype=torch.bfloat16, device=DEV)
        st["step"] = torch.full((1,), 40, dtype=torch.int64, device=DEV)
        st["norm"] = torch.zeros(2, device=DEV)
        st["decay"], st["seed"], st["hyper"] = decay, int(seed) & 0x7FFFFFFF, dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8)
        if own:   # the plan that a training program makes once, when it has its tensors
            from mxfp8_block_scaled_rowwise_gb300 import binding as mx
            cut = [(a, a + n) for a, n in zip(first, sizes)]

            def part(t, blocks=False):
                return [t[a // 32:-(-b // 32)] if blocks else t[a:b] for a, b in cut]
            eight = case["bits"] == 8
            st["plan"] = mx.adamw_plan(part(st["p"]), part(st["g"]), part(st["m"]), part(st["r"] if eight else st["v"]),
                                       scale_m=part(st["ms"], True) if eight else None,
                                       scale_r=part(st["rs"], True) if eight else None,
                                       copies=part(st["copy"]) if "copy" in st else None, weight_decay=st["wd"])
        return st
    counts = _routing(case, seed)
    E, K, N = case["E"], case["K"], case["N"]
    R = int(counts.sum())
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(counts, 0)
    st["off"], st["most"], st["R"] = off.to(DEV), max(1, int(counts.max())), R
    st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op == "fwd":
        st["a"], st["w"] = _bf16((R, K), g), _bf16((E, N, K), g, K ** -0.5)
        st["out"] = torch.empty(R, N, dtype=torch.bfloat16, device=DEV)
    elif op == "dgrad":
        st["a"], st["w"] = _bf16((R, K), g, 1e-2), _bf16((E, K, N), g, N ** -0.5)
        st["out"] = torch.empty(R, N, dtype=torch.bfloat16, device=DEV)
    else:
        st["a"], st["w"] = _bf16((R, N), g, 1e-2), _bf16((R, K), g)
        st["out"] = torch.empty(E, N, K, dtype=torch.float32, device=DEV)
    return st


# ------------------------------------------------------------------ 8-bit states: codes, scales, random bits
# Both codes hold 32 elements to one power-of-two scale, a byte b for 2^(b - 127); b = 0 is a block of zeros.
# First moment: E4M3 codes, the smallest scale that keeps the block's largest value at 448 or below.
# Root of the second moment: code c > 0 stands for (1 + (c & 15) / 16) 2^((c >> 4) - 15), 0 for 0; the largest value is 31/16 at most.
# Rounding: up where the 16 random bits u exceed what the fraction lacks, code = floor(x + u / 2^16); no u rounds to nearest.
def _exponent(x):
    return (x.contiguous().view(torch.int32) >> 23) - 127


def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _block_scale(x, top):
    amax = x.abs().view(-1, 32).amax(1, keepdim=True)
    e = _exponent(amax) - int(math.log2(top))
    e = torch.where(amax > top * _pow2(e.clamp(min=-126)), e + 1, e).clamp(min=-126).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, -127)), amax > 0


def _encode_m(m, u):
    e, some = _block_scale(m, 448.0)
    y = (m.view(-1, 32) * _pow2(-e.clamp(min=-126))).abs_()
    small = y < 2.0 ** -6
    bits = torch.where(small, y + 2.0 ** -6, y).view(torch.int32)
    bits = bits + (0x7FFFF + ((bits >> 20) & 1) if u is None else u.view(-1, 32) << 4)
    y = (bits & ~0xFFFFF).view(torch.float32)
    y = torch.where(small, y - 2.0 ** -6, y)
    return torch.copysign(y, m.view(-1, 32)).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), (e + 127).to(torch.uint8).view(-1)


def _encode_r(r, u):
    e, some = _block_scale(r, 1.9375)
    y = r.view(-1, 32) * _pow2(-e.clamp(min=-126))
    bits = y.view(torch.int32)
    bits = bits + (0x3FFFF + ((bits >> 19) & 1) if u is None else u.view(-1, 32) << 3)
    c = ((bits >> 19) - (112 << 4)).clamp(1, 255)
    return torch.where(r.view(-1, 32) > 0, c, torch.zeros_like(c)).to(torch.uint8).view(-1), (e + 127).to(torch.uint8).view(-1)


def _scales(b):
    b = b.to(torch.int32)
    return torch.where(b > 0, (b << 23).view(torch.float32), torch.zeros((), device=b.device)).view(-1, 1)


def _decode_m(c, b):
    return (c.view(torch.float8_e4m3fn).float().view(-1, 32) * _scales(b)).view(-1)


def _decode_r(c, b):
    i = c.to(torch.int32)
    x = torch.where(i > 0, ((i << 19) + (112 << 23)).view(torch.float32), torch.zeros((), device=c.device))
    return (x.view(-1, 32) * _scales(b)).view(-1)


def _hash(x, c1, s1, c2, s2):
    """Multiply, shift, multiply, shift on 32-bit words held in 64 bits."""
    x = (x * c1) & 0xFFFFFFFF
    x = x ^ (x >> s1)
    x = (x * c2) & 0xFFFFFFFF
    return x ^ (x >> s2)


def _key(seed, t, hi):
    k = _hash((seed + 0x9E3779B9 * t) & 0xFFFFFFFF, 0x9E3779B1, 15, 0x85EBCA77, 13)
    return _hash((k ^ (t >> 32)) + hi & 0xFFFFFFFF, 0x9E3779B1, 15, 0x85EBCA77, 13)


def _random_bits(P, seed, t):
    """Three 16-bit numbers for every element: for the first moment, the root of the second, and the parameter."""
    pos = torch.arange(P, device=DEV, dtype=torch.int64)
    x = _hash((pos & 0xFFFFFFFF) ^ _key(seed, t, 0), 0x9E3779B1, 15, 0x85EBCA77, 13)
    y = ((x ^ (x >> 7)) * 0xC2B2AE3D) & 0xFFFFFFFF
    return (x >> 16).int(), (x & 0xFFFF).int(), (y >> 16).int()


# ------------------------------------------------------------------ one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from mxfp8_block_scaled_rowwise_gb300 import binding as mx
    c = st["case"]
    op = c["op"]
    if op == "swiglu_fwd":
        mx.moe_swiglu_fwd(st["a"], c["R"], c["I"], st["h"])
        return st["h"]
    if op == "swiglu_bwd":
        mx.moe_swiglu_bwd(st["dh"], st["a"], c["R"], c["I"], st["da"])
        return st["da"]
    if op == "adamw":
        clip = c["clip"] > 0
        if clip:
            mx.adamw_grad_norm(st["plan"], c["clip"], st["norm"])
        mx.adamw_step(st["plan"], st["step"], grad_scale=st["norm"][1:] if clip else None, seed=st["seed"],
                      stochastic=c["stochastic"], **st["hyper"])
        if c["bits"] == 8:
            mx.adamw_state_values(st["plan"], st["values"][0], st["values"][1])
        return _adamw_outputs(st)
    call = dict(fwd=mx.grouped_gemm_bf16_fwd, dgrad=mx.grouped_gemm_bf16_dgrad, wgrad=mx.grouped_gemm_bf16_wgrad)[op]
    call(st["a"], st["w"], st["off"], c["E"], st["R"], c["N"], c["K"], st["out"], st["err"])
    return st["out"]


def _adamw_outputs(st):
    out = dict(param=st["p"], step=st["step"])
    if st["case"]["clip"] > 0:
        out["norm"] = st["norm"]
    if "copy" in st:
        out["copy"] = st["copy"]
    if st["case"]["bits"] == 8:
        out["moment"], out["root"] = st["values"][0], st["values"][1]
    else:
        out["moment"], out["second"] = st["m"], st["v"]
    return out


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op.startswith("swiglu"):
        gate, up = st["a"].float().chunk(2, dim=1)
        s = 1.0 / (1.0 + torch.exp(-gate))
        if op == "swiglu_fwd":
            st["h"].copy_(gate * s * up)
            return st["h"]
        dh = st["dh"].float()
        st["da"][:, : c["I"]].copy_(dh * up * s * (1.0 + gate * (1.0 - s)))
        st["da"][:, c["I"]:].copy_(dh * gate * s)
        return st["da"]
    if op == "adamw":
        return _plain_adamw(st)
    off, most, R = st["off"].long(), st["most"], st["R"]
    row = torch.arange(R, device=DEV)
    expert = torch.searchsorted(off[1:], row, right=True)
    place = row - off[expert]
    at = off[:-1, None] + torch.arange(most, device=DEV)           # each expert's rows, padded to the fullest one's
    there = (at < off[1:, None])[:, :, None]
    at = at.clamp_(max=R - 1)
    a = torch.where(there, st["a"][at], 0).float()
    if op == "wgrad":
        b = torch.where(there, st["w"][at], 0).float()
        st["out"].copy_(torch.bmm(a.transpose(1, 2), b))
    else:
        w = st["w"].float()
        st["out"].copy_(torch.bmm(a, w.transpose(1, 2) if op == "fwd" else w)[expert, place])
    return st["out"]


def _plain_adamw(st):
    c, h = st["case"], st["hyper"]
    t = int(st["t"]) + 1 if "t" in st else 41                      # the program's own count of steps
    st["t"] = t
    st["step"] += 1
    b1, b2 = h["beta1"], h["beta2"]
    g = st["g"].float()
    if c["clip"] > 0:
        norm = g.square().sum(dtype=torch.float32).sqrt()
        scale = torch.clamp(c["clip"] / norm, max=1.0)
        st["norm"].copy_(torch.stack([norm, scale]))
        g = g * scale
    eight = c["bits"] == 8
    u = _random_bits(g.numel(), st["seed"], t) if eight or c["stochastic"] else None
    m = _decode_m(st["m"], st["ms"]) if eight else st["m"]
    v = _decode_r(st["r"], st["rs"]).square() if eight else st["v"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g.square()
    r = v.sqrt()
    p = st["p"].float()
    p = (p.view(-1, 32) * (1.0 - h["lr"] * st["decay"])[:, None]).view(-1)
    p = p - h["lr"] / (1.0 - b1 ** t) * m / (r / math.sqrt(1.0 - b2 ** t) + h["eps"])
    if c["stochastic"]:
        p = ((p.view(torch.int32) + u[2]) & ~0xFFFF).view(torch.float32)
    st["p"].copy_(p)
    if "copy" in st:
        st["copy"].copy_(p)
    if eight:
        cm, sm = _encode_m(m, u[0])
        cr, sr = _encode_r(r, u[1])
        st["m"].copy_(cm)
        st["ms"].copy_(sm)
        st["r"].copy_(cr)
        st["rs"].copy_(sr)
        st["values"][0].copy_(_decode_m(cm, sm))
        st["values"][1].copy_(_decode_r(cr, sr))
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _adamw_outputs(st)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op.startswith("swiglu"):
        n = case["R"] * case["I"]
        return dict(bytes=n * (6 if op == "swiglu_fwd" else 10), flops=n * (8 if op == "swiglu_fwd" else 14))
    if op == "adamw":
        n = sum(_sizes(case))
        p, g = (2 if case["param"] == "bf16" else 4), (2 if case["grad"] == "bf16" else 4)
        states = 16 if case["bits"] == 32 else 4 + 4 / 32 + 4      # read and written; 8 bits: and the values they stand for
        return dict(bytes=n * (2 * p + g + states + (2 if case["param"] == "fp32" else 0)), flops=n * 20)
    T, k, E, K, N = (case[x] for x in ("T", "k", "E", "K", "N"))
    R = T * k
    flops = 2 * R * N * K
    if op == "wgrad":
        return dict(bytes=2 * R * (N + K) + 4 * E * N * K, flops=flops)
    return dict(bytes=2 * R * (N + K) + 2 * min(E, R) * N * K, flops=flops)


# ------------------------------------------------------------------ the same from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(dict(case), seed)
    op = case["op"]
    if op.startswith("swiglu"):
        I = case["I"]
        outs = []
        for r0 in range(0, case["R"], 16384):
            a = st["a"][r0:r0 + 16384].double()
            gate, up = a[:, :I], a[:, I:]
            sig = torch.sigmoid(gate)
            if op == "swiglu_fwd":
                outs.append((up * gate * sig).float())
            else:
                dh = st["dh"][r0:r0 + 16384].double()
                outs.append(torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], 1).float())
        return torch.cat(outs)
    if op == "adamw":
        return _exact_adamw(st)
    off = st["off"].tolist()
    E, K, N = case["E"], case["K"], case["N"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = st["a"][a:b].double()
        if op == "wgrad":
            out[e] = x.mT @ st["w"][a:b].double()
        elif op == "fwd":
            out[a:b] = torch.einsum("rk,nk->rn", x, st["w"][e].double())
        else:
            out[a:b] = x @ st["w"][e].double()
    return out


def _exact_adamw(st):
    c, h = st["case"], st["hyper"]
    t, eight = 41, c["bits"] == 8
    g = st["g"].double()
    out = dict(step=None)
    scale = 1.0
    if c["clip"] > 0:
        norm = float(torch.dot(g, g)) ** 0.5
        scale = min(1.0, c["clip"] / norm)
        out["norm"] = torch.tensor([norm, scale], dtype=torch.float64, device=DEV)
    g = g * scale

    def values(codes, scales, table):
        return (torch.tensor(table, dtype=torch.float64, device=DEV)[codes.long()].view(-1, 32)
                * torch.where(scales > 0, torch.exp2(scales.double() - 127), 0.0)[:, None]).view(-1)
    e4m3 = [math.nan if x & 127 == 127 else (-1.0) ** (x >> 7) * ((x & 7) / 8 * 2.0 ** -6 if x & 120 == 0 else (1 + (x & 7) / 8) * 2.0 ** ((x >> 3 & 15) - 7))
            for x in range(256)]
    root = [0.0] + [(1 + (x & 15) / 16) * 2.0 ** ((x >> 4) - 15) for x in range(1, 256)]
    m = values(st["m"], st["ms"], e4m3) if eight else st["m"].double()
    v = values(st["r"], st["rs"], root) ** 2 if eight else st["v"].double()
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + g * g * (1 - h["beta2"])
    del g
    mhat, vhat = m / (1 - h["beta1"] ** t), v / (1 - h["beta2"] ** t)
    p = st["p"].double()
    p -= h["lr"] * (st["decay"].double().repeat_interleave(32) * p + mhat / (vhat.sqrt() + h["eps"]))
    del mhat, vhat
    u = [x.double() / 65536 for x in _random_bits(p.numel(), st["seed"], t)] if eight or c["stochastic"] else None
    if c["stochastic"]:
        ulp = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
        out["param"] = torch.copysign(torch.floor(p.abs() / ulp + u[2]) * ulp, p)
    else:
        out["param"] = p
    if "copy" in st:
        out["copy"] = p
    if not eight:
        out["moment"], out["second"] = m, v
        return out

    def rounded(x, u, top, mantissa, lowest, floor_exp):
        """x >= 0 to a code's grid under its block's scale, from u in [0, 1)."""
        x = x.view(-1, 32)
        X = torch.exp2(torch.ceil(torch.log2(x.amax(1, keepdim=True).clamp(min=1e-60) / top)))
        y = x / X
        ulp = torch.exp2(torch.floor(torch.log2(y.clamp(min=1e-60))).clamp(min=floor_exp) - mantissa)
        y = torch.floor(y / ulp + u.view(-1, 32)) * ulp
        return (torch.where(x > 0, y.clamp(min=lowest), 0.0) * X).view(-1)
    out["moment"] = torch.copysign(rounded(m.abs(), u[0], 448.0, 3, 0.0, -6), m)
    out["root"] = rounded(v.sqrt(), u[1], 1.9375, 4, 17 / 16 * 2.0 ** -15, -15)
    return out
