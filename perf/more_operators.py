"""More serving operators, measured: what a decoder layer does between its products. The root-mean-square norm with
the residual's addition, the gate of a feed-forward layer (both with outputs in 8 bits and scales, as the fp8 products
take them), the rotation of queries and keys by their positions on the way into a paged cache, and the fp8 products of
rows grouped by expert.

A case is a dict of plain values. `prepare` makes what a user's program holds before the call, `run` makes the
call (the library's where `own` is true, elementary torch operations in 32 bits otherwise), `exact` computes the
same outputs from the definitions in 64 bits and `work` counts the bytes and operations that cannot be saved."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one conversation between two layers: latency
        dict(name="norm one token", op="norm", M=1, K=4096, x="bf16", res="bf16", w="bf16", y="fp8", offset=0.0),
        # a small batch of a layer of an odd width, f32 for a product with 4-bit weights, weights around 0
        dict(name="norm ragged f32", op="norm", M=37, K=5201, x="f32", res="f32", w="f32", y="f32", offset=1.0),
        # a prompt between two layers, the residual stream kept in f32
        dict(name="norm prompt", op="norm", M=8192, K=4096, x="bf16", res="f32", w="bf16", y="fp8", offset=0.0),
        # behind a fused dual projection of one token (f32), before the next one
        dict(name="gate one token", op="gate", M=1, K=12288, x="f32", y="f32"),
        # a prompt between the two products of the feed-forward layer: gate and up are halves of one product's rows
        dict(name="gate prompt", op="gate", M=4096, K=12288, x="bf16", y="fp8"),
        # one conversation, one token: the smallest call, all latency
        dict(name="rope one token", op="rope", T=1, Hq=32, Hkv=8, D=128, rot=128, page=64, x="bf16", dtype="bf16", far=700,
             inter=False, skip=0.0, base=10000.0),
        # an odd batch of single tokens at far positions, neighbouring pairs, half of each head rotated, from f32
        dict(name="rope batch far", op="rope", T=131, Hq=20, Hkv=4, D=64, rot=32, page=16, x="f32", dtype="f16",
             far=1000000, inter=True, skip=0.05, base=500000.0),
        # a prompt's queries, keys and values, parts of one fused projection, with padding tokens
        dict(name="rope prompt", op="rope", T=8192, Hq=32, Hkv=8, D=128, rot=128, page=64, x="bf16", dtype="bf16", far=131072,
             inter=False, skip=0.02, base=500000.0),
        # one token's eight experts of 64: bound by the weights of those experts
        dict(name="experts one token", op="experts", E=64, tokens=1, top=8, N=4096, K=2048, y="bf16", tail=0, route=1),
        # a decode batch: nearly every expert has a few rows, all weights are read once
        dict(name="experts decode batch", op="experts", E=64, tokens=32, top=8, N=4096, K=4096, y="bf16", tail=0, route=2),
        # a batch on few experts, sizes that are no multiples of a block, rows behind the last expert's, f32
        dict(name="experts ragged f32", op="experts", E=9, tokens=151, top=2, N=2200, K=5200, y="f32", tail=5, route=3),
        # a prompt: about 512 rows for each expert, unevenly; bound by the tensor cores
        dict(name="experts prompt", op="experts", E=32, tokens=4096, top=4, N=4096, K=4096, y="bf16", tail=0, route=4),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm", "gate", "gate", "rope", "rope", "experts", "experts", "experts"])
    if op in ("norm", "gate"):
        K = 8 * log(4, 2048) if rng.random() < 0.7 else log(17, 16384)
        M = min(log(1, 16384), max(1, 33000000 // K))
        x, y = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["fp8", "fp8", "f32", "bf16", "f16"])
        if op == "gate":
            return dict(op=op, M=M, K=K, x=x, y=y)
        return dict(op=op, M=M, K=K, x=x, res=rng.choice(["", x, x, "f32"]), w=rng.choice([x, "f32"]), y=y,
                    offset=rng.choice([0.0, 0.0, 1.0]))
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        T = min(log(1, 8192), 300000 // D)
        return dict(op=op, T=T, Hq=rng.choice([0, Hkv, 4 * Hkv, 4 * Hkv]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]), page=rng.choice([8, 16, 32, 64, 128]),
                    x=rng.choice(["f32", "bf16", "bf16", "f16"]), dtype=rng.choice(["bf16", "f16"]), far=log(2, 2000000),
                    inter=rng.random() < 0.4, skip=rng.choice([0.0, 0.1]), base=rng.choice([10000.0, 500000.0]))
    E = log(2, 128)
    N, K = log(64, 4096), 16 * log(8, 256) if rng.random() < 0.8 else log(100, 3000)
    N = max(64, min(N, 1000000000 // (E * K)))
    top = rng.randint(1, min(E, 8))
    tokens = max(1, min(log(1, 4096), 16384 // top))
    return dict(op=op, E=E, tokens=tokens, top=top, N=N, K=K, y=rng.choice(["bf16", "bf16", "f32"]), tail=rng.choice([0, 0, 3]),
                route=rng.randint(0, 10**6))


def counts(c):
    """How many rows each expert has: every token goes to `top` different ones, some of which are more popular."""
    r = np.random.RandomState(c["route"])
    score = r.randn(c["E"]) * 0.5 + r.gumbel(size=(c["tokens"], c["E"]))
    chosen = np.argpartition(-score, c["top"] - 1, axis=1)[:, :c["top"]]
    return np.bincount(chosen.ravel(), minlength=c["E"])


# ------------------------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    return globals()["prepare_" + case["op"]](case, torch.Generator("cuda").manual_seed(seed))


def normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def prepare_norm(c, g):
    M, K = c["M"], c["K"]
    # a few channels stand out, and rows differ in size, as in the middle of a model
    loud = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    size = torch.exp(normal(g, M, 1))
    x = (normal(g, M, K) * size).to(DTYPES[c["x"]])
    res = (normal(g, M, K) * loud * size).to(DTYPES[c["res"]]) if c["res"] else None
    w = (normal(g, K) * 0.2 + 1.0 - c["offset"]).to(DTYPES[c["w"]])
    return dict(c, xs=x, rs=res, ws=w, eps=1e-6)


def prepare_gate(c, g):
    both = normal(g, c["M"], 2 * c["K"]) * 2.0
    both = both.to(DTYPES[c["x"]])
    return dict(c, gate=both[:, :c["K"]], up=both[:, c["K"]:])


def prepare_rope(c, g):
    T, page, D, dt = c["T"], c["page"], c["D"], DTYPES[c["dtype"]]
    num_pages = -(-T // page) * 2 + 1
    qkv = normal(g, T, c["Hq"] + 2 * c["Hkv"], D).to(DTYPES[c["x"]])
    slots = torch.randperm(num_pages * page, generator=g, device="cuda")[:T].clone()
    slots[torch.rand(T, generator=g, device="cuda") < c["skip"]] = -1  # padding tokens
    positions = torch.randint(0, c["far"], (T,), generator=g, device="cuda")
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
    inv_freq = torch.pow(torch.full((), c["base"], dtype=torch.float64, device="cuda"), -i / c["rot"]).float()
    return dict(c, q=qkv[:, :c["Hq"]] if c["Hq"] else None, k=qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], v=qkv[:, c["Hq"] + c["Hkv"]:],
                slots=slots, positions=positions, inv_freq=inv_freq,
                k_cache=normal(g, num_pages, c["Hkv"], page, D, dtype=dt), v_cache=normal(g, num_pages, c["Hkv"], page, D, dtype=dt))


def prepare_experts(c, g):
    E, N, K = c["E"], c["N"], c["K"]
    n = counts(c)
    M = int(n.sum()) + c["tail"]
    nb, kb = -(-N // 128), -(-K // 128)
    a = (normal(g, M, K) * 110.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    a_scales = torch.rand(M, kb, generator=g, device="cuda") * 0.01 + 0.004
    w = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        w[e] = (normal(g, N, K) * 110.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    w_scales = (torch.rand(E, nb, kb, generator=g, device="cuda") + 0.5) * 0.0002
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
    return dict(c, a=a, a_scales=a_scales, ws=w, w_scales=w_scales, offsets=offsets, most=int(n.max()),
                out=torch.zeros(M, N, dtype=DTYPES[c["y"]], device="cuda"))


# --------------------------------------------------------------------------------------------------- the calls
def run(state):
    return globals()[("own_" if own else "plain_") + state["op"]](state)


def coded(y):
    """e4m3 codes of rows and one scale per 128 values."""
    M, K = y.shape
    kb = -(-K // 128)
    blocks = torch.cat([y, y.new_zeros(M, kb * 128 - K)], 1).view(M, kb, 128)
    scales = blocks.abs().amax(2) / torch.full((), 448.0, device=y.device)
    scales = torch.where(scales == 0, torch.ones_like(scales), scales)
    codes = (blocks / scales[:, :, None]).to(torch.float8_e4m3fn).view(M, kb * 128)
    return {"codes": codes.view(torch.uint8)[:, :K].contiguous().view(torch.float8_e4m3fn), "scales": scales}


def own_norm(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    if s["y"] == "fp8":
        r = qg.rms_norm_fp8_b128(s["xs"], s["ws"], s["rs"], eps=s["eps"], weight_offset=s["offset"])
        return dict(zip(("codes", "scales", "res"), r))
    r = qg.rms_norm(s["xs"], s["ws"], s["rs"], eps=s["eps"], weight_offset=s["offset"], out_dtype=DTYPES[s["y"]])
    return {"y": r} if s["rs"] is None else dict(zip(("y", "res"), r))


def plain_norm(s):
    h = s["xs"].float()
    if s["rs"] is not None:
        h = h + s["rs"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * (s["ws"].float() + s["offset"])
    out = coded(y) if s["y"] == "fp8" else {"y": y.to(DTYPES[s["y"]])}
    return out if s["rs"] is None else dict(out, res=h.to(s["rs"].dtype))


def own_gate(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    if s["y"] == "fp8":
        return dict(zip(("codes", "scales"), qg.silu_mul_fp8_b128(s["gate"], s["up"])))
    return {"y": qg.silu_mul(s["gate"], s["up"], out_dtype=DTYPES[s["y"]])}


def plain_gate(s):
    g = s["gate"].float()
    y = g / (1.0 + torch.exp(-g)) * s["up"].float()
    return coded(y) if s["y"] == "fp8" else {"y": y.to(DTYPES[s["y"]])}


def own_rope(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    q = qg.kv_append_rope(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"], s["slots"],
                          interleaved=s["inter"])
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def turned(x, cos, sin, inter):
    """x [T, heads, D] in f32, its first 2 n values of each head rotated, n angles per token."""
    x, n = x.float(), cos.shape[1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([a, b], 3).flatten(2) if inter else torch.cat([a, b], 2)
    return torch.cat([head, x[..., 2 * n:]], 2)


def plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dt = s["k_cache"].dtype
    live = s["slots"] >= 0
    at = s["slots"][live]
    page, place = at // s["page"], at % s["page"]
    s["k_cache"][page, :, place] = turned(s["k"], cos, sin, s["inter"])[live].to(dt)
    s["v_cache"][page, :, place] = s["v"][live].to(dt)
    q = None if s["q"] is None else turned(s["q"], cos, sin, s["inter"]).to(dt)
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def own_experts(s):
    import bit_quantized_gemv_dequant_gb300 as qg
    return {"y": qg.qmm_fp8_b128_grouped(s["a"], s["a_scales"], s["ws"], s["w_scales"], s["offsets"], s["out"])}


def plain_experts(s):
    E, N, K = s["ws"].shape
    at = s["offsets"].long()
    j = torch.arange(s["most"], device=at.device)
    real = j[None, :] < (at[1:] - at[:-1])[:, None]  # [E, most]
    row = (at[:-1, None] + j[None, :]).clamp(max=s["a"].shape[0] - 1)
    a = s["a"].float() * s["a_scales"].repeat_interleave(128, 1)[:, :K]
    w = s["ws"].float() * s["w_scales"].repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    s["out"][row[real]] = torch.matmul(a[row], w.transpose(1, 2))[real].to(s["out"].dtype)
    return {"y": s["out"]}


# --------------------------------------------------------------------------------------------- the definitions
def exact(case, seed):
    return globals()["exact_" + case["op"]](prepare(case, seed))


def codes_of(y):
    """The codes' values and scales of y in 64 bits; the nearest e4m3 value by arithmetic: 4 significant bits, steps of
    2**-9 at least, ties to even."""
    codes, scales = [], []
    for part in torch.split(y, 128, 1):
        top = part.abs().amax(1, keepdim=True)
        scale = torch.where(top > 0, top / 448.0, 1.0)
        v = part / scale
        step = torch.exp2(torch.clamp(torch.frexp(v).exponent - 4, min=-9).double())
        codes.append((torch.round(v / step) * step).clamp(-448.0, 448.0))
        scales.append(scale)
    return {"codes": torch.cat(codes, 1), "scales": torch.cat(scales, 1)}


def exact_norm(s):
    h = s["xs"].double() if s["rs"] is None else s["xs"].double() + s["rs"].double()
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / s["K"] + s["eps"]) * (s["ws"].double() + s["offset"])
    out = codes_of(y) if s["y"] == "fp8" else {"y": y}
    if s["rs"] is not None:
        out["res"] = h
    return out


def exact_gate(s):
    y = s["gate"].double() * torch.sigmoid(s["gate"].double()) * s["up"].double()
    return codes_of(y) if s["y"] == "fp8" else {"y": y}


def exact_rope(s):
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None, None] * s["inv_freq"].double())
    n, D = s["rot"] // 2, s["D"]
    pair = torch.arange(n, device="cuda")
    first, second = (2 * pair, 2 * pair + 1) if s["inter"] else (pair, pair + n)

    def rotate(x):
        y = x.double().clone()
        w = torch.complex(y[:, :, first], y[:, :, second]) * z
        y[:, :, first], y[:, :, second] = w.real, w.imag
        return y

    T, page = s["T"], s["page"]
    out = {"q": None if s["q"] is None else rotate(s["q"])}
    for name, rows in (("k", rotate(s["k"])), ("v", s["v"].double())):
        cache = s[name + "_cache"].double()
        flat = cache.transpose(1, 2).reshape(-1, s["Hkv"], D)
        live = torch.nonzero(s["slots"] >= 0).flatten()
        flat[s["slots"][live]] = rows[live]
        out[name] = flat.view(-1, page, s["Hkv"], D).transpose(1, 2)
    return out


def exact_experts(s):
    y = torch.zeros(s["a"].shape[0], s["N"], dtype=torch.float64, device="cuda")
    at = s["offsets"].tolist()
    of = torch.arange(s["N"], device="cuda") // 128
    for e in range(s["E"]):
        rows = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        for b, (a, w) in enumerate(zip(s["a"][rows].double().split(128, 1), s["ws"][e].double().split(128, 1))):
            y[rows] += (a @ w.t()) * s["a_scales"][rows, b, None].double() * s["w_scales"][e, of, b].double()
    return {"y": y}


# -------------------------------------------------------------------------------------------------- the floors
def work(case):
    return globals()["work_" + case["op"]](case)


def out_bytes(c):
    return c["M"] * (c["K"] * SIZE[c["y"]] + (4 * -(-c["K"] // 128) if c["y"] == "fp8" else 0))


def work_norm(c):
    n = c["M"] * c["K"]
    return {"bytes": n * (SIZE[c["x"]] + 2 * SIZE.get(c["res"], 0)) + c["K"] * SIZE[c["w"]] + out_bytes(c), "flops": 5 * n}


def work_gate(c):
    n = c["M"] * c["K"]
    return {"bytes": 2 * n * SIZE[c["x"]] + out_bytes(c), "flops": 5 * n}


def work_rope(c):
    n = c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
    return {"bytes": n * (SIZE[c["x"]] + SIZE[c["dtype"]]) + 16 * c["T"], "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}


def work_experts(c):
    n = counts(c)
    M, N, K, used = int(n.sum()), c["N"], c["K"], int((n > 0).sum())
    nb, kb = -(-N // 128), -(-K // 128)
    return {"bytes": M * (K + 4 * kb + N * SIZE[c["y"]]) + used * (N * K + 4 * nb * kb), "flops": 2 * M * N * K}
